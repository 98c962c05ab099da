// The places that the join of spec_tree_attention reads, by the library's own arithmetic.  Per line of input
// "from rounds stretch side" a line of output: the pair's parts, then each place read, in the order of the join's lanes.
// With an argument: per line "total groups" the stretch.
#include <cstdio>

#include "sv_tree_deal.hpp"

int main(int argc, char**)
{
    int total, groups;
    while (argc > 1 && std::scanf("%d %d", &total, &groups) == 2) std::printf("%d\n", sv::deal_stretch(total, groups));
    int from, rounds, stretch, side;
    while (std::scanf("%d %d %d %d", &from, &rounds, &stretch, &side) == 4) {
        const sv::PairParts parts = sv::pair_parts(from, rounds, stretch);
        std::printf("%d", parts.count);
        const int most = sv::join_batch(parts.count, side);
        for (int p0 = 0; most > 0 && p0 < (most == 8 ? parts.count : 1); p0 += 8 * side)
            for (int j = 0; j < most; ++j)
                for (int sub = 0; sub < side; ++sub)
                    std::printf(" %lld", (long long)sv::part_place(parts, sv::join_part(parts.count, p0 + j * side + sub)));
        std::printf("\n");
    }
    return 0;
}
