"""Where spec_tree_attention's join looks for the parts of a pair: inside the workspace, and at the places that its
workgroups write, whatever the lengths."""
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "rejection_sampling_verify_07_amd", "csrc")
ROUND = 64  # keys


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("deal") / "tree_deal")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, "-o", out,
                    os.path.join(HERE, "tree_deal_helper.cpp")], check=True, capture_output=True)
    return out


@pytest.fixture(scope="module")
def places(exe):
    def run(rows):
        text = "".join("%d %d %d %d\n" % r for r in rows)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        found = [[int(x) for x in line.split()] for line in out.splitlines()]
        assert len(found) == len(rows)
        return [(f[0], f[1:]) for f in found]

    return run


def dealt(lengths, heads, groups, extra):
    """The line of all pairs' rounds as the workgroups walk it: its stretch, each pair's first round and number of
    rounds, and the places that its parts are written to (None: one workgroup has all of it)."""
    rounds = [-(-n // ROUND) for n in lengths for _ in range(heads)]
    if sum(rounds) < 8 * groups:
        extra = 0
    start = np.concatenate([[0], np.cumsum([n + extra for n in rounds])])
    stretch = max(1, -(-int(start[-1]) // groups))
    written = [[] for _ in rounds]
    for g in range(groups):
        at, end, first = g * stretch, min((g + 1) * stretch, int(start[-1])), True
        while at < end:
            p = int(np.searchsorted(start, at, side="right")) - 1
            j = at - int(start[p])
            step = min(rounds[p] + extra - j, end - at)
            take = min(step, rounds[p] - j)
            if take > 0:
                written[p].append(None if j == 0 and take == rounds[p] else 2 * g + (0 if first else 1))
            at, first = at + step, False
    return stretch, [int(x) for x in start[:-1]], rounds, written


BATCHES = [
    # lengths, key heads, workgroups, extra rounds of a pair
    ([0, 500], 8, 128, 2),
    ([0, 1024], 1, 32, 2),
    ([0, 0, 0, 0], 8, 512, 2),
    ([0], 1, 64, 4),
    ([8000, 0, 0, 3], 8, 512, 2),
    ([0, 9000, 0, 16000, 0], 8, 512, 4),
    ([0] * 60 + [3000], 8, 512, 2),
    ([1] + [0] * 300 + [70000] + [0] * 9, 1, 512, 2),
    ([0, 64, 0, 65, 0, 63], 2, 256, 2),
    ([0, 40000], 8, 1, 4),
]


@pytest.mark.parametrize("lengths,heads,groups,extra", BATCHES)
def test_places_of_batches_with_empty_sequences(places, lengths, heads, groups, extra):
    check(places, lengths, heads, groups, extra)


def test_stretches_of_the_longest_line(exe):
    """Up to the 2^31 - 1 rounds that the entry point admits."""
    rows = [(t, g) for g in (1, 2, 7, 8, 511, 512) for t in (0, 1, 2, g, g + 1, 10 ** 6, 2 ** 31 - g, 2 ** 31 - 2, 2 ** 31 - 1)
            if t < 2 ** 31]
    out = subprocess.run([exe, "stretch"], input="".join("%d %d\n" % r for r in rows), capture_output=True, text=True,
                         check=True).stdout
    assert [int(x) for x in out.split()] == [max(1, -(-t // g)) for t, g in rows]


def test_places_of_random_batches(places):
    rng = np.random.default_rng(3)
    for _ in range(150):
        n = int(rng.integers(1, 40))
        lengths = rng.integers(0, 2 ** rng.integers(1, 16), n) * (rng.random(n) < rng.random())
        check(places, lengths.tolist(), int(rng.integers(1, 9)), int(rng.choice([1, 2, 7, 64, 256, 512])),
              int(rng.choice([2, 4])))


def check(places, lengths, heads, groups, extra):
    stretch, start, rounds, written = dealt(lengths, heads, groups, extra)
    for side in (1, 2, 4):
        got = places([(f, n, stretch, side) for f, n in zip(start, rounds)])
        for (count, read), n, wrote in zip(got, rounds, written):
            assert all(0 <= x < 2 * groups for x in read), (lengths, read)
            assert count == len(wrote)
            if n == 0:
                assert read == []
            elif None in wrote:
                assert wrote == [None]  # (the join leaves the pair alone)
            else:
                assert read[:count] == wrote and set(read) == set(wrote)
