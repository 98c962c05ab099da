"""Plain forms of the calls on trees of guesses and paged caches (numpy, loops),
and input makers of their tests."""
import numpy as np

INT_MAX = 2 ** 31 - 1


# --------------------------------------------------------------------------
# paged caches: pools as numpy arrays [slabs, pages, heads, page_size, row]
# --------------------------------------------------------------------------
def compact_ref(pool, table, lengths, path, nacc, cu, kmax):
    """The pool after spec_cache_compact (a copy) and the new lengths."""
    out, (_, pages, _, size, _) = pool.copy(), pool.shape
    total = len(path) - len(nacc)
    new = np.zeros(len(nacc), np.int64)
    for b in range(len(nacc)):
        cap = size if table is None else table.shape[1] * size
        length = cap if lengths is None else min(max(int(lengths[b]), 0), cap)
        k0, k1 = (b * kmax, (b + 1) * kmax) if cu is None else (int(cu[b]), int(cu[b + 1]))
        kb, n = k1 - k0, int(nacc[b])
        bad = k0 < 0 or kb < 0 or kb > kmax or k1 > total
        if bad or n < 0 or n > kb:
            new[b] = length
            continue
        first = length - 1 - kb
        new[b] = max(first + 1 + n, 0)
        own = path[k0 + b:k0 + b + n + 1]
        moves = []
        for i in range(1, n + 1):
            if own[i] <= own[i - 1] or own[i] > kb or own[0] != 0:
                break
            at = []
            for p in (first + own[i], first + i):
                page = -1 if p < 0 else (b if table is None else table[b, p // size])
                at.append((int(page), int(p) % size) if 0 <= page < pages else None)
            if own[i] != i and first + i >= 0 and None not in at:
                moves.append(at)
        was = pool
        for (sp, so), (tp, to) in moves:
            out[:, tp, :, to] = was[:, sp, :, so]
    return out, new


def fork_ref(pool, table, lengths, parents, refs, new_lengths=None, beams=0, places=None):
    """spec_page_fork: the pool (a copy), the new tables, counts and free pages."""
    out, (_, pages, _, size, _) = pool.copy(), pool.shape
    old, most = table.shape
    places = (len(parents) if parents is not None else old) if places is None else places
    refs = refs.astype(np.int64).copy()
    new = np.full((places, most), -1, np.int64)
    for p in table.reshape(-1):
        if 0 <= p < pages:
            refs[p] -= 1
    plan = []
    for w in range(places):
        s = w if parents is None else int(parents[w])
        if beams and parents is not None:
            s = w // beams * beams + s if 0 <= s < beams else -1
        if not 0 <= s < old:
            plan.append(None)
            continue
        length = min(max(int(lengths[s]), 0), most * size)
        want = length if new_lengths is None else max(length, int(new_lengths[w]))
        plan.append((s, length // size, length % size, min(-(-want // size), most)))
        for i in range(length // size):
            new[w, i] = table[s, i]
            if 0 <= table[s, i] < pages:
                refs[table[s, i]] += 1
    opened, begin = {}, {}
    for w, pl in enumerate(plan):
        if pl is None:
            continue
        s, full, rest, _ = pl
        begin[w] = full
        if rest and 0 <= table[s, full] < pages:
            page = int(table[s, full])
            if page not in opened:
                opened[page] = refs[page] == 0
                if opened[page]:
                    new[w, full] = page
                    begin[w] += 1
    for page, kept in opened.items():
        if kept:
            refs[page] = 1
    free = [p for p in range(pages) if refs[p] == 0]
    left = len(free)
    for w, pl in enumerate(plan):
        if pl is None:
            continue
        s, full, rest, need = pl
        for i in range(begin[w], need):
            left -= 1
            if free:
                new[w, i] = free.pop(0)
                refs[new[w, i]] = 1
        if rest and begin[w] == full and 0 <= table[s, full] < pages and new[w, full] >= 0:
            out[:, new[w, full], :, :rest] = pool[:, table[s, full], :, :rest]
    return out, new, refs, left


def random_tables(rng, sequences, most, pages, lengths, size, share=0.4):
    """Tables of sequences that hold `lengths`, some pages shared between neighbours, and their counts."""
    spare = list(rng.permutation(pages))
    table, refs = np.full((sequences, most), -1, np.int64), np.zeros(pages, np.int64)
    for b in range(sequences):
        for i in range(-(-int(lengths[b]) // size)):
            if b > 0 and table[b - 1, i] >= 0 and (i == 0 or table[b, i - 1] == table[b - 1, i - 1]) and rng.random() < share:
                table[b, i] = table[b - 1, i]
            else:
                table[b, i] = spare.pop()
            refs[table[b, i]] += 1
    return table, refs


# --------------------------------------------------------------------------
# trees: parents[j] is the row (0 .. j) that guess j extends
# --------------------------------------------------------------------------
def random_tree(rng, k, wide=4):
    return np.array([max(0, j - int(rng.integers(0, wide))) for j in range(k)], np.int64)


def way_up(parents, row):
    """Rows from `row` up to row 0."""
    way = [row]
    while way[-1] > 0:
        way.append(int(parents[way[-1] - 1]))
    return way


def walk_ref(tokens, ids, parents, vocab):
    """The walk over one sequence: tokens [K + 1], ids and parents [K].  (tokens out, accepted, path), or None."""
    k = len(ids)
    if any(not 0 <= int(x) < vocab for x in ids) or any(not 0 <= int(p) <= j for j, p in enumerate(parents)):
        return None
    path = [0]
    while True:
        follow = [j + 1 for j in range(k) if parents[j] == path[-1] and ids[j] == tokens[path[-1]]]
        if not follow:
            break
        path.append(follow[0])
    n = len(path) - 1
    out = [int(tokens[r]) for r in path] + [-1] * (k - n)
    return out, n, path + [-1] * (k - n)


# --------------------------------------------------------------------------
# edits of logits, in 64 bits
# --------------------------------------------------------------------------
def adjust_ref(logits, cu, tokens=None, lengths=None, prompt=None, rep=None, pres=None, freq=None, bias_ids=None,
               bias_values=None, cu_bias=None, masks=None, mask_rows=None, ids=None, parents=None):
    """logits float64 [rows, V].  The edited logits, how large the terms of each are together (0: nothing touches it)."""
    out, size = logits.copy(), np.zeros(logits.shape)
    V, batch = logits.shape[1], len(cu) - 1
    for b in range(batch):
        k = int(cu[b + 1] - cu[b])
        r_, p_, f_ = (1.0 if x is None and i == 0 else 0.0 if x is None else float(x[b])
                      for i, x in enumerate((rep, pres, freq)))
        text = [] if tokens is None else [int(t) for t in tokens[b]]
        if lengths is not None:
            text = text[:max(0, int(lengths[b]))]
        first = 0 if prompt is None else int(prompt[b])
        bias = {}
        if bias_ids is not None:
            lo, hi = (0, len(bias_ids)) if cu_bias is None else (int(cu_bias[b]), int(cu_bias[b + 1]))
            bias = {int(t): float(v) for t, v in zip(bias_ids[lo:hi], bias_values[lo:hi]) if 0 <= t < V}
        up = [j if parents is None else int(parents[cu[b] + j]) for j in range(k)]
        up = [u if 0 <= u <= j else 0 for j, u in enumerate(up)]
        for r in range(k + 1):
            row = int(cu[b]) + b + r
            path = [] if ids is None else [int(ids[cu[b] + x - 1]) for x in way_up(up, r) if x > 0]
            n = np.zeros(V)
            seen = np.zeros(V, bool)
            for i, t in enumerate(text + path):
                if 0 <= t < V:
                    seen[t] = True
                    n[t] += i >= first or i >= len(text)
            if (r_, p_, f_) != (1.0, 0.0, 0.0):
                x = out[row]
                x[seen] = np.where(x[seen] > 0, x[seen] / r_, x[seen] * r_)
                size[row][seen] += np.abs(x[seen])
                met = n > 0
                x[met] -= f_ * n[met]
                x[met] -= p_
                size[row][met] += np.abs(f_ * n[met]) + abs(p_)
            for t, v in bias.items():
                out[row, t] += v
                size[row, t] += abs(logits[row, t]) + abs(v)
            if masks is not None:
                m = row if mask_rows is None else int(mask_rows[row])
                if 0 <= m < len(masks):
                    bits = np.unpackbits(np.ascontiguousarray(masks[m]).view(np.uint8), bitorder="little")[:V]
                    out[row, bits == 0] = -np.inf
    return out, size


# --------------------------------------------------------------------------
# attention of trees over paged caches, in 64 bits
# --------------------------------------------------------------------------
def tree_attention_ref(q, k, v, table, lengths, parents, cu, scale, eps, tiny):
    """q [rows, Hq, D]; k, v [pages, size, Hk, D] (float64); table [B, most] or None (page b is the cache of b).
    Returns out, lse and how far a kernel with fp32 scores, weights rounded to the element type and fp32 sums may be
    off each, with the reasons of beam_util.attention_ref: products exact in fp32 and D of them added there, 4
    roundings on the way to the exponent, a weight rounded by eps / 2 (or `tiny`), n additions, out rounded once."""
    rows, Hq, D = q.shape
    pages, size, Hk, _ = k.shape
    rep = Hq // Hk
    out, lse = np.zeros((rows, Hq, D)), np.full((rows, Hq), -np.inf)
    b_out, b_lse = np.zeros((rows, Hq, D)), np.zeros((rows, Hq))
    for b in range(len(cu) - 1):
        n = int(cu[b + 1] - cu[b]) + 1
        up = [j if parents is None else int(parents[cu[b] + j]) for j in range(n - 1)]
        up = [u if 0 <= u <= j else 0 for j, u in enumerate(up)]
        cap = size if table is None else table.shape[1] * size
        length = cap if lengths is None else min(max(int(lengths[b]), 0), cap)
        at = np.arange(length)
        page = np.full(length, b) if table is None else table[b][at // size]
        there = (page >= 0) & (page < pages)
        kk = np.where(there[:, None, None], k[np.where(there, page, 0), at % size], 0.0)
        vv = np.where(there[:, None, None], v[np.where(there, page, 0), at % size], 0.0)
        for r in range(n):
            t = int(cu[b]) + b + r
            way = np.array(way_up(up, r)) + length - n
            see = there & (at < length - n)
            see[way[way >= 0]] = there[way[way >= 0]]
            if not see.any():
                continue
            for h in range(Hq):
                ks, vs = kk[see, h // rep], vv[see, h // rep]
                a = scale * (ks @ q[t, h])
                d_s = (D + 4) * 2.0 ** -24 * scale * (np.abs(ks) @ np.abs(q[t, h])).max()
                m = a.max()
                w = np.exp(a - m)
                z = w.sum()
                w /= z
                out[t, h], lse[t, h] = w @ vs, m + np.log(z)
                d = 2 * d_s + 8 * np.abs(a).max() * 2.0 ** -24 + 2.0 ** -22
                wv, c = w @ np.abs(vs), len(ks)
                b_out[t, h] = (eps / 2 * np.abs(out[t, h]) + (eps / 2 + d + 2 * c * 2.0 ** -24) * wv
                               + c * tiny * np.abs(vs).max() + tiny) * 1.01
                b_lse[t, h] = d + c * 2.0 ** -24 + 4 * 2.0 ** -24 * (1 + np.abs(lse[t, h]))
    return out, lse, b_out, b_lse
