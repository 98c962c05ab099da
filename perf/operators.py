"""The beam-decoding operators as measured cases: what a decode step over several
continuations of one prompt does besides the model's products.

  select     spec_beam_select: the next beams of every group, out of all beams and
             the whole vocabulary
  reorder    spec_state_reorder: the beams' states (caches, token histories) put in
             the order of their parents, in place
  attention  spec_prefix_attention: attention of every sequence's newest rows over a
             prefix that its group shares and over its own suffix

`own` chooses between the plain forms in this file and the framework's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ESIZE = {"f32": 4, "bf16": 2, "f16": 2}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _select(name, groups, beams, vocab, select, dtype, temperature=1.0, finished=0, pad=0):
    """`finished`: ended beams per group; `pad`: elements between rows beyond the vocabulary."""
    return dict(name=name, op="select", groups=groups, beams=beams, vocab=vocab, select=select, dtype=dtype,
                temperature=temperature, finished=finished, pad=pad)


def _reorder(name, groups, beams, slabs, heads, positions, row, survivors, dtype):
    """States [slabs, beams, (heads,) positions, row]; heads = 0: no head dimension.
    `survivors`: distinct parents per group."""
    return dict(name=name, op="reorder", groups=groups, beams=beams, slabs=slabs, heads=heads, positions=positions,
                row=row, survivors=survivors, dtype=dtype)


def _attention(name, groups, seqs, draft, ragged, q_heads, kv_heads, dim, prefix, suffix, dtype):
    """`seqs` sequences per group, K_b = `draft` guesses each (0 .. draft when ragged)."""
    return dict(name=name, op="attention", groups=groups, seqs=seqs, draft=draft, ragged=ragged, q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, prefix=prefix, suffix=suffix, dtype=dtype)


def listed():
    return [
        # one request, four beams: the smallest step, where launches and latency count
        _select("select_g1_w4_v50304_f32", 1, 4, 50304, 8, "f32"),
        # a served batch of small beams, twice the beams kept so that ended ones can leave
        _select("select_g32_w4_v50304_bf16", 32, 4, 50304, 8, "bf16", 0.75),
        # odd sizes, rows that start off the 16-byte grid, ended beams
        _select("select_g13_w5_v32003_f16", 13, 5, 32003, 5, "f16", 1.25, 1, 7),
        # the largest: 64 requests, wide beams, a large vocabulary
        _select("select_g64_w8_v151936_bf16", 64, 8, 151936, 16, "bf16"),
        # one request's caches of a small model: 6 layers, K and V, early in the text
        _reorder("reorder_g1_w4_l12_p37", 1, 4, 12, 0, 37, 512, 3, "bf16"),
        # caches with the head dimension outside the positions, an odd row, several requests
        _reorder("reorder_g5_w6_h5_p251", 5, 6, 24, 5, 251, 90, 4, "f16"),
        # the largest: 8 requests of 8 beams, 32 layers of 8 heads of 128, 512 own positions
        _reorder("reorder_g8_w8_l64_p512", 8, 8, 64, 0, 512, 1024, 5, "bf16"),
        # one request, four beams of a small model: latency
        _attention("attn_g1_s4_p500_d64_f16", 1, 4, 0, False, 8, 8, 64, 500, 20, "f16"),
        # beam decoding of several requests: single rows, shared heads, a read of the caches
        _attention("attn_g4_s8_p4096_d128_bf16", 4, 8, 0, False, 32, 8, 128, 4096, 128, "bf16"),
        # the scoring rows of a verify with 1 to 9 rows a sequence, ragged
        _attention("attn_g2_s16_k8_p7777_d128_bf16", 2, 16, 8, True, 32, 4, 128, 7777, 515, "bf16"),
        # wide heads, few of them
        _attention("attn_g3_s5_k3_p2049_d256_f16", 3, 5, 3, True, 8, 2, 256, 2049, 100, "f16"),
        # the largest: 64 sequences with 5 rows each on one long prompt, where products count
        _attention("attn_g1_s64_k4_p16384_d128_bf16", 1, 64, 4, False, 32, 8, 128, 16384, 300, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_one(rng):
    op = rng.choice(("select", "reorder", "attention", "attention"))
    if op == "select":
        beams = rng.randint(1, 16)
        return _select("", _log_int(rng, 1, 64), beams, _log_int(rng, 1000, 160000), rng.randint(1, 2 * beams),
                       rng.choice(("f32", "bf16", "f16")), rng.choice((1.0, 0.7, 1.3)),
                       rng.randint(0, (beams - 1) // 2), rng.randint(0, 9))
    if op == "reorder":
        beams = rng.randint(2, 16)
        heads = rng.choice((0, rng.randint(1, 16)))
        row = rng.choice((64, 80, 90, 128, 256)) * (rng.randint(1, 8) if heads == 0 else 1)
        return _reorder("", _log_int(rng, 1, 32), beams, _log_int(rng, 2, 64), heads, _log_int(rng, 1, 1024), row,
                        rng.randint(1, beams), rng.choice(("f32", "bf16", "f16")))
    kv = rng.randint(1, 8)
    draft = rng.choice((0, rng.randint(1, 8)))
    return _attention("", _log_int(rng, 1, 8), _log_int(rng, 1, 64), draft, draft > 0 and rng.random() < 0.5,
                      kv * rng.choice((1, 2, 3, 4, 8)), kv, rng.choice((64, 128, 128, 256)),
                      _log_int(rng, 16, 16384), draft + _log_int(rng, 1, 600), rng.choice(("bf16", "f16")))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["op"], (0, 0))
        most[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        case = _draw_one(rng)
        w = work(case)
        if w["bytes"] <= most[case["op"]][0] and w["flops"] <= most[case["op"]][1]:
            del case["name"]
            return case


# --------------------------------------------------------------------------
# the sizes inside a case: the same numbers for every seed, in another order
# --------------------------------------------------------------------------
def _group_lengths(case):
    """reorder: own positions of each group's beams, from all of them down to half."""
    g, p = case["groups"], case["positions"]
    return [p - i * p // (2 * g) for i in range(g)]


def _drafts(case):
    b = case["groups"] * case["seqs"]
    return [i % (case["draft"] + 1) if case["ragged"] else case["draft"] for i in range(b)]


def _prefixes(case):
    g, p = case["groups"], case["prefix"]
    return [p - i * p // (4 * g) for i in range(g)]


def _suffixes(case):
    """attention: own positions of each sequence, its newest rows among them."""
    b, s, low = case["groups"] * case["seqs"], case["suffix"], case["draft"] + 1
    return [max(low, s - i * s // (2 * b)) for i in range(b)]


def work(case):
    es = ESIZE[case["dtype"]]
    if case["op"] == "select":
        rows = case["groups"] * (case["beams"] - case["finished"])
        return {"bytes": rows * case["vocab"] * es + case["groups"] * (5 * case["beams"] + 12 * case["select"]),
                "flops": 4 * rows * case["vocab"]}
    if case["op"] == "reorder":
        column = case["slabs"] * max(1, case["heads"]) * case["row"] * es
        return {"bytes": sum(_group_lengths(case)) * column * (case["survivors"] + case["beams"])
                + 4 * case["groups"] * (case["beams"] + 1), "flops": 0}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    drafts, prefixes, suffixes = _drafts(case), _prefixes(case), _suffixes(case)
    rows = sum(drafts) + len(drafts)
    mean_rows = rows / case["groups"]  # sequences are dealt to the groups at random
    seen = sum(mean_rows * p for p in prefixes) + rows / len(drafts) * sum(suffixes) - sum(k * (k + 1) / 2 for k in drafts)
    return {"bytes": (sum(prefixes) + sum(suffixes)) * hk * d * 2 * es + rows * hq * (2 * d * es + 4),
            "flops": int(4 * hq * d * seen)}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _shuffled(values, rng, dtype=torch.int32):
    return torch.tensor([values[i] for i in rng.permutation(len(values))], dtype=dtype).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)

    if case["op"] == "select":
        g, w, v = case["groups"], case["beams"], case["vocab"]
        # logits of spread 2 with 20 likely tokens a row, as a language model's
        logits = torch.randn((g * w, v + case["pad"]), generator=gen, device="cuda") * 2.0
        ids = torch.randint(0, v, (g * w, 20), generator=gen, device="cuda")
        logits.scatter_add_(1, ids, 8.0 + torch.randn((g * w, 20), generator=gen, device="cuda"))
        ended = torch.argsort(torch.rand((g, w), generator=gen, device="cuda"), dim=1) < case["finished"]
        return dict(case=case, logits=logits.to(dt)[:, :v],
                    scores=-10.0 - 6.0 * torch.rand((g * w,), generator=gen, device="cuda"),
                    finished=ended.reshape(-1).to(torch.uint8) if case["finished"] else None, pad_token=v // 2,
                    temperature=float(np.float32(case["temperature"])))
    if case["op"] == "reorder":
        g, w, p = case["groups"], case["beams"], case["positions"]
        shape = (case["slabs"], g * w) + ((case["heads"],) if case["heads"] else ()) + (p, case["row"])
        # every survivor at least once, the other places by chance, in the order of their scores
        parents = np.empty((g, w), np.int32)
        for i in range(g):
            alive = rng.permutation(w)[:case["survivors"]]
            parents[i] = rng.permutation(np.concatenate([alive, rng.choice(alive, w - len(alive))]))
        lengths = _shuffled(_group_lengths(case), rng).repeat_interleave(w).contiguous()
        return dict(case=case, states=randn(*shape), parents=torch.from_numpy(parents.reshape(-1)).cuda(),
                    lengths=lengths)
    g, b, hk, d = case["groups"], case["groups"] * case["seqs"], case["kv_heads"], case["dim"]
    drafts = rng.permutation(_drafts(case))
    cu = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
    rows = int(cu[-1]) + b
    # queries of spread 2: scores of spread 2, some keys much likelier than the rest
    return dict(case=case, q=(2.0 * randn(rows, case["q_heads"], d).float()).to(dt),
                prefix_k=randn(g, case["prefix"], hk, d), prefix_v=randn(g, case["prefix"], hk, d),
                suffix_k=randn(b, case["suffix"], hk, d), suffix_v=randn(b, case["suffix"], hk, d),
                prefix_lengths=_shuffled(_prefixes(case), rng), suffix_lengths=_shuffled(_suffixes(case), rng),
                cu_draft=torch.from_numpy(cu).cuda() if case["ragged"] else None)


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def _plain_select(s):
    c, logits = s["case"], s["logits"]
    g, w, v, n = c["groups"], c["beams"], c["vocab"], c["select"]
    # 64 bits: the order of two beams' candidates may hang on the last bits of their scores
    x = logits.double() / s["temperature"]
    top = x.max(dim=1, keepdim=True).values
    lse = top + torch.log(torch.exp(x - top).sum(dim=1, keepdim=True))
    score = s["scores"].double()[:, None] + (x - lse)
    if s["finished"] is not None:  # an ended beam has one candidate: the pad token, at its own score
        ended = s["finished"].bool()[:, None]
        at_pad = torch.arange(v, device=x.device)[None, :] == s["pad_token"]
        score = torch.where(ended, torch.where(at_pad, s["scores"].double()[:, None], -math.inf), score)
    score = score.view(g, w * v)
    # the n best; of equal ones the first: all above the n-th value, then the first of those equal to it
    last = torch.topk(score, n, dim=1).values[:, -1:]
    above, equal = score > last, score == last
    room = n - above.sum(dim=1, keepdim=True)
    chosen = above | (equal & (torch.cumsum(equal, dim=1) <= room))
    place = torch.arange(w * v, 0, -1, device=x.device, dtype=torch.int32)
    at = (w * v) - torch.topk(torch.where(chosen, place, 0), n, dim=1).values.long()
    best, order = torch.sort(torch.gather(score, 1, at), dim=1, descending=True, stable=True)
    at = torch.gather(at, 1, order)
    return {"scores": best.float(), "tokens": (at % v).int(), "parents": torch.div(at, v, rounding_mode="floor").int()}


def _plain_reorder(s):
    c, states, parents = s["case"], s["states"], s["parents"].long()
    g, w, p = c["groups"], c["beams"], c["positions"]
    source = parents + torch.arange(g, device=parents.device).repeat_interleave(w) * w
    moved = torch.arange(p, device=parents.device)[None, :] < s["lengths"][source][:, None]
    moved = moved.view((1, g * w) + ((1,) if c["heads"] else ()) + (p, 1))
    states.copy_(torch.where(moved, states.index_select(1, source), states))
    return states.view(torch.int32 if c["dtype"] == "f32" else torch.int16)


def _plain_attention(s):
    c, q = s["case"], s["q"]
    g, n, hq, hk, d = c["groups"], c["seqs"], c["q_heads"], c["kv_heads"], c["dim"]
    b, k, rep, dev = g * n, c["draft"] + 1, hq // hk, q.device
    # rows of sequence i at cu[i] + i, padded to k rows
    cu = s["cu_draft"].long() if s["cu_draft"] is not None else torch.arange(b + 1, device=dev) * c["draft"]
    rows = cu[1:] - cu[:-1] + 1
    first = cu[:-1] + torch.arange(b, device=dev)
    step = torch.arange(k, device=dev)
    padded = q.float()[(first[:, None] + torch.minimum(step[None, :], rows[:, None] - 1))]
    padded = padded.view(b, k, hk, rep, d).permute(0, 2, 1, 3, 4).reshape(b, hk, k * rep, d) / math.sqrt(d)
    shared = padded.view(g, n, hk, k * rep, d).transpose(1, 2).reshape(g, hk, n * k * rep, d)
    kp = s["prefix_k"].float().permute(0, 2, 3, 1).contiguous()
    ks = s["suffix_k"].float().permute(0, 2, 3, 1).contiguous()
    a = torch.matmul(shared, kp)
    a = torch.where(torch.arange(c["prefix"], device=dev) < s["prefix_lengths"][:, None, None, None], a, -math.inf)
    a = a.view(g, hk, n, k * rep, c["prefix"]).transpose(1, 2)
    e = torch.matmul(padded, ks).view(b, hk, k, rep, c["suffix"])
    seen = (s["suffix_lengths"] - rows)[:, None] + step[None, :] + 1  # row j of a sequence sees so many own positions
    e = torch.where(torch.arange(c["suffix"], device=dev) < seen[:, None, :, None, None], e, -math.inf)
    e = e.view(g, n, hk, k * rep, c["suffix"])
    top = torch.maximum(a.max(dim=-1, keepdim=True).values, e.max(dim=-1, keepdim=True).values)
    a, e = torch.exp(a - top), torch.exp(e - top)
    total = a.sum(dim=-1, keepdim=True) + e.sum(dim=-1, keepdim=True)
    vp = s["prefix_v"].float().transpose(1, 2).contiguous()
    vs = s["suffix_v"].float().transpose(1, 2).contiguous()
    o = torch.matmul(a.transpose(1, 2).reshape(g, hk, n * k * rep, c["prefix"]), vp)
    o = o.view(g, hk, n, k * rep, d).transpose(1, 2)
    o = (o + torch.matmul(e.reshape(b, hk, k * rep, c["suffix"]), vs).view(g, n, hk, k * rep, d)) / total
    lse = (top + torch.log(total)).reshape(b, hk, k, rep).permute(0, 2, 1, 3).reshape(b, k, hq)
    o = o.reshape(b, hk, k, rep, d).permute(0, 2, 1, 3, 4).reshape(b, k, hq, d)
    # back to the packed rows
    row = torch.arange(q.shape[0], device=dev)
    seq = torch.searchsorted(first, row, right=True) - 1
    at = row - first[seq]
    return {"out": o[seq, at].to(q.dtype), "lse": lse[seq, at]}


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------
def _plan(s):
    """The call with its arguments marshalled once, as a decoding loop keeps it."""
    import rejection_sampling_verify_07_amd as sv

    c = s["case"]
    if c["op"] == "select":
        return sv.BeamSelectPlan(s["logits"], s["scores"], beams=c["beams"], num_select=c["select"],
                                 temperature=s["temperature"], finished=s["finished"], pad_token=s["pad_token"])
    if c["op"] == "reorder":
        return sv.StateReorderPlan(s["states"], s["parents"], beams=c["beams"], lengths=s["lengths"])
    return sv.PrefixAttentionPlan(s["q"], s["prefix_k"], s["prefix_v"], s["suffix_k"], s["suffix_v"],
                                  s["prefix_lengths"], s["suffix_lengths"], cu_draft=s["cu_draft"],
                                  max_draft=c["draft"], return_lse=True)


def run(state):
    op = state["case"]["op"]
    if own:
        if "plan" not in state:
            state["plan"] = _plan(state)
        out = state["plan"]()
        return out.view(torch.int32 if state["case"]["dtype"] == "f32" else torch.int16) if op == "reorder" else out
    return {"select": _plain_select, "reorder": _plain_reorder, "attention": _plain_attention}[op](state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "reorder":  # values are moved, not computed
        return None
    s = prepare(case, seed)
    if case["op"] == "select":
        w, n = case["beams"], case["select"]
        best = []
        for i in range(case["groups"]):
            pool = []
            for j in range(i * w, (i + 1) * w):
                if s["finished"] is not None and bool(s["finished"][j]):
                    pool.append(s["scores"][j:j + 1].double())
                    continue
                row = s["logits"][j].double() / s["temperature"]
                pool.append(torch.topk(row, min(n, row.numel())).values - torch.logsumexp(row, 0) + s["scores"][j].double())
            best.append(torch.sort(torch.cat(pool), descending=True).values[:n])
        return {"scores": torch.stack(best), "tokens": None, "parents": None}
    hk, rep, d = case["kv_heads"], case["q_heads"] // case["kv_heads"], case["dim"]
    b = case["groups"] * case["seqs"]
    cu = s["cu_draft"].tolist() if s["cu_draft"] is not None else [i * case["draft"] for i in range(b + 1)]
    lp, ls = s["prefix_lengths"].tolist(), s["suffix_lengths"].tolist()
    out, lse = [], []
    for i in range(b):
        g = i // case["seqs"]
        rows = cu[i + 1] - cu[i] + 1
        keys = torch.cat([s["prefix_k"][g, :lp[g]], s["suffix_k"][i, :ls[i]]]).double()
        vals = torch.cat([s["prefix_v"][g, :lp[g]], s["suffix_v"][i, :ls[i]]]).double()
        for j in range(rows):
            seen = lp[g] + ls[i] - (rows - 1 - j)
            query = s["q"][cu[i] + i + j].double().view(hk, rep, d)
            a = torch.stack([query[h] @ keys[:seen, h].t().contiguous() for h in range(hk)]) / math.sqrt(d)
            z = torch.logsumexp(a, dim=2, keepdim=True)
            p = torch.exp(a - z)
            out.append(torch.stack([p[h] @ vals[:seen, h].contiguous() for h in range(hk)]).view(hk * rep, d))
            lse.append(z.view(hk * rep))
    return {"out": torch.stack(out), "lse": torch.stack(lse)}
