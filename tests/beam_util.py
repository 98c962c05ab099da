"""Plain 64-bit forms of the beam-decoding calls (numpy), and tensor helpers of
their tests."""
import numpy as np
import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def select_ref(logits, scores, beams, n, T=1.0, finished=None, pad_token=0):
    """logits [G*W, V] (any float dtype, widened exactly), scores [G*W] fp32.
    Returns scores (fp64), tokens, parents [G, n]."""
    x = logits.astype(np.float64)
    T = float(np.float32(T))
    rows, V = x.shape
    G = rows // beams
    cum = scores.reshape(-1).astype(np.float64)
    s = np.full((rows, V), -np.inf)
    for r in range(rows):
        if not np.isfinite(cum[r]):
            continue
        if finished is not None and finished.reshape(-1)[r]:
            s[r, pad_token] = cum[r]
            continue
        m = x[r].max()
        if not np.isfinite(m):  # NaN, +inf, or nothing finite
            continue
        S = np.exp((x[r] - m) / T).sum()
        s[r] = (cum[r] - np.log(S)) + (x[r] - m) / T
    out_s = np.full((G, n), -np.inf)
    out_t = np.full((G, n), -1, np.int32)
    out_p = np.full((G, n), -1, np.int32)
    for g in range(G):
        flat = s[g * beams:(g + 1) * beams].reshape(-1)
        order = np.argsort(-flat, kind="stable")[:n]
        order = order[flat[order] > -np.inf]
        k = len(order)
        out_s[g, :k] = flat[order]
        out_t[g, :k] = order % V
        out_p[g, :k] = order // V
    return out_s, out_t, out_p


def widen(t):
    """A tensor's values as float64 on the host (exact for the 16-bit types)."""
    return t.detach().cpu().double().numpy()


def reorder_ref(states, parents, beams, lengths=None):
    """The reorder of a host tensor [slabs, batch, heads, positions, row], out of place."""
    out = states.clone()
    _, batch, _, positions, _ = states.shape
    for b in range(batch):
        g, q = b // beams, int(parents[b])
        if q < 0 or q >= beams:
            continue
        src = g * beams + q
        n = positions if lengths is None else max(0, min(positions, int(lengths[src])))
        out[:, b, :, :n] = states[:, src, :, :n]
    return out


def attention_ref(q, pk, pv, sk, sv, plen, slen, drafts, groups, scale, eps, tiny):
    """Attention in 64 bits, sequence by sequence.  q [rows, Hq, D]; pk, pv [G,
    P, Hk, D]; sk, sv [B, S, Hk, D] (float64 arrays); drafts [B]; groups: the
    group of each sequence.  eps: finfo(dtype).eps of the element type; tiny:
    half its smallest step (0 where it does not matter).

    Returns out, lse and how far a kernel with fp32 scores, weights rounded to
    the element type and fp32 sums may be off each:
      a score's products are exact in fp32 and added in fp32, D of them:
        d_s = (D + 4) 2^-24 scale sum |q k|, and 4 roundings of |a| on the way to
        the exponent, so a weight is off by d = 2 d_s + 8 |a| 2^-24 + 2^-22 relative
        (numerator and denominator);
      rounding a weight: eps / 2 relative, or `tiny` of the largest weight's scale;
      sums of n weights in fp32: n 2^-24 relative at most; out rounded once: eps / 2."""
    rows, Hq, D = q.shape
    Hk = sk.shape[2]
    rep = Hq // Hk
    out, lse = np.zeros((rows, Hq, D)), np.full((rows, Hq), -np.inf)
    b_out, b_lse = np.zeros((rows, Hq, D)), np.zeros((rows, Hq))
    t = 0
    for b, K in enumerate(drafts):
        g = groups[b]
        lp = max(0, min(pk.shape[1], int(plen[g])))
        ls = max(0, min(sk.shape[1], int(slen[b])))
        for k in range(K + 1):
            n2 = max(0, ls - K + k)
            for h in range(Hq):
                kk = np.concatenate([pk[g, :lp, h // rep], sk[b, :n2, h // rep]])
                vv = np.concatenate([pv[g, :lp, h // rep], sv[b, :n2, h // rep]])
                n = len(kk)
                if n == 0:
                    continue
                a = scale * (kk @ q[t, h])
                d_s = (D + 4) * 2.0 ** -24 * scale * (np.abs(kk) @ np.abs(q[t, h])).max()
                m = a.max()
                w = np.exp(a - m)
                z = w.sum()
                w /= z
                out[t, h], lse[t, h] = w @ vv, m + np.log(z)
                d = 2 * d_s + 8 * np.abs(a).max() * 2.0 ** -24 + 2.0 ** -22
                wv = w @ np.abs(vv)
                b_out[t, h] = (eps / 2 * np.abs(out[t, h]) + (eps / 2 + d + 2 * n * 2.0 ** -24) * wv
                               + n * tiny * np.abs(vv).max() + tiny) * 1.01
                b_lse[t, h] = d + n * 2.0 ** -24 + 4 * 2.0 ** -24 * (1 + np.abs(lse[t, h]))
            t += 1
    return out, lse, b_out, b_lse
