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
