"""The serving-step operators (norm, block-scaled product, latent append,
latent decode attention) in float64, one plain restatement each (test
infrastructure only).  Inputs are numpy arrays of real values; e4m3 codes are
decoded from the format's definition."""
import numpy as np

from .numerics import decode_e4m3

GROUP = 128
LATENT = 512
FP8_MAX = 448.0
FP8_TINY = float(np.float32(1e-30))


def rms_norm(x, weight, eps, residual=None):
    """(h, y, scales): h = x + residual, y the weighted norm, one scale per 128
    columns of a row of y."""
    h = x.astype(np.float64) + (0.0 if residual is None else residual)
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * weight
    groups = -(-y.shape[1] // GROUP)
    scales = np.stack([np.abs(y[:, g * GROUP:(g + 1) * GROUP]).max(axis=1) for g in range(groups)], axis=1)
    return h, y, np.maximum(scales, FP8_TINY) / FP8_MAX


def spread(scales, k):
    """[rows, ceil(k / 128)] scales, one per column of k."""
    return np.repeat(scales.astype(np.float64), GROUP, axis=1)[:, :k]


def matmul_fp8(x_codes, x_scales, w_codes, w_scales):
    """(out, sum of the terms' magnitudes), [M, N] each."""
    k, n = x_codes.shape[1], w_codes.shape[0]
    x = decode_e4m3(x_codes) * spread(x_scales, k)
    w = decode_e4m3(w_codes) * np.repeat(spread(w_scales, k), GROUP, axis=0)[:n]
    return x @ w.T, np.abs(x) @ np.abs(w).T


def slot(page_table, b, a, page_size):
    return int(page_table[b, a // page_size]) * page_size + a % page_size


def append(rows, page_table, row_offsets, cache_lens, page_size):
    """{slot: (real row / scale in float32, scale)} of every appended token."""
    out = {}
    for b in range(len(cache_lens)):
        for i in range(int(row_offsets[b + 1]) - int(row_offsets[b])):
            row = rows[int(row_offsets[b]) + i].astype(np.float32)
            scale = np.float32(max(np.abs(row).max(), np.float32(1e-30))) / np.float32(448)
            out[slot(page_table, b, int(cache_lens[b]) + i, page_size)] = (row / scale, scale)
    return out


def decode(q, codes, scales, page_table, row_offsets, cache_lens, scale, causal=True, lost=()):
    """Attention of q [Tq, H, 576] over cache codes [pages, P, 576] with scales
    [pages, P].  Returns out, lse, the weighted magnitudes sum_j p_j |c_j| and
    the largest scaled score's term sum (NaN rows: not covered by the offsets).
    `lost`: (sequence, page-table column) pairs whose keys count as masked."""
    Tq, H, W = q.shape
    P = codes.shape[1]
    out = np.full((Tq, H, LATENT), np.nan)
    mag, lse = out.copy(), np.full((Tq, H), np.nan)
    terms = np.zeros((Tq, H))
    flat, sc = codes.reshape(-1, W), scales.reshape(-1).astype(np.float64)
    for b in range(len(cache_lens)):
        q0, q1, prior = int(row_offsets[b]), int(row_offsets[b + 1]), int(cache_lens[b])
        L = prior + q1 - q0
        if q1 == q0:
            continue
        keys = [j for j in range(L) if (b, j // P) not in lost]
        slots = np.array([slot(page_table, b, j, P) for j in keys], dtype=np.int64)
        c = decode_e4m3(flat[slots]) * sc[slots][:, None]
        for t in range(q0, q1):
            n = sum(1 for j in keys if j <= prior + t - q0) if causal else len(keys)
            if n == 0:
                out[t], mag[t], lse[t] = 0.0, 0.0, -np.inf
                continue
            x = scale * (q[t].astype(np.float64) @ c[:n].T)
            top = x.max(axis=1, keepdims=True)
            e = np.exp(x - top)
            p = e / e.sum(axis=1, keepdims=True)
            out[t] = p @ c[:n, :LATENT]
            mag[t] = p @ np.abs(c[:n, :LATENT])
            lse[t] = top[:, 0] + np.log(e.sum(axis=1))
            terms[t] = scale * (np.abs(q[t]).astype(np.float64) @ np.abs(c[:n]).T).max(axis=1)
    return out, lse, mag, terms
