"""The 4-bit latent cache's row format, and norm and position rotation of heads,
in float64, one plain restatement each (test infrastructure only).

A row of W elements: W / 2 bytes of e2m1 codes (element 2 i in the low half of byte
i), the exponent E (255: NaNs), W / 64 bytes of shifts of its blocks of 32 (block 2 i
in the low half), zeros up to a multiple of 16 bytes; an element is
e2m1(code) * 2^(E - 127 - shift)."""
import numpy as np

from .numerics import E4M3_VALUES

BLOCK = 32
# e2m1: sign, two exponent bits with bias 1, one mantissa bit; exponent 0 is subnormal.
MAGNITUDES = np.array([(m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)) for e in range(4) for m in range(2)])


def row_bytes(width):
    return -(-(width // 2 + width // 64 + 1) // 16) * 16


def encode(rows):
    """uint8 [n, row_bytes(W)] of real rows [n, W] (exactly float32 values)."""
    n, W = rows.shape
    out = np.zeros((n, row_bytes(W)), dtype=np.uint8)
    for r in range(n):
        x = rows[r].astype(np.float64)
        if not np.isfinite(x).all():
            out[r, W // 2] = 255
            continue
        e = []
        for blk in x.reshape(-1, BLOCK):
            a, k = float(np.abs(blk).max()), -200
            if a:
                k = int(np.floor(np.log2(a))) - 5
                while a > 7 * 2.0 ** k:
                    k += 1
            e.append(k)
        top = min(max(max(e), -100), 125)
        shift = np.clip(top - np.array(e), 0, 14)
        y = np.abs(x) / np.repeat(2.0 ** (top - shift.astype(np.float64)), BLOCK)
        far = np.abs(y[:, None] - MAGNITUDES)
        near = far == far.min(axis=1, keepdims=True)
        # Of two equally near codes the even one (argmax takes the first of the preferred).
        code = np.argmax(near * (2 - np.arange(8) % 2), axis=1) + 8 * np.signbit(x)
        out[r, :W // 2] = code[0::2] | code[1::2] << 4
        out[r, W // 2] = top + 127
        out[r, W // 2 + 1:W // 2 + 1 + W // 64] = shift[0::2] | shift[1::2] << 4
    return out


def _parts(raw, width):
    codes = np.empty(raw.shape[:-1] + (width,), dtype=np.uint8)
    codes[..., 0::2], codes[..., 1::2] = raw[..., :width // 2] & 15, raw[..., :width // 2] >> 4
    s = raw[..., width // 2 + 1:width // 2 + 1 + width // 64]
    shift = np.empty(raw.shape[:-1] + (width // BLOCK,), dtype=np.int64)
    shift[..., 0::2], shift[..., 1::2] = s & 15, s >> 4
    unsigned = MAGNITUDES[codes & 7]
    return np.where(codes & 8, -unsigned, unsigned), raw[..., width // 2].astype(np.int64), np.repeat(shift, BLOCK, axis=-1)


def decode(raw, width):
    """float64 [..., W] of cached rows."""
    v, e, shift = _parts(raw, width)
    out = v * 2.0 ** (e[..., None] - 127 - shift).astype(np.float64)
    return np.where(e[..., None] == 255, np.nan, out)


def to_e4m3(raw, width):
    """(uint8 e4m3 codes [..., W], float32 scales [...]): the same values as codes of
    e2m1 * 2^(6 - shift) and one scale 2^(E - 133) a row; raises if one is not exact."""
    v, e, shift = _parts(raw, width)
    units = v * 2.0 ** (6 - shift).astype(np.float64)
    positive = E4M3_VALUES[:127]
    code = np.searchsorted(positive, np.abs(units))
    if not np.array_equal(positive[code], np.abs(units)):
        raise ValueError("not exact in e4m3")
    code = (code | np.where(np.signbit(units), 128, 0)).astype(np.uint8)
    scale = np.where(e == 255, np.nan, 2.0 ** (e - 133).astype(np.float64)).astype(np.float32)
    return np.where((e == 255)[..., None], 0x7F, code).astype(np.uint8), scale


def norm_rope(x, weight, eps, positions, inv_freq, scale, halves):
    """(out, magnitude of what was turned) of rows x [T, H, D]."""
    y = x.astype(np.float64).copy()
    if weight is not None:
        n = len(weight)
        y[..., :n] = y[..., :n] / np.sqrt((y[..., :n] ** 2).mean(axis=-1, keepdims=True) + eps) * weight
    mag = np.abs(y)
    if inv_freq is not None:
        angle = np.asarray(positions, dtype=np.longdouble)[:, None] * np.asarray(inv_freq, dtype=np.longdouble)
        angle = angle - 2 * PI * np.floor(angle / (2 * PI))
        c, s = (np.asarray(f(angle.astype(np.float64)))[:, None, :] * scale for f in (np.cos, np.sin))
        first, half = x.shape[-1] - 2 * len(inv_freq), len(inv_freq)
        a = slice(first, first + half) if halves else slice(first, None, 2)
        b = slice(first + half, None) if halves else slice(first + 1, None, 2)
        u, v = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = u * c - v * s, u * s + v * c
        mag[..., a] = mag[..., b] = (np.abs(u) + np.abs(v)) * abs(scale)
    return y, mag


# pi to long double's precision, as two float64 terms.
PI = np.longdouble(3.141592653589793) + np.longdouble(1.2246467991473532e-16)
