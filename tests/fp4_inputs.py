"""Seeded decode problems over the 4-bit latent cache (torch CPU tensors)."""
import numpy as np
import torch

from oracle import latent_fp4 as ora
from serving_inputs import WIDTH, Decode, page_table


class DecodeFp4(Decode):
    """A decode problem: new tokens n[b] over prior[b] cached ones in `raw` [pages, P, 304].
    Slots past a context and the spare page are rows of NaN.  `blocks`: block sizes differ by
    up to 2^blocks either way.  codes and scales say the same cache in e4m3, for the oracle."""

    def __init__(self, n, prior, heads, P, seed, spread=0.5, q_std=1.0, sink=0.0, blocks=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.n, self.prior, self.heads, self.P = n, prior, heads, P
        L = [a + b for a, b in zip(n, prior)]
        self.table, pages = page_table(L, P, gen)
        self.ro = np.concatenate([[0], np.cumsum(n)]).astype(np.int64)
        self.raw = torch.zeros((pages, P, 304), dtype=torch.uint8)
        self.raw[:, :, 288] = 255
        for b in range(len(n)):
            x = torch.randn(L[b], WIDTH, generator=gen)
            x *= torch.exp2(torch.empty(L[b], 1).uniform_(-spread, spread, generator=gen))
            x *= torch.exp2(torch.empty(L[b], 18).uniform_(-blocks, blocks, generator=gen)).repeat_interleave(32, 1)
            if sink and L[b]:
                x[0] += sink
            self.put(b, x)
        self.q = (torch.randn(int(self.ro[-1]), heads, WIDTH, generator=gen) * q_std).to(torch.bfloat16)
        self.scale = 192 ** -0.5

    def put(self, b, x):
        """Rows x as sequence b's context."""
        pos = torch.arange(len(x))
        raw = torch.from_numpy(fast_encode(x.to(torch.bfloat16).float().numpy()))
        self.raw[self.table[b, pos // self.P].long(), pos % self.P] = raw

    @property
    def codes(self):
        return torch.from_numpy(ora.to_e4m3(self.raw.numpy(), WIDTH)[0])

    @property
    def scales(self):
        return torch.from_numpy(ora.to_e4m3(self.raw.numpy(), WIDTH)[1])


def fast_encode(x):
    """oracle.latent_fp4.encode of finite rows, vectorised (a test compares the two)."""
    n, W = x.shape
    if n == 0:
        return np.zeros((0, ora.row_bytes(W)), dtype=np.uint8)
    x = x.astype(np.float64)
    m, e = np.frexp(np.maximum(np.abs(x).reshape(n, -1, 32).max(axis=2), 2.0 ** -150))
    e = e - np.where(m <= 0.875, 3, 2)
    top = np.clip(e.max(axis=1), -100, 125)
    shift = np.clip(top[:, None] - e, 0, 14)
    y = np.abs(x) * np.repeat(np.ldexp(1.0, shift - top[:, None]), 32, axis=1)
    code = np.searchsorted([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], y, side="left")
    for tie, even in ((0.75, 2), (1.75, 4), (3.5, 6)):
        code[y == tie] = even
    code = (code + 8 * np.signbit(x)).astype(np.uint8)
    out = np.zeros((n, ora.row_bytes(W)), dtype=np.uint8)
    out[:, :W // 2] = code[:, 0::2] | code[:, 1::2] << 4
    out[:, W // 2] = top + 127
    out[:, W // 2 + 1:W // 2 + 1 + W // 64] = (shift[:, 0::2] | shift[:, 1::2] << 4).astype(np.uint8)
    return out
