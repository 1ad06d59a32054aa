"""Seeded inputs of the serving-step operator tests (torch CPU tensors)."""
import numpy as np
import torch

E4M3 = torch.float8_e4m3fn
WIDTH, LATENT = 576, 512


def quantise_rows(x, group=None):
    """(uint8 codes, float32 scales) of fp32 rows: one scale per row, or per
    `group` columns."""
    if group is None:
        s = x.abs().amax(dim=1, keepdim=True).clamp_min(1e-30) / 448
        return (x / s).to(E4M3).view(torch.uint8), s[:, 0]
    rows, k = x.shape
    g = -(-k // group)
    y = torch.nn.functional.pad(x, (0, g * group - k)).view(rows, g, group)
    s = y.abs().amax(dim=2, keepdim=True).clamp_min(1e-30) / 448
    return (y / s).to(E4M3).view(torch.uint8).view(rows, -1)[:, :k].contiguous(), s.view(rows, g)


def blocks(n, k, gen, spread=2.0):
    """(codes [n, k], scales [ceil(n/128), ceil(k/128)]) with block scales that
    differ by factors, so a scale on the wrong block shows."""
    codes = (torch.randn(n, k, generator=gen) * 60).clamp(-448, 448).to(E4M3).view(torch.uint8)
    scales = torch.exp2(torch.empty(-(-n // 128), -(-k // 128)).uniform_(-spread, spread, generator=gen)) / 64
    return codes, scales


def page_table(lengths, P, gen, spare=1):
    """Shuffled pages: (uint32-valued int32 table [B, cols], pages in the pool)."""
    cols = [-(-n // P) for n in lengths]
    order = torch.randperm(sum(cols) + spare, generator=gen)
    table = torch.full((len(lengths), max(max(cols), 1)), 0, dtype=torch.int32)
    at = 0
    for b, c in enumerate(cols):
        table[b, :c] = order[at:at + c].to(torch.int32)
        at += c
    return table, sum(cols) + spare


class Decode:
    """A decode problem: new tokens n[b] over prior[b] cached ones.  Slots past a
    context, the spare page and its scales hold NaN."""

    def __init__(self, n, prior, heads, P, seed, spread=0.5, q_std=1.0, sink=0.0):
        gen = torch.Generator().manual_seed(seed)
        self.n, self.prior, self.heads, self.P = n, prior, heads, P
        L = [a + b for a, b in zip(n, prior)]
        self.table, pages = page_table(L, P, gen)
        self.ro = np.concatenate([[0], np.cumsum(n)]).astype(np.int64)
        self.codes = torch.full((pages, P, WIDTH), 0x7F, dtype=torch.uint8)
        self.scales = torch.full((pages, P), float("nan"))
        for b in range(len(n)):
            x = torch.randn(L[b], WIDTH, generator=gen) * torch.exp2(
                torch.empty(L[b], 1).uniform_(-spread, spread, generator=gen))
            if sink and L[b]:
                x[0] += sink
            c, s = quantise_rows(x)
            pos = torch.arange(L[b])
            pg = self.table[b, pos // P].long()
            self.codes[pg, pos % P] = c
            self.scales[pg, pos % P] = s
        self.q = (torch.randn(int(self.ro[-1]), heads, WIDTH, generator=gen) * q_std).to(torch.bfloat16)
        self.scale = 192 ** -0.5

    def offsets(self):
        return (torch.from_numpy(self.ro.astype(np.int32)),
                torch.tensor(self.prior, dtype=torch.int32))
