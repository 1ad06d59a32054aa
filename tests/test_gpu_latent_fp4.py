"""The 4-bit latent cache's operators (mla_norm_rope, mla_append_latent_fp4,
mla_gather_latent_fp4, mla_decode_latent_fp4) on the GPU against
oracle/latent_fp4.py and oracle/serving.py in float64.

Tolerances, all derived before the first run (half a step: bf16 2^-8, relative):
* norm and rotation: a row's sum of squares is a chain of at most 32 products and 5 additions
  of partial sums, 2^-18 relative with the few products after it; an angle is off by at most
  2^-24 of a turn and its sine and cosine by two steps (2^-22 together is 2 pi 2^-24 rounded
  up), so a turned pair (u, v) by 2^-17 (|u| + |v|) with all of it; then the output's rounding.
* append, gather: powers of two and one conversion whose ties are defined, so equal.
* attention: as for the 8-bit cache, whose e4m3 form of the same rows is the oracle's input:
  the softmax weights may carry a rounding to 8 significant bits (2^-8 of each weight), on
  both sides of the normalisation 2^-7 of sum_j p_j |c_j|; the scores 600 fp32 additions
  (2^-23 of their terms' magnitudes), which move each weight by that much, and the smallest
  query elements an absolute 2^-17 of the row's largest; then the output's rounding.  A key's
  weight times its row's unit, p_j s_j, that is below 2^-10 of the row's largest W is documented
  to be within 2^-18 W: it enters column d with |code_jd| = |c_jd| / s_j, so column d may be off by
  2^-18 W sum_j |code_jd| over those keys.  (That is below 2^-7 sum_j p_j |c_jd| wherever the keys of large
  weight hold a nonzero code of the column: the least is 0.5 * 2^(6 - shift).  A 4-bit row has many zeros, so it
  is the whole error where all of them hold a zero.)
"""
import numpy as np
import pytest
import torch

from fp4_inputs import DecodeFp4, fast_encode
from oracle import latent_fp4 as ora
from oracle import serving as ora8
from serving_inputs import E4M3, LATENT, WIDTH, blocks, page_table

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _within(got, ref, tol, what):
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} out of tolerance, worst "
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300)):.3g} x, first at {np.argwhere(bad)[0]}")


# ------------------------------------------------------------------ norm and rotation

def _positions(n, gen, far):
    p = torch.randint(0, far, (n,), generator=gen)
    return p


def _rope_inputs(T, H, D, norm, pairs, seed, far=200000, w_dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g).to(torch.bfloat16)
    w = (1 + 0.2 * torch.randn(norm, generator=g)).to(w_dtype) if norm else None
    f = (10000.0 ** -(torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))).float() if pairs else None
    pos = torch.randint(0, far, (T,), generator=g)
    return x, w, f, pos


def _check_rope(got, x, w, f, pos, eps=1e-6, scale=1.0, halves=False, what="out"):
    ref, mag = ora.norm_rope(_f64(x), None if w is None else _f64(w), eps, np.asarray(pos),
                             None if f is None else f.cpu().numpy(), scale, halves)
    _within(_f64(got), ref, 2.0 ** -8 * np.abs(ref) + 2.0 ** -17 * mag + 2.0 ** -133, what)


def _dev(t):
    return None if t is None else t.cuda()


def _u32(pos):
    return torch.from_numpy(np.asarray(pos).astype(np.uint32).view(np.int32)).cuda()


@pytest.mark.parametrize("T,H,D,norm,pairs", [
    (1, 1, 2, 0, 1), (1, 1, 1, 1, 0), (3, 2, 7, 7, 3), (1, 128, 64, 0, 32), (5, 1, 576, 512, 32), (70, 3, 128, 128, 64),
    (33, 128, 64, 0, 32), (257, 1, 576, 512, 32), (19, 5, 80, 80, 20), (4, 7, 50, 50, 12), (9, 2, 192, 0, 32),
    (2, 3, 1024, 1024, 512), (6, 4, 1024, 1000, 8), (40, 2, 48, 0, 24), (11, 1, 1023, 1000, 500), (300, 12, 96, 96, 0),
    (3, 200, 256, 256, 16), (130, 1, 64, 64, 32), (64, 9, 8, 8, 4), (1000, 2, 136, 136, 68), (5, 3, 576, 40, 32),
    (40, 1, 1024, 1024, 512), (350, 300, 64, 64, 32)])
@pytest.mark.parametrize("halves", [False, True])
def test_norm_rope(lib, T, H, D, norm, pairs, halves):
    from mla_ragged_paged_gb300 import binding
    x, w, f, pos = _rope_inputs(T, H, D, norm, pairs, T + H + D)
    out = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    binding.norm_rope(_u32(pos) if pairs else None, _dev(f), q=x.cuda(), q_out=out, q_weight=_dev(w),
                      interleaved=not halves)
    _check_rope(out, x, w, f, pos, halves=halves)
    again = torch.empty_like(out)
    binding.norm_rope(_u32(pos) if pairs else None, _dev(f), k=x.cuda(), k_out=again, k_weight=_dev(w),
                      interleaved=not halves)
    assert torch.equal(out, again)


@pytest.mark.parametrize("T,Hq,Dq,Hk,Dk", [(1, 128, 64, 1, 576), (300, 128, 64, 1, 576), (77, 12, 128, 3, 128),
                                           (5003, 1, 64, 1, 64), (10, 3, 70, 2, 66), (50, 257, 64, 2, 70), (30, 1, 70, 1, 576)])
@pytest.mark.parametrize("halves", [False, True])
def test_norm_rope_queries_and_keys(lib, T, Hq, Dq, Hk, Dk, halves):
    from mla_ragged_paged_gb300 import binding
    whole = Dq == Dk
    q, qw, f, pos = _rope_inputs(T, Hq, Dq, Dq if whole else 0, 32, 1)
    k, kw, _, _ = _rope_inputs(T, Hk, Dk, Dk if whole else min(Dk, LATENT), 32, 2, w_dtype=torch.float32)
    qo, ko = (torch.empty_like(t, device="cuda") for t in (q, k))
    binding.norm_rope(_u32(pos), f.cuda(), q=q.cuda(), q_out=qo, q_weight=_dev(qw), k=k.cuda(), k_out=ko,
                      k_weight=kw.cuda(), eps=1e-5, rope_scale=1.25, interleaved=not halves)
    _check_rope(qo, q, qw, f, pos, 1e-5, 1.25, halves, "q")
    _check_rope(ko, k, kw, f, pos, 1e-5, 1.25, halves, "k")


@pytest.mark.parametrize("freqs", [[1.0, 0.1], [1e-4, 3.7e-9], [2.5, 100.0], [6.5, 1e6], [-0.75, -1e-3], [0.0, 1e-38],
                                   [1e-42, 3e38]])
def test_norm_rope_far_positions(lib, freqs):
    """Every 32-bit position, and frequencies of any size: what is left of whole turns stays exact."""
    from mla_ragged_paged_gb300 import binding
    pos = np.array([0, 1, 2, 3, 1000, 65535, 10 ** 6, 2 ** 24 + 1, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1], dtype=np.int64)
    f = np.array(freqs, dtype=np.float32)
    x = torch.ones(len(pos), 1, 4, dtype=torch.bfloat16)
    x[:, :, 1::2] = 0
    out = torch.empty(len(pos), 1, 4, dtype=torch.bfloat16, device="cuda")
    binding.norm_rope(_u32(pos), torch.from_numpy(f).cuda(), q=x.cuda(), q_out=out)
    # Exactly, in whole numbers: f is m 2^e, a turn 2 pi to 1200 bits.
    from fractions import Fraction
    two_pi = _two_pi()
    ref = np.empty((len(pos), 1, 4))
    for i, p in enumerate(pos):
        for j, v in enumerate(f):
            turns = Fraction(int(p)) * Fraction(float(v)) / two_pi
            a = 2 * np.pi * float(turns - turns.__floor__())
            ref[i, 0, 2 * j], ref[i, 0, 2 * j + 1] = np.cos(a), np.sin(a)
    # (2^-24 of a turn relative to inv_freq's own value: the fixed point keeps 2^-64 of a turn times the
    # position, 2^-32 at most, and 64 bits of 1 / (2 pi), 2^-64 of the angle.)
    angle = np.abs(pos[:, None] * f.astype(np.float64)) * 2.0 ** -63
    tol = np.repeat(2.0 ** -21 + angle, 2, axis=1)[:, None, :] + 2.0 ** -8 * np.abs(ref)
    _within(_f64(out), ref, np.minimum(tol, 3.0), "out")


def _two_pi():
    from fractions import Fraction
    # Machin: pi = 16 atan(1/5) - 4 atan(1/239)
    def atan_inv(n, bits=1200):
        one, total, k = 1 << bits, 0, 0
        term = one // n
        while term:
            total += (term // (2 * k + 1)) * (-1 if k & 1 else 1)
            term //= n * n
            k += 1
        return Fraction(total, one)
    return 2 * (16 * atan_inv(5) - 4 * atan_inv(239))


@pytest.mark.parametrize("offset,pad,halves", [(0, 0, False), (1, 3, False), (8, 8, True), (0, 64, True), (3, 0, True)])
def test_norm_rope_strides(lib, offset, pad, halves):
    """Views of wider rows on both sides, heads before tokens, an input shared by all heads."""
    from mla_ragged_paged_gb300 import binding
    T, H, D = 37, 6, 64
    x, w, f, pos = _rope_inputs(T, H, D, D, 16, 5)
    wide = torch.full((T, H, D + pad + offset + 8), 3.0, dtype=torch.bfloat16)
    wide[:, :, offset:offset + D] = x
    wide = wide.cuda()
    buf = torch.full((H, T, D + pad + offset + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :, offset:offset + D].transpose(0, 1)
    binding.norm_rope(_u32(pos), f.cuda(), q=wide[:, :, offset:offset + D], q_out=out, q_weight=w.cuda(),
                      interleaved=not halves)
    _check_rope(out, x, w, f, pos, halves=halves)
    out.fill_(7.0)
    assert (buf == 7).all()
    one = x[:, :1].cuda().expand(T, H, D)
    binding.norm_rope(_u32(pos), f.cuda(), q=one, q_out=out, q_weight=w.cuda(), interleaved=not halves)
    _check_rope(out, x[:, :1].expand(T, H, D), w, f, pos, halves=halves)


@pytest.mark.parametrize("D,norm,pairs", [(576, 512, 32), (128, 128, 64), (70, 70, 11)])
@pytest.mark.parametrize("halves", [False, True])
def test_norm_rope_in_place(lib, D, norm, pairs, halves):
    from mla_ragged_paged_gb300 import binding
    x, w, f, pos = _rope_inputs(50, 3, D, norm, pairs, 6)
    y = x.cuda()
    binding.norm_rope(_u32(pos), f.cuda(), q=y, q_out=y, q_weight=w.cuda(), interleaved=not halves)
    _check_rope(y, x, w, f, pos, halves=halves)


def test_norm_rope_zero_nan_and_large_rows(lib):
    from mla_ragged_paged_gb300 import binding
    x, w, f, pos = _rope_inputs(6, 2, 576, 512, 32, 8)
    x[1] = 0
    x[2, 0, 5] = float("nan")
    x[3, 1, 520] = float("inf")
    x[4, 0] *= 1e30
    out = torch.empty_like(x, device="cuda")
    binding.norm_rope(_u32(pos), f.cuda(), k=x.cuda(), k_out=out, k_weight=w.cuda())
    assert (out[1] == 0).all()
    assert torch.isnan(out[2, 0, :512]).all() and (out[4, 0, :512] == 0).all()
    pair = (520 - 512) // 2 * 2 + 512
    assert not torch.isfinite(out[3, 1, pair:pair + 2]).any()
    rest = torch.ones(6, 2, 576, dtype=torch.bool)
    rest[2, 0, :512] = rest[4, 0, :512] = False
    rest[3, 1, pair:pair + 2] = False
    ref, mag = ora.norm_rope(np.nan_to_num(_f64(x), posinf=0), _f64(w), 1e-6, pos.numpy(), f.numpy(), 1.0, False)
    ok = rest.numpy()
    _within(_f64(out)[ok], ref[ok], (2.0 ** -8 * np.abs(ref) + 2.0 ** -17 * mag)[ok], "the others")
    bad = torch.tensor([float("nan"), float("inf")] + [1.0] * 30, device="cuda")
    binding.norm_rope(_u32(pos), bad, k=x.cuda(), k_out=out, k_weight=w.cuda())
    assert torch.isnan(out[0, :, 512:516]).all() and torch.isfinite(out[0, :, 516:]).all()


def test_norm_rope_no_tokens_and_other_stream(lib):
    from mla_ragged_paged_gb300 import binding
    none = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    f = torch.ones(8, device="cuda")
    binding.norm_rope(torch.empty(0, dtype=torch.int32, device="cuda"), f, q=none, q_out=none)
    x, w, f, pos = _rope_inputs(400, 16, 128, 128, 64, 12)
    dev, p, f_d, w_d = x.cuda(), _u32(pos), f.cuda(), w.cuda()
    a, b = torch.empty_like(dev), torch.empty_like(dev)
    binding.norm_rope(p, f_d, q=dev, q_out=a, q_weight=w_d)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    binding.norm_rope(p, f_d, q=dev, q_out=b, q_weight=w_d, stream=side)
    side.synchronize()
    assert torch.equal(a, b)
    with pytest.raises(binding.MlaError):
        binding.norm_rope(p[:-1], f_d, q=dev, q_out=a)


@pytest.mark.parametrize("heads", [2 ** 31 - 1, 2 ** 31 - 15])
def test_norm_rope_most_heads(lib, heads):
    """As many heads as a call takes: the angles' place is counted in 64 bits."""
    from mla_ragged_paged_gb300 import binding
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough memory")
    part = 1 << 20
    base, w, f, pos = _rope_inputs(1, part, 2, 2, 1, 13)
    buf = torch.empty(2048, part * 2, dtype=torch.bfloat16, device="cuda")
    buf[:] = base.cuda().view(1, -1)
    q = buf.view(-1)[:2 * heads].view(1, heads, 2)
    binding.norm_rope(_u32(pos), f.cuda(), q=q, q_out=q, q_weight=w.cuda())
    _check_rope(q[:, :part], base, w, f, pos)
    left = 2 ** 31 - heads
    assert (buf[:-1] == buf[0]).all()
    assert torch.equal(buf[-1, :-2 * left], buf[0, :-2 * left]) and torch.equal(buf[-1, -2 * left:].cpu(), base.view(-1)[-2 * left:])


_THREADS = """
import threading, torch
from mla_ragged_paged_gb300 import binding
# 64 KB of angles (1024 columns in items) and 128 KB (1024 columns two bytes past 16), halves and pairs.
T = 64
x = torch.randn(T, 1, 1024, device="cuda").to(torch.bfloat16)
odd = torch.empty(T, 1, 1032, dtype=torch.bfloat16, device="cuda")[:, :, 1:1025]
odd.copy_(x)
f = torch.rand(512, device="cuda")
pos = torch.arange(T, dtype=torch.int32, device="cuda")
outs, errors = [torch.zeros(T, 1, 1024, dtype=torch.bfloat16, device="cuda") for _ in range(16)], []
torch.cuda.synchronize()
start = threading.Barrier(16)
def work(i):
    try:
        start.wait()
        for _ in range(50):
            binding.norm_rope(pos, f, q=odd if i & 1 else x, q_out=outs[i], interleaved=i & 2 == 0)
    except Exception as e:
        errors.append(e)
threads = [threading.Thread(target=work, args=(i,)) for i in range(16)]
[t.start() for t in threads], [t.join() for t in threads]
torch.cuda.synchronize()
assert not errors, errors
assert all(torch.equal(outs[i], outs[i & 2]) for i in range(16))
"""


def test_norm_rope_sizes_from_several_threads(lib):
    """Calls of different shared-memory sizes, the first ones of their process, in 16 threads at once: all are
    launched."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", _THREADS], cwd=root, capture_output=True, text=True, timeout=200)
        assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------------ append and gather

def _bf16_rows(n, W, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, W, generator=g)
    x *= torch.exp2(torch.empty(n, W // 32).uniform_(-spread, spread, generator=g)).repeat_interleave(32, 1)
    return x.to(torch.bfloat16)


def _slot(table, b, a, P):
    return int(table[b, a // P]), a % P


@pytest.mark.parametrize("W", [64, 256, 320, 576, 768, 832, 1024])
@pytest.mark.parametrize("P,new,prior", [(16, [1, 1, 1], [0, 15, 31]), (12, [40, 0, 7], [5, 9, 0]), (1, [3], [2]),
                                         (64, [130, 1], [60, 700])])
def test_append_and_gather(lib, W, P, new, prior):
    from mla_ragged_paged_gb300 import binding
    g = torch.Generator().manual_seed(W + P)
    L = [a + b for a, b in zip(new, prior)]
    table, pages = page_table(L, P, g)
    rows = _bf16_rows(sum(new), W, W + P + 1)
    before = torch.randint(0, 256, (pages, P, ora.row_bytes(W)), generator=g).to(torch.uint8)
    cache = before.cuda()
    ro = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    cl = torch.tensor(prior, dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.append_latent_fp4(cache, rows.cuda(), table.cuda(), ro, cl, status)
    assert int(status) == 0
    want, raw = before.clone(), torch.from_numpy(ora.encode(rows.float().numpy()))
    t = 0
    for b in range(len(new)):
        for i in range(new[b]):
            want[_slot(table, b, prior[b] + i, P)] = raw[t]
            t += 1
    assert torch.equal(cache.cpu(), want)
    # The new rows, and a window that begins inside each sequence's context, in both forms.
    back = torch.full((sum(new) + 3, W), 7.0, dtype=torch.bfloat16, device="cuda")
    binding.gather_latent_fp4(back, cache, table.cuda(), ro, cl, status=status)
    assert np.array_equal(_f64(back[:-3]), ora.decode(raw.numpy(), W)) and (back[-3:] == 7).all()
    codes = torch.full((sum(new) + 3, W + 16), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((sum(new) + 3,), 5.0, device="cuda")
    binding.gather_latent_fp4(codes[:, :W].view(E4M3), cache, table.cuda(), ro, cl, dst_scales=scales, status=status)
    c, s = ora.to_e4m3(raw.numpy(), W)
    assert np.array_equal(codes[:-3, :W].cpu().numpy(), c) and np.array_equal(scales[:-3].cpu().numpy(), s)
    assert (codes[-3:] == 9).all() and (codes[:, W:] == 9).all() and (scales[-3:] == 5).all()
    assert int(status) == 0


def test_append_every_tie_and_exponent(lib):
    """Every bf16 mantissa against every block maximum's, so that each value next to a tie occurs; rows of
    every exponent."""
    from mla_ragged_paged_gb300 import binding
    W = 1024
    x = torch.empty(128 * 8, W)
    small = (1 + torch.arange(128) / 128.0)                                # every mantissa
    for m in range(128):
        for s in range(8):
            row = torch.zeros(W // 32, 32)
            vals = (small * 2.0 ** -s).repeat(W // 128 + 1)[:(W // 32) * 31].view(W // 32, 31)
            row[:, 0], row[:, 1:] = small[m] * 4, vals * torch.where(torch.arange(31) % 2 == 0, 1.0, -1.0)
            x[m * 8 + s] = row.view(-1)
    exps = torch.exp2(torch.arange(-133, 128).double()).float()[:, None] * x[torch.arange(261) * 3]
    exps[exps.abs() > 3.38e38] = 3.38e38
    x = torch.cat([x, exps]).to(torch.bfloat16)
    cache = torch.zeros(1, len(x), ora.row_bytes(W), dtype=torch.uint8, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    ro = torch.tensor([0, len(x)], dtype=torch.int32, device="cuda")
    binding.append_latent_fp4(cache, x.cuda(), zero[None], ro, zero)
    assert np.array_equal(cache[0].cpu().numpy(), fast_encode(x.float().numpy()))
    back = torch.empty(len(x), W, dtype=torch.bfloat16, device="cuda")
    binding.gather_latent_fp4(back, cache, zero[None], ro, zero)
    assert np.array_equal(_f64(back), ora.decode(cache[0].cpu().numpy(), W))


def test_gather_reads_any_row(lib):
    """Rows of random bytes with every exponent and shift (15, which is never written, reads as zeros)."""
    from mla_ragged_paged_gb300 import binding
    g = torch.Generator().manual_seed(4)
    raw = torch.randint(0, 256, (1, 600, 304), generator=g).to(torch.uint8)
    raw[0, :256, 288] = torch.arange(256).to(torch.uint8)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    ro = torch.tensor([0, 600], dtype=torch.int32, device="cuda")
    back = torch.empty(600, WIDTH, dtype=torch.bfloat16, device="cuda")
    binding.gather_latent_fp4(back, raw.cuda(), zero[None], ro, zero)
    v, e, shift = ora._parts(raw[0].numpy(), WIDTH)
    want = np.where(shift == 15, 0.0, ora.decode(raw[0].numpy(), WIDTH))
    want[e == 255] = np.nan
    with np.errstate(over="ignore"):
        want = torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16)
    assert torch.equal(torch.nan_to_num(back.cpu().float(), nan=1.5), torch.nan_to_num(want.float(), nan=1.5))


def test_append_and_gather_bad_pages_and_nan(lib):
    from mla_ragged_paged_gb300 import binding
    table = torch.tensor([[1, 99], [0, 2]], dtype=torch.int32, device="cuda")
    cache = torch.full((3, 4, 304), 5, dtype=torch.uint8, device="cuda")
    rows = torch.ones(13, WIDTH, dtype=torch.bfloat16, device="cuda")
    rows[0, 7], rows[1, 570] = float("nan"), float("-inf")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ro = torch.tensor([0, 6, 13], dtype=torch.int32, device="cuda")
    lens = torch.tensor([2, 3], dtype=torch.int32, device="cuda")
    # Sequence 0: tokens 2, 3 on page 1, tokens 4..7 on page 99; sequence 1: tokens
    # 3..9, of which 8 and 9 lie past its two page-table columns.
    binding.append_latent_fp4(cache, rows, table, ro, lens, status)
    assert int(status) == 0x3
    one = torch.from_numpy(ora.encode(np.ones((1, WIDTH), dtype=np.float32))).cuda()[0]
    for r in (cache[1, 2], cache[1, 3]):
        assert int(r[288]) == 255 and int(r.sum()) == 255
    assert (cache[1, :2] == 5).all() and (cache[0, :3] == 5).all()
    assert torch.equal(cache[0, 3], one) and all(torch.equal(cache[2, i], one) for i in range(4))
    for dt in ("bf16", "e4m3"):
        status.zero_()
        back = torch.full((13, WIDTH), 3.0, dtype=torch.bfloat16, device="cuda")
        codes, scales = torch.full((13, WIDTH), 9, dtype=torch.uint8, device="cuda"), torch.full((13,), 5.0, device="cuda")
        if dt == "bf16":
            binding.gather_latent_fp4(back, cache, table, ro, lens, status=status)
        else:
            binding.gather_latent_fp4(codes, cache, table, ro, lens, dst_scales=scales, status=status)
            assert (codes[2:6] == 9).all() and (scales[2:6] == 5).all() and (codes[11:] == 9).all()
            assert torch.isnan(scales[:2]).all() and (codes[:2] & 0x7F == 0x7F).all()
            back[:2] = float("nan")
            keep = [6, 7, 8, 9, 10]
            back[keep] = (codes[keep].view(E4M3).float() * scales[keep][:, None]).to(torch.bfloat16)
        assert int(status) == 0x3
        assert torch.isnan(back[:2]).all() and (back[2:6] == 3).all() and (back[11:] == 3).all()
        assert (back[6:11] == 1).all()
    lens.fill_(-1)                                   # a length no context can have
    before = cache.clone()
    binding.append_latent_fp4(cache, rows, table, ro, lens, status)
    assert torch.equal(cache, before)


def test_append_and_gather_padded_cache_and_rows_outside(lib):
    """Slots outside pages in memory, padded slots, padded rows; rows before the first and behind the last
    sequence are neither read nor written."""
    from mla_ragged_paged_gb300 import binding
    P, pages = 8, 5
    store = torch.full((P, pages, 336), 5, dtype=torch.uint8, device="cuda")
    cache = store[:, :, :304].transpose(0, 1)
    wide = torch.full((20, WIDTH + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = _bf16_rows(15, WIDTH, 3)
    wide[3:18, :WIDTH] = x.cuda()
    table = torch.tensor([[4, 0, 9, 9], [2, 3, 1, 9]], dtype=torch.int32, device="cuda")
    ro = torch.tensor([3, 9, 18], dtype=torch.int32, device="cuda")
    lens = torch.tensor([5, 11], dtype=torch.int32, device="cuda")
    binding.append_latent_fp4(cache, wide[:, :WIDTH], table, ro, lens)
    raw = torch.from_numpy(ora.encode(x.float().numpy()))
    want = torch.full((pages, P, 304), 5, dtype=torch.uint8)
    for t in range(15):
        b, i = (0, t) if t < 6 else (1, t - 6)
        want[_slot(table, b, int(lens[b]) + i, P)] = raw[t]
    assert torch.equal(cache.cpu(), want) and (store[:, :, 304:] == 5).all()
    back = torch.full((20, WIDTH + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    binding.gather_latent_fp4(back[:, :WIDTH], cache, table, ro, lens)
    assert np.array_equal(_f64(back[3:18, :WIDTH]), ora.decode(raw.numpy(), WIDTH))
    back[3:18, :WIDTH] = 3
    assert (back == 3).all()
    none = torch.empty(0, WIDTH, dtype=torch.bfloat16, device="cuda")
    binding.append_latent_fp4(cache, none, table, ro, lens)
    binding.gather_latent_fp4(none, cache, table, ro, lens)


# ------------------------------------------------------------------ attention

def _run_decode(d, mask="causal", lse=True, workspace=None, out=None, q=None, cache=None, status=None):
    from mla_ragged_paged_gb300 import binding
    ro, cl = (t.cuda() for t in d.offsets())
    q = d.q.cuda() if q is None else q
    cache = d.raw.cuda() if cache is None else cache
    if out is None:
        out = torch.full((q.shape[0], d.heads, LATENT), float("nan"), dtype=torch.bfloat16, device="cuda")
    L = torch.full((q.shape[0], d.heads), float("nan"), device="cuda") if lse else None
    binding.decode_latent_fp4(out, q, cache, d.table.cuda(), ro, cl, d.scale,
                              binding.MLA_MASK_CAUSAL if mask == "causal" else binding.MLA_MASK_NULL,
                              workspace=workspace, lse=L, status=status)
    return out, L


def _small_weights(d, mask, lost):
    """2^-18 W sum of |code| over the keys whose p_j s_j is below 2^-10 W, of every query and column."""
    raw = d.raw.view(-1, 304).numpy()
    add = np.zeros((d.q.shape[0], d.heads, LATENT))
    for b in range(len(d.prior)):
        q0, n = int(d.ro[b]), int(d.ro[b + 1] - d.ro[b])
        keys = [j for j in range(d.prior[b] + n) if (b, j // d.P) not in lost]
        slots = np.array([int(d.table[b, j // d.P]) * d.P + j % d.P for j in keys], dtype=np.int64)
        c = np.nan_to_num(ora.decode(raw[slots], WIDTH))
        unit = 2.0 ** (raw[slots, WIDTH // 2].astype(np.float64) - 133)
        for i in range(n):
            m = sum(1 for j in keys if j <= d.prior[b] + i) if mask == "causal" else len(keys)
            if not m:
                continue
            x = d.scale * (_f64(d.q[q0 + i]) @ c[:m].T)
            p = np.exp(x - x.max(axis=1, keepdims=True))
            w = p / p.sum(axis=1, keepdims=True) * unit[:m]
            top = w.max(axis=1, keepdims=True)
            add[q0 + i] = 2.0 ** -18 * top * ((w < 2.0 ** -10 * top) @ (np.abs(c[:m, :LATENT]) / unit[:m, None]))
    return add


def _check_decode(d, out, lse, mask="causal", lost=()):
    ref, z, mag, terms = ora8.decode(d.q.float().numpy(), d.codes.numpy(), d.scales.numpy(), d.table.numpy(), d.ro, d.prior,
                                     d.scale, mask == "causal", lost)
    move = 600 * 2.0 ** -23 * terms + 2.0 ** -17 * terms
    tol = (2.0 ** -7 + 4 * move)[:, :, None] * mag + 2.0 ** -8 * np.abs(ref) + _small_weights(d, mask, lost) + 1e-30
    _within(_f64(out), ref, tol, "out")
    if lse is not None:
        got = _f64(lse)
        empty = np.isneginf(z)
        assert np.array_equal(np.isneginf(got), empty)
        z, got = np.where(empty, 0, z), np.where(empty, 0, got)
        _within(got, z, 2 * move + 2.0 ** -20 * (1 + np.abs(z)) + 2.0 ** -9, "lse")


@pytest.mark.parametrize("n,prior,heads,P", [
    ([1], [0], 1, 16), ([1], [0], 16, 64), ([1], [1], 128, 64), ([1], [126], 16, 64), ([1], [127], 4, 64),
    ([1], [128], 16, 128), ([1, 1, 1], [5, 300, 64], 16, 16), ([1] * 9, [3, 1000, 0, 129, 63, 64, 65, 255, 700], 128, 64),
    ([2, 0, 4, 1], [100, 7, 0, 380], 16, 12), ([3], [50], 24, 24), ([5, 1], [1, 2000], 40, 128), ([1, 0], [40, 0], 8, 1),
    ([2], [3000], 128, 256), ([70], [0], 3, 16), ([130, 3], [60, 200], 1, 32), ([1] * 200, list(range(200)), 4, 8),
    ([1], [20000], 16, 64), ([1, 1], [9000, 4], 65, 64), ([2], [777], 200, 20)])
@pytest.mark.parametrize("mask", ["causal", "null"])
def test_decode(lib, n, prior, heads, P, mask):
    d = DecodeFp4(n, prior, heads, P, seed=sum(n) + sum(prior) + heads)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _run_decode(d, mask, status=status)
    assert int(status) == 0
    _check_decode(d, out, lse, mask)


@pytest.mark.parametrize("n,prior,heads", [
    ([1] * 170, [0, 200, 20, 127, 128] * 34, 128), ([1] * 151, [0] * 151, 16), ([1, 0, 1] * 100, [130, 9, 300] * 100, 8),
    ([1] * 31, [0] * 31, 64), ([1] * 30 + [2], [0] * 30 + [4000], 64), ([1] * 77, list(range(100, 870, 10)), 65)])
def test_decode_shares_that_end_anywhere(lib, n, prior, heads):
    """Row tiles of one to a few key tiles, so that the SMs' shares end before, behind and inside them."""
    d = DecodeFp4(n, prior, heads, 16, seed=sum(prior) + heads)
    out, lse = _run_decode(d)
    _check_decode(d, out, lse)


@pytest.mark.parametrize("q_std,spread,sink,blocks", [
    (0.0, 0.5, 0.0, 1.0), (4.0, 0.5, 0.0, 1.0), (12.0, 3.0, 0.0, 1.0), (1.0, 6.0, 0.0, 0.0), (1.5, 0.5, 3.0, 0.0),
    (1e-20, 0.5, 0.0, 1.0), (60.0, 0.1, 0.0, 0.0), (1.0, 0.5, 0.0, 7.0), (0.5, 2.0, 0.0, 12.0)])
def test_decode_value_ranges(lib, q_std, spread, sink, blocks):
    """Flat, wide and peaked softmaxes; rows and blocks of very different sizes (every shift); one early
    key far above the rest (its tail must keep its precision)."""
    d = DecodeFp4([1, 2], [1500, 300], 20, 64, seed=31, spread=spread, q_std=q_std, sink=sink, blocks=blocks)
    if sink:
        d.q += torch.tensor(0.25, dtype=torch.bfloat16)
    if blocks > 6:
        assert len(np.unique(d.raw[d.raw[..., 288] != 255][:, 289:298].numpy() & 15)) == 15
    out, lse = _run_decode(d)
    _check_decode(d, out, lse)


@pytest.mark.parametrize("spread", [12.0, 20.0, 40.0])
@pytest.mark.parametrize("n,prior", [([1, 2], [1500, 300]), ([1], [9000]), ([1] * 170, [100] * 170)])
def test_decode_scales_far_apart(lib, n, prior, spread):
    """Keys of similar softmax weight whose scales differ by up to 2^80: those with small scales add
    little to the numerator and all of their weight to the denominator, in row tiles that one CTA takes
    whole and in joined ones."""
    d = DecodeFp4(n, prior, 20, 64, seed=41, spread=spread, q_std=2.0 ** -spread)
    out, lse = _run_decode(d)
    _check_decode(d, out, lse)


@pytest.mark.parametrize("q_std", [0.0, 1.0])
@pytest.mark.parametrize("lengths,zeros", [
    ([2], "late"), ([2], "early"), ([300], "early"), ([300], "late"), ([300], "odd"), ([5000], "odd"), ([5000], "early"),
    ([5000], "all but one"), ([200] * 160, "odd"), ([200] * 160, "early"), ([70], "all")])
def test_decode_rows_of_zeros(lib, lengths, zeros, q_std):
    """Rows of zeros, as the append caches them, among ordinary ones: in an opening key tile that holds
    nothing else, in later ones, in every one."""
    from mla_ragged_paged_gb300 import binding
    d = DecodeFp4([1] * len(lengths), [n - 1 for n in lengths], 16, 16, seed=42, q_std=q_std)
    g = torch.Generator().manual_seed(43)
    rows = []
    for n in lengths:
        x = torch.randn(n, WIDTH, generator=g)
        zero = {"early": slice(0, (n + 1) // 2), "late": slice(n // 2, n), "odd": slice(1, n, 2), "all": slice(0, n),
                "all but one": slice(1, n)}[zeros]
        x[zero] = 0
        rows.append(x)
    cache = d.raw.cuda()
    ro = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
    binding.append_latent_fp4(cache, torch.cat(rows).to(torch.bfloat16).cuda(), d.table.cuda(), ro,
                              torch.zeros(len(lengths), dtype=torch.int32, device="cuda"))
    d.raw = cache.cpu()
    out, lse = _run_decode(d)
    _check_decode(d, out, lse)


def test_decode_tail_behind_a_sink(lib):
    """One key takes e^12 times the weight of each of 40 000 others, which together outweigh it in the
    first 512 columns: weights rounded to steps of the largest would lose them."""
    d = DecodeFp4([1], [40000], 16, 64, seed=8, spread=0.0, blocks=0.0)
    x = torch.zeros(40001, WIDTH)
    x[:, :LATENT] = 1.0                      # every key: ones, but for the sink's zeros
    x[0, :LATENT] = 0.0
    x[:, LATENT:] = 0.01 * torch.randn(40001, 64, generator=torch.Generator().manual_seed(3))
    x[0, LATENT:] = 1.0
    d.put(0, x)
    d.q.zero_()
    d.q[:, :, LATENT:] = 12.0 / (64 * d.scale)
    out, lse = _run_decode(d)
    _check_decode(d, out, lse)


@pytest.mark.parametrize("P", [16, 12])
def test_decode_strides_and_rows_outside(lib, P):
    """Padded queries, outputs and cache rows; rows before the first and
    behind the last sequence stay as they were."""
    d = DecodeFp4([2, 1], [100, 300], 6, P, seed=14)
    tq = int(d.ro[-1])
    big = torch.full((tq + 5, 8, 600), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[2:2 + tq, 1:7, :576] = d.q.cuda()
    q = big[:, 1:7, :576]
    buf = torch.full((tq + 5, 7, 520), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :6, :512]
    pages = d.raw.shape[0]
    cache = torch.full((pages, P, 336), 0xFF, dtype=torch.uint8, device="cuda")[:, :, :304]
    cache.copy_(d.raw.cuda())
    ref_ro = d.ro.copy()
    d.ro = d.ro + 2
    _, lse = _run_decode(d, out=out, q=q, cache=cache)
    d.ro = ref_ro
    _check_decode(d, out[2:2 + tq], lse[2:2 + tq])
    assert torch.isnan(lse[:2]).all() and torch.isnan(lse[2 + tq:]).all()
    out[2:2 + tq] = 3
    assert (buf == 3).all()


def test_decode_bad_pages(lib):
    """Keys on bad pages or past the page table count as masked; a query left without keys gets 0 and -inf."""
    d = DecodeFp4([1, 1, 1], [500, 20, 40], 16, 16, seed=15)
    good = d.table.clone()
    d.table[0, 3] = 10 ** 6
    d.table[1, :] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _run_decode(d, status=status)
    assert int(status) == 0x1
    d.table = good
    _check_decode(d, out, lse, lost={(0, 3), (1, 0), (1, 1)})
    d.table = good[:, :2].contiguous()
    status.zero_()
    out, lse = _run_decode(d, status=status)
    assert int(status) == 0x2
    _check_decode(d, out, lse, lost={(0, c) for c in range(2, 32)} | {(2, 2)})


def test_decode_nan_stays_in_its_rows(lib):
    """A NaN query gives NaN in its own rows only; a NaN row of one sequence leaves the others and the
    tokens before it alone."""
    d = DecodeFp4([2, 1, 1], [130, 40, 200], 16, 16, seed=16)
    d.q[2, 5, 17] = float("nan")
    at = d.table[0, 131 // 16].long(), 131 % 16                  # visible to token 1 of sequence 0 only
    kept = d.raw[at].clone()
    d.raw[at] = torch.from_numpy(ora.encode(np.full((1, WIDTH), np.nan, dtype=np.float32)))[0]
    out, lse = _run_decode(d)
    out, lse = out.cpu(), lse.cpu()
    assert torch.isnan(lse[1]).all() and torch.isnan(out[1]).any(dim=1).all()
    assert torch.isnan(out[2, 5]).all() and torch.isnan(lse[2, 5])
    d.q[2, 5, 17] = 1.0
    d.raw[at] = kept
    ref, z, mag, _ = ora8.decode(d.q.float().numpy(), d.codes.numpy(), d.scales.numpy(), d.table.numpy(), d.ro,
                                 d.prior, d.scale)
    for t in (0, 2, 3):
        heads = [h for h in range(16) if (t, h) != (2, 5)]
        tol = 2.0 ** -6 * mag[t, heads] + 2.0 ** -8 * np.abs(ref[t, heads])
        _within(_f64(out[t, heads]), ref[t, heads], tol, f"token {t}")


def test_decode_repeats_and_shares_a_workspace(lib):
    """Bit-identical repeats, with other problems in between on one workspace whose contents start as
    garbage, an 8-bit cache's call among them; also on a stream of its own."""
    from mla_ragged_paged_gb300 import binding
    ws = torch.full((binding.decode_workspace_size(),), 0xA5, dtype=torch.uint8, device="cuda")
    a, b = DecodeFp4([1, 1], [5000, 70], 64, 64, seed=1), DecodeFp4([1] * 30, [200] * 30, 16, 64, seed=2)
    first, lse = _run_decode(a, workspace=ws)
    _check_decode(a, first, lse)
    ro, cl = (t.cuda() for t in a.offsets())
    eight = torch.empty_like(first)
    codes, scales = a.codes.cuda(), a.scales.cuda()
    side = torch.cuda.Stream()
    for i in range(10):
        out_b, lse_b = _run_decode(b, workspace=ws)
        again, _ = _run_decode(a, workspace=ws, lse=False)
        assert torch.equal(again, first)
        binding.decode_latent(eight, a.q.cuda(), codes, scales, a.table.cuda(), ro, cl, a.scale, workspace=ws)
    _check_decode(b, out_b, lse_b)
    _check_decode(a, eight, None)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again, _ = _run_decode(a)
    side.synchronize()
    assert torch.equal(again, first)


def test_decode_graph_follows_lengths(lib):
    """A captured call reads lengths, offsets and pages when it runs: replays after the sequences have
    grown, and with one of them gone."""
    from mla_ragged_paged_gb300 import binding
    d = DecodeFp4([1, 1, 1], [700, 90, 2000], 16, 16, seed=61)
    ro, cl = (t.cuda() for t in d.offsets())
    q, cache, table = d.q.cuda(), d.raw.cuda(), d.table.cuda()
    out = torch.empty(3, 16, LATENT, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, 16, device="cuda")
    ws = binding.alloc_decode_workspace()
    call = lambda: binding.decode_latent_fp4(out, q, cache, table, ro, cl, d.scale, workspace=ws, lse=lse)
    call()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        call()
    for prior, offsets in [([3, 90, 1200], [0, 1, 2, 3]), ([700, 0, 2000], [0, 1, 2, 3]), ([700, 90, 15], [0, 1, 1, 3])]:
        cl.copy_(torch.tensor(prior, dtype=torch.int32))
        ro.copy_(torch.tensor(offsets, dtype=torch.int32))
        d.prior, d.ro = prior, np.array(offsets)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        _check_decode(d, out, lse)


def test_decode_on_two_streams(lib):
    """Two calls that overlap, each with its own workspace."""
    a, b = DecodeFp4([1], [9000], 64, 64, seed=62), DecodeFp4([1] * 6, [1500] * 6, 16, 64, seed=63)
    ref_a, ref_b = _run_decode(a)[0], _run_decode(b)[0]
    _check_decode(a, ref_a, None)
    _check_decode(b, ref_b, None)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(6):
        for d, st in ((a, streams[0]), (b, streams[1])):
            with torch.cuda.stream(st):
                outs.append((d, _run_decode(d, lse=False)[0]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref_a if d is a else ref_b) for d, o in outs)


def test_decode_impossible_lengths_and_offsets(lib):
    """A length past the page table masks the keys there; offsets that decrease or leave the queries skip
    their sequence; the others are right."""
    d = DecodeFp4([1, 1, 1, 1], [40, 100, 60, 30], 8, 16, seed=64)
    d.prior = [40, -1, 60, 30]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _run_decode(d, status=status)
    assert int(status) & 0x2
    d.prior[1] = 100
    keep = [0, 2, 3]
    ref, _, mag, _ = ora8.decode(d.q.float().numpy(), d.codes.numpy(), d.scales.numpy(), d.table.numpy(), d.ro, d.prior,
                                 d.scale)
    tol = 2.0 ** -6 * mag + 2.0 ** -8 * np.abs(ref)
    _within(_f64(out)[keep], ref[keep], tol[keep], "out")
    for bad in ([0, 3, 2, 3, 4], [0, 1, 2, 3, 9]):
        d.ro = np.array(bad)
        status.zero_()
        out, _ = _run_decode(d, status=status)
        assert int(status) & 0x4
        if bad[1] == 1:                         # sequence 0 has its offsets still
            _within(_f64(out)[0], ref[0], tol[0], "out")


def test_decode_many_heads(lib):
    d = DecodeFp4([1, 2], [70, 300], 1024, 64, seed=65)
    out, lse = _run_decode(d)
    _check_decode(d, out, lse)


def test_offsets_past_32_bits(lib):
    """Cache rows whose byte offsets pass 2^32, in decode, append and gather."""
    from mla_ragged_paged_gb300 import binding
    P, pages = 4096, 3600
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough memory")
    d = DecodeFp4([1, 1], [6000, 300], 16, P, seed=21)
    cache = torch.full((pages, P, 304), 0xFF, dtype=torch.uint8, device="cuda")
    move = torch.tensor([pages - 1, 3, pages - 2, 900])
    cache[move[:d.raw.shape[0]].cuda()] = d.raw.cuda()
    small, d.table = d.table, move[d.table.long()].to(torch.int32)
    ro, cl = (t.cuda() for t in d.offsets())
    out = torch.empty(2, 16, LATENT, dtype=torch.bfloat16, device="cuda")
    binding.decode_latent_fp4(out, d.q.cuda(), cache, d.table.cuda(), ro, cl, d.scale)
    rows = _bf16_rows(2, WIDTH, 1)
    binding.append_latent_fp4(cache, rows.cuda(), d.table.cuda(), ro, cl)
    raw = torch.from_numpy(ora.encode(rows.float().numpy()))
    for b in range(2):
        assert torch.equal(cache[_slot(d.table, b, d.prior[b], P)].cpu(), raw[b])
    back = torch.empty(2, WIDTH, dtype=torch.bfloat16, device="cuda")
    binding.gather_latent_fp4(back, cache, d.table.cuda(), ro, cl)
    assert np.array_equal(_f64(back), ora.decode(raw.numpy(), WIDTH))
    d.table = small
    _check_decode(d, out, None)


# ------------------------------------------------------------------ together

def _step_inputs(seed, B=5, heads=16, prior=(40, 0, 129, 300, 7), P=16):
    g = torch.Generator().manual_seed(seed)
    d = DecodeFp4([1] * B, list(prior), heads, P, seed=seed)
    s = dict(d=d, heads=heads, B=B)
    s["kv"] = torch.randn(B, 1, WIDTH, generator=g).to(torch.bfloat16)
    s["q"] = torch.randn(B, heads, 192, generator=g).to(torch.bfloat16)
    s["absorbed"] = torch.randn(B, heads, LATENT, generator=g).to(torch.bfloat16)
    s["w"] = (1 + 0.1 * torch.randn(LATENT, generator=g)).to(torch.bfloat16)
    s["f"] = (10000.0 ** -(torch.arange(32, dtype=torch.float64) / 32)).float()
    return s


def test_serving_step(lib):
    """Rotation and norm of a step's queries and latent rows, append and attention, directly and captured
    into a graph that is replayed on new inputs.  The rope dims of the queries go where the absorbed ones
    have them, the positions are the lengths.  Each stage is checked on its own inputs."""
    from mla_ragged_paged_gb300 import binding
    s = _step_inputs(40)
    d, B, H = s["d"], s["B"], s["heads"]
    dev = {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}
    cache, table = d.raw.cuda(), d.table.cuda()
    ro, cl = (t.cuda() for t in d.offsets())
    q = torch.empty(B, H, WIDTH, dtype=torch.bfloat16, device="cuda")
    rows = torch.empty(B, 1, WIDTH, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(B, H, LATENT, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, H, device="cuda")
    ws = binding.alloc_decode_workspace()

    def step():
        q[:, :, :LATENT].copy_(dev["absorbed"])
        binding.norm_rope(cl, dev["f"], q=dev["q"][:, :, 128:], q_out=q[:, :, LATENT:], k=dev["kv"], k_out=rows,
                          k_weight=dev["w"])
        binding.append_latent_fp4(cache, rows[:, 0], table, ro, cl)
        binding.decode_latent_fp4(out, q, cache, table, ro, cl, d.scale, workspace=ws, lse=lse)

    def check():
        torch.cuda.synchronize()
        pos = np.array(d.prior)
        _check_rope(q[:, :, LATENT:], dev["q"][:, :, 128:], None, s["f"], pos)
        _check_rope(rows, dev["kv"], s["w"], s["f"], pos)
        raw = torch.from_numpy(ora.encode(rows[:, 0].float().cpu().numpy()))
        for b in range(B):
            assert torch.equal(cache[_slot(d.table, b, d.prior[b], d.P)].cpu(), raw[b])
        d.raw, d.q = cache.cpu(), q.cpu()
        _check_decode(d, out, lse)

    step()
    check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in (41, 42):
        new = _step_inputs(seed)
        for k in ("kv", "q", "absorbed"):
            dev[k].copy_(new[k])
        out.fill_(float("nan"))
        graph.replay()
        check()


def test_prefill_over_the_4_bit_latent_cache(lib):
    """A prompt's chunk over rows kept in 4 bits: read back in e4m3 with a scale a row, up-projected by the
    8-bit product, prefilled with the contiguous K_rope of the same rows in bf16.  Each stage is
    checked on its own inputs."""
    from mla_ragged_paged_gb300 import binding
    B, H, P = 2, 4, 16
    n, prior = [40, 25], [30, 100]
    d = DecodeFp4(n, prior, H, P, seed=50)
    L = [a + b for a, b in zip(n, prior)]
    S = sum(L)
    g = torch.Generator().manual_seed(51)
    wk, wv = ([t.cuda() for t in blocks(H * 128, LATENT, g, spread=0.5)] for _ in range(2))
    ro, cl = (t.cuda() for t in d.offsets())
    bro, co, _, _ = binding.plan(ro, cl, S, 1)
    cache, table = d.raw.cuda(), d.table.cuda()
    rows = torch.empty(S, WIDTH, dtype=E4M3, device="cuda")
    scales = torch.empty(S, device="cuda")
    values = torch.empty(S, WIDTH, dtype=torch.bfloat16, device="cuda")
    binding.gather_latent_fp4(rows, cache, table, bro[0], co[0], dst_scales=scales)
    binding.gather_latent_fp4(values, cache, table, bro[0], co[0])
    slots = torch.cat([d.table[b, torch.arange(L[b]) // P].long() * P + torch.arange(L[b]) % P for b in range(B)])
    want = ora.decode(d.raw.view(-1, 304)[slots].numpy(), WIDTH)
    assert np.array_equal(_f64(values), want)
    assert torch.equal(rows.float() * scales[:, None], values.float())
    wide = scales[:, None].expand(S, LATENT // 128)
    k_nope = torch.empty(S, H, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k_nope)
    for out, w in ((k_nope, wk), (v, wv)):
        binding.matmul_fp8(out.view(S, -1), rows[:, :LATENT], wide, *w)
        ref, mag = ora8.matmul_fp8(rows[:, :LATENT].view(torch.uint8).cpu().numpy(), wide.cpu().numpy(),
                                   w[0].cpu().numpy(), w[1].cpu().numpy())
        _within(_f64(out.view(S, -1)), ref, 2.0 ** -8 * np.abs(ref) + 600 * 2.0 ** -23 * mag, "projection")
    q = (torch.randn(sum(n), H, 192, generator=g) * 0.3).to(torch.bfloat16)
    out = torch.empty(sum(n), H, 128, dtype=torch.bfloat16, device="cuda")
    rope = values[:, LATENT:].contiguous()
    binding.prefill_ragged_contiguous(out, q.cuda(), k_nope, v, rope, ro, cl, d.scale)
    for b in range(B):
        rows_b = slice(sum(L[:b]), sum(L[:b + 1]))
        k = torch.cat([k_nope[rows_b].cpu(), rope[rows_b, None, :].cpu().expand(-1, H, -1)], 2).double()
        qb = q[d.ro[b]:d.ro[b + 1]].double().transpose(0, 1)
        allowed = torch.arange(L[b])[None] <= prior[b] + torch.arange(n[b])[:, None]
        k, vb = k.transpose(0, 1), v[rows_b].cpu().double().transpose(0, 1)
        p = torch.softmax((qb @ k.transpose(1, 2) * d.scale).masked_fill(~allowed, float("-inf")), dim=2)
        # The prefill rounds each weight to bf16 (2^-8 of it, on both sides of the normalisation 2^-7 of
        # sum p |v|), adds 192 products per score in fp32 (2^-23 of the terms each, which moves a
        # weight by that much) and rounds the output.
        move = 4 * 192 * 2.0 ** -23 * d.scale * (qb.abs() @ k.abs().transpose(1, 2)).amax(dim=2, keepdim=True)
        ref = p @ vb
        tol = (2.0 ** -7 + move) * (p @ vb.abs()) + 2.0 ** -8 * ref.abs()
        got = out[d.ro[b]:d.ro[b + 1]].cpu().double().transpose(0, 1)
        _within(got.numpy(), ref.numpy(), tol.numpy(), f"sequence {b}")


@pytest.mark.parametrize("heads,P", [(64, 16), (16, 12)])
def test_decode_wait_timeout_sets_status_and_context_survives(lib, heads, P):
    """Codes that never come: the call ends, says so, and the next one is right (64- and 32-row tiles, several
    tiles a CTA, so that the warps that make the codes are stopped in mid-ring)."""
    from mla_ragged_paged_gb300 import binding
    d = DecodeFp4([1] * 60, [3000] * 60, heads, P, seed=66)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.test_inject_stall(True)
    try:
        _run_decode(d, status=status)
        assert int(status) == 0x8
    finally:
        binding.test_inject_stall(False)
    status.zero_()
    d2 = DecodeFp4([1, 1], [700, 40], heads, P, seed=67)
    out, lse = _run_decode(d2, status=status)
    assert int(status) == 0
    _check_decode(d2, out, lse)


# ------------------------------------------------------------------ the ends of the exponents

def _set_exponents(d, lo, hi, seed):
    """Every cached row an exponent E of its own in lo .. hi."""
    g = torch.Generator().manual_seed(seed)
    e = d.raw[..., WIDTH // 2]
    kept = e != 255
    e[kept] = torch.randint(lo, hi + 1, (int(kept.sum()),), generator=g).to(torch.uint8)


@pytest.mark.parametrize("lo,hi,q_std", [(223, 232, 2.0 ** -106), (200, 232, 2.0 ** -106), (122, 232, 2.0 ** -106),
                                         (245, 252, 0.0), (142, 252, 0.0), (27, 36, 1.0), (27, 137, 0.0)])
@pytest.mark.parametrize("n,prior,heads", [([1, 2], [1500, 300], 20), ([1], [9000], 16), ([1] * 170, [100] * 170, 40)])
def test_decode_rows_of_every_exponent(lib, n, prior, heads, lo, hi, q_std):
    """Rows near 2^125 and near 2^-100, within 110 of each other: the sums of the weights stay in range, in
    row tiles that one CTA takes whole and in joined ones."""
    d = DecodeFp4(n, prior, heads, 64, seed=hi, q_std=q_std)
    _set_exponents(d, lo, hi, lo)
    out, lse = _run_decode(d)
    if hi < 64:
        # The absolute part of the tolerance, made for rows near one, is above these: checked as the same
        # rows times 2^60 (exactly: a power of two).
        d.raw[..., WIDTH // 2][d.raw[..., WIDTH // 2] != 255] += 60
        out, d.q = out.float() * 2.0 ** 60, (d.q.float() * 2.0 ** -60).to(torch.bfloat16)
    _check_decode(d, out, lse)


@pytest.mark.parametrize("lo,hi,q_std", [(150, 154, 2.0 ** -20), (178, 182, 2.0 ** -48), (230, 232, 2.0 ** -98)])
@pytest.mark.parametrize("n,prior", [([1, 2], [1500, 300]), ([1], [9000])])
def test_decode_rows_of_zeros_beside_large_ones(lib, n, prior, lo, hi, q_std):
    """Rows of zeros (E = 27) more than 110 below the others, which have all the weight: no weight of theirs becomes an
    infinity or a NaN."""
    d = DecodeFp4(n, prior, 16, 64, seed=lo, q_std=q_std)
    _set_exponents(d, lo, hi, hi)
    pick = torch.rand(d.raw.shape[:2], generator=torch.Generator().manual_seed(lo)) < 0.5
    zero = torch.from_numpy(ora.encode(np.zeros((1, WIDTH))))[0]
    d.raw[pick & (d.raw[..., WIDTH // 2] != 255)] = zero
    out, lse = _run_decode(d)
    _check_decode(d, out, lse)


@pytest.mark.parametrize("nats", [40.0, 80.0, 95.0, 105.0, 140.0, 1000.0])
@pytest.mark.parametrize("zeros,others", [(100, 500), (3, 300)])
def test_decode_rows_of_zeros_far_above_the_others(lib, zeros, others, nats):
    """Rows of zeros first, then rows whose scores are far below theirs, 200 sequences of the same pages, so that CTAs
    take whole ones: the sum of the weights stays in fp32 when the others' maxima are followed downwards."""
    n = zeros + others
    d = DecodeFp4([1], [n - 1], 4, 64, seed=zeros)
    x = -torch.ones(n, WIDTH)
    x[:zeros] = 0
    d.put(0, x)
    d.n, d.prior, d.ro = [1] * 200, [n - 1] * 200, np.arange(201)
    d.table, d.q = d.table.repeat(200, 1), torch.full((200, 4, WIDTH), nats / (WIDTH * d.scale)).to(torch.bfloat16)
    out, lse = _run_decode(d)
    _check_decode(d, out, lse)


def test_decode_exponents_that_rise_and_fall(lib):
    """The largest rows first, last and in the middle of a sequence, for one token alone and beside
    keys that no row sees."""
    d = DecodeFp4([1, 1, 1, 3], [3000, 3000, 3000, 257], 16, 16, seed=5, q_std=2.0 ** -106)
    for b in range(4):
        L = d.prior[b] + d.n[b]
        pos = torch.arange(L)
        e = {0: 232 - pos * 100 // L, 1: 132 + pos * 100 // L, 2: 232 - (pos - L // 2).abs() * 100 // L,
             3: torch.where(pos >= L - 2, 252, 150)}[b]
        d.raw[d.table[b, pos // d.P].long(), pos % d.P, WIDTH // 2] = e.to(torch.uint8)
    d.q[3:] = 0
    out, lse = _run_decode(d)
    _check_decode(d, out, lse)


# ------------------------------------------------------------------ layouts and sizes that take other paths

@pytest.mark.parametrize("n,prior,heads,P,pad", [
    *[([1] * 60, [1100] * 60, heads, P, pad) for heads, P, pad in ((16, 1, 0), (16, 7, 48), (32, 3, 16), (32, 5, 0), (40, 1, 32),
                                                                   (40, 6, 0))],
    *[([1, 3, 0, 2], [127, 128, 9, 1], 8, P, 16) for P in (2, 3, 9)]])
def test_decode_row_gathers(lib, n, prior, heads, P, pad):
    """Pages of no multiple of four tokens, which are read row by row: 16-, 32- and 64-row tiles, about four tiles
    a CTA, so that the rings wrap; padded rows."""
    d = DecodeFp4(n, prior, heads, P, seed=P)
    cache = torch.full((d.raw.shape[0], P, 304 + pad), 0xFF, dtype=torch.uint8, device="cuda")[:, :, :304]
    cache.copy_(d.raw.cuda())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _run_decode(d, cache=cache, status=status)
    assert int(status) == 0
    _check_decode(d, out, lse)


@pytest.mark.parametrize("pages,P,strides", [(1, 900, (16, 320, 1)), (1, 896, (0, 304, 1)), (900, 1, (352, 16, 1)),
                                             (900, 1, (304, 0, 1)), (1, 1, (16, 0, 1))])
def test_caches_of_one_page_or_one_slot_a_page(lib, pages, P, strides):
    """The stride of a dimension of one element says nothing."""
    from mla_ragged_paged_gb300 import binding
    store = torch.full((900 * 352,), 0xFF, dtype=torch.uint8, device="cuda")
    cache = store.as_strided((pages, P, 304), strides)
    slots = pages * P
    d = DecodeFp4([1], [slots - 1], 16, P, seed=P)
    d.table = torch.randperm(pages, generator=torch.Generator().manual_seed(1))[None].to(torch.int32)
    rows = _bf16_rows(slots, WIDTH, 3)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    ro = torch.tensor([0, slots], dtype=torch.int32, device="cuda")
    binding.append_latent_fp4(cache, rows.cuda(), d.table.cuda(), ro, zero)
    raw = torch.from_numpy(ora.encode(rows.float().numpy()))
    pos = torch.arange(slots)
    d.raw = torch.zeros(pages, P, 304, dtype=torch.uint8)
    d.raw[d.table[0, pos // P].long(), pos % P] = raw
    assert torch.equal(cache.cpu(), d.raw)
    assert int((store == 0xFF).sum()) >= store.numel() - slots * 304   # nothing but the rows is written
    back = torch.empty(slots, WIDTH, dtype=torch.bfloat16, device="cuda")
    binding.gather_latent_fp4(back, cache, d.table.cuda(), ro, zero)
    assert np.array_equal(_f64(back), ora.decode(raw.numpy(), WIDTH))
    out, lse = _run_decode(d, cache=cache)
    _check_decode(d, out, lse)


def _lengths(kind, rows, g):
    """Sequence lengths that sum to `rows`: `long` ones, or `tiny` ones of 0 .. 3 with runs of 40 and 90 empty ones
    among them (for 12 000 rows, then long ones)."""
    out, left = [], rows
    while left and kind == "tiny" and rows - left < 12000:
        few = torch.randint(0, 4, (50,), generator=g).tolist() + [0] * (40 if len(out) % 3 else 90)
        for n in few:
            out.append(min(n, left))
            left -= out[-1]
    while left:
        out.append(min(left, int(torch.randint(1, 1700, (1,), generator=g))))
        left -= out[-1]
    return out


# A warp takes ceil(rows / (32 warps x SMs)) rows, 32 at most: 4864 and 155 648 rows on 152 SMs.
@pytest.mark.parametrize("rows,W", [(5000, 576), (9800, 1024), (12000, 768), (14700, 512), (20000, 64), (100001, 64),
                                    (200000, 64), (170003, 128)])
@pytest.mark.parametrize("kind", ["long", "tiny"])
def test_append_and_gather_many_rows(lib, rows, W, kind):
    """Several rows a warp: two, an odd number, the most; sequences that end anywhere in a warp's rows, more
    empty ones in a row than a warp has lanes, bad pages in their midst, rows outside the batch."""
    from mla_ragged_paged_gb300 import binding
    g = torch.Generator().manual_seed(rows + W)
    P, first, behind = 16, 5, 3
    new = _lengths(kind, rows - first - behind, g)
    prior = torch.randint(0, 40, (len(new),), generator=g)
    n = torch.tensor(new)
    table, pages = page_table((n + prior).tolist(), P, g)
    ro = first + torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    b = torch.repeat_interleave(torch.arange(len(new)), n)
    pos = prior[b] + torch.arange(len(b)) - (ro[b] - first)
    good = table.clone()
    for at in torch.randint(0, len(b), (40,), generator=g).tolist():
        table[b[at], pos[at] // P] = pages + 7
    ok = table[b, pos // P] < pages
    slots = (good[b, pos // P].long() * P + pos % P)[ok]
    x = _bf16_rows(rows, W, rows)
    raw = torch.from_numpy(fast_encode(x[first:rows - behind].float().numpy()))[ok]
    cache = torch.full((pages, P, ora.row_bytes(W)), 0xA5, dtype=torch.uint8, device="cuda")
    want = torch.full((pages * P, ora.row_bytes(W)), 0xA5, dtype=torch.uint8)
    want[slots] = raw
    args = [t.to(torch.int32).cuda() for t in (table, ro, prior)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.append_latent_fp4(cache, x.cuda(), *args, status)
    assert int(status) == 0x1
    assert torch.equal(cache.cpu().view(-1, ora.row_bytes(W)), want)
    mine = torch.zeros(rows, dtype=torch.bool)
    mine[first:rows - behind] = ok
    codes, scales = ora.to_e4m3(raw.numpy(), W)
    back = torch.full((rows, W), 3.0, dtype=torch.bfloat16, device="cuda")
    status.zero_()
    binding.gather_latent_fp4(back, cache, *args, status=status)
    assert int(status) == 0x1
    assert np.array_equal(_f64(back[mine.cuda()]), ora.decode(raw.numpy(), W)) and (back[~mine.cuda()] == 3).all()
    back8 = torch.full((rows, W), 9, dtype=torch.uint8, device="cuda")
    back_s = torch.full((rows,), 5.0, device="cuda")
    binding.gather_latent_fp4(back8, cache, *args, dst_scales=back_s, status=status)
    assert np.array_equal(back8[mine.cuda()].cpu().numpy(), codes) and (back8[~mine.cuda()] == 9).all()
    assert np.array_equal(back_s[mine.cuda()].cpu().numpy(), scales) and (back_s[~mine.cuda()] == 5).all()


@pytest.mark.parametrize("heads,P", [(16, 64), (32, 64), (40, 7)])
def test_decode_wait_timeout_in_every_row_tile(lib, heads, P):
    """Copies that never come, in 16-, 32- and 64-row tiles, in boxes and row by row: the call ends, says so, and the
    next one is right."""
    from mla_ragged_paged_gb300 import binding
    d = DecodeFp4([1] * 60, [1500] * 60, heads, P, seed=68)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.test_inject_stall(True)
    try:
        _run_decode(d, status=status)
        assert int(status) == 0x8
    finally:
        binding.test_inject_stall(False)
    status.zero_()
    d2 = DecodeFp4([1, 1], [700, 40], heads, P, seed=69)
    out, lse = _run_decode(d2, status=status)
    assert int(status) == 0
    _check_decode(d2, out, lse)


# ------------------------------------------------------------------ prompts over cached rows

def test_prefill_from_bf16_rows(lib):
    """A prompt's chunk over rows kept in 4 bits, read back once in bf16: the 16-bit up-projection of their first 512
    columns, K_rope as the tail of the same rows.  Each stage is checked on its own inputs."""
    from mla_ragged_paged_gb300 import binding
    B, H, P = 2, 4, 16
    n, prior = [40, 25], [30, 100]
    d = DecodeFp4(n, prior, H, P, seed=70)
    L = [a + b for a, b in zip(n, prior)]
    S = sum(L)
    g = torch.Generator().manual_seed(71)
    wk, wv = ((torch.randn(H * 128, LATENT, generator=g) / 16).to(torch.bfloat16).cuda() for _ in range(2))
    ro, cl = (t.cuda() for t in d.offsets())
    bro, co, _, _ = binding.plan(ro, cl, S, 1)
    rows = torch.empty(S, WIDTH, dtype=torch.bfloat16, device="cuda")
    binding.gather_latent_fp4(rows, d.raw.cuda(), d.table.cuda(), bro[0], co[0])
    slots = torch.cat([d.table[b, torch.arange(L[b]) // P].long() * P + torch.arange(L[b]) % P for b in range(B)])
    assert np.array_equal(_f64(rows), ora.decode(d.raw.view(-1, 304)[slots].numpy(), WIDTH))
    k_nope = torch.empty(S, H, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k_nope)
    for out, w in ((k_nope, wk), (v, wv)):
        binding.up_project(out.view(S, -1), rows[:, :LATENT], w)
        ref, mag = _f64(rows[:, :LATENT]) @ _f64(w).T, np.abs(_f64(rows[:, :LATENT])) @ np.abs(_f64(w)).T
        _within(_f64(out.view(S, -1)), ref, 2.0 ** -8 * np.abs(ref) + 600 * 2.0 ** -23 * mag, "projection")
    q = (torch.randn(sum(n), H, 192, generator=g) * 0.3).to(torch.bfloat16)
    out = torch.empty(sum(n), H, 128, dtype=torch.bfloat16, device="cuda")
    rope = rows[:, LATENT:]
    binding.prefill_ragged_contiguous(out, q.cuda(), k_nope, v, rope, ro, cl, d.scale)
    for b in range(B):
        rows_b = slice(sum(L[:b]), sum(L[:b + 1]))
        k = torch.cat([k_nope[rows_b].cpu(), rope[rows_b, None, :].cpu().expand(-1, H, -1)], 2).double()
        qb = q[d.ro[b]:d.ro[b + 1]].double().transpose(0, 1)
        allowed = torch.arange(L[b])[None] <= prior[b] + torch.arange(n[b])[:, None]
        k, vb = k.transpose(0, 1), v[rows_b].cpu().double().transpose(0, 1)
        p = torch.softmax((qb @ k.transpose(1, 2) * d.scale).masked_fill(~allowed, float("-inf")), dim=2)
        # (The prefill's roundings: as above.)
        move = 4 * 192 * 2.0 ** -23 * d.scale * (qb.abs() @ k.abs().transpose(1, 2)).amax(dim=2, keepdim=True)
        ref = p @ vb
        tol = (2.0 ** -7 + move) * (p @ vb.abs()) + 2.0 ** -8 * ref.abs()
        got = out[d.ro[b]:d.ro[b + 1]].cpu().double().transpose(0, 1)
        _within(got.numpy(), ref.numpy(), tol.numpy(), f"sequence {b}")


def test_fp8_prefill_over_gathered_rows(lib):
    """K_rope of an 8-bit prefill as rows kept in 4 bits and read back in e4m3 with a scale each: the rope columns of the
    gathered rows, contiguous, beside 8-bit queries, K_nope and V.  (The 8-bit prefill's tolerance.)"""
    import workloads
    from mla_ragged_paged_gb300 import binding
    from oracle import attention as oatt
    from oracle.numerics import decode_e4m3
    w = workloads.custom([140, 60], [10, 130], heads=2, page_size=16, seed=810, row_width=WIDTH, rope_col=LATENT, dtype="fp8")
    shape = w.k_rope_pool.shape
    rows = decode_e4m3(w.k_rope_pool.view(torch.uint8).numpy()) * w.k_rope_scales.numpy().astype(np.float64)[..., None]
    rows[..., :LATENT] = np.random.default_rng(811).standard_normal(shape[:2] + (LATENT,))   # (NaN in the workload: not K_rope)
    rows = torch.from_numpy(rows).to(torch.bfloat16).float().numpy().reshape(-1, WIDTH)
    raw = torch.from_numpy(ora.encode(rows)).view(shape[0], shape[1], 304)
    codes, scales = ora.to_e4m3(raw.numpy(), WIDTH)
    w.k_rope_pool = torch.from_numpy(codes).view(w.k_rope_pool.dtype)
    w.k_rope_scales = torch.from_numpy(scales)
    d = workloads.device_inputs(w)
    Sk = w.total_k
    dst = torch.empty(Sk, WIDTH, dtype=torch.uint8, device="cuda")
    dst_scales = torch.empty(Sk, device="cuda")
    bro, co, _, _ = binding.plan(d["row_offsets"], d["cache_lens"], Sk, 1)
    binding.gather_latent_fp4(dst, raw.cuda(), d["page_table"], bro[0], co[0], dst_scales=dst_scales)
    want, want_scales = workloads.contiguous_rope(w)
    assert torch.equal(dst.cpu(), want.view(torch.uint8)) and torch.equal(dst_scales.cpu(), want_scales)
    out = torch.full((w.total_q, w.heads, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = binding.alloc_workspace(w.batch, fp8_pool_slots=Sk)
    rope = dst.view(d["q"].dtype)[:, LATENT:]
    binding.prefill_ragged_contiguous(out, d["q"], d["k_nope"], d["v"], rope, d["row_offsets"], d["cache_lens"], w.scale,
                                      binding.MLA_MASK_CAUSAL, ws, q_scale=d["q_scale"], k_scale=d["k_scale"],
                                      v_scale=d["v_scale"], k_rope_scales=dst_scales)
    assert binding.device_status(ws) == 0
    ref = oatt.reference(w)
    _within(_f64(out), ref, 6e-2 + 6e-2 * np.abs(ref), "out")
