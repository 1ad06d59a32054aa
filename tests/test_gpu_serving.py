"""The serving-step operators (mla_rms_norm, mla_matmul_fp8, mla_append_latent,
mla_decode_latent) on the GPU against oracle/serving.py in float64.

Tolerances, all derived before the first run (half a step: bf16 2^-8, e4m3
2^-4, float32 2^-24, relative):
* norm: the row's sum of squares is a chain of at most 32 products and 15
  additions of partial sums, so 2^-18 relative covers it and the few products
  after it; then one rounding of the output.  Codes: half a step, and half of
  e4m3's smallest step (2^-10) of the group's scale.
* product: K fp32 additions inside the blocks, at most 2^-23 of the terms'
  magnitudes each (the tensor cores may truncate), and one per block outside;
  then one rounding of the output.
* append: the same float32 division and rounding as torch's, so equal.
* attention: the softmax weights may carry a rounding to 8 significant bits
  (2^-8 of each weight), on both sides of the normalisation 2^-7 of
  sum_j p_j |c_j|; the scores 600 fp32 additions (2^-23 of their terms'
  magnitudes), which move each weight by that much, and the smallest query
  elements an absolute 2^-17 of the row's largest; then the output's rounding.
"""
import numpy as np
import pytest
import torch

from oracle import serving as ora
from oracle.numerics import decode_e4m3
from serving_inputs import E4M3, LATENT, WIDTH, Decode, blocks, quantise_rows

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _within(got, ref, tol, what):
    assert got.shape == ref.shape, what
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} out of tolerance, worst "
                           f"{np.nanmax(err / np.maximum(tol, 1e-300)):.3g} x, first at {np.argwhere(bad)[0]}")


# ------------------------------------------------------------------ norm

def _norm_case(rows, dim, seed, x_stride=None, w_dtype=torch.bfloat16, offset=0):
    g = torch.Generator().manual_seed(seed)
    stride = x_stride or dim
    x = torch.randn(rows * stride + offset, generator=g).to(torch.bfloat16).cuda()
    x = torch.as_strided(x, (rows, dim), (stride, 1), offset)
    r = (2 * torch.randn(rows, dim, generator=g)).to(torch.bfloat16).cuda()
    w = (1 + 0.2 * torch.randn(dim, generator=g)).to(w_dtype).cuda()
    return x, r, w


def _check_norm(x, r, w, eps, out, codes, scales, res_out):
    h, y, s = ora.rms_norm(_f64(x), _f64(w), eps, None if r is None else _f64(r))
    if out is not None:
        _within(_f64(out), y, (2.0 ** -8 + 2.0 ** -17) * np.abs(y) + 2.0 ** -133, "out")
    if codes is not None:
        _within(_f64(scales), s, 2.0 ** -17 * s, "scales")
        got = decode_e4m3(codes.view(torch.uint8).cpu().numpy())
        step = ora.spread(s, y.shape[1])
        _within(got * ora.spread(_f64(scales), y.shape[1]), y, (2.0 ** -4 + 2.0 ** -15) * np.abs(y) + 2.0 ** -10 * step,
                "codes")
        cols = np.abs(got[:, :128]).max(axis=1)
        assert (cols[s[:, 0] > 1e-20] == 448).all(), "a group's largest value takes the largest code"
    if res_out is not None:
        assert torch.equal(res_out, (x.float() + r.float()).to(torch.bfloat16))


@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (9, 8), (2, 128), (5, 129), (70, 256), (17, 1000), (3, 1024),
                                      (2, 1025), (2, 4096), (1, 8192), (400, 5000), (2, 16384), (3, 20001), (1, 32768)])
def test_norm(lib, rows, dim):
    from mla_ragged_paged_gb300 import binding
    x, r, w = _norm_case(rows, dim, rows + dim)
    out, res_out = torch.empty_like(r), torch.empty_like(r)
    codes = torch.empty(rows, dim, dtype=E4M3, device="cuda")
    scales = torch.empty(rows, -(-dim // 128), device="cuda")
    binding.rms_norm(x, w, 1e-6, residual=r, residual_out=res_out, out=out, out_fp8=codes, out_scales=scales)
    _check_norm(x, r, w, 1e-6, out, codes, scales, res_out)
    only = torch.empty_like(codes)
    binding.rms_norm(x, w, 1e-6, out_fp8=only, out_scales=scales)
    _check_norm(x, None, w, 1e-6, None, only, scales, None)


@pytest.mark.parametrize("dim", [600, 2100, 4600, 5100, 6100, 7001, 9000, 9999, 12000, 14000, 18001, 24000, 26000])
def test_norm_blocks_that_walk_several_rows(lib, dim):
    from mla_ragged_paged_gb300 import binding
    rows = 900 if dim < 4000 else 330
    x, r, w = _norm_case(rows, dim, dim)
    out, res_out = torch.empty_like(r), torch.empty_like(r)
    codes = torch.empty(rows, dim, dtype=E4M3, device="cuda")
    scales = torch.empty(rows, -(-dim // 128), device="cuda")
    binding.rms_norm(x, w, 1e-6, residual=r, residual_out=res_out, out=out, out_fp8=codes, out_scales=scales)
    _check_norm(x, r, w, 1e-6, out, codes, scales, res_out)


@pytest.mark.parametrize("rows,dim,stride,offset,w_dtype", [
    (50, 512, 576, 0, torch.bfloat16), (7, 512, 513, 1, torch.float32), (6, 1100, 1112, 8, torch.float32),
    (5, 2049, 2050, 3, torch.bfloat16), (4, 640, 0, 0, torch.bfloat16)])
def test_norm_strides(lib, rows, dim, stride, offset, w_dtype):
    from mla_ragged_paged_gb300 import binding
    if stride == 0:  # one row for all: an expanded input
        x, r, w = _norm_case(1, dim, 77)
        x, r = x.expand(rows, dim), r.expand(rows, dim)
    else:
        x, r, w = _norm_case(rows, dim, 78, stride, w_dtype, offset)
    wide = torch.full((rows, dim + 5), 3.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros(rows, dim + 3, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, -(-dim // 128) + 1), 7.0, device="cuda")
    binding.rms_norm(x, w, 1e-5, residual=r, out=wide[:, 2:2 + dim], out_fp8=codes[:, 1:1 + dim],
                     out_scales=scales[:, :-1])
    _check_norm(x, r, w, 1e-5, wide[:, 2:2 + dim], codes[:, 1:1 + dim], scales[:, :-1], None)
    assert (wide[:, :2] == 3).all() and (wide[:, 2 + dim:] == 3).all() and (scales[:, -1] == 7).all()
    assert (codes[:, 0] == 0).all() and (codes[:, 1 + dim:] == 0).all()


@pytest.mark.parametrize("dim", [300, 3000])
def test_norm_in_place_zero_and_nan_rows(lib, dim):
    from mla_ragged_paged_gb300 import binding
    x, r, w = _norm_case(6, dim, 5)
    x[1], r[1] = 0, 0
    x[2, 3] = float("nan")
    x[4] *= 1e-30
    r[4] = 0
    x0, r0 = x.clone(), r.clone()
    codes = torch.empty(6, dim, dtype=E4M3, device="cuda")
    scales = torch.empty(6, -(-dim // 128), device="cuda")
    binding.rms_norm(x, w, 1e-6, residual=r, residual_out=r, out=x, out_fp8=codes, out_scales=scales)
    keep = [0, 1, 3, 4, 5]
    _check_norm(x0[keep], r0[keep], w, 1e-6, x[keep], codes[keep], scales[keep], r[keep])
    assert (codes[1].float() == 0).all() and (scales[1] > 0).all()
    assert torch.isnan(scales[2]).all() and torch.isnan(codes[2].float()).all() and torch.isnan(x[2]).all()


@pytest.mark.parametrize("dim", [256, 3000, 3001])
def test_norm_sum_of_squares_past_float32_gives_zeros(lib, dim):
    from mla_ragged_paged_gb300 import binding
    x, r, w = _norm_case(3, dim, 6)
    x[1, 5] = 1e20
    out = torch.empty_like(r)
    codes = torch.empty(3, dim, dtype=E4M3, device="cuda")
    scales = torch.empty(3, -(-dim // 128), device="cuda")
    binding.rms_norm(x, w, 1e-6, out=out, out_fp8=codes, out_scales=scales)
    assert (out[1].float() == 0).all() and (codes[1].float() == 0).all() and (scales[1] > 0).all()
    _check_norm(x[::2], None, w, 1e-6, out[::2], codes[::2], scales[::2], None)


def test_norm_no_rows(lib):
    from mla_ragged_paged_gb300 import binding
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    binding.rms_norm(x, torch.ones(256, dtype=torch.bfloat16, device="cuda"), 0.0, out=torch.empty_like(x))


# ------------------------------------------------------------------ product

def _matmul_case(m, n, k, seed, row_scale=False):
    g = torch.Generator().manual_seed(seed)
    xc, xs = quantise_rows(torch.randn(m, k, generator=g) * torch.exp2(3 * torch.randn(m, 1, generator=g)),
                           None if row_scale else 128)
    if row_scale:
        xs = xs[:, None].expand(m, -(-k // 128))
    wc, ws = blocks(n, k, g)
    return xc.cuda().view(E4M3), xs.cuda(), wc.cuda().view(E4M3), ws.cuda()


def _check_matmul(out, x, xs, w, ws, cols=None):
    k = x.shape[1]
    ref, mag = ora.matmul_fp8(x.view(torch.uint8).cpu().numpy(), _f64(xs), w.view(torch.uint8).cpu().numpy(), _f64(ws))
    got = _f64(out)
    tol = HALF[out.dtype] * np.abs(ref) + (k + 2 * -(-k // 128) + 4) * 2.0 ** -23 * mag + 1e-38
    _within(got, ref, tol, "product")


@pytest.mark.parametrize("m,n,k", [
    (1, 1, 16), (1, 128, 128), (1, 1000, 4096), (2, 130, 144), (3, 7, 48), (16, 256, 512), (17, 300, 400),
    (31, 4096, 128), (33, 129, 2048), (64, 512, 1040), (65, 384, 640), (100, 100, 2000), (127, 640, 272),
    (128, 256, 256), (129, 257, 384), (200, 1000, 16), (300, 520, 1152), (513, 896, 528), (700, 2304, 768)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matmul(lib, m, n, k, dtype):
    from mla_ragged_paged_gb300 import binding
    x, xs, w, ws = _matmul_case(m, n, k, m + n + k)
    out = torch.full((m, n), float("nan"), dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.matmul_fp8(out, x, xs, w, ws, status)
    _check_matmul(out, x, xs, w, ws)
    assert int(status) == 0


@pytest.mark.parametrize("m,n,k", [(5, 200, 272), (150, 333, 512), (600, 1000, 400)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matmul_strides(lib, m, n, k, dtype):
    """Padded operands, transposed and broadcast scales, unaligned output rows
    whose surroundings keep their values."""
    from mla_ragged_paged_gb300 import binding
    x, xs, w, ws = _matmul_case(m, n, k, 3, row_scale=True)
    nan = torch.full((1,), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)
    wide = lambda t, pad: torch.cat([t.view(torch.uint8), nan.view(torch.uint8).expand(t.shape[0], pad)], 1).view(E4M3)
    x, w = wide(x, 32)[:, :k], wide(w, 16)[:, :k]
    ws = ws.t().contiguous().t()
    buf = torch.full((m + 2, n + 5), 3.0, dtype=dtype, device="cuda")
    out = buf[1:1 + m, 3:3 + n]
    binding.matmul_fp8(out, x, xs, w, ws)
    _check_matmul(out, x, xs, w, ws)
    out.fill_(3)
    assert (buf == 3).all()


@pytest.mark.parametrize("m,n,k", [(700, 2048, 4112), (129, 8200, 6000), (760, 1000, 10000), (65, 1100, 40960)])
@pytest.mark.parametrize("dtype,pad", [(torch.bfloat16, 8), (torch.float32, 5)])
def test_matmul_few_tiles_of_a_long_k(lib, m, n, k, dtype, pad):
    """Few output tiles, whose K is shared by several CTA pairs in unequal parts; outputs stored in
    both ways, the same in every run."""
    from mla_ragged_paged_gb300 import binding
    x, xs, w, ws = _matmul_case(m, n, k, 5)
    buf = torch.full((m + 1, n + pad), 3.0, dtype=dtype, device="cuda")
    out = buf[:m, :n]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.matmul_fp8(out, x, xs, w, ws, status)
    first = out.clone()
    _check_matmul(out, x, xs, w, ws)
    out.fill_(3)
    assert (buf == 3).all() and int(status) == 0
    binding.matmul_fp8(out, x, xs, w, ws)
    assert torch.equal(out, first)


@pytest.mark.parametrize("m,n,k", [(700, 2048, 4112), (760, 1000, 10000), (129, 8200, 6000)])
def test_matmul_delayed_second_half_keeps_results(lib, m, n, k):
    """One half of a tile's columns added up far behind the other where K is shared: the first
    half's sums must not take the place of operands that the second half still needs."""
    from mla_ragged_paged_gb300 import binding
    x, xs, w, ws = _matmul_case(m, n, k, 6)
    ref, out = (torch.empty(m, n, device="cuda") for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.matmul_fp8(ref, x, xs, w, ws, status)
    _check_matmul(ref, x, xs, w, ws)
    binding.test_delay_softmax(5000)
    try:
        for _ in range(5):
            out.fill_(float("nan"))
            binding.matmul_fp8(out, x, xs, w, ws, status)
            assert torch.equal(out, ref) and int(status) == 0
    finally:
        binding.test_delay_softmax(0)


@pytest.mark.parametrize("dtype,pad", [(torch.bfloat16, 24), (torch.float32, 4), (torch.float32, 12)])
def test_matmul_aligned_padded_rows(lib, dtype, pad):
    """Output rows that start 16-byte aligned and end inside a store's width:
    what lies behind them stays."""
    from mla_ragged_paged_gb300 import binding
    m, n, k = 700, 2280, 400
    x, xs, w, ws = _matmul_case(m, n, k, 4)
    buf = torch.full((m + 1, n + pad), 3.0, dtype=dtype, device="cuda")
    out = buf[:m, :n]
    binding.matmul_fp8(out, x, xs, w, ws)
    _check_matmul(out, x, xs, w, ws)
    out.fill_(3)
    assert (buf == 3).all()


def test_matmul_accumulates_in_32_bits(lib):
    """Terms that a narrower accumulator would lose: one large product, then
    many small ones that sum to something of float32's resolution of it."""
    from mla_ragged_paged_gb300 import binding
    m, n, k = 130, 128, 256
    x = torch.full((m, k), 2.0 ** -3, device="cuda")
    w = torch.full((n, k), 2.0 ** -3, device="cuda")
    x[:, 0] = w[:, 0] = 128.0
    for rows in (m, 3):
        out = torch.empty(rows, n, device="cuda")
        binding.matmul_fp8(out, x[:rows].to(E4M3), torch.ones(rows, 2, device="cuda"), w.to(E4M3),
                           torch.ones(1, 2, device="cuda"))
        want = 128.0 ** 2 + 255 * 2.0 ** -6
        assert (out - want).abs().max().item() <= 256 * 2.0 ** -23 * want


@pytest.mark.parametrize("m", [3, 200])
def test_matmul_nan_and_infinite_scale_stay_in_their_row(lib, m):
    from mla_ragged_paged_gb300 import binding
    x, xs, w, ws = _matmul_case(m, 300, 384, 9)
    x.view(torch.uint8)[1, 200] = 0x7F
    out = torch.empty(m, 300, device="cuda")
    binding.matmul_fp8(out, x, xs, w, ws)
    assert torch.isnan(out[1]).all()
    keep = [0] + list(range(2, m))
    _check_matmul(out[keep], x[keep], xs[keep], w, ws)


@pytest.mark.parametrize("m,n,k", [(48, 640, 8192), (700, 2304, 768), (700, 2048, 4112)])
def test_matmul_wait_timeout_sets_status_and_context_survives(lib, m, n, k):
    """A copy that never comes: the call ends, says so, and the next one is right (few tokens, many, and
    a tile's K shared by a cluster)."""
    from mla_ragged_paged_gb300 import binding
    x, xs, w, ws = _matmul_case(m, n, k, 11)
    out = torch.empty(m, n, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.test_inject_stall(True)
    try:
        binding.matmul_fp8(out, x, xs, w, ws, status)
        assert int(status) == 0x8
    finally:
        binding.test_inject_stall(False)
    status.zero_()
    binding.matmul_fp8(out, x, xs, w, ws, status)
    _check_matmul(out, x, xs, w, ws)
    assert int(status) == 0


@pytest.mark.parametrize("m,n,k", [(3, 300, 384), (200, 300, 384), (700, 2048, 4112)])
def test_matmul_infinite_and_nan_scales_stay_in_their_rows(lib, m, n, k):
    """A row's scale that is infinite or NaN, in each kernel, makes that row not finite and no other."""
    from mla_ragged_paged_gb300 import binding
    x, xs, w, ws = _matmul_case(m, n, k, 10)
    xs[1, 2], xs[2, 0] = float("inf"), float("nan")
    out = torch.empty(m, n, device="cuda")
    binding.matmul_fp8(out, x, xs, w, ws)
    assert not torch.isfinite(out[1]).any() and torch.isnan(out[2]).all()
    keep = [0] + list(range(3, m))
    _check_matmul(out[keep], x[keep], xs[keep], w, ws)


def test_matmul_no_rows(lib):
    from mla_ragged_paged_gb300 import binding
    x, xs, w, ws = _matmul_case(4, 64, 128, 1)
    binding.matmul_fp8(torch.empty(0, 64, device="cuda"), x[:0], xs[:0], w, ws)


def test_matmul_repeats_bit_for_bit(lib):
    from mla_ragged_paged_gb300 import binding
    for m, n, k in [(1, 1000, 4096), (48, 640, 8192), (700, 900, 1024)]:
        x, xs, w, ws = _matmul_case(m, n, k, 2)
        outs = []
        for _ in range(20):
            outs.append(torch.empty(m, n, device="cuda"))
            binding.matmul_fp8(outs[-1], x, xs, w, ws)
        assert all(torch.equal(o, outs[0]) for o in outs)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("W", [16, 256, 576, 1024])
@pytest.mark.parametrize("P,new,prior", [(16, [1, 1, 1], [0, 15, 31]), (12, [40, 0, 7], [5, 9, 0]), (1, [3], [2]),
                                         (64, [1] * 70, list(range(70)))])
def test_append(lib, W, P, new, prior):
    from mla_ragged_paged_gb300 import binding
    g = torch.Generator().manual_seed(W + P)
    from serving_inputs import page_table
    table, pages = page_table([a + b for a, b in zip(new, prior)], P, g)
    ro = np.concatenate([[0], np.cumsum(new)]) + 2      # rows before the first and after the last sequence
    rows = (torch.randn(int(ro[-1]) + 3, W, generator=g) * 5).to(torch.bfloat16)
    rows[2] = 0
    codes = torch.randint(0, 256, (pages, P, W), dtype=torch.uint8, generator=g)
    scales = torch.rand(pages, P, generator=g)
    wide = torch.full((pages, P, W + 32), 9, dtype=torch.uint8, device="cuda")
    cache = wide[:, :, :W]
    cache.copy_(codes)
    got_scales = scales.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.append_latent(cache, got_scales, rows.cuda(), table.cuda(), torch.tensor(ro, dtype=torch.int32).cuda(),
                          torch.tensor(prior, dtype=torch.int32).cuda(), status)
    want_c, want_s = codes.view(-1, W).clone(), scales.view(-1).clone()
    for slot, (row, scale) in ora.append(rows.float().numpy(), table.numpy(), ro, prior, P).items():
        want_c[slot] = torch.from_numpy(row).to(E4M3).view(torch.uint8)
        want_s[slot] = float(scale)
    assert torch.equal(cache.cpu().view(-1, W), want_c)
    assert torch.equal(got_scales.cpu().view(-1), want_s)
    assert (wide[:, :, W:] == 9).all() and int(status) == 0


def test_append_codes_next_to_ties(lib):
    """Every bf16 mantissa at seven exponents over every mantissa of the largest number:
    quotients on both sides of a tie and on it, subnormal codes, infinities."""
    from mla_ragged_paged_gb300 import binding
    W = 896
    mantissas = torch.arange(128) / 128 + 1
    body = (mantissas[None] * 2.0 ** torch.tensor([-1, -2, -5, -11, -14, -15, -16])[:, None]).reshape(-1)
    rows = body.repeat(129, 1) * torch.where(torch.arange(W) % 3 == 0, -1.0, 1.0)
    rows[:128, 5] = 2 * mantissas
    rows[128, 5] = float("inf")
    rows = torch.cat([rows, rows[:128] * 2.0 ** -100, rows[:128] * 2.0 ** 120]).to(torch.bfloat16)
    n = rows.shape[0]
    cache = torch.zeros(1, n, W, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(1, n, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.append_latent(cache, scales, rows.cuda(), torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                          torch.tensor([0, n], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda(), status)
    want = rows.float().abs().amax(1).clamp_min(1e-30) / 448
    quotient = rows.float() / want[:, None]
    assert int(status) == 0 and torch.equal(scales.cpu()[0], want)
    assert torch.equal(cache.cpu()[0] & 0x7F, quotient.to(E4M3).view(torch.uint8) & 0x7F)
    finite = quotient == quotient
    assert torch.equal(cache.cpu()[0][finite], quotient.to(E4M3).view(torch.uint8)[finite])


def test_append_bad_pages_and_nan(lib):
    from mla_ragged_paged_gb300 import binding
    table = torch.tensor([[1, 99], [0, 2]], dtype=torch.int32, device="cuda")
    cache = torch.zeros(3, 4, 576, dtype=torch.uint8, device="cuda")
    scales = torch.full((3, 4), 5.0, device="cuda")
    rows = torch.ones(13, 576, dtype=torch.bfloat16, device="cuda")
    rows[0, 7] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ro = torch.tensor([0, 6, 13], dtype=torch.int32, device="cuda")
    lens = torch.tensor([2, 3], dtype=torch.int32, device="cuda")
    # Sequence 0: tokens 2, 3 on page 1, tokens 4..7 on page 99; sequence 1:
    # tokens 3..9, of which 8 and 9 lie past its two page-table columns.
    binding.append_latent(cache, scales, rows, table, ro, lens, status)
    assert int(status) == 0x3
    one = torch.tensor(1.0 / 448)
    assert torch.isnan(scales[1, 2]) and torch.equal(scales[1, 3].cpu(), one)
    assert (scales[1, :2] == 5).all() and (scales[0, :3] == 5).all()
    assert torch.equal(scales[0, 3].cpu(), one) and torch.equal(scales[2].cpu(), one.expand(4))
    lens.fill_(-1)                                   # a length no context can have
    before = cache.clone()
    binding.append_latent(cache, scales, rows, table, ro, lens, status)
    assert torch.equal(cache, before)


# ------------------------------------------------------------------ attention

def _run_decode(d, mask="causal", lse=True, per_tensor=None, workspace=None, out=None, q=None, cache=None, status=None):
    from mla_ragged_paged_gb300 import binding
    ro, cl = (t.cuda() for t in d.offsets())
    q = d.q.cuda() if q is None else q
    cache = d.codes.cuda() if cache is None else cache
    scales = d.scales.cuda() if per_tensor is None else torch.tensor([per_tensor], device="cuda")
    if out is None:
        out = torch.full((q.shape[0], d.heads, LATENT), float("nan"), dtype=torch.bfloat16, device="cuda")
    L = torch.full((q.shape[0], d.heads), float("nan"), device="cuda") if lse else None
    binding.decode_latent(out, q, cache, scales, d.table.cuda(), ro, cl, d.scale,
                          binding.MLA_MASK_CAUSAL if mask == "causal" else binding.MLA_MASK_NULL,
                          workspace=workspace, lse=L, status=status)
    return out, L


def _check_decode(d, out, lse, mask="causal", scales=None, lost=()):
    ref, z, mag, terms = ora.decode(d.q.float().numpy(), d.codes.numpy(),
                                    d.scales.numpy() if scales is None else scales, d.table.numpy(), d.ro, d.prior,
                                    d.scale, mask == "causal", lost)
    move = 600 * 2.0 ** -23 * terms + 2.0 ** -17 * terms
    tol = (2.0 ** -7 + 4 * move)[:, :, None] * mag + 2.0 ** -8 * np.abs(ref) + 1e-30
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
    d = Decode(n, prior, heads, P, seed=sum(n) + sum(prior) + heads)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _run_decode(d, mask, status=status)
    assert int(status) == 0
    _check_decode(d, out, lse, mask)


@pytest.mark.parametrize("n,prior,heads", [
    ([1] * 170, [0, 200, 20, 127, 128] * 34, 128), ([1] * 151, [0] * 151, 16), ([1, 0, 1] * 100, [130, 9, 300] * 100, 8),
    ([1] * 31, [0] * 31, 64), ([1] * 30 + [2], [0] * 30 + [4000], 64), ([1] * 77, list(range(100, 870, 10)), 65)])
def test_decode_shares_that_end_anywhere(lib, n, prior, heads):
    """Row tiles of one to a few key tiles, so that the SMs' shares end before, behind and inside them."""
    d = Decode(n, prior, heads, 16, seed=sum(prior) + heads)
    out, lse = _run_decode(d)
    _check_decode(d, out, lse)


@pytest.mark.parametrize("q_std,spread,sink", [(0.0, 0.5, 0.0), (4.0, 0.5, 0.0), (12.0, 3.0, 0.0), (1.0, 6.0, 0.0),
                                               (1.5, 0.5, 3.0), (1e-20, 0.5, 0.0), (60.0, 0.1, 0.0)])
def test_decode_value_ranges(lib, q_std, spread, sink):
    """Flat, wide and peaked softmaxes; rows of very different sizes; one early
    key far above the rest (its tail must keep its precision)."""
    d = Decode([1, 2], [1500, 300], 20, 64, seed=31, spread=spread, q_std=q_std, sink=sink)
    if sink:
        d.q += torch.tensor(0.25, dtype=torch.bfloat16)
    out, lse = _run_decode(d)
    _check_decode(d, out, lse)


@pytest.mark.parametrize("spread", [12.0, 20.0, 40.0])
@pytest.mark.parametrize("n,prior", [([1, 2], [1500, 300]), ([1], [9000]), ([1] * 170, [100] * 170)])
def test_decode_scales_far_apart(lib, n, prior, spread):
    """Keys of similar softmax weight whose scales differ by up to 2^80: those with small scales add
    little to the numerator and all of their weight to the denominator, in row tiles that one CTA takes
    whole and in joined ones."""
    d = Decode(n, prior, 20, 64, seed=41, spread=spread, q_std=2.0 ** -spread)
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
    d = Decode([1] * len(lengths), [n - 1 for n in lengths], 16, 16, seed=42, q_std=q_std)
    g = torch.Generator().manual_seed(43)
    rows = []
    for n in lengths:
        x = torch.randn(n, WIDTH, generator=g)
        zero = {"early": slice(0, (n + 1) // 2), "late": slice(n // 2, n), "odd": slice(1, n, 2), "all": slice(0, n),
                "all but one": slice(1, n)}[zeros]
        x[zero] = 0
        rows.append(x)
    cache, scales = d.codes.cuda(), d.scales.cuda()
    ro = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
    binding.append_latent(cache, scales, torch.cat(rows).to(torch.bfloat16).cuda(), d.table.cuda(), ro,
                          torch.zeros(len(lengths), dtype=torch.int32, device="cuda"))
    d.codes, d.scales = cache.cpu(), scales.cpu()
    out, lse = _run_decode(d)
    _check_decode(d, out, lse)


@pytest.mark.parametrize("large", [2.0 ** 8, 2.0 ** 10, 2.0 ** 14])
def test_decode_query_elements_next_to_a_large_one(lib, large):
    """One element far above the others, in a dim that the cache leaves at zero: the others must
    keep what is documented."""
    d = Decode([1, 2], [700, 40], 20, 64, seed=77, q_std=1.0)
    d.q.clamp_(-2, 2)
    d.q[:, :, 7] = large
    d.codes.view(torch.uint8)[..., 7] = 0
    out, lse = _run_decode(d)
    # The two terms: the row's largest element is scaled into [128, 256).
    q = d.q.float()
    up = 2.0 ** (7 - torch.floor(torch.log2(q.abs().amax(-1, keepdim=True))))
    first = (q * up).to(E4M3).float()
    taken = (first + (q * up - first).to(E4M3).float()) / up
    assert ((taken - q).abs() <= 2.0 ** -17 * large).all()
    assert torch.equal(taken[q.abs() >= 2.0 ** -9 * large], q[q.abs() >= 2.0 ** -9 * large])
    d.q = taken
    _check_decode(d, out, lse)


def test_decode_tail_behind_a_sink(lib):
    """One key takes e^12 times the weight of each of 40 000 others, which
    together outweigh it in the first 512 columns: weights rounded to steps of
    the largest would lose them."""
    d = Decode([1], [40000], 16, 64, seed=8, spread=0.0)
    x = torch.zeros(40001, WIDTH)
    x[:, :LATENT] = 1.0                      # every key: ones, but for the sink's zeros
    x[0, :LATENT] = 0.0
    x[:, LATENT:] = 0.01 * torch.randn(40001, 64, generator=torch.Generator().manual_seed(3))
    x[0, LATENT:] = 1.0
    codes, scales = quantise_rows(x)
    pos = torch.arange(40001)
    pg = d.table[0, pos // 64].long()
    d.codes[pg, pos % 64], d.scales[pg, pos % 64] = codes, scales
    d.q.zero_()
    d.q[:, :, LATENT:] = 12.0 / (64 * d.scale)
    out, lse = _run_decode(d)
    _check_decode(d, out, lse)


def test_decode_per_tensor_scale(lib):
    d = Decode([1, 2], [200, 33], 16, 16, seed=12)
    d.codes[d.codes == 0x7F] = 0
    out, lse = _run_decode(d, per_tensor=0.0078125)
    _check_decode(d, out, lse, scales=np.full(d.scales.shape, 0.0078125))


@pytest.mark.parametrize("P", [16, 12])
def test_decode_strides_and_rows_outside(lib, P):
    """Padded queries, outputs and cache rows; rows before the first and behind
    the last sequence stay as they were."""
    d = Decode([2, 1], [100, 300], 6, P, seed=14)
    tq = int(d.ro[-1])
    big = torch.full((tq + 5, 8, 600), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[2:2 + tq, 1:7, :576] = d.q.cuda()
    q = big[:, 1:7, :576]
    buf = torch.full((tq + 5, 7, 520), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :6, :512]
    wide = torch.full((d.codes.shape[0], P, 592), 0x7F, dtype=torch.uint8, device="cuda")
    wide[:, :, :576] = d.codes.cuda()
    ref_ro = d.ro.copy()
    d.ro = d.ro + 2
    _, lse = _run_decode(d, out=out, q=q, cache=wide[:, :, :576])
    d.ro = ref_ro
    _check_decode(d, out[2:2 + tq], lse[2:2 + tq])
    assert torch.isnan(lse[:2]).all() and torch.isnan(lse[2 + tq:]).all()
    out[2:2 + tq] = 3
    assert (buf == 3).all()


def test_decode_bad_pages(lib):
    """Keys on bad pages or past the page table count as masked; a query left
    without keys gets 0 and -inf."""
    d = Decode([1, 1, 1], [500, 20, 40], 16, 16, seed=15)
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
    """A NaN query gives NaN in its own rows only; a NaN code in one sequence
    leaves the others alone; a masked NaN key is not seen."""
    d = Decode([2, 1, 1], [130, 40, 200], 16, 16, seed=16)
    d.q[2, 5, 17] = float("nan")
    d.codes[d.table[0, 131 // 16].long(), 131 % 16, 9] = 0x7F      # visible to token 1 of sequence 0 only
    out, lse = _run_decode(d)
    out, lse = out.cpu(), lse.cpu()
    assert torch.isnan(lse[1]).all() and torch.isnan(out[1]).any(dim=1).all()
    assert torch.isnan(out[2, 5]).all() and torch.isnan(lse[2, 5])
    d.q[2, 5, 17] = 1.0
    ref, z, mag, _ = ora.decode(d.q.float().numpy(), d.codes.numpy(), d.scales.numpy(), d.table.numpy(), d.ro,
                                d.prior, d.scale)
    for t in (0, 2, 3):
        heads = [h for h in range(16) if (t, h) != (2, 5)]
        tol = 2.0 ** -6 * mag[t, heads] + 2.0 ** -8 * np.abs(ref[t, heads])
        _within(_f64(out[t, heads]), ref[t, heads], tol, f"token {t}")


def test_decode_repeats_and_shares_a_workspace(lib):
    """Bit-identical repeats, with other problems in between on one workspace
    whose contents start as garbage; also on a stream of its own."""
    from mla_ragged_paged_gb300 import binding
    ws = torch.full((binding.decode_workspace_size(),), 0xA5, dtype=torch.uint8, device="cuda")
    a, b = Decode([1, 1], [5000, 70], 64, 64, seed=1), Decode([1] * 30, [200] * 30, 16, 64, seed=2)
    first, lse = _run_decode(a, workspace=ws)
    _check_decode(a, first, lse)
    side = torch.cuda.Stream()
    for i in range(10):
        out_b, lse_b = _run_decode(b, workspace=ws)
        again, _ = _run_decode(a, workspace=ws, lse=False)
        assert torch.equal(again, first)
    _check_decode(b, out_b, lse_b)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again, _ = _run_decode(a)
    side.synchronize()
    assert torch.equal(again, first)


def test_decode_graph_follows_lengths(lib):
    """A captured call reads lengths, offsets and pages when it runs: replays
    after the sequences have grown, and with one of them gone."""
    from mla_ragged_paged_gb300 import binding
    d = Decode([1, 1, 1], [700, 90, 2000], 16, 16, seed=61)
    ro, cl = (t.cuda() for t in d.offsets())
    q, cache, scales, table = d.q.cuda(), d.codes.cuda(), d.scales.cuda(), d.table.cuda()
    out = torch.empty(3, 16, LATENT, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, 16, device="cuda")
    ws = binding.alloc_decode_workspace()
    call = lambda: binding.decode_latent(out, q, cache, scales, table, ro, cl, d.scale, workspace=ws, lse=lse)
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
    from mla_ragged_paged_gb300 import binding
    a, b = Decode([1], [9000], 64, 64, seed=62), Decode([1] * 6, [1500] * 6, 16, 64, seed=63)
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
    """A length past the page table masks the keys there; offsets that decrease
    or leave the queries skip their sequence; the others are right."""
    d = Decode([1, 1, 1, 1], [40, 100, 60, 30], 8, 16, seed=64)
    d.prior = [40, -1, 60, 30]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _run_decode(d, status=status)
    assert int(status) & 0x2
    d.prior[1] = 100
    keep = [0, 2, 3]
    ref, _, mag, _ = ora.decode(d.q.float().numpy(), d.codes.numpy(), d.scales.numpy(), d.table.numpy(), d.ro, d.prior,
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


@pytest.mark.parametrize("heads,P", [(64, 16), (16, 12)])
def test_decode_wait_timeout_sets_status_and_context_survives(lib, heads, P):
    """A copy that never comes: the call ends, says so, and the next one is right (64- and 32-row tiles,
    boxes and row gathers; several tiles a CTA, so that the producer is stopped in mid-ring)."""
    from mla_ragged_paged_gb300 import binding
    d = Decode([1] * 60, [3000] * 60, heads, P, seed=66)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.test_inject_stall(True)
    try:
        _run_decode(d, status=status)
        assert int(status) == 0x8
    finally:
        binding.test_inject_stall(False)
    status.zero_()
    d2 = Decode([1, 1], [700, 40], heads, P, seed=67)
    out, lse = _run_decode(d2, status=status)
    assert int(status) == 0
    _check_decode(d2, out, lse)


def test_decode_many_heads(lib):
    d = Decode([1, 2], [70, 300], 1024, 64, seed=65)
    out, lse = _run_decode(d)
    _check_decode(d, out, lse)


def test_decode_offsets_past_32_bits(lib):
    """Cache rows whose byte offsets pass 2^32."""
    P, pages = 4096, 1900
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough memory")
    d = Decode([1, 1], [6000, 300], 16, P, seed=21)
    cache = torch.full((pages, P, WIDTH), 0x7F, dtype=torch.uint8, device="cuda")
    scales = torch.full((pages, P), float("nan"), device="cuda")
    move = torch.tensor([pages - 1, 3, pages - 2, 900])
    cache[move[:d.codes.shape[0]].cuda()] = d.codes.cuda()
    scales[move[:d.codes.shape[0]].cuda()] = d.scales.cuda()
    small, d.table = d.table, move[d.table.long()].to(torch.int32)
    from mla_ragged_paged_gb300 import binding
    ro, cl = (t.cuda() for t in d.offsets())
    out = torch.empty(2, 16, LATENT, dtype=torch.bfloat16, device="cuda")
    binding.decode_latent(out, d.q.cuda(), cache, scales, d.table.cuda(), ro, cl, d.scale)
    # The append reaches the same slots.
    rows = torch.randn(2, WIDTH, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    binding.append_latent(cache, scales, rows.cuda(), d.table.cuda(), ro, cl)
    codes, s = quantise_rows(rows.float())
    for b in range(2):
        pg, sl = int(d.table[b, d.prior[b] // P]), d.prior[b] % P
        assert torch.equal(cache[pg, sl].cpu(), codes[b]) and scales[pg, sl].item() == s[b].item()
    d.table = small
    _check_decode(d, out, None)


# ------------------------------------------------------------------ together

def _step_inputs(seed, B=5, heads=16, hidden=1024, prior=(40, 0, 129, 300, 7), P=16):
    g = torch.Generator().manual_seed(seed)
    s = dict(B=B, heads=heads)
    s["d"] = Decode([1] * B, list(prior), heads, P, seed=seed)
    s["x"] = torch.randn(B, hidden, generator=g).to(torch.bfloat16)
    s["res"] = torch.randn(B, hidden, generator=g).to(torch.bfloat16)
    s["w_norm"] = (1 + 0.1 * torch.randn(hidden, generator=g)).to(torch.bfloat16)
    s["w_lat"] = (1 + 0.1 * torch.randn(LATENT, generator=g)).to(torch.bfloat16)
    s["w_kv"] = blocks(WIDTH, hidden, g, spread=0.0)
    s["w_q"] = blocks(heads * WIDTH, hidden, g, spread=0.0)
    return s


def test_serving_step(lib):
    """Norm, projections, latent norm in place, append and attention, as a
    serving step runs them: directly, and captured into a graph that is replayed
    on new inputs.  Each stage is checked against the oracle on the stage's own
    inputs, so no tolerance piles up."""
    from mla_ragged_paged_gb300 import binding
    s = _step_inputs(40)
    d, B, H = s["d"], s["B"], s["heads"]
    dev = {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}
    w_kv, w_q = [t.cuda() for t in s["w_kv"]], [t.cuda() for t in s["w_q"]]
    cache, scales, table = d.codes.cuda(), d.scales.cuda(), d.table.cuda()
    ro, cl = (t.cuda() for t in d.offsets())
    hidden = dev["x"].shape[1]
    y8 = torch.empty(B, hidden, dtype=E4M3, device="cuda")
    ys = torch.empty(B, hidden // 128, device="cuda")
    res_out = torch.empty_like(dev["res"])
    kv = torch.empty(B, WIDTH, dtype=torch.bfloat16, device="cuda")
    raw = torch.empty_like(kv)
    q = torch.empty(B, H, WIDTH, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(B, H, LATENT, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, H, device="cuda")
    ws = binding.alloc_decode_workspace()

    def step():
        binding.rms_norm(dev["x"], dev["w_norm"], 1e-6, residual=dev["res"], residual_out=res_out, out_fp8=y8,
                         out_scales=ys)
        binding.matmul_fp8(raw, y8, ys, *w_kv)
        binding.matmul_fp8(q.view(B, H * WIDTH), y8, ys, *w_q)
        kv.copy_(raw)
        binding.rms_norm(kv[:, :LATENT], dev["w_lat"], 1e-6, out=kv[:, :LATENT])
        binding.append_latent(cache, scales, kv, table, ro, cl)
        binding.decode_latent(out, q, cache, scales, table, ro, cl, d.scale, workspace=ws, lse=lse)

    def check():
        torch.cuda.synchronize()
        _check_norm(dev["x"], dev["res"], dev["w_norm"], 1e-6, None, y8, ys, res_out)
        _check_matmul(raw, y8, ys, *(t.view(E4M3) if t.dtype == torch.uint8 else t for t in w_kv))
        _check_matmul(q.view(B, -1), y8, ys, *(t.view(E4M3) if t.dtype == torch.uint8 else t for t in w_q))
        _check_norm(raw[:, :LATENT], None, dev["w_lat"], 1e-6, kv[:, :LATENT], None, None, None)
        assert torch.equal(kv[:, LATENT:], raw[:, LATENT:])
        codes, sc = quantise_rows(kv.float().cpu())
        for b in range(B):
            pg, sl = int(d.table[b, d.prior[b] // d.P]), d.prior[b] % d.P
            assert torch.equal(cache[pg, sl].cpu(), codes[b]) and scales[pg, sl].item() == sc[b].item()
        d.codes, d.scales, d.q = cache.cpu(), scales.cpu(), q.cpu()
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
        dev["x"].copy_(new["x"])
        dev["res"].copy_(new["res"])
        out.fill_(float("nan"))
        graph.replay()
        check()


def test_prefill_over_the_8_bit_latent_cache(lib):
    """A prompt's chunk over rows kept in the 8-bit cache: the gather, the
    up-projections with one scale per row, then the prefill; K_rope is the
    dequantised tail of the same rows."""
    import workloads
    from mla_ragged_paged_gb300 import binding
    from oracle import plan as oplan
    B, H, P = 2, 4, 16
    n, prior = [40, 25], [30, 100]
    d = Decode(n, prior, H, P, seed=50)
    L = [a + b for a, b in zip(n, prior)]
    S = sum(L)
    g = torch.Generator().manual_seed(51)
    wk, wv = ([t.cuda() for t in blocks(H * 128, LATENT, g, spread=0.5)] for _ in range(2))
    ro, cl = (t.cuda() for t in d.offsets())
    bro, co, _, _ = oplan.plan_formula(d.ro.astype(np.uint32), np.array(prior, dtype=np.uint32), S, 1)
    bro_d, co_d = (torch.from_numpy(a[0].astype(np.int32)).cuda() for a in (bro, co))
    rows = torch.empty(S, WIDTH, dtype=torch.uint8, device="cuda")
    binding.gather_rows(rows, d.codes.cuda(), d.table.cuda(), bro_d, co_d)
    slots = torch.cat([d.table[b, torch.arange(L[b]) // P].long() * P + torch.arange(L[b]) % P for b in range(B)])
    row_scales = d.scales.view(-1)[slots].cuda()
    wide = row_scales[:, None].expand(S, LATENT // 128)
    k_nope = torch.empty(S, H, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k_nope)
    binding.matmul_fp8(k_nope.view(S, -1), rows[:, :LATENT], wide, *wk)
    binding.matmul_fp8(v.view(S, -1), rows[:, :LATENT], wide, *wv)
    lat = rows[:, :LATENT].view(E4M3)
    _check_matmul(k_nope.view(S, -1), lat, wide, wk[0].view(E4M3), wk[1])
    _check_matmul(v.view(S, -1), lat, wide, wv[0].view(E4M3), wv[1])
    rope = (rows[:, LATENT:].view(E4M3).float() * row_scales[:, None]).to(torch.bfloat16)
    q = (torch.randn(sum(n), H, 192, generator=g) * 0.3).to(torch.bfloat16)
    out = torch.empty(sum(n), H, 128, dtype=torch.bfloat16, device="cuda")
    binding.prefill_ragged_contiguous(out, q.cuda(), k_nope, v, rope, ro, cl, d.scale)
    for b in range(B):
        rows_b = slice(sum(L[:b]), sum(L[:b + 1]))
        k = torch.cat([k_nope[rows_b].cpu(), rope[rows_b, None, :].cpu().expand(-1, H, -1)], 2).double()
        qb = q[d.ro[b]:d.ro[b + 1]].double().transpose(0, 1)
        allowed = torch.arange(L[b])[None] <= prior[b] + torch.arange(n[b])[:, None]
        k, vb = k.transpose(0, 1), v[rows_b].cpu().double().transpose(0, 1)
        p = torch.softmax((qb @ k.transpose(1, 2) * d.scale).masked_fill(~allowed, float("-inf")), dim=2)
        # The prefill rounds each weight to bf16 (2^-8 of it, on both sides of
        # the normalisation 2^-7 of sum p |v|), adds 192 products per score in
        # fp32 (2^-23 of the terms each, which moves a weight by that much) and
        # rounds the output: the values here reach 60, so an absolute tolerance
        # made for values of size one says nothing.
        move = 4 * 192 * 2.0 ** -23 * d.scale * (qb.abs() @ k.abs().transpose(1, 2)).amax(dim=2, keepdim=True)
        ref = p @ vb
        tol = (2.0 ** -7 + move) * (p @ vb.abs()) + 2.0 ** -8 * ref.abs()
        got = out[d.ro[b]:d.ro[b + 1]].cpu().double().transpose(0, 1)
        _within(got.numpy(), ref.numpy(), tol.numpy(), f"sequence {b}")
