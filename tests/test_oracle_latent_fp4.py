"""Pins of oracle/latent_fp4.py (CPU): the format's numbers, exactness, and the
rotation against complex arithmetic."""
import numpy as np
import pytest
import torch

from oracle import latent_fp4 as ora
from oracle.numerics import decode_e4m3


def _bf16(x):
    return torch.as_tensor(x, dtype=torch.float32).to(torch.bfloat16).float().numpy()


def test_numbers_of_the_format():
    assert ora.MAGNITUDES.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert [ora.row_bytes(w) for w in (64, 512, 576, 1024)] == [48, 272, 304, 544]
    row = np.zeros((1, 64), dtype=np.float32)
    row[0, :8] = [6, -3, 0.25, 0.75, 2.5, 3.5, 5, 7]          # ties go to the even code; 7 becomes 6
    row[0, 32:36] = [0.75, -0.375, 0.03125, -0.0]               # a block 8 times smaller
    raw = ora.encode(row)[0]
    assert raw[:4].tolist() == [0xD7, 0x20, 0x64, 0x76] and raw[32] == 127 and raw[33] == 0x30
    assert raw[16:18].tolist() == [0xD7, 0x80] and not raw[34:].any()
    assert ora.decode(raw, 64)[:8].tolist() == [6, -3, 0, 1, 2, 4, 4, 6]


@pytest.mark.parametrize("spread", [0.0, 3.0, 12.0])
def test_rows_are_near_and_exact_in_e4m3(spread):
    g = np.random.default_rng(int(spread))
    x = _bf16(g.standard_normal((20, 576)) * np.repeat(np.exp2(spread * g.uniform(-1, 1, (20, 18))), 32, axis=1))
    raw = ora.encode(x)
    v = ora.decode(raw, 576)
    amax = np.repeat(np.abs(x).reshape(20, 18, 32).max(axis=2), 32, axis=1)
    floor = np.abs(x).max(axis=1, keepdims=True) * 2.0 ** -14 / 3.5
    assert (np.abs(v - x) <= np.maximum(amax / 3.5, floor)).all()
    codes, scales = ora.to_e4m3(raw, 576)
    assert np.array_equal(decode_e4m3(codes) * scales[:, None].astype(np.float64), v)


def test_how_far_values_are_held():
    """Every mantissa of a block's largest value, with values of every mantissa and smaller exponents beside it, in
    blocks up to 2^20 below the row's largest and in rows at both ends of the exponents."""
    least = np.inf
    for row_exp in (0, -90, -105, -115, 125, 127):
        worst = 0.0
        for block_exp in (0, 3, 13, 14, 15, 20):
            x = np.zeros((128, 64))
            m = 1 + np.arange(128) / 128
            x[:, 0] = 1.75 * 2.0 ** row_exp                            # the row's largest, exact
            x[:, 32] = m * 2.0 ** (row_exp - block_exp) if block_exp else np.minimum(m, 1.9921875) * 2.0 ** row_exp
            for j in range(31):
                x[:, 33 + j] = -m[(np.arange(128) * 5 + 37 * j) % 128] * 2.0 ** (row_exp - block_exp - j // 8)
            x[:, 33:] = np.clip(x[:, 33:], -x[:, 32:33], 0)
            x = np.clip(x, -3.3895e38, 3.3895e38)
            if row_exp - block_exp < -126:
                continue
            x = _bf16(x).astype(np.float64)
            raw = ora.encode(x)
            v, top = ora.decode(raw, 64), 2.0 ** (raw[:, 32].astype(np.float64) - 127)
            amax = np.abs(x[:, 32:]).max(axis=1)
            past = amax > 7 * 2.0 ** 125
            share = np.where(past, 0.25, 0.2)
            err = np.abs(v - x)[:, 32:].max(axis=1)
            assert (err <= np.maximum(share * amax, top * 2.0 ** -14 / 4)).all(), (row_exp, block_exp)
            worst = max(worst, float((err / amax)[~past].max()) if (~past).any() else 0.0)
        least = min(least, worst) if row_exp == 0 else least
    assert least >= 0.2                                                  # a largest value of 5 becomes 4
    assert ora.encode(np.zeros((1, 64)))[0, 32] == 27


def test_special_rows():
    x = np.zeros((5, 64), dtype=np.float32)
    x[1, 3], x[2, 40] = np.nan, -np.inf
    x[3, 0] = _bf16(3.3e38)
    x[4, 0], x[4, 32] = 1e-37, 2.0 ** -126
    raw = ora.encode(x)
    assert raw[:, 32].tolist() == [27, 255, 255, 252, 27]
    v = ora.decode(raw, 64)
    assert not v[0].any() and np.isnan(v[1:3]).all() and v[3, 0] == 6 * 2.0 ** 125
    assert v[4].any() == (2.0 ** -126 >= 2.0 ** -115)


@pytest.mark.parametrize("halves", [False, True])
def test_rotation_is_a_complex_product(halves):
    g = np.random.default_rng(3)
    x = g.standard_normal((4, 2, 10))
    f = np.array([1.0, 0.1, 0.01], dtype=np.float32)
    pos = np.array([0, 1, 1000, 4000000000])
    y, _ = ora.norm_rope(x, np.full(4, 2.0), 1e-5, pos, f, 1.5, halves)
    n = x.copy()
    n[..., :4] = 2 * x[..., :4] / np.sqrt((x[..., :4] ** 2).mean(-1, keepdims=True) + 1e-5)
    a, b = ((4, 5, 6), (7, 8, 9)) if halves else ((4, 6, 8), (5, 7, 9))
    z = (n[..., a] + 1j * n[..., b]) * np.exp(1j * (pos[:, None] * f.astype(np.float64)))[:, None, :] * 1.5
    assert np.allclose(y[..., a], z.real, atol=1e-6) and np.allclose(y[..., b], z.imag, atol=1e-6)
    assert np.array_equal(y[..., :4], n[..., :4])


def test_vectorised_encoder_is_the_oracles():
    from fp4_inputs import fast_encode
    g = np.random.default_rng(9)
    x = _bf16(g.standard_normal((40, 576)) * np.repeat(np.exp2(g.uniform(-20, 20, (40, 18))), 32, axis=1))
    x[3], x[4, :64], x[5] = 0, -0.0, _bf16(g.integers(-28, 29, 576) / 4)
    x[6] = 3.3e38
    x = _bf16(x)
    assert np.array_equal(fast_encode(x), ora.encode(x))
