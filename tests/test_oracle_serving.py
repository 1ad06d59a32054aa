"""Pins of oracle/serving.py against independent torch float64 forms (CPU)."""
import numpy as np
import pytest
import torch

from oracle import serving as ora
from serving_inputs import E4M3, LATENT, Decode, blocks, quantise_rows


@pytest.mark.parametrize("rows,dim", [(3, 1), (2, 130), (4, 512)])
def test_norm(rows, dim):
    g = torch.Generator().manual_seed(dim)
    x, r, w = (torch.randn(rows, dim, generator=g, dtype=torch.float64) for _ in range(3))
    w = w[0]
    h, y, s = ora.rms_norm(x.numpy(), w.numpy(), 1e-5, r.numpy())
    ref = torch.nn.functional.rms_norm(x + r, (dim,), w, 1e-5)
    assert np.allclose(h, (x + r).numpy(), rtol=0, atol=0)
    assert np.allclose(y, ref.numpy(), rtol=1e-12)
    pad = torch.nn.functional.pad(ref, (0, -dim % 128)).view(rows, -1, 128)
    assert np.allclose(s, (pad.abs().amax(2) / 448).numpy(), rtol=1e-12)


@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (3, 130, 144), (5, 257, 400)])
def test_matmul(m, n, k):
    g = torch.Generator().manual_seed(k)
    xc, xs = quantise_rows(torch.randn(m, k, generator=g), 128)
    wc, ws = blocks(n, k, g)
    out, mag = ora.matmul_fp8(xc.numpy(), xs.numpy(), wc.numpy(), ws.numpy())
    x, w = xc.view(E4M3).double(), wc.view(E4M3).double()
    ref = torch.zeros(m, n, dtype=torch.float64)
    for i in range(m):
        for j in range(n):
            for kb in range(-(-k // 128)):
                c = slice(128 * kb, 128 * kb + 128)
                ref[i, j] += xs[i, kb].double() * ws[j // 128, kb].double() * (x[i, c] * w[j, c]).sum()
    assert np.allclose(out, ref.numpy(), rtol=1e-11, atol=1e-11)
    assert (mag >= np.abs(out) - 1e-9).all()


@pytest.mark.parametrize("causal", [True, False])
def test_decode(causal):
    d = Decode([1, 3, 0, 2], [5, 0, 4, 17], heads=3, P=4, seed=5)
    out, lse, mag, _ = ora.decode(d.q.float().numpy(), d.codes.numpy(), d.scales.numpy(), d.table.numpy(), d.ro,
                                  d.prior, d.scale, causal)
    for b in range(4):
        L = d.n[b] + d.prior[b]
        c = torch.stack([d.codes[d.table[b, j // 4].long(), j % 4].view(E4M3).double()
                         * d.scales[d.table[b, j // 4].long(), j % 4].double() for j in range(L)])
        q = d.q[d.ro[b]:d.ro[b + 1]].double().transpose(0, 1)
        allowed = torch.ones(d.n[b], L, dtype=torch.bool)
        if causal:
            allowed = torch.arange(L)[None] <= d.prior[b] + torch.arange(d.n[b])[:, None]
        if d.n[b] == 0:
            continue
        x = (q @ c.T * d.scale).masked_fill(~allowed, float("-inf"))
        ref = torch.nn.functional.scaled_dot_product_attention(
            q, c.expand(3, -1, -1), c[:, :LATENT].expand(3, -1, -1), attn_mask=allowed, scale=d.scale)
        sel = slice(int(d.ro[b]), int(d.ro[b + 1]))
        assert np.allclose(out[sel], ref.transpose(0, 1).numpy(), rtol=1e-10, atol=1e-12)
        assert np.allclose(lse[sel], torch.logsumexp(x, 2).T.numpy(), rtol=1e-12)
        assert (mag[sel] >= np.abs(out[sel]) - 1e-12).all()


def test_append_places_every_row():
    g = torch.Generator().manual_seed(1)
    rows = torch.randn(5, 32, generator=g).to(torch.bfloat16)
    table = np.array([[2, 0], [3, 1]], dtype=np.int64)
    got = ora.append(rows.float().numpy(), table, [0, 2, 5], [1, 0], 2)
    assert sorted(got) == [0, 2, 5, 6, 7]
    assert np.array_equal(got[0][0], (rows[1].float() / torch.tensor(got[0][1])).numpy())
    assert np.abs(got[2][0]).max() <= 448.01
