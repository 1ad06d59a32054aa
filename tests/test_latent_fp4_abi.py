"""Refusals of the 4-bit latent cache's entry points (norm and rotation, append,
gather, decode): host checks, no GPU needed."""
import ctypes

import pytest
import torch

import mla_ragged_paged_gb300 as pkg
from mla_ragged_paged_gb300 import binding

F8, F32, U32, BYTES = (binding.MLA_DTYPE_FP8_E4M3, binding.MLA_DTYPE_F32, binding.MLA_DTYPE_U32,
                       binding.MLA_DTYPE_BYTES)


@pytest.fixture(scope="module")
def lib():
    pkg.build()
    return binding.load()


def _desc(shape, dtype=binding.MLA_DTYPE_BF16, ptr=0x10000, stride=None, scale=None, gran=0):
    d = binding.MlaTensor()
    d.data, d.dtype, d.ndim = ptr, dtype, len(shape)
    step = 1
    for i in reversed(range(len(shape))):
        d.shape[i] = shape[i]
        d.stride[i] = step if stride is None else stride[i]
        step *= shape[i]
    d.scale, d.scale_gran = scale, gran
    return d


def _ref(d):
    return None if d is None else ctypes.addressof(d)


def test_row_bytes(lib):
    assert [binding.latent_fp4_row_bytes(w) for w in (64, 512, 576, 1024)] == [48, 272, 304, 544]
    assert [lib.mla_latent_fp4_row_bytes(w) for w in (0, 32, 63, 100, 1088, 1 << 31)] == [0] * 6
    for w in (0, -64, 100, 1 << 40):
        with pytest.raises(binding.MlaError):
            binding.latent_fp4_row_bytes(w)


# ------------------------------------------------------------------ norm and rotation

def _rope(lib, **over):
    a = dict(qo=_desc([6, 4, 192]), q=_desc([6, 4, 192]), qw=None, ko=_desc([6, 1, 576]), k=_desc([6, 1, 576]),
             kw=_desc([512]), eps=1e-6, pos=0x20000, f=_desc([32], F32), scale=1.0, flags=0)
    a.update(over)
    return lib.mla_norm_rope(_ref(a["qo"]), _ref(a["q"]), _ref(a["qw"]), _ref(a["ko"]), _ref(a["k"]), _ref(a["kw"]),
                             a["eps"], a["pos"], _ref(a["f"]), a["scale"], a["flags"], None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(q=None, qo=None, k=None, ko=None, kw=None),
    dict(k=None, ko=None), dict(q=None, qo=None, qw=_desc([192])),
    dict(q=_desc([6, 4, 192], F32)), dict(qo=_desc([6, 4, 192], F8)), dict(qo=_desc([6, 4, 128])),
    dict(qo=_desc([5, 4, 192])), dict(qo=_desc([6, 3, 192])), dict(q=_desc([24, 192]), qo=_desc([24, 192])),
    dict(q=_desc([7, 4, 192]), qo=_desc([7, 4, 192])), dict(q=_desc([6, 0, 192]), qo=_desc([6, 0, 192])),
    dict(q=_desc([6, 4, 1025]), qo=_desc([6, 4, 1025])), dict(q=_desc([6, 4, 62]), qo=_desc([6, 4, 62])),
    dict(q=_desc([6, 4, 192], ptr=0x10001)), dict(qo=_desc([6, 4, 192], ptr=0x10001)),
    dict(q=_desc([6, 4, 192], stride=[768, 192, 2])), dict(qo=_desc([6, 4, 192], stride=[768, 0, 1])),
    dict(qo=_desc([6, 4, 192], stride=[0, 192, 1])), dict(qo=_desc([6, 4, 192], stride=[700, 192, 1])),
    dict(qo=_desc([6, 4, 192], stride=[768, -192, 1])), dict(kw=_desc([0])), dict(kw=_desc([577])),
    dict(kw=_desc([512], F8)), dict(kw=_desc([1, 512])), dict(kw=_desc([512], F32, ptr=0x10002)),
    dict(kw=_desc([512], ptr=0x10001)), dict(kw=_desc([512], stride=[2])), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(pos=None), dict(pos=0x20002), dict(f=_desc([0], F32)), dict(f=_desc([97], F32)),
    dict(f=_desc([32])), dict(f=_desc([32], F32, ptr=0x10002)), dict(f=_desc([1, 32], F32)),
    dict(f=None), dict(f=None, kw=None), dict(scale=float("nan")), dict(scale=float("inf")), dict(flags=2),
    dict(q=_desc([1 << 30, 4, 192]), qo=_desc([1 << 30, 4, 192]), k=None, ko=None, kw=None),
])
def test_norm_rope_refuses(lib, change):
    assert _rope(lib, **change) == binding.MLA_ERR_INVALID_ARG
    assert lib.mla_last_error_string()


@pytest.mark.parametrize("change", [
    dict(), dict(q=None, qo=None), dict(k=None, ko=None, kw=None), dict(flags=1), dict(scale=-0.5),
    dict(f=None, pos=None, qw=_desc([192], F32)), dict(qo=_desc([6, 4, 192], stride=[192, 1152, 1])),
    dict(q=_desc([6, 4, 192], stride=[0, 0, 1])), dict(q=_desc([6, 4, 192], ptr=0x10002)),
    dict(f=_desc([96], F32)),
])
def test_norm_rope_takes(lib, change):
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    assert _rope(lib, **change) in (binding.MLA_ERR_UNSUPPORTED, binding.MLA_ERR_CUDA)


# ------------------------------------------------------------------ append, gather

def _cache(shape=(8, 16, 304), **kw):
    return _desc(list(shape), kw.pop("dtype", BYTES), **kw)


CACHES = [
    dict(cache=None), dict(cache=_cache(dtype=F8)), dict(cache=_cache((8, 16, 576))), dict(cache=_cache((8, 16, 320))),
    dict(cache=_cache((0, 16, 304))), dict(cache=_cache((8, 0, 304))), dict(cache=_cache(ptr=0x10008)),
    dict(cache=_cache(stride=[16 * 312, 312, 1])), dict(cache=_cache(stride=[16 * 288, 288, 1])),
    dict(cache=_cache(stride=[304, 304, 1])), dict(cache=_cache(stride=[304, 7 * 304, 1])),
    dict(cache=_cache(stride=[16 * 304, 304, 2])), dict(cache=_cache((1 << 20, 1 << 12, 304))),
    dict(cache=_desc([128, 304], BYTES)), dict(pt=None), dict(pt=_desc([0, 4], U32)), dict(pt=_desc([2, 0], U32)),
    dict(pt=_desc([2, 4])), dict(pt=_desc([2, 4], U32, ptr=0x10002)), dict(ro=None), dict(cl=None), dict(ro=0x20002),
    dict(cl=0x30001), dict(status=0x60002),
]


def _append(lib, **over):
    a = dict(cache=_cache(), rows=_desc([6, 576]), pt=_desc([2, 4], U32), ro=0x20000, cl=0x30000, status=None)
    a.update(over)
    return lib.mla_append_latent_fp4(_ref(a["cache"]), _ref(a["rows"]), _ref(a["pt"]), a["ro"], a["cl"], a["status"], None)


@pytest.mark.parametrize("change", CACHES + [
    dict(rows=None), dict(rows=_desc([6, 576], F8)), dict(rows=_desc([6, 512])), dict(rows=_desc([6, 560])),
    dict(rows=_desc([6, 1088]), cache=_cache((8, 16, 576))), dict(rows=_desc([6, 32]), cache=_cache((8, 16, 32))),
    dict(rows=_desc([6, 576], ptr=0x10008)), dict(rows=_desc([6, 576], stride=[580, 1])),
])
def test_append_refuses(lib, change):
    assert _append(lib, **change) == binding.MLA_ERR_INVALID_ARG
    assert lib.mla_last_error_string()


def _to8(shape=(6, 576), **kw):
    return _desc(list(shape), F8, **dict(dict(scale=0x50000, gran=binding.MLA_SCALE_PER_TOKEN), **kw))


def _gather(lib, **over):
    a = dict(dst=_desc([6, 576]), cache=_cache(), pt=_desc([2, 4], U32), ro=0x20000, cl=0x30000, status=None)
    a.update(over)
    return lib.mla_gather_latent_fp4(_ref(a["dst"]), _ref(a["cache"]), _ref(a["pt"]), a["ro"], a["cl"], a["status"], None)


@pytest.mark.parametrize("change", CACHES + [
    dict(dst=None), dict(dst=_desc([6, 576], F32)), dict(dst=_desc([6, 512])), dict(dst=_desc([6, 576], ptr=0x10008)),
    dict(dst=_desc([6, 576], stride=[580, 1])), dict(dst=_desc([6, 576], stride=[568, 1])),
    dict(dst=_desc([6, 576], stride=[0, 1])), dict(dst=_to8(scale=None)), dict(dst=_to8(scale=0x50002)),
    dict(dst=_to8(gran=binding.MLA_SCALE_PER_TENSOR)), dict(dst=_to8(ptr=0x10008)), dict(dst=_to8(stride=[584, 1])),
])
def test_gather_refuses(lib, change):
    assert _gather(lib, **change) == binding.MLA_ERR_INVALID_ARG
    assert lib.mla_last_error_string()


# ------------------------------------------------------------------ attention

def _decode(lib, **over):
    a = dict(out=_desc([6, 4, 512]), lse=_desc([6, 4], F32), q=_desc([6, 4, 576]), cache=_cache(),
             pt=_desc([2, 4], U32), ro=0x20000, cl=0x30000, scale=0.07, mask=0, status=None, ws=0x40000,
             ws_bytes=binding.decode_workspace_size())
    a.update(over)
    return lib.mla_decode_latent_fp4(_ref(a["out"]), _ref(a["lse"]), _ref(a["q"]), _ref(a["cache"]), _ref(a["pt"]),
                                     a["ro"], a["cl"], a["scale"], a["mask"], a["status"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("change", CACHES + [
    dict(out=None), dict(q=None), dict(ws=None), dict(ws=0x40010), dict(ws_bytes=16),
    dict(out=_desc([6, 4, 576])), dict(out=_desc([6, 4, 512], F32)), dict(out=_desc([6, 4, 512], ptr=0x10008)),
    dict(out=_desc([6, 4, 512], stride=[2048, 516, 1])), dict(out=_desc([6, 4, 512], stride=[2048, 0, 1])),
    dict(out=_desc([6, 4, 512], stride=[1024, 512, 1])), dict(q=_desc([6, 4, 512])), dict(q=_desc([6, 3, 576])),
    dict(q=_desc([6, 4, 576], ptr=0x10004)), dict(q=_desc([6, 4, 576], stride=[2304, 580, 1])),
    dict(q=_desc([6, 0, 576]), out=_desc([6, 0, 512]), lse=None),
    dict(q=_desc([6, 1025, 576]), out=_desc([6, 1025, 512]), lse=None),
    dict(lse=_desc([6, 5], F32)), dict(lse=_desc([6, 4])), dict(lse=_desc([6, 4], F32, ptr=0x10002)),
    dict(lse=_desc([6, 4], F32, stride=[0, 1])), dict(pt=_desc([16385, 4], U32)),
    dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(mask=7),
    dict(cache=_cache(stride=[17 * 304, 304, 1])), dict(cache=_cache(stride=[304, 8 * 304, 1])),
])
def test_decode_refuses(lib, change):
    assert _decode(lib, **change) == binding.MLA_ERR_INVALID_ARG
    assert lib.mla_last_error_string()


def test_good_arguments_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    later = (binding.MLA_ERR_UNSUPPORTED, binding.MLA_ERR_CUDA)
    for call in (_append, _gather, _decode):
        assert call(lib) in later
        assert call(lib, cache=_cache(stride=[16 * 320, 320, 1])) in later       # padded rows
    for call in (_append, _gather):
        assert call(lib, cache=_cache(stride=[17 * 320, 320, 1])) in later       # padded pages too
        assert call(lib, cache=_cache(stride=[304, 8 * 304, 1])) in later        # slots outside, pages inside
    for call in (_append, _gather, _decode):
        assert call(lib, cache=_cache((1, 1, 304), stride=[0, 0, 1])) in later
    assert _gather(lib, dst=_to8()) in later
    assert _gather(lib, dst=_desc([0, 576], ptr=0)) in later


def test_binding_refuses_host_tensors_and_other_types(lib):
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    for call in (lambda: binding.norm_rope(None, None, q=x, q_out=x), lambda: binding.norm_rope(None, None),
                 lambda: binding.append_latent_fp4(x, x, x, x, x), lambda: binding.gather_latent_fp4(x, x, x, x, x),
                 lambda: binding.decode_latent_fp4(x, x, x, x, x, x, 1.0)):
        with pytest.raises(binding.MlaError):
            call()
