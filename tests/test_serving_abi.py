"""Refusals of the serving-step entry points (norm, block-scaled product,
latent append, latent decode): host checks, no GPU needed."""
import ctypes
import os

import pytest
import torch

import mla_ragged_paged_gb300 as pkg
from mla_ragged_paged_gb300 import binding

F8, F32, U32 = binding.MLA_DTYPE_FP8_E4M3, binding.MLA_DTYPE_F32, binding.MLA_DTYPE_U32


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


def _norm(lib, **over):
    a = dict(out=_desc([4, 256]), out8=_desc([4, 256], F8), scales=_desc([4, 2], F32), x=_desc([4, 256]),
             res=_desc([4, 256]), res_out=_desc([4, 256]), w=_desc([256]), eps=1e-6)
    a.update(over)
    return lib.mla_rms_norm(_ref(a["out"]), _ref(a["out8"]), _ref(a["scales"]), _ref(a["x"]), _ref(a["res"]),
                            _ref(a["res_out"]), _ref(a["w"]), a["eps"], None)


@pytest.mark.parametrize("change", [
    dict(x=None), dict(w=None), dict(out=None, out8=None, scales=None), dict(out8=None), dict(scales=None),
    dict(res=None), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(x=_desc([4, 0])), dict(x=_desc([4, 32769])), dict(x=_desc([4, 256], F32)), dict(x=_desc([4, 256], ptr=0x10001)),
    dict(out=_desc([4, 255])), dict(out=_desc([3, 256])), dict(out8=_desc([4, 256])), dict(scales=_desc([4, 3], F32)),
    dict(scales=_desc([4, 2], F32, ptr=0x10002)), dict(scales=_desc([4, 2], F32, stride=[1, 1])),
    dict(out=_desc([4, 256], stride=[128, 1])), dict(out8=_desc([4, 256], F8, stride=[0, 1])),
    dict(res_out=_desc([4, 256], stride=[0, 1])), dict(x=_desc([4, 256], stride=[512, 2])),
    dict(w=_desc([255])), dict(w=_desc([256], F8)), dict(w=_desc([1, 256])), dict(res=_desc([4, 128])),
    dict(w=_desc([256], F32, ptr=0x10002)),
])
def test_norm_refuses(lib, change):
    assert _norm(lib, **change) == binding.MLA_ERR_INVALID_ARG
    assert lib.mla_last_error_string()


def _matmul(lib, **over):
    a = dict(out=_desc([5, 300]), x=_desc([5, 272], F8), xs=_desc([5, 3], F32), w=_desc([300, 272], F8),
             ws=_desc([3, 3], F32))
    a.update(over)
    return lib.mla_matmul_fp8(_ref(a["out"]), _ref(a["x"]), _ref(a["xs"]), _ref(a["w"]), _ref(a["ws"]), None, None)


@pytest.mark.parametrize("change", [
    dict(out=None), dict(x=None), dict(xs=None), dict(w=None), dict(ws=None),
    dict(out=_desc([5, 301])), dict(out=_desc([5, 300], F8)), dict(out=_desc([5, 300], stride=[299, 1])),
    dict(out=_desc([5, 300], ptr=0x10001)), dict(out=_desc([5, 300], F32, ptr=0x10002)),
    dict(x=_desc([5, 272])), dict(x=_desc([5, 256], F8)), dict(x=_desc([5, 272], F8, ptr=0x10008)),
    dict(x=_desc([5, 272], F8, stride=[280, 1])), dict(x=_desc([5, 272], F8, stride=[256, 1])),
    dict(w=_desc([300, 256], F8)), dict(w=_desc([300, 272], F8, ptr=0x10008)),
    dict(x=_desc([5, 264], F8), w=_desc([300, 264], F8)), dict(x=_desc([5, 0], F8), w=_desc([300, 0], F8)),
    dict(xs=_desc([5, 2], F32)), dict(xs=_desc([5, 3])), dict(xs=_desc([5, 3], F32, ptr=0x10002)),
    dict(xs=_desc([5, 3], F32, stride=[3, -1])), dict(ws=_desc([2, 3], F32)), dict(ws=_desc([3, 2], F32)),
    dict(w=_desc([0, 272], F8), out=_desc([5, 0]), ws=_desc([0, 3], F32)),
])
def test_matmul_refuses(lib, change):
    assert _matmul(lib, **change) == binding.MLA_ERR_INVALID_ARG
    assert lib.mla_last_error_string()


def _cache(shape=(8, 16, 576), **kw):
    kw = dict(dict(scale=0x50000, gran=binding.MLA_SCALE_PER_TOKEN), **kw)
    return _desc(list(shape), kw.pop("dtype", F8), **kw)


def _append(lib, **over):
    a = dict(cache=_cache(), rows=_desc([6, 576]), pt=_desc([2, 4], U32), ro=0x20000, cl=0x30000)
    a.update(over)
    return lib.mla_append_latent(_ref(a["cache"]), _ref(a["rows"]), _ref(a["pt"]), a["ro"], a["cl"], None, None)


@pytest.mark.parametrize("change", [
    dict(cache=None), dict(rows=None), dict(pt=None), dict(ro=None), dict(cl=None),
    dict(cache=_cache(scale=None)), dict(cache=_cache(gran=binding.MLA_SCALE_PER_TENSOR)),
    dict(cache=_cache(scale=0x50002)), dict(cache=_cache(dtype=binding.MLA_DTYPE_BF16)),
    dict(cache=_cache((8, 16, 512))), dict(cache=_cache((8, 16, 24)), rows=_desc([6, 24])),
    dict(cache=_cache((8, 16, 1040)), rows=_desc([6, 1040])), dict(cache=_cache((0, 16, 576))),
    dict(cache=_cache(ptr=0x10008)), dict(cache=_cache(stride=[16 * 584, 584, 1])),
    dict(cache=_cache(stride=[16 * 560, 560, 1])), dict(cache=_cache(stride=[576, 576, 1])),
    dict(cache=_cache((1 << 20, 1 << 12, 576))), dict(rows=_desc([6, 576], F8)),
    dict(rows=_desc([6, 576], ptr=0x10004)), dict(rows=_desc([6, 576], stride=[580, 1])),
    dict(pt=_desc([0, 4], U32)), dict(pt=_desc([2, 0], U32)), dict(pt=_desc([2, 4])),
])
def test_append_refuses(lib, change):
    assert _append(lib, **change) == binding.MLA_ERR_INVALID_ARG
    assert lib.mla_last_error_string()


def _decode(lib, **over):
    a = dict(out=_desc([6, 4, 512]), lse=_desc([6, 4], F32), q=_desc([6, 4, 576]), cache=_cache(),
             pt=_desc([2, 4], U32), ro=0x20000, cl=0x30000, scale=0.07, mask=0, ws=0x40000,
             ws_bytes=binding.decode_workspace_size())
    a.update(over)
    return lib.mla_decode_latent(_ref(a["out"]), _ref(a["lse"]), _ref(a["q"]), _ref(a["cache"]), _ref(a["pt"]),
                                 a["ro"], a["cl"], a["scale"], a["mask"], None, a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("change", [
    dict(out=None), dict(q=None), dict(cache=None), dict(pt=None), dict(ro=None), dict(cl=None), dict(ws=None),
    dict(out=_desc([6, 4, 576])), dict(out=_desc([6, 4, 512], F32)), dict(out=_desc([6, 4, 512], ptr=0x10008)),
    dict(out=_desc([6, 4, 512], stride=[2048, 516, 1])), dict(q=_desc([6, 4, 512])), dict(q=_desc([6, 3, 576])),
    dict(q=_desc([6, 4, 576], ptr=0x10004)), dict(q=_desc([6, 4, 576], stride=[2304, 580, 1])),
    dict(q=_desc([6, 0, 576]), out=_desc([6, 0, 512]), lse=None),
    dict(q=_desc([6, 1025, 576]), out=_desc([6, 1025, 512]), lse=None),
    dict(lse=_desc([6, 5], F32)), dict(lse=_desc([6, 4])), dict(lse=_desc([6, 4], F32, ptr=0x10002)),
    dict(cache=_cache((8, 16, 512))), dict(cache=_cache(scale=None)), dict(cache=_cache(gran=0)),
    dict(cache=_cache(dtype=binding.MLA_DTYPE_BF16)), dict(cache=_cache(ptr=0x10008)),
    dict(cache=_cache(stride=[17 * 576, 576, 1])), dict(cache=_cache(stride=[16 * 584, 584, 1])),
    dict(cache=_cache((0, 16, 576))), dict(cache=_cache((1 << 20, 1 << 12, 576))),
    dict(pt=_desc([2, 0], U32)), dict(pt=_desc([16385, 4], U32)),
    dict(q=_desc([1 << 29, 8, 576]), out=_desc([1 << 29, 8, 512]), lse=None), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(mask=7), dict(ws=0x40010), dict(ws_bytes=16),
])
def test_decode_refuses(lib, change):
    assert _decode(lib, **change) == binding.MLA_ERR_INVALID_ARG
    assert lib.mla_last_error_string()


@pytest.mark.parametrize("change", [
    dict(ro=0x20002), dict(cl=0x30001), dict(status=0x60002), dict(pt=_desc([2, 4], U32, ptr=0x10002)),
    dict(cache=_cache(scale=0x50001)),
    dict(out=_desc([6, 4, 512], stride=[2048, 0, 1])), dict(out=_desc([6, 4, 512], stride=[0, 512, 1])),
    dict(out=_desc([6, 4, 512], stride=[1024, 512, 1])), dict(out=_desc([6, 4, 512], stride=[512, 2560, 1])),
    dict(lse=_desc([6, 4], F32, stride=[0, 1])), dict(lse=_desc([6, 4], F32, stride=[3, 1])),
])
def test_decode_refuses_stray_addresses_and_shared_rows(lib, change):
    a = dict(dict(out=_desc([6, 4, 512]), lse=_desc([6, 4], F32), cache=_cache(), pt=_desc([2, 4], U32), ro=0x20000,
                  cl=0x30000, status=0x60000), **change)
    assert lib.mla_decode_latent(_ref(a["out"]), _ref(a["lse"]), _ref(_desc([6, 4, 576])), _ref(a["cache"]), _ref(a["pt"]),
                                 a["ro"], a["cl"], 0.07, 0, a["status"], 0x40000, binding.decode_workspace_size(),
                                 None) == binding.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("shape,stride", [([6, 4, 512], [512, 3200, 1]), ([1, 4, 512], [0, 512, 1]),
                                          ([6, 1, 512], [512, 0, 1]), ([6, 4, 512], [1 << 45, 1 << 40, 1])])
def test_decode_takes_rows_in_any_order(lib, shape, stride):
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    assert _decode(lib, out=_desc(shape, stride=stride), q=_desc([shape[0], shape[1], 576]),
                   lse=None) in (binding.MLA_ERR_UNSUPPORTED, binding.MLA_ERR_CUDA)


def test_append_and_matmul_refuse_stray_addresses(lib):
    for change in (dict(ro=0x20002), dict(cl=0x30001), dict(pt=_desc([2, 4], U32, ptr=0x10002))):
        assert _append(lib, **change) == binding.MLA_ERR_INVALID_ARG
    assert lib.mla_append_latent(_ref(_cache()), _ref(_desc([6, 576])), _ref(_desc([2, 4], U32)), 0x20000, 0x30000,
                                 0x60002, None) == binding.MLA_ERR_INVALID_ARG
    assert lib.mla_matmul_fp8(_ref(_desc([5, 300])), _ref(_desc([5, 272], F8)), _ref(_desc([5, 3], F32)),
                              _ref(_desc([300, 272], F8)), _ref(_desc([3, 3], F32)), 0x60002,
                              None) == binding.MLA_ERR_INVALID_ARG


def test_good_arguments_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    for call in (_norm, _matmul, _append, _decode):
        assert call(lib) in (binding.MLA_ERR_UNSUPPORTED, binding.MLA_ERR_CUDA)


def test_no_kernel_copies_by_multicast():
    """Ranks of multi-GPU jobs load the library: every copy lands in the CTA that issued it."""
    csrc = os.path.join(os.path.dirname(pkg.__file__), "csrc")
    for name in os.listdir(csrc):
        with open(os.path.join(csrc, name)) as f:
            assert "multicast" not in f.read(), name


def test_packed_descriptors_have_the_structs_layout():
    for n in range(1, 5):
        t = torch.zeros([3, 4, 5, 6][:n], dtype=torch.bfloat16).transpose(0, n - 1)
        raw = binding._pack(t, 1, 0x50000, 2)
        d = binding.MlaTensor.from_buffer_copy(raw)
        assert len(raw) == ctypes.sizeof(binding.MlaTensor)
        assert (d.data, d.dtype, d.ndim, d.scale, d.scale_gran) == (t.data_ptr(), 1, n, 0x50000, 2)
        assert list(d.shape)[:n] == list(t.shape) and list(d.stride)[:n] == list(t.stride())
    with pytest.raises(binding.MlaError):
        binding._pack(torch.zeros(()), 1)
    assert binding._pack(None, 1) is None


def test_binding_refuses_host_tensors_and_other_types(lib):
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(binding.MlaError):
        binding.rms_norm(x, x[0], 1e-6, out=x)
    with pytest.raises(binding.MlaError):
        binding.matmul_fp8(x, x, x, x, x)
    with pytest.raises(binding.MlaError):
        binding.append_latent(x, x, x, x, x, x)
    with pytest.raises(binding.MlaError):
        binding.decode_latent(x, x, x, x, x, x, x, 1.0)
    with pytest.raises(binding.MlaError):
        binding._typed(x, "x", torch.float32)
    with pytest.raises(binding.MlaError):
        binding._indices(torch.zeros(4, dtype=torch.int64), "row_offsets", 4)
    with pytest.raises(binding.MlaError):
        binding._indices(torch.zeros(4, dtype=torch.int32), "row_offsets", 5)
