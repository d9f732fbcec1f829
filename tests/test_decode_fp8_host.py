"""Host side of the 8-bit-cache decode: refusals before anything is enqueued
(no GPU)."""
import ctypes

import pytest

from mla_decode_attention_07_gb300 import libmla


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return libmla.load()


def _call(lib, fn="mla_decode_fp8", **kw):
    a = dict(q=0x1000, kv=0x2000, sc=0x3000, g=1, pages=4, bt=0x4000, max_pages=4, sl=0x5000,
             batch=1, s_q=1, h_q=16, meta=0x6000, out=0x7000, lse=0x8000, scale=0.07, ws=0x9000,
             ws_bytes=1 << 30)
    a.update(kw)
    return getattr(lib, fn)(a["q"], a["kv"], a["sc"], a["g"], a["pages"], a["bt"], a["max_pages"],
                            a["sl"], a["batch"], a["s_q"], a["h_q"], a["meta"], a["out"], a["lse"],
                            ctypes.c_float(a["scale"]), a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("fn", ["mla_decode_fp8", "mla_decode_fp8_f32"])
@pytest.mark.parametrize("kw", [
    dict(q=None), dict(kv=None), dict(sc=None), dict(bt=None), dict(sl=None), dict(meta=None),
    dict(out=None), dict(lse=None), dict(g=0), dict(g=3), dict(g=128), dict(g=-2), dict(batch=0),
    dict(s_q=0), dict(s_q=9), dict(h_q=0), dict(h_q=129), dict(pages=0), dict(max_pages=0),
    dict(pages=1 << 25), dict(q=0x1008), dict(kv=0x2004), dict(sc=0x3002), dict(out=0x7008),
    dict(lse=0x8002), dict(bt=0x4001), dict(sl=0x5002), dict(meta=0x6004),
    dict(scale=float("nan")), dict(scale=0.0), dict(scale=-0.1), dict(batch=1 << 25, h_q=64),
], ids=str)
def test_decode_fp8_rejects_bad_args_on_host(lib, fn, kw):
    assert _call(lib, fn, **kw) == libmla.MLA_ERR_INVALID_ARG


def test_decode_fp8_plan_rejects_bad_args_on_host(lib):
    E = libmla.MLA_ERR_INVALID_ARG
    assert lib.mla_decode_fp8_plan(None, 1, 1, 16, 0x5000, 4096, None) == E
    assert lib.mla_decode_fp8_plan(0x4000, 1, 1, 0, 0x5000, 4096, None) == E
    assert lib.mla_decode_fp8_plan(0x4000, 1, 9, 16, 0x5000, 4096, None) == E
    assert lib.mla_decode_fp8_plan(0x4000, 1, 1, 16, 0x5004, 4096, None) == E
    assert lib.mla_decode_fp8_plan_size(0, 1, 16, 0) == 0
    assert lib.mla_decode_fp8_workspace_size(1, 1, 129, 0) == 0


def test_decode_fp8_needs_a_device(lib):
    from conftest import gpu_available
    if gpu_available():
        pytest.skip("a GPU is present")
    assert _call(lib) in (libmla.MLA_ERR_CUDA, libmla.MLA_ERR_UNSUPPORTED_DEVICE)
    assert lib.mla_decode_fp8_plan_size(1, 1, 16, 0) == 0
    with pytest.raises(libmla.MlaError):
        libmla.alloc_fp8_plan_and_workspace(1, 1, 16)


def test_decode_fp8_binding_refuses_wrong_types_and_tables(lib):
    torch = pytest.importorskip("torch")
    bf, i32 = torch.bfloat16, torch.int32
    good = dict(q=torch.zeros(2, 1, 5, 576, dtype=bf), kv_cache=torch.zeros(4, 64, 1, 576, dtype=torch.uint8),
                scales=torch.zeros(4, 4), block_table=torch.zeros(2, 2, dtype=i32),
                cache_seqlens=torch.zeros(2, dtype=i32), tile_meta=torch.zeros(4, dtype=i32),
                out=torch.zeros(2, 1, 5, 512, dtype=bf), lse=torch.zeros(2, 5, 1),
                workspace=torch.zeros(4), softmax_scale=0.07, stream=0)
    bad = [dict(q=good["q"].float()), dict(out=good["out"].float()), dict(lse=good["lse"].to(bf)),
           dict(kv_cache=good["kv_cache"].to(bf)), dict(scales=good["scales"].double()),
           dict(block_table=good["block_table"].long()), dict(block_table=good["block_table"][:1]),
           dict(block_table=torch.zeros(2, 4, dtype=i32)[:, :2]),
           dict(cache_seqlens=good["cache_seqlens"].long()), dict(cache_seqlens=good["cache_seqlens"][:1])]
    for kw in bad:
        with pytest.raises(libmla.MlaError) as e:
            libmla.mla_decode_fp8(**{**good, **kw})
        assert e.value.code == libmla.MLA_ERR_INVALID_ARG
    with pytest.raises(libmla.MlaError):
        libmla.mla_decode_fp8_f32(**good)                       # its out is fp32
    with pytest.raises(libmla.MlaError):
        libmla.mla_decode_fp8_plan(good["cache_seqlens"].long(), 1, 5, good["tile_meta"], stream=0)


class OnDevice:
    """A tensor as the compiled marshalling sees it, on a device of choice."""

    def __init__(self, t, device):
        self.t, self.device_index = t, device
        self.shape, self.dtype, self.itemsize, self.nbytes = tuple(t.shape), t.dtype, t.itemsize, t.nbytes

    def stride(self):
        return self.t.stride()

    def is_contiguous(self):
        return self.t.is_contiguous()

    def data_ptr(self):
        return self.t.data_ptr()

    def get_device(self):
        return self.device_index


def _decode_args(torch):
    bf, i32 = torch.bfloat16, torch.int32
    return dict(q=torch.zeros(2, 1, 5, 576, dtype=bf),
                kv_cache=torch.zeros(4, 64, 1, 576, dtype=torch.uint8), scales=torch.zeros(4, 4),
                block_table=torch.zeros(2, 2, dtype=i32), cache_seqlens=torch.zeros(2, dtype=i32),
                tile_meta=torch.zeros(4, dtype=i32), out=torch.zeros(2, 1, 5, 512, dtype=bf),
                lse=torch.zeros(2, 5, 1), workspace=torch.zeros(4))


def test_decode_fp8_binding_refuses_host_tensors(lib):
    """Every tensor on the host, or one of them among tensors of a device."""
    torch = pytest.importorskip("torch")
    good = _decode_args(torch)
    for host in [set(good)] + [{k} for k in good]:
        a = {k: t if k in host else OnDevice(t, 0) for k, t in good.items()}
        with pytest.raises(libmla.MlaError, match="current CUDA device") as e:
            libmla.mla_decode_fp8(**a, softmax_scale=0.07, stream=0)
        assert e.value.code == libmla.MLA_ERR_INVALID_ARG
    for a in ((good["cache_seqlens"], good["tile_meta"]),
              (OnDevice(good["cache_seqlens"], 0), good["tile_meta"]),
              (good["cache_seqlens"], OnDevice(good["tile_meta"], 0))):
        with pytest.raises(libmla.MlaError, match="current CUDA device"):
            libmla.mla_decode_fp8_plan(a[0], 1, 5, a[1], stream=0)


def test_decode_fp8_binding_refuses_two_devices(lib):
    torch = pytest.importorskip("torch")
    good = _decode_args(torch)
    for other in good:
        a = {k: OnDevice(t, int(k == other)) for k, t in good.items()}
        with pytest.raises(libmla.MlaError, match="current CUDA device"):
            libmla.mla_decode_fp8(**a, softmax_scale=0.07, stream=0)


def test_decode_fp8_binding_refuses_types_of_the_same_size(lib):
    """A type is more than its size: each tensor in every other type of as many
    bytes an element, on the device and else as it should be."""
    torch = pytest.importorskip("torch")
    same = {1: [torch.int8, torch.float8_e5m2, torch.float8_e4m3fnuz, torch.bool],
            2: [torch.float16, torch.int16], 4: [torch.int32, torch.float32]}
    good = _decode_args(torch)
    needs = dict(q="q must be bf16", kv_cache="kv_cache must be float8_e4m3fn or uint8",
                 scales="scales must be fp32", block_table="block_table must be int32",
                 cache_seqlens="must be int32", out="out must be", lse="lse must be fp32")
    for k, why in needs.items():
        for other in same[good[k].itemsize]:
            if other == good[k].dtype:
                continue
            a = {**{n: OnDevice(t, 0) for n, t in good.items()}, k: OnDevice(good[k].view(other), 0)}
            with pytest.raises(libmla.MlaError, match=why) as e:
                libmla.mla_decode_fp8(**a, softmax_scale=0.07, stream=0)
            assert e.value.code == libmla.MLA_ERR_INVALID_ARG
    with pytest.raises(libmla.MlaError, match="out must be"):        # its own type is fp32
        libmla.mla_decode_fp8_f32(**good, softmax_scale=0.07, stream=0)
    with pytest.raises(libmla.MlaError, match="must be int32"):
        libmla.mla_decode_fp8_plan(OnDevice(torch.zeros(2), 0), 1, 5, OnDevice(good["tile_meta"], 0),
                                   stream=0)
    # both types of codes reach the check of devices
    for codes in (good["kv_cache"], good["kv_cache"].view(torch.float8_e4m3fn)):
        with pytest.raises(libmla.MlaError, match="current CUDA device"):
            libmla.mla_decode_fp8(**{**good, "kv_cache": codes}, softmax_scale=0.07, stream=0)
