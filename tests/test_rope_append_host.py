"""Host side of the rotating cache appends: refusals before anything is
enqueued, and the 64-bit model's e4m3 arithmetic (no GPU)."""
import numpy as np
import pytest

import fp8_model as M
from mla_decode_attention_07_gb300 import libmla


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return libmla.load()


def _call(lib, fp8, **kw):
    a = dict(kv=0x1000, kb=576, ks=576, q=0x2000, qb=64, qs=64, qh=64, o=0x3000, ob=64, os=64,
             oh=64, cache=0x4000, scales=0x5000, g=1, pages=4, bt=0x6000, max_pages=4, sl=0x7000,
             new=None, cs=0x8000, max_pos=256, il=1, batch=1, s_new=1, h=16)
    a.update(kw)
    lead = [a[k] for k in ("kv", "kb", "ks", "q", "qb", "qs", "qh", "o", "ob", "os", "oh", "cache")]
    tail = [a[k] for k in ("pages", "bt", "max_pages", "sl", "new", "cs", "max_pos", "il", "batch",
                           "s_new", "h")]
    if fp8:
        return lib.mla_rope_append_fp8(*lead, a["scales"], a["g"], *tail, None)
    return lib.mla_rope_append(*lead, *tail, None)


BAD = [
    dict(kv=None), dict(cache=None), dict(bt=None), dict(sl=None), dict(cs=None), dict(q=None),
    dict(o=None), dict(batch=0), dict(s_new=0), dict(h=0), dict(pages=0), dict(max_pages=0),
    dict(max_pos=0), dict(pages=1 << 25), dict(batch=1 << 16, s_new=1 << 15), dict(kv=0x1008),
    dict(cache=0x4008), dict(q=0x2008), dict(o=0x3004), dict(cs=0x8004), dict(bt=0x6002),
    dict(sl=0x7001), dict(new=0x9002), dict(kb=4), dict(ks=580), dict(ks=-576), dict(qh=60),
    dict(qs=-64), dict(ob=12), dict(oh=0), dict(oh=56), dict(s_new=2, os=0), dict(batch=2, ob=0),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", BAD, ids=str)
def test_rope_append_rejects_bad_args_on_host(lib, fp8, kw):
    assert _call(lib, fp8, **kw) == libmla.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(scales=None), dict(scales=0x5002), dict(g=0), dict(g=3),
                                dict(g=128), dict(g=-1)])
def test_rope_append_fp8_rejects_bad_scales_on_host(lib, kw):
    assert _call(lib, True, **kw) == libmla.MLA_ERR_INVALID_ARG


def test_rope_append_needs_a_device(lib):
    from conftest import gpu_available
    if gpu_available():
        pytest.skip("a GPU is present")
    for fp8 in (False, True):
        assert _call(lib, fp8) in (libmla.MLA_ERR_CUDA, libmla.MLA_ERR_UNSUPPORTED_DEVICE)


def test_binding_refuses_wrong_shapes():
    torch = pytest.importorskip("torch")
    kv = torch.zeros(2, 3, 576, dtype=torch.bfloat16)
    cache = torch.zeros(4, 64, 1, 576, dtype=torch.uint8)
    sc = torch.zeros(4, 4)
    bt, sl = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cs = torch.zeros(64, 64)
    q = torch.zeros(2, 3, 5, 64, dtype=torch.bfloat16)
    bad = [
        dict(kv=kv[..., :512]), dict(kv=kv.transpose(1, 2)), dict(q=q, o=None), dict(q=None, o=q),
        dict(q=q[:, :2], o=q[:, :2]), dict(q=q, o=q[..., :32]), dict(cs=cs[:, :32]),
        dict(cache=cache.to(torch.bfloat16)), dict(cache=cache[:, :32]), dict(sc=sc[:3]),
        dict(sc=torch.zeros(4, 3)), dict(sc=torch.zeros(4, 4, dtype=torch.float64)),
    ]
    for kw in bad:
        a = dict(kv=kv, cache=cache, sc=sc, cs=cs, q=q, o=q)
        a.update(kw)
        with pytest.raises(libmla.MlaError) as e:
            libmla.mla_rope_append_fp8(a["kv"], a["cache"], a["sc"], bt, sl, a["cs"], a["q"],
                                       a["o"], stream=0)
        assert e.value.code == libmla.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("fp8", [False, True])
def test_binding_refuses_wrong_types_and_tables(fp8):
    torch = pytest.importorskip("torch")
    bf, i32 = torch.bfloat16, torch.int32
    good = dict(kv=torch.zeros(2, 3, 576, dtype=bf), bt=torch.zeros(2, 2, dtype=i32),
                sl=torch.zeros(2, dtype=i32), cs=torch.zeros(64, 64), nl=torch.zeros(2, dtype=i32),
                q=torch.zeros(2, 3, 5, 64, dtype=bf), o=torch.zeros(2, 3, 5, 64, dtype=bf),
                cache=torch.zeros(4, 64, 1, 576, dtype=torch.uint8 if fp8 else bf))
    bad = [dict(kv=good["kv"].float()), dict(q=good["q"].float()), dict(o=good["o"].float()),
           dict(cs=good["cs"].to(bf)), dict(bt=good["bt"].long()), dict(bt=good["bt"][:1]),
           dict(bt=torch.zeros(2, 4, dtype=i32)[:, :2]), dict(sl=good["sl"].long()),
           dict(sl=good["sl"][:1]), dict(nl=good["nl"].long()), dict(nl=good["nl"][:1]),
           dict(cache=good["cache"].to(bf if fp8 else torch.uint8)),
           dict(cache=torch.zeros(4, 64, 1, 640, dtype=good["cache"].dtype)[..., :576])]
    for kw in bad:
        a = {**good, **kw}
        cache = (a["cache"], torch.zeros(4, 4)) if fp8 else (a["cache"],)
        with pytest.raises(libmla.MlaError) as e:
            (libmla.mla_rope_append_fp8 if fp8 else libmla.mla_rope_append)(
                a["kv"], *cache, a["bt"], a["sl"], a["cs"], a["q"], a["o"], new_lens=a["nl"],
                stream=0)
        assert e.value.code == libmla.MLA_ERR_INVALID_ARG


def test_model_e4m3_matches_torch():
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(vals, nan=999.0), np.nan_to_num(M.E4M3, nan=999.0))
    x = np.concatenate([np.linspace(-448, 448, 20001), np.linspace(-0.05, 0.05, 5001),
                        (M.E4M3[:0x7E] + M.E4M3[1:0x7F]) / 2]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = M.e4m3_codes(x)
    assert np.array_equal(M.E4M3[got], M.E4M3[want])


@pytest.mark.parametrize("fp8", [False, True])
def test_binding_refuses_host_tensors(lib, fp8):
    """Every tensor on the host, or one of them among tensors of a device, or
    one on another device."""
    from test_decode_fp8_host import OnDevice
    torch = pytest.importorskip("torch")
    bf, i32 = torch.bfloat16, torch.int32
    good = dict(kv_new=torch.zeros(2, 3, 576, dtype=bf),
                kv_cache=torch.zeros(4, 64, 1, 576, dtype=torch.uint8 if fp8 else bf),
                block_table=torch.zeros(2, 2, dtype=i32), cache_seqlens=torch.zeros(2, dtype=i32),
                cos_sin=torch.zeros(64, 64), q_rope=torch.zeros(2, 3, 5, 64, dtype=bf),
                q_out=torch.zeros(2, 3, 5, 64, dtype=bf), new_lens=torch.zeros(2, dtype=i32))
    if fp8:
        good["scales"] = torch.zeros(4, 4)
    fn = libmla.mla_rope_append_fp8 if fp8 else libmla.mla_rope_append
    for odd in [set(good)] + [{k} for k in good]:
        for other in (None, 1):
            if other and len(odd) > 1:
                continue
            a = {k: OnDevice(t, 0) if k not in odd else OnDevice(t, other) if other else t
                 for k, t in good.items()}
            with pytest.raises(libmla.MlaError, match="current CUDA device") as e:
                fn(**a, stream=0)
            assert e.value.code == libmla.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("fp8", [False, True])
def test_binding_refuses_types_of_the_same_size(lib, fp8):
    """Each tensor in every other type of as many bytes an element."""
    torch = pytest.importorskip("torch")
    bf, i32 = torch.bfloat16, torch.int32
    same = {1: [torch.int8, torch.float8_e5m2, torch.float8_e4m3fnuz], 2: [torch.float16, torch.int16],
            4: [torch.int32, torch.float32]}
    good = dict(kv_new=torch.zeros(2, 3, 576, dtype=bf),
                kv_cache=torch.zeros(4, 64, 1, 576, dtype=torch.uint8 if fp8 else bf),
                block_table=torch.zeros(2, 2, dtype=i32), cache_seqlens=torch.zeros(2, dtype=i32),
                cos_sin=torch.zeros(64, 64), q_rope=torch.zeros(2, 3, 5, 64, dtype=bf),
                q_out=torch.zeros(2, 3, 5, 64, dtype=bf), new_lens=torch.zeros(2, dtype=i32))
    needs = dict(kv_new="kv_new must be bf16", kv_cache="kv_cache must be", cos_sin="cos_sin must be fp32",
                 block_table="block_table must be int32", cache_seqlens="must be int32",
                 new_lens="must be int32", q_rope="bf16", q_out="bf16")
    if fp8:
        good["scales"], needs["scales"] = torch.zeros(4, 4), "scales must be fp32"
    fn = libmla.mla_rope_append_fp8 if fp8 else libmla.mla_rope_append
    for k, why in needs.items():
        for other in same[good[k].itemsize]:
            if other == good[k].dtype:
                continue
            with pytest.raises(libmla.MlaError, match=why) as e:
                fn(**{**good, k: good[k].view(other)}, stream=0)
            assert e.value.code == libmla.MLA_ERR_INVALID_ARG
    with pytest.raises(libmla.MlaError, match="current CUDA device"):
        fn(**good, stream=0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [
    dict(s_new=2, os=64, oh=64), dict(s_new=3, os=512, oh=64, h=16), dict(batch=2, ob=64, oh=64),
    dict(batch=2, s_new=2, ob=1024, os=1024), dict(batch=3, s_new=2, h=1, ob=64, os=128),
    dict(batch=2, s_new=1, h=2, ob=96, oh=64)], ids=str)
def test_rope_append_rejects_query_rows_on_one_another(lib, fp8, kw):
    """Strides of q_out that put two rows on the same elements."""
    assert _call(lib, fp8, **kw) == libmla.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [
    dict(s_new=2, os=1024, oh=64), dict(batch=2, s_new=3, ob=64 * 6 * 16, os=64, oh=64 * 6, qs=64),
    dict(batch=2, s_new=2, os=128 * 16, ob=64, oh=128),          # entries inside the heads
    dict(batch=1, s_new=2, ob=0, os=576 * 16, oh=576), dict(batch=4, s_new=1, os=0, ob=1024, oh=64),
    dict(batch=2, s_new=1, h=1, ob=64, oh=0, os=0)], ids=str)
def test_rope_append_takes_query_rows_in_any_order(lib, fp8, kw):
    from conftest import gpu_available
    if gpu_available():
        pytest.skip("the addresses are made up")
    assert _call(lib, fp8, **kw) in (libmla.MLA_ERR_CUDA, libmla.MLA_ERR_UNSUPPORTED_DEVICE)
