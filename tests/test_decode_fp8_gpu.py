"""MLA decode over the 8-bit cache on the GPU against the 64-bit model, whose
bounds follow from the arithmetic (fp8_model.decode); the bf16 output is the
fp32 output rounded to nearest even, bit for bit."""
import numpy as np
import pytest

import fp8_model as M
import plan_model
from mla_decode_attention_07_gb300 import libmla
from mla_decode_attention_07_gb300 import workloads as W
from test_parity_gpu import assert_bf16_is_rounded_f32

pytestmark = pytest.mark.gpu
SCALE = 192.0 ** -0.5


@pytest.fixture(scope="module")
def torch_cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch


class Inputs:
    """Seeded inputs; what an entry must not use holds NaN codes, NaN or
    infinite scales and block-table entries outside the pool."""

    def __init__(self, seed, s_q, h_q, lens, G, spread=0.5, q_scale=1.0):
        self.s_q, self.h_q, self.G = s_q, h_q, G
        self.lens = np.asarray(lens, dtype=np.int32)
        B = len(lens)
        per = [(int(n) + 63) // 64 for n in lens]
        self.pages = sum(per) + 2
        perm = W.permutation(seed, 1, self.pages)
        self.bt = np.full((B, max(max(per), 1)), self.pages, dtype=np.int32)
        k = 0
        for b, p in enumerate(per):
            self.bt[b, :p] = perm[k:k + p]
            k += p
        x = W.bf16_bits_to_float32(W.normal_bf16(seed, 2, self.pages * 64 * 576)).astype(np.float64)
        x = x.reshape(self.pages, 64 // G, G * 576)
        z = W.splitmix64(seed ^ 77, 0, self.pages * (64 // G))
        u = (z >> np.uint64(11)).astype(np.float64) * 2.0 ** -53 - 0.5
        x *= np.exp2(2 * spread * u).reshape(self.pages, 64 // G, 1)
        self.scales = (np.abs(x).max(-1) / 448).astype(np.float32)
        self.codes = M.e4m3_codes(x / self.scales[..., None]).reshape(self.pages, 64, 1, 576)
        self.q = (W.bf16_bits_to_float32(W.normal_bf16(seed, 3, B * s_q * h_q * 576))
                  .reshape(B, s_q, h_q, 576) * np.float32(q_scale))
        self.q = W.bf16_bits_to_float32(W.float32_to_bf16_bits(self.q))
        self.codes_gpu, self.scales_gpu = self.codes.copy(), self.scales.copy()
        used = np.zeros(self.pages * 64, dtype=bool)
        for b in range(B):
            t = np.arange(int(lens[b]))
            used[self.bt[b, t // 64] * 64 + t % 64] = True
        used = used.reshape(self.pages, 64)
        self.codes_gpu[~used] = 0x7F
        dead = ~used.reshape(self.pages, 64 // G, G).any(-1)
        self.scales_gpu[dead] = np.where(np.arange(int(dead.sum())) % 2, np.nan, np.inf)

    def model(self):
        return M.decode(self.q, self.codes, self.scales, self.bt, self.lens, SCALE)


def to_gpu(torch, x):
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return dict(q=t(x.q).to(torch.bfloat16), codes=t(x.codes_gpu), scales=t(x.scales_gpu),
                bt=t(x.bt), lens=t(x.lens))


def run(torch, x, f32=False, d=None, check=True):
    d = d or to_gpu(torch, x)
    B = len(x.lens)
    out = torch.full((B, x.s_q, x.h_q, 512), float("nan"),
                     dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    lse = torch.full((B, x.h_q, x.s_q), float("nan"), dtype=torch.float32, device="cuda")
    meta, ws = libmla.alloc_fp8_plan_and_workspace(B, x.s_q, x.h_q)
    ws.fill_(float("nan"))
    libmla.mla_decode_fp8_plan(d["lens"], x.s_q, x.h_q, meta)
    fn = libmla.mla_decode_fp8_f32 if f32 else libmla.mla_decode_fp8
    fn(d["q"], d["codes"], d["scales"], d["bt"], d["lens"], meta, out, lse, SCALE, ws)
    rc = libmla.mla_check_device_error()
    if check:
        assert rc == 0, libmla.mla_strerror(rc)
    return out.float().cpu().numpy(), lse.cpu().numpy(), rc


def compare(x, out, lse, bars=False):
    ref, rl, otol, ltol = x.model()
    assert not np.isnan(out).any() and not np.isnan(lse).any()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty)
    el = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, rl))
    assert np.all(el <= ltol), f"lse: {np.max(el - ltol):.3e} past its bound, {el.max():.3e} off"
    eo = np.abs(out - ref)
    assert np.all(eo <= otol), f"out: {np.max(eo - otol):.3e} past its bound, {eo.max():.3e} off"
    if bars:      # the bf16 decode's fixed bars, far inside those worst cases
        assert eo.max() <= 1e-2 and el.max() <= 1e-3, f"out {eo.max():.3e}, lse {el.max():.3e}"


ragged = lambda seed, n, lo, hi: list(W.uniform_int(seed, W.TENSOR_SEQLENS, n, lo, hi))
CASES = [
    # seed, s_q, h_q, lengths, tokens to a scale
    (1, 1, 16, [64], 1),                       # one whole page
    (2, 1, 1, [1], 1),                         # one token, one head
    (3, 1, 16, [256, 63, 65, 1], 1),
    (4, 1, 32, [200, 64], 16),
    (5, 1, 64, [130, 511], 64),
    (6, 1, 128, [300, 90], 1),                 # two tiles
    (7, 2, 128, [1, 127, 300], 2),             # four tiles, rows that see nothing
    (8, 8, 128, [5, 700], 4),                  # sixteen tiles
    (9, 8, 5, [3, 200, 64], 8),                # 40 rows of 64
    (10, 3, 7, [1000, 2], 32),                 # 21 rows of 32
    (11, 2, 3, [77, 0, 400], 1),               # 6 rows of 16, an empty entry
    (12, 1, 100, [333, 90, 1], 16),            # the second tile has 36 rows
    (13, 1, 16, [20000], 1),                   # split over every CTA
    (14, 1, 64, [9000, 10], 64),
    (15, 1, 128, [5000], 1),
    (16, 1, 16, ragged(16, 300, 1, 64), 1),    # many one-page entries
    (17, 1, 33, ragged(17, 170, 0, 200), 4),
    (18, 1, 16, [0, 0], 1),                    # nothing at all
    (19, 1, 64, ragged(19, 40, 1500, 3000), 1),   # several long entries a CTA, 64 rows
    (20, 1, 16, ragged(20, 250, 200, 900), 1),    # the same with 16 rows
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"s{c[0]}_sq{c[1]}_h{c[2]}_g{c[4]}")
def test_decode_fp8(torch_cuda, case):
    x = Inputs(*case)
    d = to_gpu(torch_cuda, x)
    out32, lse32, _ = run(torch_cuda, x, f32=True, d=d)
    compare(x, out32, lse32, bars=True)
    out16, lse16, _ = run(torch_cuda, x, d=d)
    assert np.array_equal(lse16, lse32)
    assert_bf16_is_rounded_f32(out16, out32)


@pytest.mark.parametrize("h_q", [16, 32, 64])
def test_decode_fp8_scales_far_apart(torch_cuda, h_q):
    """Scales over 2^40: the running maximum is that of p c, not of p."""
    x = Inputs(31, 1, h_q, [700, 1500], 1, spread=20.0, q_scale=2.0 ** -10)
    compare(x, *run(torch_cuda, x, f32=True)[:2])


def test_decode_fp8_sharp_and_flat(torch_cuda):
    """Scores of +-100 (the maximum moves often) and of almost nothing."""
    for q_scale in (12.0, 1e-3):
        for h_q in (16, 32, 64):
            x = Inputs(32, 2, h_q, [1500, 640], 16, q_scale=q_scale)
            compare(x, *run(torch_cuda, x, f32=True)[:2])


def test_decode_fp8_rising_scores(torch_cuda):
    """Every page raises the maximum: O and the sums are rescaled each time."""
    for h_q in (5, 32, 64):
        x = Inputs(33, 1, h_q, [64 * 12 + 5], 1)
        x.q[:] = np.abs(x.q)
        t = np.arange(64 * 12 + 5)
        rise = (t / 64.0).astype(np.float32)
        x.codes[x.bt[0, t // 64], t % 64, 0] &= 0x7F         # all positive: scores grow with c
        x.scales[x.bt[0, t // 64], t % 64] = 0.002 * (1 + rise)
        x.codes_gpu[x.bt[0, t // 64], t % 64] = x.codes[x.bt[0, t // 64], t % 64]
        x.scales_gpu[x.bt[0, t // 64], t % 64] = x.scales[x.bt[0, t // 64], t % 64]
        compare(x, *run(torch_cuda, x, f32=True)[:2])


def test_decode_fp8_zero_rows_and_zero_scales(torch_cuda):
    x = Inputs(34, 1, 16, [100], 1)
    for t in range(0, 100, 3):
        x.scales[x.bt[0, t // 64], t % 64] = (0.0, 2.0 ** -100)[t % 2]
        x.scales_gpu[x.bt[0, t // 64], t % 64] = (0.0, 2.0 ** -100)[t % 2]
    x.q[0, 0, 3] = 0.0
    compare(x, *run(torch_cuda, x, f32=True)[:2])


def test_decode_fp8_query_outliers(torch_cuda):
    """A query element 2^12 times the others."""
    x = Inputs(35, 1, 20, [300], 1, q_scale=2.0 ** -6)
    x.q[..., 100] *= 4096.0
    compare(x, *run(torch_cuda, x, f32=True)[:2])


@pytest.mark.parametrize("length", [130, 5000])                 # 5000: many splits
@pytest.mark.parametrize("h_q", [8, 16, 64])
def test_decode_fp8_infinite_query(torch_cuda, h_q, length):
    """An infinity or a NaN in a query row makes that row NaN, or leaves it
    empty where it sees no key; the other rows keep their bits."""
    x = Inputs(44, 2, h_q, [1, length], 1)
    clean = run(torch_cuda, x)
    x.q[0, 0, 1, 7] = np.inf                                    # sees no key
    x.q[1, 0, 3, 5], x.q[1, 0, 4, 575], x.q[1, 1, 2, 570] = np.inf, -np.inf, np.nan
    out, lse, _ = run(torch_cuda, x)
    for i, h in ((0, 3), (0, 4), (1, 2)):
        assert np.isnan(out[1, i, h]).all() and np.isnan(lse[1, h, i])
        out[1, i, h], lse[1, h, i] = clean[0][1, i, h], clean[1][1, h, i]
    assert np.array_equal(out, clean[0]) and np.array_equal(lse, clean[1])
    assert np.all(out[0, 0] == 0) and np.all(np.isneginf(lse[0, :, 0]))


def test_decode_fp8_same_bits_again(torch_cuda):
    for h_q, lens in ((16, [3000, 900]), (128, [3000, 900])):
        x = Inputs(36, 1, h_q, lens, 1)
        d = to_gpu(torch_cuda, x)
        a, b = run(torch_cuda, x, d=d), run(torch_cuda, x, d=d)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_decode_fp8_scales_by_block_are_scales_by_token(torch_cuda):
    """A cache with one scale a page gives the bits of the same cache with the
    scale written out for each token."""
    x = Inputs(37, 1, 32, [500, 70], 64)
    d = to_gpu(torch_cuda, x)
    a = run(torch_cuda, x, d=d)
    d["scales"] = d["scales"].repeat_interleave(64, 1).contiguous()
    b = run(torch_cuda, x, d=d)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_decode_fp8_bad_page_and_wrong_plan_are_flagged(torch_cuda):
    torch, x = torch_cuda, Inputs(38, 1, 16, [300], 1)
    d = to_gpu(torch, x)
    d["bt"][0, 2] = x.pages
    libmla.mla_check_device_error()
    assert run(torch, x, d=d, check=False)[2] == libmla.MLA_ERR_DEVICE_BOUNDS
    d = to_gpu(torch, x)
    out = torch.zeros(1, 1, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(1, 16, 1, dtype=torch.float32, device="cuda")
    meta, ws = libmla.alloc_fp8_plan_and_workspace(1, 1, 16)
    libmla.mla_decode_plan(d["lens"], 1, 16, meta)           # the other kernel's plan
    libmla.mla_decode_fp8(d["q"], d["codes"], d["scales"], d["bt"], d["lens"], meta, out, lse,
                          SCALE, ws)
    assert libmla.mla_check_device_error() == libmla.MLA_ERR_PLAN


def test_decode_fp8_refuses_on_host(torch_cuda):
    torch, x = torch_cuda, Inputs(39, 1, 16, [100], 4)
    d = to_gpu(torch, x)
    out = torch.zeros(1, 1, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(1, 16, 1, dtype=torch.float32, device="cuda")
    meta, ws = libmla.alloc_fp8_plan_and_workspace(1, 1, 16)
    good = dict(q=d["q"], kv_cache=d["codes"], scales=d["scales"], block_table=d["bt"],
                cache_seqlens=d["lens"], tile_meta=meta, out=out, lse=lse, softmax_scale=SCALE,
                workspace=ws)
    for kw, code in [(dict(workspace=ws[:64]), libmla.MLA_ERR_WORKSPACE),
                     (dict(scales=d["scales"][:1]), libmla.MLA_ERR_INVALID_ARG),
                     (dict(out=out[..., :256]), libmla.MLA_ERR_INVALID_ARG),
                     (dict(q=d["q"].expand(2, 1, 16, 576)), libmla.MLA_ERR_INVALID_ARG),
                     (dict(softmax_scale=float("inf")), libmla.MLA_ERR_INVALID_ARG)]:
        with pytest.raises(libmla.MlaError) as e:
            libmla.mla_decode_fp8(**{**good, **kw})
        assert e.value.code == code
    with pytest.raises(libmla.MlaError) as e:
        libmla.mla_decode_fp8_plan(d["lens"], 1, 16, meta[:8])
    assert e.value.code == libmla.MLA_ERR_WORKSPACE


def test_decode_fp8_two_graphs_on_two_streams(torch_cuda):
    """Captured calls with workspaces of their own, replayed together."""
    torch = torch_cuda
    jobs = []
    for seed, h_q, lens in ((40, 16, [4000, 200]), (41, 128, [900, 2500])):
        x = Inputs(seed, 1, h_q, lens, 1)
        d = to_gpu(torch, x)
        ref = run(torch, x, d=d)
        out = torch.zeros(2, 1, h_q, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(2, h_q, 1, dtype=torch.float32, device="cuda")
        meta, ws = libmla.alloc_fp8_plan_and_workspace(2, 1, h_q)
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            libmla.mla_decode_fp8_plan(d["lens"], 1, h_q, meta)
            libmla.mla_decode_fp8(d["q"], d["codes"], d["scales"], d["bt"], d["lens"], meta, out,
                                  lse, SCALE, ws)
        jobs.append((graph, side, out, lse, ref, d, meta, ws))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, side, *_ in jobs:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    assert libmla.mla_check_device_error() == 0
    for _, _, out, lse, ref, *_ in jobs:
        assert np.array_equal(out.float().cpu().numpy(), ref[0])
        assert np.array_equal(lse.cpu().numpy(), ref[1])


@pytest.mark.parametrize("G", [1, 16])
def test_decode_step_append_absorb_attend(torch_cuda, G):
    """The run of calls of a decode step: rotate and append in 8 bits, absorb
    the query into the same 576-wide rows, attend; against the 64-bit model on
    the cache the append left."""
    torch = torch_cuda
    B, s_q, h = 3, 2, 16
    x = Inputs(42, s_q, h, [130, 66, 2], G)
    x.codes_gpu[x.codes_gpu == 0x7F] = 0                       # the new tokens' pages are fresh
    x.scales_gpu[~np.isfinite(x.scales_gpu)] = 1.0
    d = to_gpu(torch, x)
    p = W.make_prologue_inputs(43, B, s_q, h, [130, 66, 2])
    bf = lambda a: torch.from_numpy(np.ascontiguousarray(a.view(np.int16))).cuda().view(torch.bfloat16)
    kv_new, q_rope = bf(p.kv_new), bf(p.q_rope)
    a = np.arange(130)[:, None] * 10000.0 ** (-np.arange(32) / 32.0)
    cs = torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()
    turned = torch.empty_like(q_rope)
    libmla.mla_rope_append_fp8(kv_new, d["codes"], d["scales"], d["bt"], d["lens"], cs, q_rope, turned)
    libmla.mla_q_absorb(bf(p.q_nope), turned, bf(p.w_uk), d["q"])
    out, lse, _ = run(torch, x, f32=True, d=d)
    x.q = d["q"].float().cpu().numpy()
    x.codes, x.scales = d["codes"].cpu().numpy(), d["scales"].cpu().numpy()
    compare(x, out, lse)
    # the turned part of the query and the newest cache row, from the formula
    want, mag = M.rotated(W.bf16_bits_to_float32(p.q_rope)[0, 1], cs.cpu().numpy()[129], True)
    assert np.all(np.abs(x.q[0, 1, :, 512:] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * mag)
    row = M.dequant(x.codes, x.scales)[x.bt[0, 129 // 64], 129 % 64, 0]
    new = W.bf16_bits_to_float32(p.kv_new)[0, 1].astype(np.float64)
    new[512:] = M.rotated(new[512:], cs.cpu().numpy()[129], True)[0]
    size = np.abs(x.scales).max()
    assert np.all(np.abs(row - new) <= np.maximum(2.0 ** -4 * np.abs(new), 2.0 ** -10 * size) * 1.01)


@pytest.mark.parametrize("h", [16, 128])
def test_decode_steps_back_to_back(torch_cuda, h):
    """Steps of a decode loop (lengths, append, plan, attend) on a side stream
    with one plan and workspace and no host synchronisation between them: the
    bits of the same steps with one after every call."""
    torch, B, steps = torch_cuda, 24, 5
    final = ragged(45, B, steps, 900)
    x = Inputs(45, 1, h, final, 16)
    bf = lambda t, *s: torch.from_numpy(W.bf16_bits_to_float32(
        W.normal_bf16(46, t, int(np.prod(s)))).reshape(s)).cuda().bfloat16()
    kv_new, q_rope = bf(1, steps, B, 1, 576), bf(2, steps, B, 1, h, 64)
    a = np.arange(1000)[:, None] * 10000.0 ** (-np.arange(32) / 32.0)
    cs = torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()
    got = []
    for sync in (True, False):
        d = to_gpu(torch, x)
        d["lens"] -= steps
        out = torch.zeros(steps, B, 1, h, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(steps, B, h, 1, dtype=torch.float32, device="cuda")
        meta, ws = libmla.alloc_fp8_plan_and_workspace(B, 1, h)
        wait = torch.cuda.synchronize if sync else (lambda: None)
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            for i in range(steps):
                d["lens"] += 1
                wait()
                libmla.mla_rope_append_fp8(kv_new[i], d["codes"], d["scales"], d["bt"], d["lens"], cs,
                                           q_rope[i], d["q"][..., 512:])
                wait()
                libmla.mla_decode_fp8_plan(d["lens"], 1, h, meta)
                wait()
                libmla.mla_decode_fp8(d["q"], d["codes"], d["scales"], d["bt"], d["lens"], meta,
                                      out[i], lse[i], SCALE, ws)
                wait()
        torch.cuda.synchronize()
        assert libmla.mla_check_device_error() == 0
        got.append([t.cpu() for t in (out.float(), lse, d["codes"], d["scales"])])
    assert torch.isfinite(got[0][0]).all()
    for one, other in zip(*got):
        assert torch.equal(one.nan_to_num(7.0) if one.is_floating_point() else one,
                           other.nan_to_num(7.0) if other.is_floating_point() else other)


@pytest.mark.parametrize("h", [16, 128])
def test_decode_fp8_pages_past_4_gb(torch_cuda, h):
    """The pages at the end of a pool of 4.4 GB: the bits of a small pool."""
    torch = torch_cuda
    x = Inputs(47, 1, h, [200, 64, 700], 4)
    d = to_gpu(torch, x)
    ref = run(torch, x, d=d)
    pool = 120000
    codes = torch.full((pool, 64, 1, 576), 0x7F, dtype=torch.uint8, device="cuda")
    scales = torch.full((pool, 16), float("nan"), device="cuda")
    codes[pool - x.pages:], scales[pool - x.pages:] = d["codes"], d["scales"]
    far = dict(d, codes=codes, scales=scales, bt=d["bt"] + (pool - x.pages))
    out, lse, _ = run(torch, x, d=far)
    assert np.array_equal(out, ref[0]) and np.array_equal(lse, ref[1])


def test_decode_fp8_thousands_of_entries(torch_cuda):
    """More entries than the planner keeps in shared memory, a hundredth of them
    empty, some split."""
    lens = ragged(48, 4500, 1, 40)
    for i in range(0, 4500, 100):
        lens[i] = 0
    lens[77], lens[4400] = 9000, 5000
    x = Inputs(48, 1, 4, lens, 8)
    compare(x, *run(torch_cuda, x, f32=True)[:2])


def test_decode_fp8_replayed_with_other_lengths(torch_cuda):
    """A captured plan and decode, replayed on a stream of its own after the
    lengths changed in place; two entries share their first page."""
    torch = torch_cuda
    x = Inputs(49, 1, 64, [900, 640, 100], 16)
    x.bt[1, 0] = x.bt[0, 0]
    x.codes_gpu[:], x.scales_gpu[:] = x.codes, x.scales
    d, side = to_gpu(torch, x), torch.cuda.Stream()
    out = torch.zeros(3, 1, 64, 512, dtype=torch.float32, device="cuda")
    lse = torch.zeros(3, 64, 1, dtype=torch.float32, device="cuda")
    meta, ws = libmla.alloc_fp8_plan_and_workspace(3, 1, 64)
    call = lambda: (libmla.mla_decode_fp8_plan(d["lens"], 1, 64, meta, stream=side),
                    libmla.mla_decode_fp8_f32(d["q"], d["codes"], d["scales"], d["bt"], d["lens"],
                                              meta, out, lse, SCALE, ws, stream=side))
    torch.cuda.synchronize()
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for lens in ([900, 640, 100], [1, 0, 99], [64, 577, 37]):
        x.lens[:] = lens
        with torch.cuda.stream(side):
            d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
            graph.replay()
        torch.cuda.synchronize()
        assert libmla.mla_check_device_error() == 0
        compare(x, out.cpu().numpy(), lse.cpu().numpy())


@pytest.mark.parametrize("h, lens", [(4, [40000]), (16, [20000, 30, 0]), (32, [12000, 9000]),
                                     (64, [20000]), (128, [6000])])
def test_decode_fp8_many_splits(torch_cuda, h, lens):
    """Long entries split over all the workers: 16 warps merge an entry's splits."""
    x = Inputs(50 + h, 1, h, lens, 16)
    out, lse, _ = run(torch_cuda, x, f32=True)
    compare(x, out, lse, bars=True)


@pytest.mark.parametrize("other", ["bf16", "heads", "batch", "none"])
@pytest.mark.parametrize("h, lens", [(16, [300]), (128, [5000, 70]), (5, [40] * 300)])
def test_decode_fp8_plan_of_another_call_leaves_outputs(torch_cuda, other, h, lens):
    """A plan made for another call, and so shorter than this one's: what lies
    behind it (here numbers that pass for split counts) is not used, the call is
    reported, and out and lse stay as they were."""
    torch, x = torch_cuda, Inputs(51, 1, h, lens, 1)
    d, B, lib = to_gpu(torch, x), len(lens), libmla.load()
    stream = torch.cuda.current_stream().cuda_stream
    need = lib.mla_decode_fp8_plan_size(B, 1, h, 0)
    buf = torch.full((need // 4 + 64,), 2, dtype=torch.int32, device="cuda")
    one = d["lens"][:1].contiguous()
    if other == "bf16":
        n = lib.mla_plan_size(B, 1, h, 0)
        rc = lib.mla_decode_plan(d["lens"].data_ptr(), B, 1, h, buf.data_ptr(), n, stream)
    elif other == "heads":                                       # more tiles, fewer workers in each
        n = lib.mla_decode_fp8_plan_size(1, 8, 128, 0)
        rc = lib.mla_decode_fp8_plan(one.data_ptr(), 1, 8, 128, buf.data_ptr(), n, stream)
    elif other == "batch":
        n = lib.mla_decode_fp8_plan_size(B + 1, 1, 128, 0)
        lens2 = torch.cat([d["lens"], d["lens"][:1]])
        buf = torch.full((max(n, need) // 4 + 64,), 2, dtype=torch.int32, device="cuda")
        rc = lib.mla_decode_fp8_plan(lens2.data_ptr(), B + 1, 1, 128, buf.data_ptr(), n, stream)
    else:
        rc = libmla.MLA_OK
    assert rc == libmla.MLA_OK
    out = torch.full((B, 1, h, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, h, 1), 7.0, device="cuda")
    ws = torch.ones(lib.mla_decode_fp8_workspace_size(B, 1, h, 0) // 4 + 64, device="cuda")
    libmla.mla_check_device_error()
    rc = lib.mla_decode_fp8(d["q"].data_ptr(), d["codes"].data_ptr(), d["scales"].data_ptr(), 1,
                            x.pages, d["bt"].data_ptr(), d["bt"].shape[1], d["lens"].data_ptr(), B,
                            1, h, buf.data_ptr(), out.data_ptr(), lse.data_ptr(), SCALE,
                            ws.data_ptr(), ws.numel() * 4, stream)
    assert rc == libmla.MLA_OK
    assert libmla.mla_check_device_error() == libmla.MLA_ERR_PLAN
    assert torch.all(out == 7) and torch.all(lse == 7)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("h, lens", [(16, [20000]), (128, [5000, 70]), (64, [3000, 10, 2000])])
def test_bf16_decode_refuses_the_8bit_plan(torch_cuda, h, lens, f32):
    """The two plans are not interchangeable: that of the 8-bit decode has more
    workers and so more slots than the bf16 decode's workspace; the call is
    reported, and out and lse stay as they were."""
    torch, B = torch_cuda, len(lens)
    inp = W.make_inputs(131, B, 1, h, lens)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    bf = lambda a: t(a.view(np.int16)).view(torch.bfloat16)
    sl = t(np.asarray(lens, dtype=np.int32))
    meta, _ = libmla.alloc_fp8_plan_and_workspace(B, 1, h)
    _, ws = libmla.alloc_plan_and_workspace(B, 1, h)
    ws.fill_(1.0)
    libmla.mla_decode_fp8_plan(sl, 1, h, meta)
    out = torch.full((B, 1, h, 512), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    lse = torch.full((B, h, 1), 7.0, device="cuda")
    libmla.mla_check_device_error()
    (libmla.mla_decode_f32 if f32 else libmla.mla_decode)(
        bf(inp.q), bf(inp.kv_cache), t(inp.block_table), sl, meta, out, lse, inp.softmax_scale, ws)
    assert libmla.mla_check_device_error() == libmla.MLA_ERR_PLAN
    assert torch.all(out == 7) and torch.all(lse == 7)


def test_decode_fp8_refuses_short_plans_and_host_tensors(torch_cuda):
    """A plan's buffer of another shape, strided buffers, and single tensors on
    the host are refused before anything is enqueued."""
    torch, x = torch_cuda, Inputs(52, 1, 16, [100], 4)
    d = to_gpu(torch, x)
    out = torch.full((1, 1, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, 16, 1), 7.0, device="cuda")
    meta, ws = libmla.alloc_fp8_plan_and_workspace(1, 1, 16)
    short = libmla.alloc_fp8_plan_and_workspace(1, 1, 128)[0]     # fewer workers in a group
    good = dict(q=d["q"], kv_cache=d["codes"], scales=d["scales"], block_table=d["bt"],
                cache_seqlens=d["lens"], tile_meta=meta, out=out, lse=lse, softmax_scale=SCALE,
                workspace=ws)
    bad = [dict(tile_meta=short), dict(tile_meta=meta[::2]), dict(tile_meta=meta[:1].expand(1 << 20)),
           dict(workspace=ws[:1].expand(1 << 28))]
    bad += [{k: t.cpu()} for k, t in good.items() if k != "softmax_scale"]
    for kw in bad:
        with pytest.raises(libmla.MlaError) as e:
            libmla.mla_decode_fp8(**{**good, **kw})
        assert e.value.code == libmla.MLA_ERR_INVALID_ARG
    for a in ((d["lens"].cpu(), meta), (d["lens"], meta.cpu()), (d["lens"], meta[:1].expand(1 << 20))):
        with pytest.raises(libmla.MlaError) as e:
            libmla.mla_decode_fp8_plan(a[0], 1, 16, a[1])
        assert e.value.code == libmla.MLA_ERR_INVALID_ARG
    assert libmla.mla_check_device_error() == 0
    assert torch.all(out == 7) and torch.all(lse == 7)
    assert not np.isnan(run(torch, x, d=d)[0]).any()


@pytest.mark.parametrize("h_q", [16, 32, 64])
@pytest.mark.parametrize("exps", [(-70,), (-85,), (-100,), (-70, -85, -100)])
@pytest.mark.parametrize("q_exp", [0, 1])
def test_decode_fp8_all_scales_small(torch_cuda, h_q, exps, q_exp):
    """Every scale of an entry far below one, down to the least that the append
    stores: the weights keep their bits and out is the small average it is.  With
    q_exp the query is as large as the scales are small, so that scores spread."""
    x = Inputs(53, 2, h_q, [700, 90, 1], 1)
    z = np.asarray(W.splitmix64(54, 0, x.scales.size) % np.uint64(len(exps))).reshape(x.scales.shape)
    fresh = np.exp2(np.array(exps, dtype=np.float64))[z.astype(np.int64)].astype(np.float32)
    x.scales = fresh * (1 + x.scales / x.scales.max()).astype(np.float32)
    x.scales_gpu = np.where(np.isfinite(x.scales_gpu), x.scales, x.scales_gpu)
    if q_exp:
        x.q *= np.float32(2.0 ** (-max(exps) - 8))
    d = to_gpu(torch_cuda, x)
    out, lse, _ = run(torch_cuda, x, f32=True, d=d)
    compare(x, out, lse)
    ref = x.model()[0]
    assert np.abs(out - ref).max() <= 0.25 * np.abs(ref).max()      # not near zero
    assert_bf16_is_rounded_f32(run(torch_cuda, x, d=d)[0], out)


@pytest.mark.parametrize("h_q", [16, 32, 64])
@pytest.mark.parametrize("gain", [20.0, 60.0, 125.0])
def test_decode_fp8_small_scales_that_weigh_most(torch_cuda, h_q, gain):
    """Tokens of scale 1 with nothing in them first, then tokens of scale 2^-100
    whose scores are up to `gain` higher in log2: their p is 2^100 times their
    p c, far over the first tokens' reference."""
    n = 64 * 20 + 9
    x = Inputs(55, 1, h_q, [n], 1)
    t = np.arange(n)
    page, at = x.bt[0, t // 64], t % 64
    x.codes[page, at, 0] &= 0x7F
    first = (t // 64) % 4 < 2                                    # two pages of each kind in turn
    x.codes[page[first], at[first], 0] = 0
    x.scales[page, at] = np.where(first, 1.0, 2.0 ** -100)
    x.q = np.abs(x.q)
    k = M.E4M3[x.codes[page[~first], at[~first], 0]] * 2.0 ** -100
    top = (x.q[0, 0].astype(np.float64) @ k.T).max() * SCALE * np.log2(np.e)
    x.q = W.bf16_bits_to_float32(W.float32_to_bf16_bits((x.q.astype(np.float64) * (gain / top)).astype(np.float32)))
    x.codes_gpu[page, at], x.scales_gpu[page, at] = x.codes[page, at], x.scales[page, at]
    out, lse, _ = run(torch_cuda, x, f32=True)
    compare(x, out, lse)
    ref = x.model()[0]
    assert np.abs(out - ref).max() <= 0.05 * ref.max()              # not near zero


@pytest.mark.parametrize("s_q, h_q", [(1, 5), (1, 32), (2, 16), (1, 64), (1, 128)])
def test_decode_fp8_rescales_in_long_segments(torch_cuda, s_q, h_q):
    """Workers that hold ten and more consecutive pages of an entry, rows whose
    scores pass the running reference by more than 2^40 on every page, on every
    second, once by 2^130, or never (flat, falling): the factors reach their own
    rows' columns of O and sums.  The moves are counted on the host, from the
    model's scores and the plan's page ranges."""
    torch, B, L = torch_cuda, 170, 64 * 12 + 5
    x = Inputs(56, s_q, h_q, [L], 1)
    t = np.arange(L)
    page, at = x.bt[0, t // 64], t % 64
    c = 2.0 ** -6
    x.scales[page, at] = c
    x.codes[page, at, 0, 7] = M.e4m3_codes(16.0 * (t // 64))      # exact
    x.codes[page, at, 0, 9] = M.e4m3_codes(np.where(t >= 64 * 6, 128.0, 0.0))
    x.codes_gpu[page, at], x.scales_gpu[page, at] = x.codes[page, at], x.scales[page, at]
    rng = np.random.default_rng(57)
    q = rng.standard_normal((B, s_q, h_q, 576)) * 0.25
    kind = (np.arange(h_q)[None, None] + np.arange(s_q)[None, :, None] + np.arange(B)[:, None, None]) % 5
    per_page = np.choose(kind, [0.0, 50.0, -50.0, 30.0, 0.0])      # log2 units
    q[..., 7] = per_page / (SCALE * np.log2(np.e) * c * 16)
    q[..., 9] = np.where(kind == 4, 130.0, 0.0) / (SCALE * np.log2(np.e) * c * 128)
    x.q = W.bf16_bits_to_float32(W.float32_to_bf16_bits(q.astype(np.float32)))
    x.lens, x.bt = np.full(B, L, dtype=np.int32), np.repeat(x.bt, B, 0)
    d = to_gpu(torch, x)
    out, lse, _ = run(torch, x, f32=True, d=d)
    compare(x, out, lse)
    # what the kernel's reference does, from the page ranges
    meta, _ = libmla.alloc_fp8_plan_and_workspace(B, s_q, h_q)
    libmla.mla_decode_fp8_plan(d["lens"], s_q, h_q, meta)
    plan = plan_model.decode(meta.cpu().numpy())
    k = M.E4M3[x.codes[page, at, 0]] * c
    longest, moves = 0, np.zeros((5, 13), dtype=int)
    for w in range(plan["gused"]):
        for b, pb, pe, _ in plan_model.segments(plan, w):
            if pe - pb < 10:
                continue
            longest = max(longest, pe - pb)
            z = (x.q[b].reshape(-1, 576).astype(np.float64) @ k.T) * SCALE * np.log2(np.e) + np.log2(c)
            for i in range(s_q):
                z[i * h_q:(i + 1) * h_q, L - s_q + 1 + i:] = -np.inf
            ref = np.ceil(z[:, 64 * pb:64 * pb + 64].max(-1))
            for pg in range(pb + 1, pe):
                top = z[:, 64 * pg:64 * pg + 64].max(-1)
                move = top > ref + 40
                np.add.at(moves[:, pg], kind[b].reshape(-1)[move], 1)
                ref = np.where(move, np.ceil(top), ref)
    assert longest >= 10
    assert (moves[1, 2:] > 0).all() and (moves[3, 2:] > 0).sum() >= 5 and moves[4, 6] > 0
    assert not moves[0].any() and not moves[2].any()


@pytest.mark.parametrize("h, pages", [
    (16, [38, 45, 47, 16, 47, 47, 27]),          # 17 splits of an entry
    (16, [17, 44, 44, 44, 44]), (5, [44]), (16, [4, 5]), (16, [50, 50, 50]), (16, [1]),
    (32, [30, 30, 30]), (32, [5, 5, 5, 5]), (32, [4, 32, 5, 32, 17]), (20, [28, 28]),
    (64, [28, 27, 28, 9]), (64, [300]), (128, [30, 30, 30]), (128, [29, 60]), (16, [20] * 30)])
def test_decode_fp8_table_width_changes_no_bit(torch_cuda, h, pages):
    """A block table just as wide as its longest entry, and one as wide as a
    context limit."""
    torch = torch_cuda
    lens = [64 * p - 7 * (i % 3) for i, p in enumerate(pages)]
    x = Inputs(58, 1, h, lens, 1)
    d = to_gpu(torch, x)
    tight = run(torch, x, f32=True, d=d)
    for width in (len(x.bt[0]) + 1, 2 * len(x.bt[0]), 2048):
        bt = torch.full((len(lens), width), x.pages, dtype=torch.int32, device="cuda")
        bt[:, :d["bt"].shape[1]] = d["bt"]
        out, lse, _ = run(torch, x, f32=True, d=dict(d, bt=bt))
        assert np.array_equal(out, tight[0]) and np.array_equal(lse, tight[1]), width
