"""The rotating cache appends on the GPU against the 64-bit model.

Bars, derived from the arithmetic:
* latent dims into bf16 pages: bit for bit.
* turned dims in bf16: two products and a sum in fp32 (each within 2^-24 of
  its size, so 2^-22 sum |terms| covers them), then half a bf16 step, at most
  2^-8 of the value.
* scales: amax / 448 in fp32: 2^-24 for the quotient, 2^-22 sum |terms| / amax
  (at most 2 * 2^-22) for a turned amax.
* codes: half an e4m3 step of x / scale, at most 2^-4 of the value or 2^-10
  below the smallest normal number, plus the fp32 product and reciprocal
  (2^-22 relative).
"""
import numpy as np
import pytest

import fp8_model as M
from mla_decode_attention_07_gb300 import libmla
from mla_decode_attention_07_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch


def table_of_angles(n, theta=10000.0):
    a = np.arange(n)[:, None] * theta ** (-np.arange(32) / 32.0)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class Case:
    """Seeded inputs on the host: s_new rows for each entry after `starts`."""

    def __init__(self, seed, starts, news, s_new, h, interleaved, pitch=576, G=1, spare=2,
                 rope_scale=1.0):
        B = len(starts)
        self.s_new, self.h, self.il, self.G = s_new, h, interleaved, G
        self.lens = np.array([a + n for a, n in zip(starts, news)], dtype=np.int32)
        self.new_lens = np.array(news, dtype=np.int32)
        per = [(int(n) + 63) // 64 for n in self.lens]
        self.pages = sum(per) + spare
        perm = W.permutation(seed, 1, self.pages)
        self.bt = np.full((B, max(max(per), 1)), self.pages + 5, dtype=np.int32)
        k = 0
        for b, p in enumerate(per):
            self.bt[b, :p] = perm[k:k + p]
            k += p
        self.cos_sin = table_of_angles(max(int(self.lens.max()), 1))
        f = lambda tid, *shape: W.bf16_bits_to_float32(
            W.normal_bf16(seed, tid, int(np.prod(shape)))).reshape(shape).copy()
        self.kv_wide = f(2, B, s_new, pitch)
        self.kv_wide[..., pitch - 64:] = W.bf16_bits_to_float32(W.float32_to_bf16_bits(
            self.kv_wide[..., pitch - 64:] * np.float32(rope_scale)))
        self.kv = self.kv_wide[..., pitch - 576:]
        self.q_wide = f(3, B, s_new, h, 192)
        self.cache16 = f(4, self.pages, 64, 1, 576)
        self.codes = (W.splitmix64(seed ^ 9, 0, self.pages * 64 * 576) % np.uint64(0x7F)).astype(
            np.uint8).reshape(self.pages, 64, 1, 576)
        z = W.splitmix64(seed ^ 10, 0, self.pages * (64 // G))
        self.scales = np.exp2(-9.0 + 4.0 * (z >> np.uint64(40)).astype(np.float64) / 2 ** 24).astype(
            np.float32).reshape(self.pages, 64 // G)

    def rows(self):
        return list(M.new_rows(self.kv, self.q_wide[..., 128:], self.bt, self.lens, self.new_lens,
                               self.cos_sin, self.il, self.pages))


def to_gpu(torch, c, padded=True):
    bf = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda().to(torch.bfloat16)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    kv = bf(c.kv_wide)[..., c.kv_wide.shape[-1] - 576:]
    q_in = bf(c.q_wide)[..., 128:]
    q_full = torch.full((*c.q_wide.shape[:3], 576), 7.0, dtype=torch.bfloat16, device="cuda")
    return dict(kv=kv, q=q_in, q_full=q_full, q_out=q_full[..., 512:], bt=t(c.bt), lens=t(c.lens),
                new=t(c.new_lens) if padded else None, cs=t(c.cos_sin), cache16=bf(c.cache16),
                codes=t(c.codes), scales=t(c.scales))


def check_queries(c, g, rows):
    got = g["q_full"].float().cpu().numpy().astype(np.float64)
    want = np.full(got.shape, 7.0)
    slack = np.zeros(got.shape)
    for b, i, _, _, _, _, q, mag in rows:
        want[b, i, :, 512:] = q
        slack[b, i, :, 512:] = 2.0 ** -8 * np.abs(q) + 2.0 ** -22 * mag
    assert np.all(np.abs(got - want) <= slack)


CASES = [
    # seed, starts, news, s_new, heads, interleaved, row pitch, tokens to a scale
    (1, [0], [1], 1, 1, True, 576, 1),
    (2, [255], [1], 1, 16, False, 576, 64),
    (3, [0, 63, 64, 130], [1, 1, 1, 1], 1, 128, True, 584, 2),
    (4, [61, 5, 127], [5, 0, 3], 5, 3, False, 1152, 4),
    (5, [0, 100, 7], [130, 64, 1], 130, 5, True, 576, 8),
    (6, [31, 0], [200, 199], 200, 33, False, 640, 16),
    (7, [1, 40], [77, 150], 150, 128, True, 576, 32),
    (8, [63, 64, 10], [70, 128, 0], 128, 20, False, 576, 64),
    (9, [3] * 40, [2] * 40, 2, 128, True, 576, 16),
    (10, [5, 9], [300, 250], 300, 129, True, 576, 1),     # more heads than one CTA takes
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"s{c[0]}_h{c[4]}_g{c[7]}")
def test_append_bf16(torch_cuda, case):
    torch, c = torch_cuda, Case(*case)
    g, rows = to_gpu(torch, c), c.rows()
    libmla.mla_rope_append(g["kv"], g["cache16"], g["bt"], g["lens"], g["cs"], g["q"], g["q_out"],
                           new_lens=g["new"], interleaved=c.il)
    assert libmla.mla_check_device_error() == 0
    got = g["cache16"].float().cpu().numpy().astype(np.float64).reshape(-1, 576)
    want = c.cache16.reshape(-1, 576).astype(np.float64)
    slack = np.zeros(want.shape)
    for _, _, _, row, val, mag, _, _ in rows:
        want[row] = val
        slack[row, 512:] = 2.0 ** -8 * np.abs(val[512:]) + 2.0 ** -22 * mag[512:]
    assert np.all(np.abs(got - want) <= slack)
    check_queries(c, g, rows)


@pytest.mark.parametrize("rope_scale", [0.25, 8.0])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"s{c[0]}_h{c[4]}_g{c[7]}")
def test_append_fp8(torch_cuda, case, rope_scale):
    torch, c = torch_cuda, Case(*case, rope_scale=rope_scale)
    g, rows = to_gpu(torch, c), c.rows()
    libmla.mla_rope_append_fp8(g["kv"], g["codes"], g["scales"], g["bt"], g["lens"], g["cs"],
                               g["q"], g["q_out"], new_lens=g["new"], interleaved=c.il)
    assert libmla.mla_check_device_error() == 0
    _, scales, fresh, again = M.append_fp8(c.codes, c.scales, rows, c.lens, c.new_lens, c.s_new)
    got_s = g["scales"].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got_s - scales) <= 2.0 ** -20 * scales)
    got = g["codes"].cpu().numpy().reshape(-1, 576)
    touched = np.zeros(len(got), dtype=bool)
    for row, val in {**again, **fresh}.items():
        touched[row] = True
        v = M.E4M3[got[row]]
        slack = np.maximum(2.0 ** -4 * np.abs(val), 2.0 ** -10) + 2.0 ** -19 * np.abs(val)
        assert np.all(np.abs(v - val) <= slack), row
    before = c.codes.reshape(-1, 576)
    assert np.array_equal(got[~touched], before[~touched])
    # with an amax in the latent dims every bit of the codes is determined
    if rope_scale < 1 and c.G == 1:
        lat = c.kv.astype(np.float32)
        for b, i, _, row, val, *_ in rows:
            x = lat[b, i, :512]
            if np.abs(x).max() > np.abs(val[512:]).max():
                quotient = x.astype(np.float64) * 448 / np.float64(np.abs(x).max())
                assert np.array_equal(got[row, :512], M.e4m3_codes(quotient))
    check_queries(c, g, rows)


def test_append_without_queries_and_counts(torch_cuda):
    torch, c = torch_cuda, Case(21, [10, 70], [4, 4], 4, 2, True)
    g = to_gpu(torch, c, padded=False)
    libmla.mla_rope_append(g["kv"], g["cache16"], g["bt"], g["lens"], g["cs"])
    assert libmla.mla_check_device_error() == 0
    got = g["cache16"].float().cpu().numpy().reshape(-1, 576)
    for _, _, _, row, val, mag, _, _ in c.rows():
        assert np.all(np.abs(got[row] - val) <= 2.0 ** -8 * np.abs(val) + 2.0 ** -22 * mag)


def test_append_turns_queries_in_place(torch_cuda):
    torch, c = torch_cuda, Case(22, [10, 70], [3, 2], 3, 40, False)
    g, rows = to_gpu(torch, c), c.rows()
    g["q_full"][..., 512:] = g["q"]
    libmla.mla_rope_append(g["kv"], g["cache16"], g["bt"], g["lens"], g["cs"], g["q_out"],
                           g["q_out"], new_lens=g["new"], interleaved=False)
    assert libmla.mla_check_device_error() == 0
    got = g["q_full"].float().cpu().numpy()
    for b, i, _, _, _, _, q, mag in rows:
        assert np.all(np.abs(got[b, i, :, 512:] - q) <= 2.0 ** -8 * np.abs(q) + 2.0 ** -22 * mag)
    assert np.array_equal(got[1, 2, :, 512:], c.q_wide[1, 2, :, 128:])       # a padded row
    assert np.all(got[..., :512] == 7.0)


def test_append_fp8_twice_is_once(torch_cuda):
    """The second append of the same rows finds its own scales and changes nothing."""
    torch, c = torch_cuda, Case(23, [10, 50], [9, 30], 30, 2, True, G=64, rope_scale=6.0)
    g = to_gpu(torch, c)
    call = lambda: libmla.mla_rope_append_fp8(g["kv"], g["codes"], g["scales"], g["bt"], g["lens"],
                                              g["cs"], g["q"], g["q_out"], new_lens=g["new"])
    call()
    codes, scales, q = g["codes"].clone(), g["scales"].clone(), g["q_full"].clone()
    call()
    assert libmla.mla_check_device_error() == 0
    assert torch.equal(g["codes"], codes) and torch.equal(g["scales"], scales)
    assert torch.equal(g["q_full"], q)


@pytest.mark.parametrize("G", [1, 8, 64])
def test_append_fp8_half_way_values(torch_cuda, G):
    """448 x / amax half way between two codes goes to the even one, for every
    scale (amax over all 128 fractions of a bf16 number)."""
    torch = torch_cuda
    c = Case(25, [0], [128], 128, 1, True, G=G, rope_scale=0.0)
    grid = M.E4M3[8:0x7E]                                          # 2^-6 .. 416
    ties = (grid + M.E4M3[9:0x7F]) / 2
    for i in range(128):
        top = (1 + (i if G == 1 else i // G * G) / 128) * 2.0 ** 3
        x = ties * top / 448
        x = x[x == W.bf16_bits_to_float32(W.float32_to_bf16_bits(x.astype(np.float32)))]
        c.kv_wide[0, i, -576:] = 0.0
        c.kv_wide[0, i, -576] = top
        c.kv_wide[0, i, -575:-575 + len(x)] = x
    g = to_gpu(torch, c)
    libmla.mla_rope_append_fp8(g["kv"], g["codes"], g["scales"], g["bt"], g["lens"], g["cs"],
                               g["q"], g["q_out"], new_lens=g["new"])
    assert libmla.mla_check_device_error() == 0
    got, checked = g["codes"].cpu().numpy(), 0
    for i in range(128):
        top = (1 + (i if G == 1 else i // G * G) / 128) * 2.0 ** 3
        quotient = c.kv_wide[0, i, -576:-64].astype(np.float64) * 448 / top   # a turned 0 may be -0
        assert np.array_equal(got[c.bt[0, i // 64], i % 64, 0, :512], M.e4m3_codes(quotient)), i
        checked += int(np.isin(quotient, ties).sum())
    assert checked > 0


def test_append_fp8_zero_and_tiny_rows(torch_cuda):
    torch, c = torch_cuda, Case(24, [0], [3], 3, 1, True)
    c.kv_wide[0, 0] = 0.0
    c.kv_wide[0, 1] = W.bf16_bits_to_float32(np.full(576, 1, dtype=np.uint16))   # 2^-133
    g = to_gpu(torch, c)
    libmla.mla_rope_append_fp8(g["kv"], g["codes"], g["scales"], g["bt"], g["lens"], g["cs"],
                               g["q"], g["q_out"], new_lens=g["new"])
    assert libmla.mla_check_device_error() == 0
    page = int(c.bt[0, 0])
    s = g["scales"].cpu().numpy()[page]
    assert s[0] == 2.0 ** -100 and s[1] == 2.0 ** -100 and s[2] > 2.0 ** -9
    assert not (g["codes"].cpu().numpy()[page, :2] & 0x7F).any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("what", ["before_start", "page", "angles", "count"])
def test_append_out_of_range_is_flagged_and_skipped(torch_cuda, fp8, what):
    torch, c = torch_cuda, Case(25, [20, 60], [4, 8], 8, 2, True, G=8)
    if what == "before_start":
        c.lens[0] = 2                       # four new tokens, two positions
    elif what == "page":
        c.bt[1, 1] = c.pages                # positions 64..67 of entry 1
    elif what == "angles":
        c.cos_sin = c.cos_sin[:66]          # positions 66, 67 of entry 1
    else:
        c.new_lens[0] = 9
    g, rows = to_gpu(torch, c), c.rows()
    libmla.mla_check_device_error()
    if fp8:
        libmla.mla_rope_append_fp8(g["kv"], g["codes"], g["scales"], g["bt"], g["lens"], g["cs"],
                                   g["q"], g["q_out"], new_lens=g["new"])
    else:
        libmla.mla_rope_append(g["kv"], g["cache16"], g["bt"], g["lens"], g["cs"], g["q"],
                               g["q_out"], new_lens=g["new"])
    assert libmla.mla_check_device_error() == libmla.MLA_ERR_DEVICE_BOUNDS
    good = {r[3]: r for r in rows if r[3] is not None}
    if fp8:
        want, scales, fresh, again = M.append_fp8(c.codes, c.scales, rows, c.lens, c.new_lens, 8)
        assert np.allclose(g["scales"].cpu().numpy(), scales, rtol=2.0 ** -20, atol=0)
        got, before = g["codes"].cpu().numpy().reshape(-1, 576), c.codes.reshape(-1, 576)
        keep = [r for r in range(len(got)) if r not in fresh and r not in again]
        assert set(fresh) == set(good)
        for row, val in fresh.items():
            slack = np.maximum(2.0 ** -4 * np.abs(val), 2.0 ** -10) + 2.0 ** -19 * np.abs(val)
            assert np.all(np.abs(M.E4M3[got[row]] - val) <= slack)
    else:
        got = g["cache16"].float().cpu().numpy().reshape(-1, 576)
        before = c.cache16.reshape(-1, 576)
        keep = [r for r in range(len(got)) if r not in good]
        for row, r in good.items():
            assert np.all(np.abs(got[row] - r[4]) <= 2.0 ** -8 * np.abs(r[4]) + 2.0 ** -22 * r[5])
    assert np.array_equal(got[keep], before[keep])
    check_queries(c, g, rows)


def test_append_captured_and_replayed(torch_cuda):
    """A captured append replays with what the buffers hold then."""
    torch, c, d = torch_cuda, Case(26, [10], [2], 2, 16, True, G=16), None
    g = to_gpu(torch, c)
    call = lambda s: libmla.mla_rope_append_fp8(g["kv"], g["codes"], g["scales"], g["bt"],
                                                g["lens"], g["cs"], g["q"], g["q_out"],
                                                new_lens=g["new"], stream=s)
    libmla.mla_num_clusters(0)                      # the device's one-time set-up, not captured
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(torch.cuda.current_stream())
    d = Case(27, [30], [2], 2, 16, True, G=16)
    h = to_gpu(torch, d)
    for k in ("codes", "scales", "kv", "q", "q_full", "cs", "lens"):
        src = h[k]
        if k == "cs":
            g[k].copy_(src[:g[k].shape[0]])
        elif k != "lens":
            g[k].copy_(src)
    graph.replay()
    assert libmla.mla_check_device_error() == 0
    libmla.mla_rope_append_fp8(h["kv"], h["codes"], h["scales"], g["bt"], g["lens"], g["cs"],
                               h["q"], h["q_out"], new_lens=g["new"])
    assert libmla.mla_check_device_error() == 0
    for k in ("codes", "scales", "q_full"):
        assert torch.equal(g[k].view(torch.uint8), h[k].view(torch.uint8)), k


@pytest.mark.parametrize("fp8", [False, True])
def test_append_pages_past_4_gb(torch_cuda, fp8):
    """The pages at the end of a pool of 4.4 GB get the bits of a small pool."""
    torch, c = torch_cuda, Case(26, [3, 70], [130, 9], 130, 2, True, G=16)
    pool = 120000 if fp8 else 60000
    got = []
    for far in (False, True):
        g = to_gpu(torch, c)
        cache, scales = g["codes"] if fp8 else g["cache16"], g["scales"]
        if far:
            big = torch.zeros((pool, 64, 1, 576), dtype=cache.dtype, device="cuda")
            sbig = torch.zeros((pool, 4), device="cuda")
            big[pool - c.pages:], sbig[pool - c.pages:] = cache, scales
            cache, scales, g["bt"] = big, sbig, g["bt"] + (pool - c.pages)
        lead = (g["kv"], cache, scales) if fp8 else (g["kv"], cache)
        (libmla.mla_rope_append_fp8 if fp8 else libmla.mla_rope_append)(
            *lead, g["bt"], g["lens"], g["cs"], g["q"], g["q_out"], new_lens=g["new"])
        assert libmla.mla_check_device_error() == 0
        got.append([cache[cache.shape[0] - c.pages:].clone(), scales[scales.shape[0] - c.pages:].clone()])
        if far:
            assert not cache[:pool - c.pages].view(torch.int32).any()
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"s{c[0]}_h{c[4]}_g{c[7]}")
def test_append_fp8_bits_of_scales_and_latents(torch_cuda, case):
    """Where the largest magnitude of a block lies in its latent dims (bf16, not
    turned), the scale, every latent code and every code that is stored anew are
    determined: quotients rounded to fp32, then codes to the nearest, halves to
    even."""
    torch, c = torch_cuda, Case(*case, rope_scale=0.125)
    g, f32 = to_gpu(torch, c), np.float32
    libmla.mla_rope_append_fp8(g["kv"], g["codes"], g["scales"], g["bt"], g["lens"], g["cs"],
                               g["q"], g["q_out"], new_lens=g["new"], interleaved=c.il)
    assert libmla.mla_check_device_error() == 0
    codes, scales = g["codes"].cpu().numpy().reshape(-1, 576), g["scales"].cpu().numpy().reshape(-1)
    blocks = {}
    for b, i, t, row, val, *_ in c.rows():
        blocks.setdefault((b, row // c.G), []).append((t, row, val))
    checked = grown = 0
    for (b, blk), toks in blocks.items():
        if max(np.abs(v[512:]).max() for _, _, v in toks) > max(np.abs(v[:512]).max() for _, _, v in toks) / 2:
            continue
        amax = max(np.abs(v[:512]).max() for _, _, v in toks)
        fresh = max(f32(amax / 448), f32(M.SCALE_MIN))
        start, t0 = int(c.lens[b] - c.new_lens[b]), toks[0][0] - toks[0][1] % c.G
        old = c.scales.reshape(-1)[blk] if t0 < start else f32(0)
        scale = max(fresh, old)
        assert scales[blk] == scale
        for _, row, v in toks:
            quotient = v[:512] * 448 / amax if scale == fresh else v[:512] / np.float64(scale)
            assert np.array_equal(codes[row, :512], M.e4m3_codes(quotient.astype(f32))), row
        before = c.codes.reshape(-1, 576)[blk * c.G:blk * c.G + max(start - t0, 0)]
        if scale > old:
            ratio = f32(np.float64(old) / np.float64(scale))
            before = M.e4m3_codes(M.E4M3[before].astype(f32) * ratio)
            grown += len(before) > 0
        assert np.array_equal(codes[blk * c.G:blk * c.G + len(before)], before)
        checked += 1
    assert checked > 0
    if c.G == 16:
        assert grown > 0
