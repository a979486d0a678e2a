"""MXFP4 quantiser, dequantisers and grouped product on the GPU, against plain
definitions in 64 bits."""
import numpy as np
import pytest
import torch

import sigmoid_top_routing_02_amd as moe
from helpers import dev, np_, say

pytestmark = pytest.mark.gpu

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
F8 = torch.float64


# ------------------------------------------------------------------ the definition, on the host

def ref_quant(x):
    """x float64 [n, 32] (values of bf16 or binary32) -> (codes [n, 32], scale bytes [n])."""
    bad = ~np.isfinite(x).all(1)
    z = np.where(bad[:, None], 0.0, x)
    amax = np.abs(z).max(1)
    e = np.where(amax == 0, -127, np.frexp(np.where(amax == 0, 1.0, amax))[1] - 1 - 2)
    e = np.clip(e, -127, 125)
    v = np.abs(z) * np.exp2(-e.astype(np.float64))[:, None]
    up = np.minimum(np.searchsorted(GRID, v, side="left"), 7)          # first grid value >= v, or 6
    dn = np.maximum(up - 1, 0)
    du, dd = np.abs(GRID[up] - v), np.abs(v - GRID[dn])
    pick_dn = (dd < du) | ((dd == du) & (dn % 2 == 0))                 # ties to the even code
    c = np.where(v >= 6.0, 7, np.where(pick_dn, dn, up))
    c = c + 8 * np.signbit(z)
    return np.where(bad[:, None], 0, c).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def unpack(q):
    q = np_(q)
    return np.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], -1)


def check_quant(x):
    rows, cols = x.shape
    q, s = moe.mxfp4_quant_1x32(x)
    torch.cuda.synchronize()
    c, b = ref_quant(np_(x.float()).astype(np.float64).reshape(-1, 32))
    assert np.array_equal(np_(s).reshape(-1), b)
    assert np.array_equal(unpack(q).reshape(-1, 32), c)


def all_bf16():
    return torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.uint16).view(torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_every_bf16_value(dtype):
    """Every bf16 pattern among its neighbours, among random others, and in a block whose scale is 1."""
    dev()
    x = all_bf16()
    check_quant(x.view(-1, 64).to(dtype))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    check_quant(x[torch.randperm(65536, generator=g, device="cuda")].view(-1, 64).to(dtype))
    fin = x[x.abs() < 8]
    head = torch.full((fin.numel(), 1), 4.0, device="cuda", dtype=torch.bfloat16)
    check_quant(torch.cat((head, fin[:, None].expand(-1, 31)), 1).to(dtype).contiguous())


def test_quant_f32_about_the_midpoints():
    """binary32 values at each midpoint of the grid and the five on either side, under scales over the whole range."""
    dev()
    mid = ((GRID[1:] + GRID[:-1]) / 2).astype(np.float32)
    near = np.concatenate([(mid.view(np.int32) + k).view(np.float32) for k in range(-5, 6)])
    near = np.concatenate([near, -near, GRID.astype(np.float32)])
    blocks = []
    for e in list(range(-127, -118)) + [-60, -1, 0, 1, 60] + list(range(118, 126)):
        v = np.ldexp(near.astype(np.float64), e)
        v = v[np.abs(v) < np.finfo(np.float32).max]
        pad = np.zeros(-len(v) % 31)
        v = np.concatenate([v, pad]).reshape(-1, 31)
        blocks.append(np.concatenate([np.full((len(v), 1), np.ldexp(4.0, e)), v], 1))
    check_quant(torch.from_numpy(np.concatenate(blocks).astype(np.float32)).cuda())


@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 64), (3, 96), (7, 32), (256, 7168), (1021, 2080)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_shapes_and_values_back(rows, cols, dtype):
    dev()
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 1e-2, x * 100, x).to(dtype)
    check_quant(x)
    q, s = moe.mxfp4_quant_1x32(x)
    for out in (torch.bfloat16, torch.float32):
        v = moe.mxfp4_dequant_1x32(q, s, dtype=out)
        torch.cuda.synchronize()
        c = unpack(q).astype(np.int64)
        want = np.where(c & 8, -1.0, 1.0) * GRID[c & 7] * np.repeat(np.exp2(np_(s).astype(np.float64) - 127), 32, 1)
        assert np.array_equal(np_(v.to(F8)), want)


def test_quant_no_rows():
    dev()
    q, s = moe.mxfp4_quant_1x32(torch.empty((0, 64), device="cuda"))
    assert q.shape == (0, 32) and s.shape == (0, 2)
    assert moe.mxfp4_dequant_1x32(q, s).shape == (0, 64)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_dequant_every_code_and_scale(out):
    dev()
    s = torch.arange(256, dtype=torch.uint8, device="cuda").view(256, 1)
    q = torch.arange(0, 256, 1, dtype=torch.int32, device="cuda")[:16].to(torch.uint8)
    q = (q | ((15 - q) << 4)).expand(256, 16).contiguous()
    v = np_(moe.mxfp4_dequant_1x32(q, s, dtype=out).to(F8))
    c = unpack(q).astype(np.int64)
    want = np.where(c & 8, -1.0, 1.0) * GRID[c & 7] * np.exp2(np.arange(256.0) - 127)[:, None]
    want[np.abs(want) >= 2.0 ** 128] *= np.inf
    assert np.isnan(v[255]).all()
    assert np.array_equal(v[:255], want[:255]) and np.array_equal(np.signbit(v[:255]), np.signbit(want[:255]))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_fp8_dequant(out):
    """Every code under a few scales: E4M3(q) * scale in binary32, rounded once for bf16."""
    dev()
    q = torch.arange(256, dtype=torch.int32, device="cuda").to(torch.uint8).repeat(5, 1)
    s = torch.tensor([[1.0, 0.37], [2.0 ** -120, 3e-39], [1e30, 7.7], [0.0, 1e36], [123.456, 2.0 ** -7]], device="cuda")
    v = moe.fp8_dequant_1x128(q, s, dtype=out)
    want = (q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 1)).to(out)
    assert torch.equal(torch.isnan(v), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(v[ok], want[ok])
    assert moe.fp8_dequant_1x128(q[:0], s[:0], dtype=out).shape == (0, 256)


# ------------------------------------------------------------------ the grouped product

def operands(M, a_rows, G, N, K, seed, low=126, high=129):
    """Random codes under scales 2^(low - 127) .. 2^(high - 128): with the three scales 1/2, 1, 2 every
    product is a multiple of 2^-4 of at most 144, so that sums of fewer than 7281 are binary32 numbers and
    the product has one right answer, whatever its order."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def r(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    aq, bq = r(0, 256, a_rows, K // 2).to(torch.uint8), r(0, 256, G, N, K // 2).to(torch.uint8)
    a_s, b_s = r(low, high, a_rows, K // 32).to(torch.uint8), r(low, high, G, N, K // 32).to(torch.uint8)
    return aq, a_s, bq, b_s, r(0, a_rows, M)


def values(q, s):
    lut = torch.tensor(np.concatenate([GRID, -GRID]), device="cuda")
    c = torch.stack((q & 15, q >> 4), -1).flatten(-2)
    e = torch.where(s == 255, float("nan"), torch.exp2(s.to(F8) - 127))
    return lut[c.int()] * e.repeat_interleave(32, -1)


def ref_product(aq, a_s, bq, b_s, idx, sizes):
    """float64 [M, N]; rows of A that idx does not name inside A are zeros."""
    out, m = [], 0
    a = torch.cat((values(aq, a_s), torch.zeros((1, aq.shape[1] * 2), dtype=F8, device="cuda")))
    for g, n in enumerate(sizes):
        if n:
            i = torch.arange(m, m + n, device="cuda") if idx is None else idx[m:m + n].long()
            i = torch.where((i < 0) | (i >= aq.shape[0]), aq.shape[0], i)
            out.append(a.index_select(0, i) @ values(bq[g], b_s[g]).t())
            m += n
    return torch.cat(out) if out else torch.empty((0, bq.shape[1]), dtype=F8, device="cuda")


def offsets(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


RAGGED = [0, 1, 15, 16, 17, 0, 31, 33, 64, 65, 2, 0]
SIZES = {
    "one_row": [1],
    "one_row_of_many": [0, 0, 1, 0],
    "few": [3, 0, 16, 1, 7, 0, 12, 9],
    "ragged": RAGGED,
    "dense": [300],
    "uneven": [700, 1, 0, 257, 128],
    "full_tiles": [256, 512],
    "none": [0, 0, 0],
}
SHAPES = [(1, 32), (3, 64), (16, 96), (100, 160), (250, 128), (256, 512), (300, 544), (1000, 1056), (130, 2048),
          (272, 640), (515, 7168)]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("N,K", SHAPES)
def test_product_exact(sizes, N, K):
    dev()
    sz = SIZES[sizes]
    M, G = sum(sz), len(sz)
    say(f"  {sizes} M={M} N={N} K={K}")
    aq, a_s, bq, b_s, idx = operands(M, max(M // 2, 5), G, N, K, N + K + M)
    ref = ref_product(aq, a_s, bq, b_s, idx, sz)
    off = offsets(sz)
    got = moe.grouped_gemm_mxfp4(aq, a_s, off, M, bq, b_s, a_row_index=idx)
    half = moe.grouped_gemm_mxfp4(aq, a_s, off, M, bq, b_s, a_row_index=idx, epi=moe.MOE_MX_STORE_BF16)
    torch.cuda.synchronize()
    assert torch.equal(got.to(F8), ref)
    assert torch.equal(half, ref.float().bfloat16())


# Sizes that the other kernels take: a wave's 16, 32 and 64 rows, whole and half
# tiles; K with and without a whole number of 128s and of 512s.
MANY = [
    ([13] * 31 + [0], 4096, 640), ([12] * 30 + [1, 39], 4096, 1056),
    ([1200, 0, 500, 300], 1500, 1056), ([700, 1, 0, 1100, 199], 1536, 2048), ([129, 128, 127, 1616], 1280, 1152),
    ([6000], 4096, 544), ([3500, 0, 2500], 4000, 672), ([2600, 1, 0, 255, 257, 2300, 31], 3840, 1024),
    ([5000, 256], 3840, 1152), ([12] * 30 + [0, 9], 4608, 1152), ([11] * 30 + [1, 39], 4608, 1056),
    ([10] * 13 + [0, 2, 0], 4608, 4128), ([10] * 15 + [21], 4608, 4096), ([0, 0, 1, 0] * 16, 1024, 640),
    ([0] * 280 + [3, 0, 17] + [0] * 17, 512, 672),
    ([217, 183], 1536, 4096), ([200, 0, 143, 1], 1536, 4128),
]


@pytest.mark.parametrize("sz,N,K", MANY)
def test_product_exact_of_many_rows(sz, N, K):
    dev()
    M, G = sum(sz), len(sz)
    say(f"  M={M} G={G} N={N} K={K}")
    aq, a_s, bq, b_s, idx = operands(M, M // 2 + 5, G, N, K, N + K + M)
    idx[[0, M // 3, M - 1]] = torch.tensor([-1, M // 2 + 5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    ref = ref_product(aq, a_s, bq, b_s, idx, sz)
    off = offsets(sz)
    out = torch.full((M + 2, N), 7.0, device="cuda")
    moe.grouped_gemm_mxfp4(aq, a_s, off, M, bq, b_s, a_row_index=idx, out=out[:M])
    half = torch.full((M + 2, N), 7.0, device="cuda", dtype=torch.bfloat16)
    moe.grouped_gemm_mxfp4(aq, a_s, off, M, bq, b_s, a_row_index=idx, epi=moe.MOE_MX_STORE_BF16, out=half[:M])
    torch.cuda.synchronize()
    assert torch.equal(out[:M].to(F8), ref) and (out[M:] == 7.0).all()
    assert torch.equal(half[:M], ref.float().bfloat16()) and (half[M:] == 7.0).all()
    a_s[4, K // 32 - 1] = 255                       # a NaN scale stays in its rows and its column
    b_s[G - 1 if sz[-1] else G - 2, N - 1, K // 32 - 1] = 255
    got = moe.grouped_gemm_mxfp4(aq, a_s, off, M, bq, b_s, a_row_index=idx)
    torch.cuda.synchronize()
    nan = (idx == 4)[:, None].expand(M, N).clone()
    nan[M - (sz[-1] or sz[-2]):, N - 1] = True
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan].to(F8), ref[~nan])
    again = moe.grouped_gemm_mxfp4(aq, a_s, off, M, bq, b_s, a_row_index=idx)
    assert torch.equal(again.view(torch.int32), got.view(torch.int32))


@pytest.mark.parametrize("sz,N,K", [m for m in MANY if m[1] % 256 == 0])
def test_swiglu_of_many_rows(sz, N, K):
    dev()
    check_swiglu(sz, N, K)


@pytest.mark.parametrize("sizes", ["few", "dense", "uneven"])
def test_product_without_a_row_index(sizes):
    dev()
    sz = SIZES[sizes]
    M = sum(sz)
    aq, a_s, bq, b_s, _ = operands(M, M + 3, len(sz), 272, 640, 5)
    got = moe.grouped_gemm_mxfp4(aq, a_s, offsets(sz), M, bq, b_s)
    torch.cuda.synchronize()
    assert torch.equal(got.to(F8), ref_product(aq, a_s, bq, b_s, None, sz))


@pytest.mark.parametrize("sizes", ["few", "ragged", "uneven"])
@pytest.mark.parametrize("K", [1056, 7168])
def test_product_of_wide_scales(sizes, K):
    """Scales over 2^+-12: the sum is within binary32's accumulation error, one rounding of the running
    sum per term: K 2^-24 of the sum of magnitudes."""
    dev()
    sz = SIZES[sizes]
    M, N = sum(sz), 272
    aq, a_s, bq, b_s, idx = operands(M, M, len(sz), N, K, 9, low=115, high=140)
    got = moe.grouped_gemm_mxfp4(aq, a_s, offsets(sz), M, bq, b_s, a_row_index=idx)
    torch.cuda.synchronize()
    ref = ref_product(aq, a_s, bq, b_s, idx, sz)
    size = ref_product(aq & 0x77, a_s, bq & 0x77, b_s, idx, sz)
    assert ((got.to(F8) - ref).abs() <= K * 2.0 ** -24 * size).all()


def swiglu64(c):
    t = c.view(c.shape[0], c.shape[1] // 256, 256)
    return (torch.nn.functional.silu(t[:, :, :128]) * t[:, :, 128:]).reshape(c.shape[0], c.shape[1] // 2)


@pytest.mark.parametrize("sizes", ["one_row", "few", "ragged", "uneven", "none"])
@pytest.mark.parametrize("N,K", [(256, 32), (512, 640), (768, 1056), (512, 2048)])
def test_swiglu(sizes, N, K):
    """C is exact (see operands), so h = SiLU(C_gate) C_up is off by its own few binary32 operations: the
    exponential, the reciprocal and the products, 16 2^-24 where the exponential's argument is small; its
    argument's rounding adds |gate| 2^-24.  bf16 then rounds by 2^-8; the MXFP4 codes are the nearest to
    within that error."""
    dev()
    check_swiglu(SIZES[sizes], N, K)


def check_swiglu(sz, N, K):
    M = sum(sz)
    say(f"  M={M} G={len(sz)} N={N} K={K}")
    aq, a_s, bq, b_s, idx = operands(M, max(M, 1), len(sz), N, K, 11, low=121, high=124)
    off = offsets(sz)
    c = ref_product(aq, a_s, bq, b_s, idx, sz)
    h = swiglu64(c)
    gate = c.view(M, N // 256, 256)[:, :, :128].reshape(h.shape).abs()
    rel = (16 + gate) * 2.0 ** -23
    got = moe.grouped_gemm_mxfp4(aq, a_s, off, M, bq, b_s, a_row_index=idx, epi=moe.MOE_MX_SWIGLU_BF16)
    q, s = moe.grouped_gemm_mxfp4(aq, a_s, off, M, bq, b_s, a_row_index=idx, epi=moe.MOE_MX_SWIGLU_QUANT)
    torch.cuda.synchronize()
    tiny = 2.0 ** -126
    assert ((got.to(F8) - h).abs() <= (2.0 ** -8 + rel) * h.abs() + tiny).all()
    if M == 0:
        return
    rows = np.unique(np.linspace(0, M - 1, 1500).astype(np.int64))        # of many, these
    at = torch.from_numpy(rows).cuda()
    q, s, h, rel = q[at], s[at], h[at], rel[at]
    hb, rb = np_(h).reshape(-1, 32), np_(rel).reshape(-1, 32)
    e = np_(s).reshape(-1).astype(np.int64) - 127
    _, lo = ref_quant((np.abs(hb) * (1 - rb)).astype(np.float64))
    _, hi = ref_quant((np.abs(hb) * (1 + rb)).astype(np.float64))
    assert ((e + 127 >= lo) & (e + 127 <= hi)).all()
    cc = unpack(q).reshape(-1, 32).astype(np.int64)
    val = np.where(cc & 8, -1.0, 1.0) * GRID[cc & 7]
    v = np.clip(hb / np.exp2(e)[:, None], -6.0, 6.0)
    # no grid value is nearer than the one taken, by more than the error of h
    best = np.abs(v[..., None] - np.concatenate([GRID, -GRID])).min(-1)
    assert (np.abs(val - v) <= best + 2 * rb * np.abs(v) + tiny).all()


def test_empty_and_bad_rows():
    """A row index outside A is a row of zeros; rows outside every group are not written."""
    dev()
    for sz in ([5, 0, 30], [200, 90]):
        M = sum(sz)
        aq, a_s, bq, b_s, idx = operands(M, 40, len(sz), 272, 160, 3)
        idx[[0, 3, M - 1]] = torch.tensor([-1, 40, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
        out = torch.full((M + 2, 272), 7.0, device="cuda")
        moe.grouped_gemm_mxfp4(aq, a_s, offsets(sz), M, bq, b_s, a_row_index=idx, out=out[:M])
        torch.cuda.synchronize()
        assert torch.equal(out[:M].to(F8), ref_product(aq, a_s, bq, b_s, idx, sz)) and (out[M:] == 7.0).all()
        assert (out[[0, 3, M - 1]] == 0).all()


@pytest.mark.parametrize("K", [96, 640, 1056])
@pytest.mark.parametrize("sz", [[5, 0, 30], [200, 90]])
def test_nan_scales_stay_in_their_row_and_column(sz, K):
    dev()
    M, N = sum(sz), 272
    aq, a_s, bq, b_s, _ = operands(M, M, len(sz), N, K, 3)
    ref = ref_product(aq, a_s, bq, b_s, None, sz)
    a_s[4, K // 32 - 1] = 255
    b_s[0, 17, 0] = 255
    b_s[len(sz) - 1, N - 1, K // 32 - 1] = 255
    got = moe.grouped_gemm_mxfp4(aq, a_s, offsets(sz), M, bq, b_s)
    torch.cuda.synchronize()
    nan = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    nan[4] = True
    nan[:sz[0], 17] = True
    nan[M - sz[-1]:, N - 1] = True
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan].to(F8), ref[~nan])


def test_many_groups():
    dev()
    rng = np.random.default_rng(0)
    sz = (rng.integers(0, 4, 1024) * (rng.random(1024) < 0.3)).tolist()
    sz[1023] = 70
    M = sum(sz)
    aq, a_s, bq, b_s, idx = operands(M, 99, 1024, 48, 160, 2)
    got = moe.grouped_gemm_mxfp4(aq, a_s, offsets(sz), M, bq, b_s, a_row_index=idx)
    torch.cuda.synchronize()
    assert torch.equal(got.to(F8), ref_product(aq, a_s, bq, b_s, idx, sz))


def test_offsets_past_32_bits():
    """B past 4 GiB (the last group's rows), then an output past 4 GiB (its last rows)."""
    dev()
    G, N, K = 40, 16384, 16384
    bq = torch.zeros((G, N, K // 2), dtype=torch.uint8, device="cuda")
    b_s = torch.full((G, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    bq[G - 1] = 0x22                                   # ones
    bq[G - 1, N - 1] = 0x44                            # twos
    aq = torch.full((1, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    a_s = torch.full((1, K // 32), 127, dtype=torch.uint8, device="cuda")
    for rows in (3, 300):
        out = moe.grouped_gemm_mxfp4(aq, a_s, offsets([0] * (G - 1) + [rows]), rows, bq, b_s,
                                     a_row_index=torch.zeros(rows, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert (out[:, :-1] == K).all() and (out[:, -1] == 2 * K).all()
    del bq, b_s
    M, N, K = 70000, 16384, 32
    aq, a_s, bq, b_s, idx = operands(M, 50, 1, N, K, 1)
    got = moe.grouped_gemm_mxfp4(aq, a_s, offsets([M]), M, bq, b_s, a_row_index=idx)
    torch.cuda.synchronize()
    ref = ref_product(aq, a_s, bq, b_s, torch.arange(50, device="cuda"), [50])
    for m in (0, 1, 65535, 65536, M - 200, M - 1):
        assert torch.equal(got[m].to(F8), ref[int(idx[m])])


def test_repeatable_on_another_stream_and_in_a_graph():
    dev()
    for sz, N in (([3, 0, 9, 1], 512), ([300, 40], 512), ([1500, 0, 700], 1536), ([3000, 3000], 4096)):
        M = sum(sz)
        aq, a_s, bq, b_s, idx = operands(M, M, len(sz), N, 1056, 4, low=120, high=130)
        off = offsets(sz)
        x = torch.randn((M, 1056), device="cuda")

        def step():
            q, s = moe.mxfp4_quant_1x32(x)
            hq, hs = moe.grouped_gemm_mxfp4(q, s, off, M, bq, b_s, a_row_index=idx, epi=moe.MOE_MX_SWIGLU_QUANT)
            return (q, s, hq, hs, moe.mxfp4_dequant_1x32(hq, hs), moe.grouped_gemm_mxfp4(q, s, off, M, bq, b_s))

        want = step()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            got = step()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
        for i in range(3):
            x.mul_(-1.25)
            graph.replay()
            torch.cuda.synchronize()
            eager = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(held, eager)), i


def test_binding_refusals():
    dev()
    aq, a_s, bq, b_s, idx = operands(8, 8, 2, 256, 64, 1)
    off = offsets([4, 4])
    g = moe.grouped_gemm_mxfp4
    bad = [
        lambda: moe.mxfp4_quant_1x32(torch.zeros((2, 40), device="cuda")),
        lambda: moe.mxfp4_quant_1x32(torch.zeros((2, 64), device="cuda").half()),
        lambda: moe.mxfp4_quant_1x32(torch.zeros((2, 64))),
        lambda: moe.mxfp4_quant_1x32(torch.zeros((2, 128), device="cuda")[:, ::2]),
        lambda: moe.mxfp4_quant_1x32(torch.zeros((3, 68), device="cuda").view(-1)[1:129].view(2, 64)),
        lambda: moe.mxfp4_dequant_1x32(aq, a_s[:, :1].contiguous()),
        lambda: moe.mxfp4_dequant_1x32(aq, a_s, dtype=torch.float16),
        lambda: moe.fp8_dequant_1x128(aq, torch.ones((8, 1), device="cuda")),
        lambda: g(aq, a_s, off, 9, bq, b_s),
        lambda: g(aq, a_s, off[:2], 8, bq, b_s),
        lambda: g(aq, a_s, off.long(), 8, bq, b_s),
        lambda: g(aq[:, :16].contiguous(), a_s, off, 8, bq, b_s),
        lambda: g(aq, a_s, off, 8, bq, b_s[:1]),
        lambda: g(aq, a_s, off, 9, bq, b_s, a_row_index=idx),
        lambda: g(aq, a_s, off, 8, bq, b_s, epi=4),
        lambda: g(aq, a_s, off, 8, bq[:, :128].contiguous(), b_s[:, :128].contiguous(), epi=moe.MOE_MX_SWIGLU_BF16),
        lambda: g(aq, a_s, off, 8, bq, b_s, out=torch.empty((8, 256), dtype=torch.bfloat16, device="cuda")),
        lambda: g(aq.cpu(), a_s, off, 8, bq, b_s),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(moe.MoEError):
            f()
            pytest.fail(f"case {i} was taken")
