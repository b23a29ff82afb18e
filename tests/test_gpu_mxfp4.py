"""MXFP4 quantisers, read-back and products against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from _util import capi, require_cuda
from oracle import mxfp4

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def np64(t):
    return t.detach().double().cpu().numpy()


def matrix(rows, cols, dtype, seed=0, special=True):
    """Normal rows with outliers; the first rows hold the awkward values."""
    g = torch.Generator().manual_seed(seed + 7919 * rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-12, 6, (rows, 1), generator=g).float())
    x = torch.where(torch.rand(rows, cols, generator=g) < 0.01, 30 * x, x)
    if special:
        tiny = torch.finfo(dtype).smallest_normal
        if rows > 3:
            x[0] = 0.0
            x[1] = torch.arange(cols).float() % 64 / 8 - 4                   # ties
            x[2] = tiny * (torch.arange(cols).float() % 5 - 2)
            x[3, cols // 2] = torch.finfo(dtype).max
        if rows > 6:
            x[4, cols // 3] = float("inf")
            x[5, cols - 1] = float("nan")
            x[6, 0] = -float("inf")
            x[6, 1:] = -0.0
    return x.to(dtype)


def check_quantized(q, x, layout):
    """Codes and scale bytes equal the oracle's for the rows of x."""
    rows, cols = x.shape
    codes, scales = mxfp4.quantize(np64(x))
    got = q.codes.cpu().numpy().reshape(rows, -1)
    assert np.array_equal(got, codes)
    s = q.scales.cpu().numpy().reshape(-1)
    if layout == "canonical":
        assert np.array_equal(s.reshape(scales.shape), scales)
    else:
        assert np.array_equal(s[mxfp4.tiled_index(rows, cols)], scales)
        # padding blocks of data rows are zero
        pad = -(-scales.shape[1] // 4) * 4
        assert (s[mxfp4.tiled_index(rows, pad * 32)[:, scales.shape[1]:]] == 0).all()


SHAPES = [(1, 1), (1, 32), (3, 33), (16, 256), (129, 100), (7, 2049), (130, 128), (300, 514), (5000, 300), (64, 6144)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("layout", ["tiled", "canonical"])
def test_quantize_matches_oracle(rows, cols, dtype, layout):
    require_cuda()
    c = capi()
    x = matrix(rows, cols, DTYPES[dtype])
    check_quantized(c.mxfp4_quantize(x.cuda(), layout), x, layout)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES + [(1, 700), (31, 64), (513, 96), (1030, 65)])
@pytest.mark.parametrize("layout", ["tiled", "canonical"])
def test_quantize_transposed_matches_oracle(rows, cols, dtype, layout):
    require_cuda()
    c = capi()
    x = matrix(cols, rows, DTYPES[dtype]).t().contiguous()
    check_quantized(c.mxfp4_quantize_transposed(x.cuda(), layout), x.t(), layout)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("off,pad", [(0, 8), (0, 4), (0, 2), (0, 1), (8, 16), (4, 12), (2, 6), (1, 7)])
def test_strided_rows_of_every_alignment(dtype, off, pad):
    """Rows at every offset and pitch alignment: the access width changes, the
    result does not, and nothing outside the rows is read into it."""
    require_cuda()
    c = capi()
    rows, cols = 70, 200
    x = matrix(rows, cols, DTYPES[dtype])
    big = torch.full((rows, off + cols + pad), float("nan"), dtype=DTYPES[dtype], device="cuda")
    view = big[:, off:off + cols]
    view.copy_(x)
    check_quantized(c.mxfp4_quantize(view), x, "tiled")
    check_quantized(c.mxfp4_quantize_transposed(view), x.t(), "tiled")
    # read-back into the same strided rows leaves the rest alone
    q = c.mxfp4_quantize(view)
    c.mxfp4_dequantize(q, out=view)
    want = mxfp4.dequantize(*mxfp4.quantize(np64(x)), cols)
    want = torch.from_numpy(want).to(DTYPES[dtype]).double().numpy()
    assert np.array_equal(np64(view), want, equal_nan=True)
    rest = np64(big)
    assert np.isnan(rest[:, :off]).all() and np.isnan(rest[:, off + cols:]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("layout", ["tiled", "canonical"])
def test_dequantize_every_code_and_scale(rows, cols, dtype, layout):
    require_cuda()
    c = capi()
    rng = np.random.default_rng(rows * 31 + cols)
    codes = rng.integers(0, 256, (rows, -(-cols // 32) * 16), dtype=np.uint8)
    scales = rng.integers(0, 256, (rows, -(-cols // 32)), dtype=np.uint8)
    s = scales if layout == "canonical" else mxfp4.to_tiled(scales, cols)
    q = c.Mxfp4(torch.from_numpy(codes).cuda(), torch.from_numpy(s.copy()).cuda(), rows, cols, layout)
    v = torch.from_numpy(mxfp4.dequantize(codes, scales, cols))
    got = c.mxfp4_dequantize(q, dtype=DTYPES[dtype])
    # one rounding from the exact value (fp64 -> fp32 is exact or overflows like the product does)
    assert torch.equal(torch.nan_to_num(got.cpu().float(), nan=-77.0),
                       torch.nan_to_num(v.float().to(DTYPES[dtype]).float(), nan=-77.0))
    if dtype != "fp16":
        fine = v.abs() <= torch.finfo(DTYPES[dtype]).max
        assert torch.equal(got.cpu().double()[fine], v[fine])


def test_quantize_gathers_rows():
    require_cuda()
    c = capi()
    x = matrix(9, 100, torch.bfloat16)
    perm = torch.tensor([3, -1, 8, 8, 9, 0, 2 ** 31 - 1, -2 ** 31, 7] * 20, dtype=torch.int32)
    q = c.mxfp4_quantize(x.cuda(), perm=perm.cuda())
    rows = torch.zeros(perm.numel(), 100, dtype=torch.bfloat16)
    ok = (perm >= 0) & (perm < 9)
    rows[ok] = x[perm[ok].long()]
    check_quantized(q, rows, "tiled")
    empty = c.mxfp4_quantize(x.cuda(), perm=perm[:0].cuda())
    assert empty.rows == 0


def test_canonical_scales_become_tiled_by_quantising_again():
    require_cuda()
    c = capi()
    rng = np.random.default_rng(4)
    rows, cols = 300, 1000
    codes = rng.integers(0, 256, (rows, 512), dtype=np.uint8)
    scales = rng.integers(0, 253, (rows, 32), dtype=np.uint8)
    q = c.Mxfp4(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), rows, cols, "canonical")
    for dt in (torch.float32, torch.bfloat16):
        v = c.mxfp4_dequantize(q, dtype=dt)
        t = c.mxfp4_quantize(v)
        assert t.layout == "tiled" and torch.equal(c.mxfp4_dequantize(t, dtype=dt), v)


def test_zero_rows_and_stacks():
    require_cuda()
    c = capi()
    q = c.mxfp4_quantize(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert c.mxfp4_dequantize(q).shape == (0, 64)
    w = matrix(256, 96, torch.bfloat16, special=False).reshape(2, 128, 96)
    check_quantized(c.mxfp4_quantize(w.cuda()), w.reshape(256, 96), "tiled")
    y = c.mxfp4_matmul(q, c.mxfp4_quantize(w[0, :, :64].cuda()))
    assert y.shape == (0, 128)
    assert c.mxfp4_linear(torch.zeros(0, 64, device="cuda"), c.mxfp4_quantize(w[0, :, :64].cuda())).shape == (0, 128)


# --- products ----------------------------------------------------------------

def operand(rows, cols, seed, integers=False):
    """(Mxfp4 on the device, its float64 values)."""
    c = capi()
    rng = np.random.default_rng(seed)
    if integers:
        x = rng.choice([-6.0, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6], (rows, cols))
        x[:, ::32] = 4.0                       # every block's scale is 1
    else:
        x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-6, 6, (rows, 1)))
    codes, scales = mxfp4.quantize(x)
    q = c.Mxfp4(torch.from_numpy(codes).cuda(), torch.from_numpy(mxfp4.to_tiled(scales, cols)).cuda(), rows, cols)
    return q, mxfp4.dequantize(codes, scales, cols)


def product_bound(a, b, ref, dtype, row_weight=None, bias=None):
    """Largest possible |y - ref|: the products of E2M1 values are exact; K of
    them enter fp32 sums in some order, each addition off by at most 2^-23
    (truncated) of a partial sum that never passes sum |a||b|; bias and
    row_weight round once each; the store by half a step of the output type
    (or half its smallest subnormal)."""
    K = a.shape[1]
    mag = np.abs(a) @ np.abs(b).T
    if bias is not None:
        mag = mag + np.abs(bias)
    err = (K + 2) * 2.0 ** -23 * mag
    if row_weight is not None:
        err = err * np.abs(row_weight)[:, None] + 2.0 ** -24 * np.abs(ref)
    fi = torch.finfo(dtype)
    return err + fi.eps / 2 * (np.abs(ref) + err) + fi.smallest_normal * fi.eps


MNK = [(3, 5, 1), (1, 1, 32), (1, 128, 64), (1, 6144, 512), (2, 7, 33), (15, 130, 96), (16, 256, 128), (17, 500, 160),
       (31, 64, 256), (32, 129, 288), (33, 1000, 544), (64, 384, 1024), (65, 128, 100), (100, 300, 2048), (100, 300, 5000), (128, 6000, 4500),
       (128, 128, 512), (129, 255, 320), (200, 1024, 640), (256, 256, 256), (257, 130, 224), (300, 700, 384),
       (515, 129, 1056), (1024, 1536, 256), (3000, 257, 96), (16, 128, 6144), (5, 260, 4000),
       # on CTA pairs (tests/test_mxfp4.py checks that these sizes reach them), K ending with one atom and two
       (2990, 2290, 1900), (3000, 2049, 1700),
       # two CTAs on an SM, and their second wave
       (3000, 1000, 96), (2990, 2290, 300)]


@pytest.mark.parametrize("M,N,K", MNK)
def test_matmul_matches_oracle(M, N, K):
    require_cuda()
    c = capi()
    a, av = operand(M, K, M + N)
    b, bv = operand(N, K, M + K + 1)
    ref = av @ bv.T
    for name, dt in DTYPES.items():
        y = c.mxfp4_matmul(a, b, out_dtype=dt)
        assert y.dtype == dt
        if name == "fp16":
            keep = np.abs(ref) < 60000
            assert (np.abs(np64(y) - ref)[keep] <= product_bound(av, bv, ref, dt)[keep]).all()
        else:
            assert (np.abs(np64(y) - ref) <= product_bound(av, bv, ref, dt)).all(), name


@pytest.mark.parametrize("M,N,K", MNK)
def test_matmul_of_integers_is_exact(M, N, K):
    """Integer values: every partial sum is an integer below 2^24, so fp32
    accumulation has no rounding and the output is the product itself."""
    require_cuda()
    c = capi()
    a, av = operand(M, K, 3 * M + N, integers=True)
    b, bv = operand(N, K, 5 * N + K, integers=True)
    ref = av @ bv.T
    assert np.abs(ref).max() < 2 ** 24 and 36 * K < 2 ** 24
    y = c.mxfp4_matmul(a, b, out_dtype=torch.float32)
    assert np.array_equal(np64(y), ref)


def test_matmul_bias_row_weight_and_strided_out():
    require_cuda()
    c = capi()
    rng = np.random.default_rng(5)
    for M, N, K in [(3, 200, 320), (3, 200, 2048), (40, 130, 96), (300, 300, 256), (2990, 2290, 1900), (3000, 2049, 1700)]:
        a, av = operand(M, K, 1)
        b, bv = operand(N, K, 2)
        bias = rng.standard_normal(N).astype(np.float32)
        rw = rng.standard_normal(M).astype(np.float32)
        rw[0] = 0.0
        ref = rw[:, None].astype(np.float64) * (av @ bv.T + bias)
        big = torch.full((M, N + 13), 7.0, device="cuda")
        y = c.mxfp4_matmul(a, b, out=big[:, 5:5 + N], bias=torch.from_numpy(bias).cuda(),
                           row_weight=torch.from_numpy(rw).cuda())
        assert (np.abs(np64(y) - ref) <= product_bound(av, bv, ref, torch.float32, rw, bias)).all()
        assert (big[:, :5] == 7.0).all() and (big[:, 5 + N:] == 7.0).all()


@pytest.mark.parametrize("M", [1, 40, 300, 2990])
def test_a_nan_block_reaches_its_row_only(M):
    require_cuda()
    c = capi()
    N, K = (200, 300) if M < 2990 else (2290, 1900)
    a, av = operand(M, K, 3)
    b, bv = operand(N, K, 4)
    clean = c.mxfp4_matmul(a, b)
    at = int(mxfp4.tiled_index(M, K)[M - 1, K // 32])          # the last, partly filled block
    a.scales[at] = 255
    y = c.mxfp4_matmul(a, b)
    assert torch.isnan(y[M - 1]).all() and torch.equal(y[:M - 1], clean[:M - 1])
    a.scales[at] = 127
    b.scales[int(mxfp4.tiled_index(N, K)[131, 0])] = 255
    y = c.mxfp4_matmul(a, b)
    assert torch.isnan(y[:, 131]).all() and not torch.isnan(y[:, :131]).any() and not torch.isnan(y[:, 132:]).any()


def test_padding_bytes_do_not_matter():
    """Scale bytes of padding rows may hold anything, NaN included."""
    require_cuda()
    c = capi()
    for M, N, K in [(3, 70, 100), (150, 260, 300), (2990, 2290, 1900)]:
        a, av = operand(M, K, 8)
        b, bv = operand(N, K, 9)
        want = c.mxfp4_matmul(a, b, out_dtype=torch.float32)
        for q, rows in ((a, M), (b, N)):
            keep = torch.zeros_like(q.scales, dtype=torch.bool)
            keep[torch.from_numpy(mxfp4.tiled_index(rows, -(-K // 128) * 128).reshape(-1)).cuda()] = True
            q.scales[~keep] = 255
        assert torch.equal(c.mxfp4_matmul(a, b, out_dtype=torch.float32), want)


def grouped_case(counts, gaps, N, K, seed):
    """Rows in 128-row segments, E matrices of N rows."""
    segs = [-(-n // 128) * 128 + 128 * g for n, g in zip(counts, gaps)]
    off = np.concatenate([[0], np.cumsum(segs)]).astype(np.int32)
    M = int(off[-1])
    a, av = operand(M, K, seed)
    b, bv = operand(len(counts) * N, K, seed + 1)
    return off, M, a, av, b, bv


@pytest.mark.parametrize("counts,gaps,N,K", [
    ([5], [0], 128, 64),
    ([0, 1, 128, 129, 0, 300, 7], [0, 0, 0, 1, 1, 0, 2], 256, 288),
    ([3] * 40, [0] * 40, 128, 512),
    ([1000, 0, 257], [0, 0, 0], 384, 160),
    ([0, 0, 0], [0, 1, 0], 128, 96),
    ([900, 0, 385, 1900], [0, 0, 0, 0], 2048, 1700),        # on CTA pairs
    ([1000, 1024, 1, 1200], [0, 0, 0, 0], 1920, 1900),        # pairs, an odd number of 128-row b tiles per expert
])
def test_grouped_matmul(counts, gaps, N, K):
    require_cuda()
    c = capi()
    off, M, a, av, b, bv = grouped_case(counts, gaps, N, K, 11)
    E = len(counts)
    rng = np.random.default_rng(0)
    rw = rng.standard_normal(M).astype(np.float32)
    bias = rng.standard_normal(E * N).astype(np.float32)
    cu = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    for with_counts in (True, False):
        n = np.array(counts, np.int32) if with_counts else np.diff(off).astype(np.int32)
        ref = np.full((M, N), -3.0)
        bound = np.zeros((M, N))
        for e in range(E):
            r, w = slice(off[e], off[e] + n[e]), slice(e * N, (e + 1) * N)
            ref[r] = rw[r, None].astype(np.float64) * (av[r] @ bv[w].T + bias[w])
            bound[r] = product_bound(av[r], bv[w], ref[r], torch.bfloat16, rw[r], bias[w])
        out = torch.full((M, N), -3.0, dtype=torch.bfloat16, device="cuda")
        y = c.mxfp4_matmul(a, b, out=out, bias=cu(bias), row_weight=cu(rw), expert_offsets=cu(off),
                           expert_counts=cu(n) if with_counts else None)
        # rows of no expert hold -3 still
        assert (np.abs(np64(y) - ref) <= bound).all()


def test_grouped_offsets_outside_the_rows_are_clamped():
    require_cuda()
    c = capi()
    a, av = operand(256, 64, 1)
    b, bv = operand(3 * 128, 64, 2)
    off = torch.tensor([-128, 128, 1 << 30, 0], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([1 << 30, 1 << 30, -5], dtype=torch.int32, device="cuda")
    y = np64(c.mxfp4_matmul(a, b, out_dtype=torch.float32, expert_offsets=off, expert_counts=cnt))
    ref = np.concatenate([av[:128] @ bv[:128].T, av[128:] @ bv[128:256].T])
    assert (np.abs(y - ref) <= 66 * 2.0 ** -23 * 64 * 36 * np.abs(av).max() * np.abs(bv).max()).all()


@pytest.mark.parametrize("M,offsets,N,K,dtype", [
    (300, [0, 384, 384], 128, 64, torch.float32),
    (300, [0, 128, 384, 384, 512], 256, 288, torch.bfloat16),
    (1, [0, 128, 128, 256], 128, 96, torch.float16),
    (3400, [0, 1152, 3456, 3456, 3584], 2048, 1700, torch.bfloat16),      # on CTA pairs
])
def test_grouped_rows_that_end_inside_the_last_segment(M, offsets, N, K, dtype):
    """A last segment whose padding was trimmed, with empty experts behind it:
    they have no rows, with and without counts."""
    require_cuda()
    c = capi()
    E = len(offsets) - 1
    assert c.nvfp4_test_mxfp4_plan(M, N, K, E)[2] == (M == 3400)
    a, av = operand(M, K, 1)
    b, bv = operand(E * N, K, 2)
    lim = np.clip(offsets, 0, M)
    ref = np.zeros((M, N))
    bound = np.zeros((M, N))
    for e in range(E):
        r = slice(lim[e], lim[e + 1])
        ref[r] = av[r] @ bv[e * N:(e + 1) * N].T
        bound[r] = product_bound(av[r], bv[e * N:(e + 1) * N], ref[r], dtype)
    fine = np.abs(ref) < torch.finfo(dtype).max / 2
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    counts = torch.from_numpy(np.diff(lim).astype(np.int32)).cuda()
    counts[-1] = 5                                          # of a segment past the rows
    for cnt in (None, counts):
        y = c.mxfp4_matmul(a, b, out_dtype=dtype, expert_offsets=off, expert_counts=cnt)
        assert (np.abs(np64(y) - ref) <= bound)[fine].all()


def test_linear_is_quantize_then_matmul():
    require_cuda()
    c = capi()
    for M, N, K, dt in [(1, 300, 6144, torch.bfloat16), (37, 501, 201, torch.float16), (700, 256, 500, torch.float32)]:
        x = matrix(M, K + 24, dt, special=False).cuda()[:, 8:8 + K]
        w, _ = operand(N, K, N)
        y = c.mxfp4_linear(x, w)
        assert y.dtype == dt
        assert torch.equal(y, c.mxfp4_matmul(c.mxfp4_quantize(x), w, out_dtype=dt))
        perm = torch.randint(-1, M, (2 * M + 1,), dtype=torch.int32, device="cuda")
        yp = c.mxfp4_linear(x, w, perm=perm)
        assert torch.equal(yp, c.mxfp4_matmul(c.mxfp4_quantize(x, perm=perm), w, out_dtype=dt))
        assert not yp[perm < 0].any()


# (M, N, K): products that quantise their rows themselves; whole and partial K
# stages, one to four K splits, one and two CTAs an SM, rings that wrap
FUSED = [(1, 1, 1), (1, 128, 32), (2, 500, 31), (3, 501, 201), (5, 300, 257), (16, 130, 300), (13, 640, 64),
         (8, 1024, 6144), (7, 5001, 2010), (2, 12288, 4096), (1, 37000, 1000), (1, 1000, 8192), (1, 3000, 14000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", FUSED)
def test_linear_of_few_rows(M, N, K, dtype):
    """The product that quantises its rows itself: the values of the oracle,
    and bit for bit those of quantising first; rows at every alignment, gathered
    rows, rows without a source, blocks that are zero, NaN or infinite."""
    require_cuda()
    c = capi()
    dt = DTYPES[dtype]
    w, wv = operand(N, K, M + K)
    bias = torch.randn(N, device="cuda")
    rw = torch.randn(M, device="cuda")
    for off in (0, 1, 8):
        wide = off * dt.itemsize % 16 == 0
        if c.nvfp4_test_mxfp4_fuses(M, N, K, dt, wide) is None:
            assert dt == torch.float32 and M > 4 or not wide          # more passes over the rows
            continue
        base = matrix(M, (K + off + 15) // 16 * 16, dt, seed=off, special=False).cuda()
        base[:, :off] = base[:, off + K:] = float("nan")               # the neighbours of x in memory
        x = base[:, off:off + K]
        if M > 2:
            x[1, K // 2] = 0.0 if off else float("inf")
            x[2] = 0.0
        y = c.mxfp4_linear(x, w, out_dtype=torch.float32)
        assert torch.equal(y.isnan(), c.mxfp4_matmul(c.mxfp4_quantize(x), w, out_dtype=torch.float32).isnan())
        codes, scales = mxfp4.quantize(np64(x))
        xv = mxfp4.dequantize(codes, scales, K)
        good = np.isfinite(xv).all(axis=1)
        ref = xv[good] @ wv.T
        assert (np.abs(np64(y)[good] - ref) <= product_bound(xv[good], wv, ref, torch.float32)).all()
        assert torch.isnan(y[torch.from_numpy(~good).cuda()]).all()
        out = torch.full((M, N + 3), 7.0, dtype=dt, device="cuda")[:, 1:1 + N]
        c.mxfp4_linear(x, w, out=out, bias=bias, row_weight=rw)
        want = torch.full_like(out, 7.0)
        c.mxfp4_matmul(c.mxfp4_quantize(x), w, out=want, bias=bias, row_weight=rw)
        assert torch.equal(out.nan_to_num(5.0), want.nan_to_num(5.0))
        perm = torch.randint(-2, 2 * M, (M,), dtype=torch.int32, device="cuda")
        yp = c.mxfp4_linear(x, w, perm=perm)
        assert torch.equal(yp.nan_to_num(5.0), c.mxfp4_matmul(c.mxfp4_quantize(x, perm=perm), w, out_dtype=dt).nan_to_num(5.0))
        assert not yp[(perm < 0) | (perm >= M)].any()


def test_few_rows_gathered_from_many_and_none():
    require_cuda()
    c = capi()
    w, _ = operand(384, 600, 8)
    assert c.nvfp4_test_mxfp4_fuses(4, 384, 600, torch.bfloat16)
    x = matrix(5000, 600, torch.bfloat16, special=False).cuda()
    perm = torch.tensor([4999, 17, 17, 5000], dtype=torch.int32, device="cuda")
    y = c.mxfp4_linear(x, w, perm=perm)
    assert torch.equal(y, c.mxfp4_matmul(c.mxfp4_quantize(x, perm=perm), w))
    assert torch.equal(y[1], y[2]) and not y[3].any()
    assert not c.mxfp4_linear(x[:0], w, perm=perm).any()


def test_y_in_the_place_of_few_rows():
    """y over x, and y whose rows lie between x's: x is read before y is written."""
    require_cuda()
    c = capi()
    w, _ = operand(512, 512, 3)
    assert c.nvfp4_test_mxfp4_fuses(4, 512, 512, torch.bfloat16)
    both = torch.cat([matrix(4, 512, torch.bfloat16, seed=i, special=False) for i in (1, 2)], dim=1).cuda()
    x = both[:, :512]
    want = c.mxfp4_linear(x.clone(), w)
    assert torch.equal(c.mxfp4_linear(x, w, out=both[:, 512:]), want)
    for shift in (0, 1):                          # rows shifted by one: y's row i is x's row i + 1
        z = torch.cat([x, x[:1]])
        assert torch.equal(c.mxfp4_linear(z[:4], w, out=z[shift:4 + shift]), want)


@pytest.mark.parametrize("with_counts", [True, False])
def test_grouped_linear_with_padding_rows(with_counts):
    """Rows of perm without a source: inside an expert's tokens they are
    zeros (y = weight * bias); outside them nothing is read or written."""
    require_cuda()
    c = capi()
    E, N, K = 3, 128, 330
    off = torch.tensor([0, 256, 256, 512], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([130, 0, 7], dtype=torch.int32, device="cuda")
    x = matrix(50, K, torch.bfloat16, special=False).cuda()
    w, _ = operand(E * N, K, 4)
    perm = torch.full((512,), -1, dtype=torch.int32)
    perm[:130] = torch.arange(130) % 50
    perm[256:263] = torch.arange(7)
    perm[3] = perm[129] = perm[260] = -1
    perm = perm.cuda()
    rw = torch.randn(512, device="cuda")
    bias = torch.randn(E * N, device="cuda")
    out = torch.full((512, N), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((c.mxfp4_linear_workspace_size(512, K),), 255, dtype=torch.uint8, device="cuda")   # NaN scales
    kw = dict(row_weight=rw, bias=bias, expert_offsets=off, expert_counts=cnt if with_counts else None)
    c.mxfp4_linear(x, w, perm=perm, out=out, workspace=ws, **kw)
    want = torch.full_like(out, 9.0)
    c.mxfp4_matmul(c.mxfp4_quantize(x, perm=perm), w, out=want, **kw)
    assert torch.equal(out, want) and torch.isfinite(out).all()
    if with_counts:
        assert (out[130:256] == 9.0).all() and (out[263:] == 9.0).all()
    for r, e in ((3, 0), (129, 0), (260, 2)):
        assert torch.equal(out[r], (rw[r] * bias[e * N:(e + 1) * N]).to(torch.bfloat16))


@pytest.mark.parametrize("offsets,counts", [([-128, 128, 256], [100, 7]), ([-384, -128, 1 << 30], [50, 200]),
                                            ([-2 ** 31, 256, 2 ** 31 - 1], [2 ** 31 - 1, 9])])
def test_grouped_linear_with_clamped_offsets(offsets, counts):
    """Rows without a source are zeros wherever the product reads them, which
    for an offset outside the rows is counted from its clamped value."""
    require_cuda()
    c = capi()
    E, N, K, M = 2, 128, 200, 256
    x = matrix(60, K, torch.bfloat16, special=False).cuda()
    w, _ = operand(E * N, K, 4)
    bias = torch.randn(E * N, device="cuda")
    perm = torch.arange(M, dtype=torch.int32) % 60
    perm[::3] = -1
    perm = perm.cuda()
    kw = dict(bias=bias, expert_offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"),
              expert_counts=torch.tensor(counts, dtype=torch.int32, device="cuda"))
    ws = torch.full((c.mxfp4_linear_workspace_size(M, K),), 255, dtype=torch.uint8, device="cuda")   # NaN scales
    out = torch.full((M, N), 9.0, dtype=torch.bfloat16, device="cuda")
    c.mxfp4_linear(x, w, perm=perm, out=out, workspace=ws, **kw)
    want = torch.full_like(out, 9.0)
    c.mxfp4_matmul(c.mxfp4_quantize(x, perm=perm), w, out=want, **kw)
    assert torch.isfinite(out).all() and torch.equal(out, want)


def test_results_do_not_change_from_run_to_run():
    require_cuda()
    c = capi()
    for M, N, K in [(1, 1000, 4096), (48, 512, 2048), (600, 640, 1024), (2990, 2290, 1900)]:
        a, _ = operand(M, K, 1)
        b, _ = operand(N, K, 2)
        first = c.mxfp4_matmul(a, b, out_dtype=torch.float32)
        for _ in range(5):
            assert torch.equal(c.mxfp4_matmul(a, b, out_dtype=torch.float32), first)


def test_offsets_past_32_bits():
    """Matrices of more than 2^32 bytes: the last rows come out as they do by
    themselves."""
    require_cuda()
    c = capi()
    rows, cols = 66000, 33000                                  # 8.7 GB of fp32
    x = torch.empty(rows, cols, device="cuda")
    tail = matrix(300, cols, torch.float32, special=False).cuda()
    x[:-300] = 0.0
    x[-300:] = tail
    q, qt = c.mxfp4_quantize(x, "canonical"), c.mxfp4_quantize(tail, "canonical")
    assert torch.equal(q.codes[-300:], qt.codes) and torch.equal(q.scales[-300:], qt.scales)
    assert not q.codes[:-300].any() and not q.scales[:-300].any()
    back = c.mxfp4_dequantize(q, dtype=torch.float32, out=x)
    assert torch.equal(back[-300:], c.mxfp4_dequantize(qt, dtype=torch.float32)) and not back[:1000].any()
    wide = c.mxfp4_quantize_transposed(back[:, -40:], "canonical")       # rows 33000 apart, past 2^32 bytes
    alone = c.mxfp4_quantize_transposed(back[:, -40:].contiguous(), "canonical")
    assert torch.equal(wide.codes, alone.codes) and torch.equal(wide.scales, alone.scales)
    del x, back, q, wide, alone
    M, N, K = 40000, 60000, 64                                 # 4.8 GB of bf16 outputs
    a, _ = operand(M, K, 1)
    b, _ = operand(N, K, 2)
    y = c.mxfp4_matmul(a, b)
    ac, bc = c.mxfp4_dequantize(a), c.mxfp4_dequantize(b)
    part = c.mxfp4_matmul(c.mxfp4_quantize(ac[-700:].contiguous()), c.mxfp4_quantize(bc[-900:].contiguous()))
    assert torch.equal(y[-700:, -900:], part)


def test_y_may_take_the_place_of_x():
    require_cuda()
    c = capi()
    for M in (5, 600):
        x = matrix(M, 512, torch.bfloat16, special=False).cuda()
        w, _ = operand(512, 512, 3)
        want = c.mxfp4_linear(x, w)
        assert torch.equal(c.mxfp4_linear(x, w, out=x), want)


FIRST_CALLS_IN_A_CAPTURE = """
import sys, torch
sys.path.insert(0, %r)
from nvfp4_w4a4_quantized_moe_b200 import capi as c
torch.manual_seed(0)
x = [torch.randn(m, 1900, device="cuda").bfloat16() for m in (1, 300, 2990)]
w = torch.randn(2290, 1900, device="cuda").bfloat16()
l = torch.randn(3000, 64, device="cuda")
idx = l.topk(4).indices.int()
one = torch.ones(1, device="cuda")
def everything():
    q = c.mxfp4_quantize(w)
    t = c.mxfp4_quantize_transposed(w)
    b = c.moe_balance_loss(l, idx, 0.1)
    return ([c.mxfp4_linear(v, q) for v in x] + [c.mxfp4_dequantize(t), b.loss, b.probs,
            c.moe_balance_loss_backward(l, b, one), c.moe_balance_loss(l[:9], idx[:9], 0.1).loss])
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = everything()
g.replay()
torch.cuda.synchronize()
want = everything()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("same")
"""


def test_first_calls_of_a_process_may_be_captured():
    require_cuda()
    import subprocess
    import sys

    from _util import ROOT
    capi()
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS_IN_A_CAPTURE % ROOT], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


def test_calls_from_two_threads_and_streams():
    require_cuda()
    c = capi()
    import threading
    w, _ = operand(1000, 640, 1)
    xs = [matrix(m, 640, torch.bfloat16, special=False).cuda() for m in (3, 300)]
    want = [c.mxfp4_linear(x, w) for x in xs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                if not torch.equal(c.mxfp4_linear(xs[i], w), want[i]):
                    bad.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1, 0, 1)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_side_stream_and_captured_graphs_sharing_a_workspace():
    require_cuda()
    c = capi()
    w, _ = operand(500, 640, 1)
    xs = [matrix(m, 640, torch.bfloat16, special=False).cuda() for m in (3, 200)]
    want = [c.mxfp4_linear(x, w) for x in xs]
    ws = torch.empty(c.mxfp4_linear_workspace_size(200, 640), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [c.mxfp4_linear(x, w, workspace=ws) for x in xs]
    side.synchronize()
    assert all(torch.equal(g, v) for g, v in zip(got, want))
    outs = [torch.zeros_like(v) for v in want]
    graphs = []
    for x, o in zip(xs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.mxfp4_linear(x, w, out=o, workspace=ws)
        graphs.append(g)
    for x in xs:
        x.mul_(2.0)                                            # powers of two: the outputs double exactly
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, 2 * v) for o, v in zip(outs, want))
    c.nvfp4_workspace_status(ws)


def test_linear_gradients_against_the_formula_and_differences():
    """y = q(x) q(w)^T; dx = q(dy) q(w^T)^T and dw = q(dy^T) q(x^T)^T from the
    transposed quantiser, against their formulas in 64 bits.  With operands on
    the E2M1 grid quantisation changes nothing, so dx and dw are the true
    gradients of sum(dy * y): checked against exact differences (y is linear
    in each of x and w)."""
    require_cuda()
    c = capi()
    rng = np.random.default_rng(3)
    M, N, K = 70, 96, 200
    grid = np.array([-6.0, -4, -3, -2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2, 3, 4, 6])
    x, w, dy = (rng.choice(grid, s) for s in ((M, K), (N, K), (M, N)))
    for t in (x, w, dy):
        t[:, ::16] = 6.0
        t[::16, :] = 6.0                                     # every block, either way, has scale 1
    cu = lambda t: torch.from_numpy(t).to(torch.bfloat16).cuda()  # noqa: E731
    dx = c.mxfp4_matmul(c.mxfp4_quantize(cu(dy)), c.mxfp4_quantize_transposed(cu(w)), out_dtype=torch.float32)
    dw = c.mxfp4_matmul(c.mxfp4_quantize_transposed(cu(dy)), c.mxfp4_quantize_transposed(cu(x)),
                        out_dtype=torch.float32)
    assert np.array_equal(np64(dx), dy @ w) and np.array_equal(np64(dw), dy.T @ x)
    loss = lambda x_, w_: float((dy * np64(c.mxfp4_linear(cu(x_), c.mxfp4_quantize(cu(w_)),  # noqa: E731
                                                          out_dtype=torch.float32))).sum())
    for i, j in ((0, 1), (17, 33), (69, 199)):
        for arr, g in ((x, dx), (w, dw)):
            hi, lo = arr.copy(), arr.copy()
            hi[i, j], lo[i, j] = 2.0, -2.0
            d = (loss(hi, w) - loss(lo, w) if arr is x else loss(x, hi) - loss(x, lo)) / 4.0
            assert d == float(g[i, j])


def test_binding_refusals():
    require_cuda()
    c = capi()
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    q = c.mxfp4_quantize(x)
    bad = [
        lambda: c.mxfp4_quantize(x.int()), lambda: c.mxfp4_quantize(x.t()), lambda: c.mxfp4_quantize(x[0]),
        lambda: c.mxfp4_quantize(x[:1].expand(4, 64)), lambda: c.mxfp4_quantize(x, perm=torch.zeros(4, device="cuda")),
        lambda: c.mxfp4_quantize(x, out=c.mxfp4_quantize(x[:2])),
        lambda: c.mxfp4_dequantize(q, out=torch.zeros(4, 63, device="cuda")),
        lambda: c.Mxfp4(q.codes, q.scales[:100], 4, 64), lambda: c.Mxfp4(q.codes, q.scales, 5, 64),
        lambda: c.Mxfp4(q.codes, q.scales, 4, 64, "staged"),
        lambda: c.mxfp4_matmul(q, c.mxfp4_quantize(x[:, :32])),
        lambda: c.mxfp4_matmul(q, c.mxfp4_quantize(x, "canonical")),
        lambda: c.mxfp4_matmul(q, q, out=torch.zeros(4, 5, device="cuda")),
        lambda: c.mxfp4_matmul(q, q, bias=torch.zeros(5, device="cuda")),
        lambda: c.mxfp4_matmul(q, q, row_weight=torch.zeros(4, dtype=torch.float64, device="cuda")),
        lambda: c.mxfp4_matmul(q, q, expert_counts=torch.zeros(1, dtype=torch.int32, device="cuda")),
        lambda: c.mxfp4_matmul(q, q, expert_offsets=torch.zeros(4, dtype=torch.int32, device="cuda")),
        lambda: c.mxfp4_linear(x[:, :32], q),
        lambda: c.mxfp4_linear(x, q, out=torch.zeros(4, 4, dtype=torch.int32, device="cuda")),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(c.Nvfp4Error):                       # 4 rows an expert: not a multiple of 128
        c.mxfp4_matmul(q, q, expert_offsets=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(c.Nvfp4Error):
        c.mxfp4_linear(x, q, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
