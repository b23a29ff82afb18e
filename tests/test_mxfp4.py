"""MXFP4 and the balance loss on the CPU: the oracles against second
definitions, the binding's and the library's refusals, the headers."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from _util import ROOT, capi
from oracle import balance, mxfp4


# --- oracles -----------------------------------------------------------------

def test_e2m1_rounding_against_the_seven_midpoints():
    y = np.arange(-9 * 1024, 9 * 1024 + 1) / 1024.0
    a = np.abs(y)
    m = ((a > 0.25).astype(int) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    assert np.array_equal(mxfp4.round_e2m1(y), m | (np.signbit(y) << 3))


def test_mxfp4_scale_and_values():
    x = np.zeros((7, 40))
    x[0, 0] = 7.9                      # floor(log2) = 2: scale 1, clamped to 6
    x[1, :3] = [8.0, 5.0, 0.25]        # scale 2: 4 * 2, 2.5 -> tie to 2, 0.125 -> 0
    x[2, 33] = -3 * 2.0 ** -140        # below the smallest scale: 2^-127 stays
    x[3, 1] = np.inf
    x[4, 39] = np.nan
    x[5, :2] = [2.0 ** 127 * 1.75, -2.0 ** 120]
    codes, scales = mxfp4.quantize(x)
    assert codes.shape == (7, 32) and scales.shape == (7, 2)
    assert scales[:, 0].tolist() == [127, 128, 0, 255, 0, 252, 0]
    assert scales[:, 1].tolist() == [0, 0, 0, 0, 255, 0, 0]
    v = mxfp4.dequantize(codes, scales, 40)
    assert v[0, 0] == 6.0 and v[1, :3].tolist() == [8.0, 4.0, 0.0]
    assert v[2, 33] == 0.0 and np.isnan(v[3, :32]).all() and (v[3, 32:] == 0).all() and np.isnan(v[4, 32:]).all()
    assert v[5, 0] == 6 * 2.0 ** 125 and (v[6] == 0).all()
    # quantising the values again changes nothing
    ok = np.array([0, 1, 2, 5, 6])
    assert np.array_equal(mxfp4.dequantize(*mxfp4.quantize(v[ok]), 40), v[ok])


def test_quantising_values_again_keeps_them():
    """Any codes under any scale up to 2^125 (what 6 times it leaves finite):
    the block's new scale may be smaller, the values stay."""
    rng = np.random.default_rng(2)
    codes = rng.integers(0, 256, (2000, 32), dtype=np.uint8)
    codes[:500] &= 0x33                                    # blocks of small elements
    codes[500:600] &= 0x11
    codes[600:700] = 0
    scales = rng.integers(0, 253, (2000, 2), dtype=np.uint8)
    scales[:50] = 0
    v = mxfp4.dequantize(codes, scales, 64)
    assert np.array_equal(mxfp4.dequantize(*mxfp4.quantize(v), 64), v)


def test_mxfp4_error_is_within_half_a_step():
    x = np.random.default_rng(0).standard_normal((50, 320)) * 3
    codes, scales = mxfp4.quantize(x)
    v = mxfp4.dequantize(codes, scales, 320)
    s = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=1)
    y = np.abs(x) / s
    assert (y < 8).all()
    # half the local spacing (0.25, 0.5, 1), or the distance to 6 where clamped
    half = np.where(y > 6, y - 6, np.where(y > 4, 1.0, np.where(y > 2, 0.5, 0.25)))
    assert (np.abs(v - x) <= half * s * (1 + 1e-12)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(score):
    rng = np.random.default_rng(1)
    T, E, k = 12, 6, 2
    l = rng.standard_normal((T, E)) * 2
    l[3, 2] = -np.inf
    idx = np.argsort(-l, axis=1)[:, :k]
    mask = np.ones(T, bool)
    mask[5] = False
    off = np.array([0, 4, 4, 9, 11])           # an empty sequence; token 11 in none
    args = (idx, 0.3, score, mask, off)
    ref = balance.balance_loss(l, *args)
    assert ref["tokens"].tolist() == [4, 0, 4, 2, 3]
    assert (ref["dlogits"][5] == 0).all() and (ref["dlogits"][11] == 0).all() and ref["dlogits"][3, 2] == 0
    h = 1e-6
    for t in range(T):
        for e in range(E):
            if np.isinf(l[t, e]):
                continue
            up, dn = l.copy(), l.copy()
            up[t, e] += h
            dn[t, e] -= h
            num = (balance.balance_loss(up, *args)["loss"] - balance.balance_loss(dn, *args)["loss"]) / (2 * h)
            # central difference: h^2 |f'''| / 6 and the loss's rounding over 2 h
            assert abs(num - ref["dlogits"][t, e]) <= 1e-9


def test_balance_of_uniform_routing_is_coeff():
    """Equal counts and equal shares: <f, P> = E * (1/E) = 1 per sequence."""
    E, k = 8, 2
    idx = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(16)])
    for score in ("softmax", "sigmoid"):
        r = balance.balance_loss(np.zeros((16, E)), idx, 0.01, score)
        assert abs(r["loss"] - 0.01) < 1e-15 and np.abs(r["dlogits"]).max() < 1e-18


# --- refusals ----------------------------------------------------------------

FAKE = ctypes.c_void_p(0x1000)


def test_quantiser_refusals():
    lib = capi().lib
    q = lambda x=FAKE, dt=0, r=4, c=64, st=64, perm=None, n=0, lay=1, co=FAKE, sc=FAKE: \
        lib.mxfp4_quantize(x, dt, r, c, st, perm, n, lay, co, sc, None)  # noqa: E731
    assert q(x=None) == 1 and b"NULL" in lib.nvfp4_last_error()
    assert q(dt=3) == 1 and q(r=-1) == 1 and q(c=0) == 1 and q(st=63) == 1 and q(lay=2) == 1
    assert q(co=None) == 1 and q(sc=None) == 1 and q(co=ctypes.c_void_p(0x1008)) == 1
    assert q(x=ctypes.c_void_p(0x1001)) == 1 and q(perm=FAKE, n=-1) == 1
    assert q(c=(1 << 30) + 1, st=1 << 31) == 2
    assert q(r=(1 << 31) - 1, c=1 << 20, st=1 << 20) == 2            # 2^51 elements
    assert q(r=0) == 0 and q(perm=FAKE, n=0) == 0                      # nothing to do
    t = lambda r=4, c=64, st=64, lay=1, dt=0: \
        lib.mxfp4_quantize_transposed(FAKE, dt, r, c, st, lay, FAKE, FAKE, None)  # noqa: E731
    assert t(r=0) == 1 and t(lay=2) == 1 and t(st=1) == 1 and t(dt=-1) == 1 and t(r=(1 << 31) - 1) == 2
    d = lambda r=4, c=64, st=64, lay=1, dt=0, o=FAKE: \
        lib.mxfp4_dequantize(FAKE, FAKE, lay, r, c, dt, o, st, None)  # noqa: E731
    assert d(o=None) == 1 and d(lay=3) == 1 and d(st=5) == 1 and d(r=0) == 0
    # sizes
    assert lib.mxfp4_scale_bytes(3, 33, 0) == 6 and lib.mxfp4_scale_bytes(3, 33, 1) == 512
    assert lib.mxfp4_scale_bytes(129, 160, 1) == 2 * 2 * 512 and lib.mxfp4_scale_bytes(1, 32, 2) == 0
    assert lib.mxfp4_scale_bytes(-1, 32, 1) == 0


def test_product_refusals():
    lib = capi().lib

    def mm(a=FAKE, M=4, b=FAKE, N=128, K=64, E=0, off=None, cnt=None, rw=None, bias=None, dt=0, y=FAKE, st=128,
           ws=FAKE, n=256):
        return lib.mxfp4_matmul(a, FAKE, M, b, FAKE, N, K, E, off, cnt, rw, bias, dt, y, st, ws, n, None)
    assert mm(a=None) == 1 and mm(b=None) == 1 and mm(y=None) == 1
    assert mm(M=-1) == 1 and mm(N=0) == 1 and mm(K=0) == 1 and mm(dt=3) == 1 and mm(st=127) == 1
    assert mm(E=2) == 1 and mm(off=FAKE) == 1 and mm(cnt=FAKE) == 1            # E and the offsets go together
    assert mm(E=2, off=FAKE, N=130, st=130) == 2 and mm(E=1025, off=FAKE) == 2
    assert mm(a=ctypes.c_void_p(0x1008)) == 1 and mm(y=ctypes.c_void_p(0x1001)) == 1
    assert mm(n=255) == 5 and mm(ws=None) == 5 and mm(ws=ctypes.c_void_p(0x1010)) == 5
    assert mm(K=(1 << 30) + 1) == 2 and mm(M=(1 << 30) + 1, N=1, st=1) == 2 and mm(M=1 << 30, N=1 << 20, st=1 << 20) == 2
    assert mm(M=0) == 0

    def lin(x=FAKE, dt=0, r=4, st=64, perm=None, n=0, N=128, K=64, ws=FAKE, wsn=1 << 20):
        return lib.mxfp4_linear(x, dt, r, st, perm, n, FAKE, FAKE, N, K, 0, None, None, None, None, 0, FAKE, 128, ws,
                                wsn, None)
    assert lin(x=None) == 1 and lin(st=63) == 1 and lin(perm=FAKE, n=-2) == 1 and lin(wsn=256) == 5
    assert lin(r=0) == 0
    c = capi()
    assert c.mxfp4_linear_workspace_size(4, 64) == 256 + 256 + 512
    assert c.mxfp4_linear_workspace_size(-1, 64) == 0


def test_product_plans():
    """Host arithmetic: every plan fits the kernels' limits, and the sizes
    that the GPU tests use reach each of their variants."""
    c = capi()
    plan = c.nvfp4_test_mxfp4_plan
    sizes = (1, 2, 15, 16, 17, 64, 65, 128, 129, 255, 256, 257, 384, 385, 1000, 4096, 8192, 100000)
    for M in sizes:
        for N in sizes:
            for K in (1, 32, 256, 257, 2048, 6144, 16384):
                nt, splits, pair, stages = plan(M, N, K)
                kt = -(-K // 256)
                assert 1 <= splits <= 8 and splits <= kt
                assert nt % 16 == 0 and (nt == 384) == pair
                assert nt >= min(M, 128) and stages >= 3
                if not pair:
                    assert nt <= 128
                    # the split's partial sums fit the stages they overlay
                    stage = 16384 + nt * 128 + 2048
                    assert splits == 1 or nt * 512 <= stages * stage
                    assert stages * stage + 1024 <= 227 * 1024 - 256
            for E in (1, 8, 80, 481, 1024):
                if N % 128 == 0 and M % 128 == 0:
                    nt, splits, pair, stages = plan(M, N, 2048, E)
                    assert nt in (128, 384) and splits == 1 and not (pair and E > 480) and stages >= 3
                    if not pair:
                        assert stages * 34816 + (3 * E + 1) * 4 + 1024 <= 227 * 1024 - 256
    assert plan(1, 6144, 512)[1] == 1 and plan(16, 128, 6144)[1] == 4 and plan(100, 300, 2048)[1] == 1 and plan(100, 300, 6144)[1] == 4
    assert plan(1, 1000, 4096) == (16, 4, False, 5)
    for M, N, K in ((2990, 2290, 1900), (3000, 2049, 1700)):
        assert plan(M, N, K)[2]
    assert plan(3456, 2048, 1700, 4)[2] and plan(3456, 1920, 1900, 4)[2] and plan(1152, 512, 96, 3)[0] == 128
    # alone on an SM (six stages), and two on an SM (three)
    assert plan(256, 256, 256) == (128, 1, False, 6) and plan(3000, 1000, 96) == (128, 1, False, 3)
    for bad in ((0, 1, 1), ((1 << 30) + 1, 1, 1), (1, 1, 1, 1025)):
        with pytest.raises(ValueError):
            plan(*bad)


def test_products_that_share_an_sm_fit_it():
    """Host arithmetic: the CTAs that a plan puts on an SM fit its shared
    memory (228 KiB, 1 KiB of it taken by each CTA, and 256 bytes of static
    variables) and its 512 columns of tensor memory, whose allocation would
    otherwise wait for the other CTA's end."""
    c = capi()
    seen = set()
    sizes = (1, 16, 17, 32, 33, 48, 64, 65, 128, 129, 256, 1000, 3000, 4096, 20000, 100000)
    for M in sizes:
        for N in (1, 128, 384, 1024, 6144, 12288, 18944, 100096):
            for K in (1, 256, 300, 2048, 6144, 20000):
                for E in (0, 1, 8, 80, 480, 481, 1024):
                    if E and N % 128:
                        continue
                    nt, splits, pair, stages = c.nvfp4_test_mxfp4_plan(M, N, K, E)
                    ctas, smem, columns = c.nvfp4_test_mxfp4_residency(M, N, K, E)
                    seen.add((ctas, columns, splits > 1, pair))
                    assert ctas in (1, 2) and columns in (64, 128, 256, 512)
                    assert smem <= 228 * 1024 // ctas - 1024 - 256
                    assert ctas * columns <= 512 and (not pair or columns == 512)
                    # an accumulator's columns and two 4-column scale atoms of either operand
                    assert pair or columns >= max(nt, 32) + 16
                    # what a few tokens are planned for
                    assert pair or nt > 64 or E or ctas == 2
    assert {(2, 128, True, False), (2, 256, False, False), (1, 512, False, False), (1, 512, False, True)} <= seen
    for M in (1, 16):                                    # fused: one accumulator of 32 columns and the scales
        ctas = c.nvfp4_test_mxfp4_fuses(M, 1024, 6144, torch.bfloat16)[1]
        assert ctas * 64 <= 512
    with pytest.raises(ValueError):
        c.nvfp4_test_mxfp4_residency(0, 1, 1)


def test_segments_of_grouped_products():
    """Host arithmetic shared with the kernels: whatever the number of rows,
    each expert has the clamped rows of its own segment and no others."""
    seg = capi().nvfp4_test_mxfp4_segments
    rows = lambda s: [(a, n) for a, n in s if n]  # noqa: E731
    # segments that start at or past the rows' end are empty: no 128-row tile is taken twice
    assert rows(seg([0, 384, 384], None, 300)) == [(0, 300)]
    assert rows(seg([0, 384, 384], [300, 0], 300)) == [(0, 300)]
    assert rows(seg([0, 384, 512, 512], [300, 77, 9], 300)) == [(0, 300)]
    assert rows(seg([0, 128, 256, 384, 640], None, 257)) == [(0, 128), (128, 128), (256, 1)]
    assert rows(seg([-128, 128, 1 << 30, 0], [1 << 30, 1 << 30, -5], 256)) == [(0, 128), (128, 128)]
    assert rows(seg([-2 ** 31, 2 ** 31 - 1], None, 1)) == [(0, 1)] and rows(seg([0, 128], None, 0)) == []
    assert rows(seg([0, 100, 256], None, 256)) == [(0, 100)]           # a start inside a scale tile
    rng = np.random.default_rng(0)
    for _ in range(2000):
        E, M = int(rng.integers(1, 12)), int(rng.integers(0, 1500))
        off = np.concatenate([[rng.integers(-2, 2)], rng.integers(0, 4, E)]).cumsum() * 128
        cnt = [int(v) for v in rng.integers(-10, 500, E)] if rng.random() < 0.5 else None
        owner = np.full(M, -1)
        for e, (a, n) in enumerate(seg([int(v) for v in off], cnt, M)):
            assert n >= 0 and (n == 0 or (a % 128 == 0 and 0 <= a and a + n <= M))
            assert (owner[a:a + n] == -1).all()
            owner[a:a + n] = e
        lim = np.clip(off, 0, M)
        want = np.full(M, -1)
        for e in range(E):
            n = lim[e + 1] - lim[e] if cnt is None else min(lim[e + 1] - lim[e], max(cnt[e], 0))
            want[lim[e]:lim[e] + n] = e
        assert np.array_equal(owner, want)
    with pytest.raises(ValueError):
        seg([0, 128], None, -1)


def test_products_that_quantise_their_rows():
    """Host arithmetic: shared memory and tiles of a fused mxfp4_linear fit."""
    c = capi()
    fuses = c.nvfp4_test_mxfp4_fuses
    seen = 0
    for M in (1, 2, 3, 5, 8, 12, 15, 16, 17, 64):
        for N in (1, 128, 1000, 1024, 6144, 12288, 18000, 18944, 37888, 100000):
            for K in (1, 32, 256, 257, 300, 2010, 2048, 4096, 6144, 8192, 16384, 1 << 20):
                for dt in (torch.bfloat16, torch.float16, torch.float32):
                    for wide in (True, False):
                        f = fuses(M, N, K, dt, wide)
                        if f is None:
                            continue
                        seen += 1
                        stages, per_sm = f
                        nt, splits, pair, _ = c.nvfp4_test_mxfp4_plan(M, N, K)
                        share = -(-(-(-K // 256)) // splits)           # K stages of a CTA
                        assert M <= 16 and nt == 16 and not pair and 3 <= stages <= 8 and share <= 32
                        assert -(-N // 128) * splits <= 148 * per_sm
                        smem = stages * 17408 + share * (16 * 128 + 1024) + 1024
                        assert smem <= (227 * 1024 - 512 if per_sm == 1 else 228 * 512 - 1024 - 512)
                        assert nt * 512 <= stages * 17408              # the split's partial sums
    assert seen > 500
    for M, N, K in ((17, 1024, 6144), (16, 6144, 6144), (1, 100000, 512), (1, 128, 1 << 20)):
        assert fuses(M, N, K, torch.bfloat16) is None
    with pytest.raises(ValueError):
        fuses(0, 1, 1, torch.float32)


def test_balance_refusals():
    lib = capi().lib

    def f(l=FAKE, dt=2, T=4, E=8, st=8, idx=FAKE, k=2, sc=0, off=None, S=1, loss=FAKE, ws=FAKE, n=1 << 20):
        return lib.moe_balance_loss(l, dt, T, E, st, idx, k, sc, None, off, S, 0.1, loss, FAKE, FAKE, FAKE, ws, n,
                                    None)
    assert f(l=None) == 1 and f(idx=None) == 1 and f(loss=None) == 1 and f(dt=3) == 1 and f(sc=2) == 1
    assert f(T=-1) == 1 and f(S=0) == 1 and f(S=2) == 1 and f(st=7) == 1 and f(l=ctypes.c_void_p(0x1002)) == 1
    assert f(E=0) == 2 and f(E=1025, st=1025) == 2 and f(k=0) == 2 and f(k=33) == 2
    assert f(n=256) == 5 and f(ws=None) == 5

    other = ctypes.c_void_p(0x2000)

    def b(T=4, E=8, gs=8, d=other, g=FAKE):
        return lib.moe_balance_loss_backward(FAKE, 2, T, E, 8, 2, 0, None, None, 1, 0.1, FAKE, FAKE, g, d, gs, None)
    assert b(d=FAKE) == 1 and b"place" in lib.nvfp4_last_error()
    assert b(gs=7) == 1 and b(d=None) == 1 and b(g=None) == 1 and b(E=2000) == 2 and b(T=0) == 0
    c = capi()
    assert c.moe_balance_loss_workspace_size(0, 8) > 0 and c.moe_balance_loss_workspace_size(4, 0) == 0


def test_balance_gradient_over_part_of_the_logits_is_refused():
    """Logits of 4 x 8 fp32, rows `st` elements apart, at 0x10000.  A call that
    is not refused for its memory is refused for the misaligned grad_loss
    behind it, so nothing is launched."""
    lib = capi().lib
    base = 0x10000

    def refused(by, st=8, gs=None, T=4, dt=2, E=8):
        r = lib.moe_balance_loss_backward(ctypes.c_void_p(base), dt, T, E, st, 2, 0, None, None, 1, 0.1, FAKE, FAKE,
                                          ctypes.c_void_p(0x1001), ctypes.c_void_p(base + by), gs or st, None)
        assert r == 1
        return b"place" in lib.nvfp4_last_error()
    assert refused(0) and refused(0, T=1) and refused(0, st=20)
    for rows in (1, 2, 3, -1, -3):                       # shifted by rows
        assert refused(32 * rows) and refused(80 * rows, st=20)
    assert not refused(128) and not refused(-128) and not refused(32, T=1) and refused(28, T=1)
    assert refused(4) and refused(-4) and refused(124) and refused(-124)
    # other columns of one buffer: apart while the rows do not meet
    assert not refused(32, st=20) and not refused(48, st=20) and refused(28, st=20) and refused(52, st=20)
    assert not refused(32, st=16) and not refused(-32, st=16) and refused(36, st=16)
    assert not refused(80 + 40, st=20) and not refused(-80 + 40, st=20) and refused(-80 + 52, st=20)
    # other strides over the same memory are refused, over other memory not
    assert refused(32, st=20, gs=24) and refused(0, st=16, gs=8) and not refused(320, st=20, gs=8)
    # two-byte elements; T and strides whose extent passes 32 bits
    assert refused(16, dt=0) and not refused(64, dt=0) and not refused(16, st=16, dt=0)
    big = 1 << 20
    assert refused(4 * big * 4095, st=big, T=4096) and not refused(4 * big * 4095 + 32, st=big, T=4096)


class ShapeOnly(torch.Tensor):
    """A tensor without memory that the binding takes for one on the device."""
    is_cuda = True

    @staticmethod
    def of(*shape, dtype):
        return torch.Tensor._make_subclass(ShapeOnly, torch.empty(*shape, dtype=dtype, device="meta"))


def test_sizes_past_32_bits_are_refused():
    """2^32 + 4 rows must not reach the library as 4."""
    c = capi()
    n = 2 ** 32 + 4
    t = ShapeOnly.of
    small, idx = t(4, 8, dtype=torch.float32), t(4, 2, dtype=torch.int32)
    long_idx = t(n, dtype=torch.int32)
    q = c.Mxfp4.__new__(c.Mxfp4)
    q.codes, q.scales, q.rows, q.cols, q.layout = t(4, 16, dtype=torch.uint8), t(512, dtype=torch.uint8), 4, 8, "tiled"
    for call in (lambda: c.mxfp4_quantize(t(n, 8, dtype=torch.bfloat16)),
                 lambda: c.mxfp4_quantize(t(4, n, dtype=torch.bfloat16)),
                 lambda: c.mxfp4_quantize(t(2 ** 31, 2, 2, dtype=torch.float16)),
                 lambda: c.mxfp4_quantize(small, perm=long_idx),
                 lambda: c.mxfp4_quantize_transposed(t(n, 8, dtype=torch.float32)),
                 lambda: c.mxfp4_dequantize(q, out=t(n, 8, dtype=torch.float32)),
                 lambda: c.Mxfp4(t(n, 16, dtype=torch.uint8), t(2 ** 40, dtype=torch.uint8), n, 8),
                 lambda: c.mxfp4_linear(t(n, 8, dtype=torch.float32), q),
                 lambda: c.mxfp4_linear(small, q, perm=long_idx),
                 lambda: c.mxfp4_matmul(q, q, expert_offsets=long_idx),
                 lambda: c.mxfp4_linear_workspace_size(n, 8), lambda: c.mxfp4_linear_workspace_size(8, n),
                 lambda: c.moe_balance_loss(t(n, 8, dtype=torch.float32), t(n, 2, dtype=torch.int32), 0.1),
                 lambda: c.moe_balance_loss(small, t(4, n, dtype=torch.int32), 0.1),
                 lambda: c.moe_balance_loss(small, idx, 0.1, seq_offsets=long_idx),
                 lambda: c.moe_balance_loss_workspace_size(n, 8), lambda: c.moe_balance_loss_workspace_size(4, 8, n)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_backward_refuses_logits_of_another_length():
    """The counts hold for the forward call's tokens; without a mask nothing
    else tells the two calls' lengths apart."""
    c = capi()
    t = ShapeOnly.of
    fwd = c.BalanceLoss(t(1, dtype=torch.float32), t(1, 8, dtype=torch.int32), t(2, dtype=torch.int32),
                        t(1, 8, dtype=torch.float32), 2, "sigmoid", 0.1, None, None, 6)
    for T in (0, 5, 7):
        with pytest.raises(ValueError, match=f"{T} tokens"):
            c.moe_balance_loss_backward(t(T, 8, dtype=torch.float32), fwd, t(1, dtype=torch.float32))


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    c = capi()
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: c.mxfp4_quantize(x), lambda: c.mxfp4_quantize_transposed(x),
                 lambda: c.Mxfp4(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 4, 64),
                 lambda: c.moe_balance_loss(x.float(), torch.zeros(4, 2, dtype=torch.int32), 0.1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("header", ["mxfp4.h", "moe_balance.h"])
@pytest.mark.parametrize("lang", [("c", "-std=c99"), ("c++", "-std=c++17")])
def test_headers_compile_as_plain_c_and_cpp(header, lang):
    cc = shutil.which("gcc" if lang[0] == "c" else "g++")
    if cc is None:
        pytest.skip("no host compiler")
    r = subprocess.run([cc, "-fsyntax-only", lang[1], "-Wall", "-Wextra", "-Werror", "-x", lang[0],
                        os.path.join(ROOT, "include", header)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
