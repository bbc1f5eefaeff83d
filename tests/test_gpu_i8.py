"""GPU parity of the 8-bit operators against the 64-bit oracle, through the
Python binding.

Codes and token scales are compared exactly.  Products are held to the
oracle's bound (the fp32 roundings that include/q4i8.h allows) plus half a
step of the output's type.  Sizes cover one row to many, rows and columns that
end inside a tile, K that ends inside a step, and groups that are empty, of
one row, or cross tiles.
"""

import sys
import threading

import numpy as np
import pytest
import torch

import memory_bandwidth_amd as q4
from oracle import i8

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def codes(seed, *shape):
    """Every int8 value, -128 among them."""
    return np.random.default_rng(seed).integers(-128, 128, shape, dtype=np.int8)


def scales(seed, *shape):
    return np.random.default_rng(seed).uniform(0.0005, 0.02, shape).astype(np.float32)


def small_scales(seed, K, *shape):
    """Scales that bring products of random codes near 1, whatever K."""
    return (np.random.default_rng(seed).uniform(0.5, 2, shape) / (74 * K ** 0.25)).astype(np.float32)


def check(y, want, bound, t, label):
    got = y.float().cpu().numpy().astype(np.float64)
    tol = i8.tolerance(want, bound, t)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{label}: {int(bad.sum())} of {bad.size} outside, first at {np.argwhere(bad)[0]}, worst "
                           f"{np.nanmax(np.abs(got - want) / tol):.3g} of the tolerance")


# ---------------------------------------------------------------- quant_i8

@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (65, 128), (7, 896), (33, 1040), (2, 4096), (5, 14336), (3, 32784),
                                 (1, 131056), (1030, 272)])
def test_quant(t, M, K):
    x = torch.from_numpy(np.random.default_rng(M * K).standard_normal((M, K)).astype(np.float32)).to(TYPES[t])
    x[:, 5] *= 11
    c, s = q4.quant_i8(x.to(DEV))
    cw, sw = i8.quant(x.double().numpy())
    assert np.array_equal(s.cpu().numpy(), sw)
    assert np.array_equal(c.cpu().numpy(), cw)


@pytest.mark.parametrize("t", TYPES)
def test_quant_ties_and_special_rows(t):
    K = 528
    rng = np.random.default_rng(9)
    x = np.zeros((12, K), dtype=np.float32)
    x[0] = rng.integers(-254, 255, K) / 2                  # scale 1: half of the values are ties
    x[0, 3] = 127
    x[1] = rng.integers(-254, 255, K) * 0.375              # scale 0.75
    x[1, 3] = -127 * 0.75
    x[3] = rng.standard_normal(K)
    x[3, 100] = np.inf
    x[4] = rng.standard_normal(K)
    x[4, K - 1] = np.nan
    x[5, 0] = -np.inf
    x[6] = rng.standard_normal(K) * 1e-6
    x[7] = rng.standard_normal(K) * 100
    x[8, 17] = 2.0 ** -24                                  # alone in its row
    x[9] = 1.0
    x[10, K - 1] = -3.0
    x[11] = rng.standard_normal(K)
    if t == "f32":
        x[6] = rng.integers(-9, 10, K) * 2.0 ** -149       # subnormal
        x[7] = rng.standard_normal(K) * 8e37
        x[8] = rng.integers(-254, 255, K) * 2.0 ** -127    # scale 2^-126, ties
        x[8, 1] = 127 * 2.0 ** -126
    xt = torch.from_numpy(x).to(TYPES[t])
    c, s = q4.quant_i8(xt.to(DEV))
    cw, sw = i8.quant(xt.double().numpy())
    assert np.array_equal(s.cpu().numpy(), sw, equal_nan=True)
    assert np.array_equal(c.cpu().numpy(), cw)


def test_quant_near_ties():
    """Quotients within a few ulp of n + 1/2, on both sides and on it."""
    K = 4096
    rng = np.random.default_rng(4)
    s = np.float32(0.0123456789)
    x = ((rng.integers(-126, 126, K) + 0.5) * np.float64(s)).astype(np.float32)
    x = (x.view(np.int32) + rng.integers(-2, 3, K).astype(np.int32)).view(np.float32)
    x[0] = np.float32(127) * s
    c, got = q4.quant_i8(dev(x[None]))
    cw, sw = i8.quant(x[None].astype(np.float64))
    assert np.array_equal(got.cpu().numpy(), sw) and np.array_equal(c.cpu().numpy(), cw)


# ---------------------------------------------------------------- gemm_i8

GEMM = [(1, 1, 16), (1, 17, 48), (1, 896, 896), (1, 300, 4096), (2, 64, 128), (3, 129, 144), (8, 1000, 1040),
        (15, 33, 4096), (16, 16, 64), (17, 257, 272), (31, 130, 14336), (32, 512, 2816), (48, 100, 912),
        (64, 64, 128), (65, 127, 256), (100, 896, 4864), (128, 256, 1024), (129, 300, 1040), (200, 333, 2064),
        (256, 256, 256), (257, 511, 528), (300, 1024, 896), (511, 520, 4112), (700, 777, 1296), (1025, 1030, 400),
        (2049, 260, 144), (260, 4100, 208)]


@pytest.mark.parametrize("M,N,K", GEMM)
@pytest.mark.parametrize("t", TYPES)
def test_gemm(M, N, K, t):
    a, w, sa, sw = codes(1, M, K), codes(2, N, K), small_scales(3, K, M), small_scales(4, K, N)
    y = q4.gemm_i8(dev(a), dev(sa), dev(w), dev(sw), dtype=TYPES[t])
    assert y.dtype == TYPES[t]
    check(y, *i8.gemm(a, sa, w, sw), t, f"{M} {N} {K}")


# Every tile that the products choose from, with rows and columns that end
# inside tiles and K inside steps, and more tiles than workgroups.
LARGE = [(64, 4100, 2064), (500, 2050, 2064), (330, 4870, 912), (1090, 5000, 528), (3775, 1827, 1056),
         (3984, 3781, 656), (2900, 5050, 528), (4100, 4100, 272), (5000, 300, 4112), (64, 3999, 4112),
         (230, 3313, 400), (36, 1373, 32), (126, 2093, 6016), (64, 4090, 14336), (128, 3990, 4112)]
LARGE_SWIGLU = [(64, 2100, 2064), (300, 1000, 2064), (200, 2320, 912), (1060, 2500, 528), (2593, 1533, 800),
                (2365, 3095, 432), (1500, 4100, 400), (96, 999, 4112), (67, 3422, 368), (40, 1100, 1040),
                (40, 499, 8208), (40, 1373, 48), (100, 1789, 6160)]


@pytest.mark.parametrize("M,N,K", LARGE)
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_gemm_large(M, N, K, t):
    a, w, sa, sw = codes(1, M, K), codes(2, N, K), small_scales(3, K, M), small_scales(4, K, N)
    y = q4.gemm_i8(dev(a), dev(sa), dev(w), dev(sw), dtype=TYPES[t])
    check(y, *i8.gemm(a, sa, w, sw), t, f"{M} {N} {K}")


@pytest.mark.parametrize("M,N,K", LARGE_SWIGLU)
def test_swiglu_large(M, N, K):
    a, sa = codes(1, M, K), small_scales(3, K, M)
    gate, up = (codes(2, N, K), small_scales(4, K, N) * 3), (codes(5, N, K), small_scales(6, K, N))
    y = q4.gemm_i8_swiglu(dev(a), dev(sa), tuple(map(dev, gate)), tuple(map(dev, up)), dtype=torch.float16)
    check(y, *i8.swiglu(a, sa, gate, up), "f16", f"{M} {N} {K}")


def exact_rows(a, sa, w, sw):
    """P in float64 on the GPU, where the sums are exact as in the oracle, for sizes too large for it."""
    return (dev(a).double() @ dev(w).double().t()) * dev(sa).double()[:, None] * dev(sw).double()


@pytest.mark.parametrize("M,N,K", [(4300, 4100, 2064), (4096, 5300, 2000), (8200, 4097, 1040), (4300, 5000, 2064)])
@pytest.mark.parametrize("groups", [0, 3])
@pytest.mark.parametrize("swiglu", [False, True])
def test_last_round_halved(M, N, K, groups, swiglu):
    """A last round of few tiles, taken by halved ones, whose quarters may lie past the rows or columns."""
    N = (N + 1) // 2 if swiglu else N
    E = max(groups, 1)
    K = K * 5 if groups else K                              # long enough for the largest tiles
    off = [0, M // 2 - 3, M - 1500, M] if groups else [0, M]
    a, sa = codes(1, M, K), small_scales(3, K, M)
    gate, up = (codes(2, E, N, K), small_scales(4, K, E, N)), (codes(5, E, N, K), small_scales(6, K, E, N))
    mats = 2 if swiglu else 1
    g = q4.gemm_i8_geometry(mats, M, N, K, groups)
    assert (g["tile_rows"], g["tile_cols"]) == (256, 256 // mats)
    if groups:
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        y = (q4.gemm_i8_grouped_swiglu(dev(a), dev(sa), tuple(map(dev, gate)), tuple(map(dev, up)), o) if swiglu else
             q4.gemm_i8_grouped(dev(a), dev(sa), *map(dev, gate), o))
    else:
        y = (q4.gemm_i8_swiglu(dev(a), dev(sa), (dev(gate[0][0]), dev(gate[1][0])), (dev(up[0][0]), dev(up[1][0])))
             if swiglu else q4.gemm_i8(dev(a), dev(sa), dev(gate[0][0]), dev(gate[1][0])))
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        p = exact_rows(a[rows], sa[rows], gate[0][e], gate[1][e])
        bound = 3.1 * i8.U * p.abs()
        if swiglu:                                          # as i8.swiglu
            u = exact_rows(a[rows], sa[rows], up[0][e], up[1][e])
            s = p * torch.sigmoid(p)
            ds = 1.1 * bound + s.abs() * (2 * p.abs() + 9) * i8.U
            p, bound = s * u, 1.01 * (u.abs() * ds + s.abs() * 3.1 * i8.U * u.abs()) + u.abs() * 2.0 ** -118
        tol = bound + 2.0 ** -24 * (p.abs() + bound)
        assert ((y[rows].double() - p).abs() <= tol).all(), f"expert {e}"


def test_sizes_take_every_tile():
    for mats, shapes, tiles in ((1, GEMM + LARGE, {(8,), (16,), (32,), (64, 32), (64, 64), (64, 128), (128, 128),
                                                   (128, 256), (256, 256)}),
                                (2, LARGE_SWIGLU, {(8,), (16,), (32,), (64, 16), (64, 32), (64, 64), (128, 64),
                                                   (128, 128), (256, 128)})):
        got = [q4.gemm_i8_geometry(mats, *s) for s in shapes]
        seen = {(g["tile_rows"], g["tile_cols"]) for g in got} | {(g["tile_rows"],) for g in got}
        assert tiles <= seen, tiles - seen
        assert {g["block"] for g in got if g["tile_rows"] <= 32} == {256, 512}
        # Both kinds of launch: a workgroup for each tile, and workgroups that go through several.
        many = [g["grid"] < -(-s[0] // g["tile_rows"]) * -(-s[1] // g["tile_cols"]) for g, s in zip(got, shapes)]
        assert any(many) and not all(many)


@pytest.mark.parametrize("M,N,K", [(1, 77, 256), (40, 520, 144), (130, 64, 1024), (600, 515, 400)])
@pytest.mark.parametrize("t", TYPES)
def test_gemm_bias(M, N, K, t):
    a, w, sa, sw = codes(1, M, K), codes(2, N, K), small_scales(3, K, M), small_scales(4, K, N)
    b = np.random.default_rng(5).standard_normal(N).astype(np.float32) * 3
    y = q4.gemm_i8(dev(a), dev(sa), dev(w), dev(sw), bias=dev(b), dtype=TYPES[t])
    check(y, *i8.gemm(a, sa, w, sw, b), t, f"{M} {N} {K}")


@pytest.mark.parametrize("M,N", [(1, 5), (20, 18), (70, 70), (300, 260)])
def test_gemm_largest_sums(M, N):
    """-128 x -128 at the longest K, and its negative: the sums reach 2147221504."""
    K = 131056
    a, w = np.full((M, K), -128, dtype=np.int8), np.full((N, K), -128, dtype=np.int8)
    w[1::2] = 127
    one = np.ones(max(M, N), dtype=np.float32)
    y = q4.gemm_i8(dev(a), dev(one[:M]), dev(w), dev(one[:N])).cpu().numpy()
    want = np.where(np.arange(N) % 2 == 0, 16384.0 * K, -128.0 * 127 * K).astype(np.float32)
    assert np.array_equal(y, np.broadcast_to(want, (M, N)))


@pytest.mark.parametrize("M", [1, 9, 40, 100, 600])
def test_gemm_rows_do_not_mix(M):
    """A NaN scale, a zero row and huge scales stay in their rows and columns."""
    N, K = 150, 400
    a, w, sa, sw = codes(1, M, K), codes(2, N, K), scales(3, M), scales(4, N)
    a[M // 2] = 0
    sa[M - 1] = np.nan
    sw[3] = np.inf
    want = i8.product(a, sa, w, sw)
    y = q4.gemm_i8(dev(a), dev(sa), dev(w), dev(sw)).cpu().numpy()
    assert np.array_equal(np.isnan(y), np.isnan(want)) and np.isnan(y[M - 1]).all()
    fine = np.isfinite(want)
    assert np.array_equal(fine, np.isfinite(y))
    assert (np.abs(y[fine] - want[fine]) <= 4.1 * i8.U * np.abs(want[fine])).all()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,N", [(1, 40), (5, 64), (70, 72), (300, 264)])
@pytest.mark.parametrize("skew", [0, 1])
def test_gemm_out_in_a_larger_buffer(t, M, N, skew):
    """Outputs that start off a 16-byte border, with guards on both sides."""
    K = 160
    a, w, sa, sw = codes(1, M, K), codes(2, N, K), small_scales(3, K, M), small_scales(4, K, N)
    buf = torch.full((M * N + 32,), 7.0, dtype=TYPES[t], device=DEV)
    out = buf[8 + skew:8 + skew + M * N].view(M, N)
    y = q4.gemm_i8(dev(a), dev(sa), dev(w), dev(sw), dtype=TYPES[t], out=out)
    assert y.data_ptr() == out.data_ptr()
    check(y, *i8.gemm(a, sa, w, sw), t, f"{M} {N}")
    assert (buf[:8 + skew] == 7).all() and (buf[8 + skew + M * N:] == 7).all()


def test_gemm_empty():
    z = torch.zeros
    y = q4.gemm_i8(z(0, 64, dtype=torch.int8, device=DEV), z(0, device=DEV), z(5, 64, dtype=torch.int8, device=DEV),
                   z(5, device=DEV))
    assert tuple(y.shape) == (0, 5)
    c, s = q4.quant_i8(z(0, 64, device=DEV))
    assert tuple(c.shape) == (0, 64) and tuple(s.shape) == (0,)


# ---------------------------------------------------------------- swiglu

@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 896, 896), (4, 300, 4096), (16, 65, 144), (30, 1000, 1040),
                                   (64, 32, 128), (100, 130, 2816), (257, 200, 528), (520, 515, 1296)])
@pytest.mark.parametrize("t", TYPES)
def test_swiglu(M, N, K, t):
    a, sa = codes(1, M, K), small_scales(3, K, M)
    gate, up = (codes(2, N, K), small_scales(4, K, N) * 3), (codes(5, N, K), small_scales(6, K, N))
    y = q4.gemm_i8_swiglu(dev(a), dev(sa), tuple(map(dev, gate)), tuple(map(dev, up)), dtype=TYPES[t])
    check(y, *i8.swiglu(a, sa, gate, up), t, f"{M} {N} {K}")


def test_swiglu_far_gates():
    """Gates far to both sides: silu(g) -> g and -> 0, no NaN."""
    M, N, K = 3, 40, 64
    a, sa = codes(1, M, K), scales(3, M)
    gate, up = (codes(2, N, K), scales(4, N) * 5000), (codes(5, N, K), scales(6, N))
    y = q4.gemm_i8_swiglu(dev(a), dev(sa), tuple(map(dev, gate)), tuple(map(dev, up)))
    check(y, *i8.swiglu(a, sa, gate, up), "f32", "far")


# ---------------------------------------------------------------- grouped

GROUPS = {
    "one": [0, 37],
    "empty ends": [0, 0, 5, 5, 21, 21],
    "all in the last": [0, 0, 0, 90],
    "single rows": list(range(0, 18)),
    "tile borders": [0, 16, 48, 112, 240, 496, 497, 1009],
    "rows outside": [3, 20, 20, 85],
    "none": [0, 0, 0],
    "none, in the middle": [4, 4, 4, 4],
    "many": np.concatenate([[0], np.cumsum(np.random.default_rng(8).integers(0, 9, 150))]).tolist(),
    "uneven": [0, 1, 400, 402, 402, 700, 701],
    "more than a lane's": np.concatenate([[0], np.cumsum(np.random.default_rng(9).integers(0, 3, 301) ** 2)]).tolist(),
    "large and small": [0, 0, 1000, 1000, 1003, 1003, 1130, 2400, 2400],
}


@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("t,N,K", [("f32", 70, 144), ("bf16", 136, 400)])
def test_grouped(name, swiglu, t, N, K):
    off = GROUPS[name]
    E, M = len(off) - 1, off[-1] + 6                       # rows behind the last group
    a, sa = codes(1, M, K), small_scales(3, K, M)
    gate, up = (codes(2, E, N, K), small_scales(4, K, E, N)), (codes(5, E, N, K), small_scales(6, K, E, N))
    out = torch.full((M, N), 7.0, dtype=TYPES[t], device=DEV)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    if swiglu:
        y = q4.gemm_i8_grouped_swiglu(dev(a), dev(sa), tuple(map(dev, gate)), tuple(map(dev, up)), o, dtype=TYPES[t],
                                      out=out)
    else:
        y = q4.gemm_i8_grouped(dev(a), dev(sa), dev(gate[0]), dev(gate[1]), o, dtype=TYPES[t], out=out)
    inside = np.zeros(M, dtype=bool)
    for e, lo, hi in i8.groups(off):
        inside[lo:hi] = True
        g, u = (gate[0][e], gate[1][e]), (up[0][e], up[1][e])
        want = i8.swiglu(a[lo:hi], sa[lo:hi], g, u) if swiglu else i8.gemm(a[lo:hi], sa[lo:hi], *g)
        check(y[lo:hi], *want, t, f"{name} expert {e}")
    assert (y[torch.from_numpy(~inside).to(DEV)] == 7).all()


@pytest.mark.parametrize("E,rows", [(5000, 1), (5000, 700), (65536, 40)])
def test_grouped_many_experts(E, rows):
    """Few rows among very many experts."""
    N, K = 24, 32
    M = rows
    rng = np.random.default_rng(E)
    chosen = np.sort(rng.integers(0, E, M))
    off = np.concatenate([[0], np.cumsum(np.bincount(chosen, minlength=E))])
    a, sa = codes(1, M, K), small_scales(3, K, M)
    w, sw = codes(2, E, N, K), small_scales(4, K, E, N)
    y = q4.gemm_i8_grouped(dev(a), dev(sa), dev(w), dev(sw), torch.tensor(off, dtype=torch.int32, device=DEV))
    want = np.concatenate([i8.product(a[lo:hi], sa[lo:hi], w[e], sw[e]) for e, lo, hi in i8.groups(off)])
    check(y, want, 3.1 * i8.U * np.abs(want), "f32", f"{E}")


@pytest.mark.parametrize("M,N,K,E", [(2500, 4200, 1040, 4), (9000, 1030, 272, 3)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_goes_through_many_tiles(M, N, K, E, swiglu):
    N = N // 2 if swiglu else N
    off = [0, M // 3 + 1, M // 3 + 1, M - 50, M][:E] + [M]
    E = len(off) - 1
    a, sa = codes(1, M, K), small_scales(3, K, M)
    gate, up = (codes(2, E, N, K), small_scales(4, K, E, N)), (codes(5, E, N, K), small_scales(6, K, E, N))
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    if swiglu:
        y = q4.gemm_i8_grouped_swiglu(dev(a), dev(sa), tuple(map(dev, gate)), tuple(map(dev, up)), o)
    else:
        y = q4.gemm_i8_grouped(dev(a), dev(sa), dev(gate[0]), dev(gate[1]), o)
    for e, lo, hi in i8.groups(off):
        g, u = (gate[0][e], gate[1][e]), (up[0][e], up[1][e])
        want = i8.swiglu(a[lo:hi], sa[lo:hi], g, u) if swiglu else i8.gemm(a[lo:hi], sa[lo:hi], *g)
        check(y[lo:hi], *want, "f32", f"expert {e}")


@pytest.mark.parametrize("off", [[0, 50, 30, 80], [-5, 10, 900, 40], [70, 60, 50, 40], [2**31 - 1, -2**31, 5, 9]])
@pytest.mark.parametrize("M", [10, 40, 300])
def test_grouped_bad_offsets_stay_inside(off, M):
    """Offsets out of order and range: nothing outside y is written."""
    N, K, E = 40, 160, 3
    a, sa = codes(1, M, K), scales(3, M)
    w, sw = codes(2, E, N, K), scales(4, E, N)
    buf = torch.full((M * N + 64,), 7.0, device=DEV)
    out = buf[32:32 + M * N].view(M, N)
    q4.gemm_i8_grouped(dev(a), dev(sa), dev(w), dev(sw), torch.tensor(off, dtype=torch.int32, device=DEV), out=out)
    torch.cuda.synchronize()
    assert (buf[:32] == 7).all() and (buf[32 + M * N:] == 7).all() and torch.isfinite(out).all()


# ---------------------------------------------------------------- streams, graphs, whole layers

def layer(x, gate, up, down):
    """A feed-forward layer: quantise, gate and up, quantise, down."""
    c, s = q4.quant_i8(x)
    h = q4.gemm_i8_swiglu(c, s, gate, up, dtype=torch.bfloat16)
    c2, s2 = q4.quant_i8(h)
    return c, s, h, c2, s2, q4.gemm_i8(c2, s2, *down, dtype=torch.bfloat16)


def layer_problem(M, D, F, seed=1):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((M, D)).astype(np.float32)).bfloat16()
    gate = (codes(2, F, D), small_scales(4, D, F) * 10)
    up = (codes(5, F, D), small_scales(6, D, F) * 10)
    down = (codes(7, D, F), small_scales(8, F, D))
    return x, gate, up, down


@pytest.mark.parametrize("M", [1, 5, 33, 150, 300])
def test_layer(M):
    x, gate, up, down = layer_problem(M, 896, 1200)
    c, s, h, c2, s2, y = layer(x.to(DEV), *(tuple(map(dev, m)) for m in (gate, up, down)))
    cw, sw = i8.quant(x.double().numpy())
    assert np.array_equal(c.cpu().numpy(), cw) and np.array_equal(s.cpu().numpy(), sw)
    check(h, *i8.swiglu(cw, sw, gate, up), "bf16", "h")
    cw, sw = i8.quant(h.double().cpu().numpy())
    assert np.array_equal(c2.cpu().numpy(), cw) and np.array_equal(s2.cpu().numpy(), sw)
    check(y, *i8.gemm(cw, sw, *down), "bf16", "y")


@pytest.mark.parametrize("T", [3, 64, 400])
def test_expert_layer(T):
    """Routed rows: quantise, grouped gate and up, quantise, grouped down."""
    E, D, F = 6, 512, 720
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).bfloat16()
    gate = (codes(2, E, F, D), small_scales(4, D, E, F) * 10)
    up = (codes(5, E, F, D), small_scales(6, D, E, F) * 10)
    down = (codes(7, E, D, F), small_scales(8, F, E, D))
    chosen = np.sort(rng.choice(E, T, p=[0.5, 0.3, 0.1, 0.1, 0, 0]))
    off = np.concatenate([[0], np.cumsum(np.bincount(chosen, minlength=E))])
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    c, s = q4.quant_i8(x.to(DEV))
    h = q4.gemm_i8_grouped_swiglu(c, s, tuple(map(dev, gate)), tuple(map(dev, up)), o, dtype=torch.bfloat16)
    c2, s2 = q4.quant_i8(h)
    y = q4.gemm_i8_grouped(c2, s2, *map(dev, down), o)
    cw, sw = i8.quant(x.double().numpy())
    cw2, sw2 = i8.quant(h.double().cpu().numpy())
    assert np.array_equal(c2.cpu().numpy(), cw2) and np.array_equal(s2.cpu().numpy(), sw2)
    for e, lo, hi in i8.groups(off):
        check(h[lo:hi], *i8.swiglu(cw[lo:hi], sw[lo:hi], (gate[0][e], gate[1][e]), (up[0][e], up[1][e])), "bf16",
              f"h {e}")
        check(y[lo:hi], *i8.gemm(cw2[lo:hi], sw2[lo:hi], down[0][e], down[1][e]), "f32", f"y {e}")


@pytest.mark.parametrize("M", [1, 24, 90, 300])
def test_a_row_does_not_depend_on_the_batch(M):
    """The sums are exact, so a row's products are the same bits at any batch."""
    N, K = 200, 2064
    a, w, sa, sw = dev(codes(1, 300, K)), dev(codes(2, N, K)), dev(scales(3, 300)), dev(scales(4, N))
    whole = q4.gemm_i8(a, sa, w, sw)
    assert torch.equal(q4.gemm_i8(a[:M], sa[:M], w, sw), whole[:M])
    o = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    assert torch.equal(q4.gemm_i8_grouped(a[:M], sa[:M], w[None], sw[None], o), whole[:M])


@pytest.mark.parametrize("t", TYPES)
def test_epilogues_do_not_depend_on_the_batch(t):
    """Scales, bias and silu are the same steps in every kernel: 2600 rows, their first ones, and groups of them."""
    R, N, K = 2600, 1500, 528
    a, sa = dev(codes(1, R, K)), dev(small_scales(3, K, R))
    gate = dev(codes(2, N, K)), dev(small_scales(4, K, N) * 4)
    up = dev(codes(5, N, K)), dev(small_scales(6, K, N))
    bias = torch.linspace(-2, 2, N, device=DEV)
    y = q4.gemm_i8(a, sa, *gate, bias=bias, dtype=TYPES[t])
    h = q4.gemm_i8_swiglu(a, sa, gate, up, dtype=TYPES[t])
    for M in (1, 12, 30, 70, 150, 330, 700, 1300):
        assert torch.equal(q4.gemm_i8(a[:M], sa[:M], *gate, bias=bias, dtype=TYPES[t]), y[:M]), M
        assert torch.equal(q4.gemm_i8_swiglu(a[:M], sa[:M], gate, up, dtype=TYPES[t]), h[:M]), M
        o = torch.tensor([0, M // 3, M], dtype=torch.int32, device=DEV)
        twice = [tuple(torch.stack([p, p]) for p in m) for m in (gate, up)]
        assert torch.equal(q4.gemm_i8_grouped_swiglu(a[:M], sa[:M], *twice, o, dtype=TYPES[t]), h[:M]), M


@pytest.mark.parametrize("M", [2, 40, 300])
def test_graph_replays(M):
    x, *mats = layer_problem(M, 512, 640)
    mats = [tuple(map(dev, m)) for m in mats]
    xs = x.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(xs, *mats)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = layer(xs, *mats)
    for k in range(4):
        xs.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(k)).bfloat16())
        want = layer(xs, *mats)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k


@pytest.mark.parametrize("T", [6, 200, 900])
def test_graph_replays_with_other_groups(T):
    """The offsets are read on the GPU: a captured call takes the groups of the moment."""
    E, D, F = 5, 512, 320
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    gate, up = [(dev(codes(k, E, F, D)), dev(small_scales(k + 1, D, E, F) * 5)) for k in (2, 4)]
    down = dev(codes(7, E, D, F)), dev(small_scales(8, F, E, D))
    o = torch.zeros(E + 1, dtype=torch.int32, device=DEV)

    def experts():
        c, s = q4.quant_i8(x)
        h = q4.gemm_i8_grouped_swiglu(c, s, gate, up, o, dtype=torch.bfloat16)
        return q4.gemm_i8_grouped(*q4.quant_i8(h), *down, o, dtype=torch.bfloat16)

    def route(seed):
        c = torch.from_numpy(np.random.default_rng(seed).multinomial(T, [0.6, 0, 0.25, 0.1, 0.05]))
        o.copy_(torch.cat([torch.zeros(1, dtype=torch.long), c.cumsum(0)]).int())

    route(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        experts()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = experts()
    for k in range(1, 5):
        route(k)
        want = experts()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want), k


def test_weights_past_32_bits():
    """Experts whose matrices start beyond 4 GiB, by a few rows and by many."""
    E, N, K = 80, 14336, 4096                              # 4.7 GB
    w = torch.empty(E, N, K, dtype=torch.int8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    for part in w.view(-1).split(1 << 28):
        part.copy_(torch.randint(-128, 128, part.shape, generator=g, device=DEV, dtype=torch.int8))
    sw = dev(small_scales(4, K, E, N))
    for T in (7, 300):
        a, sa = codes(1, T, K), small_scales(3, K, T)
        off = [0] * (E - 1) + [2, T]                       # all in the last two experts
        y = q4.gemm_i8_grouped(dev(a), dev(sa), w, sw, torch.tensor(off, dtype=torch.int32, device=DEV))
        for e, lo, hi in ((E - 2, 0, 2), (E - 1, 2, T)):
            cols = slice(N - 500, N)
            want = i8.gemm(a[lo:hi], sa[lo:hi], w[e, cols].cpu().numpy(), sw[e, cols].cpu().numpy())
            check(y[lo:hi, cols], *want, "f32", f"{T} rows, expert {e}")


def test_rows_past_32_bits():
    """Inputs, codes and outputs whose last rows lie beyond 4 GiB."""
    M, K, N = 270_000, 16384, 16
    x = torch.empty(M, K, dtype=torch.float16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    for part in x.split(1 << 14):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV, dtype=torch.float16))
    c, s = q4.quant_i8(x)
    at = [0, M // 2, M - 1]
    cw, sw = i8.quant(x[at].double().cpu().numpy())
    assert np.array_equal(c[at].cpu().numpy(), cw) and np.array_equal(s[at].cpu().numpy(), sw)
    del x
    w, ws = codes(2, N, K), small_scales(4, K, N)
    y = q4.gemm_i8(c, s, dev(w), dev(ws))
    check(y[at], *i8.gemm(cw, sw, w, ws), "f32", "a")
    del c
    M, K, N = 70_000, 256, 32_768
    a, sa, w, ws = codes(1, M, K), small_scales(3, K, M), codes(2, N, K), small_scales(4, K, N)
    for K in (256, 48):                                    # tiles, and K below a step
        y = q4.gemm_i8(dev(a[:, :K]), dev(sa), dev(w[:, :K]), dev(ws), dtype=torch.bfloat16)
        check(y[at[:1] + [M - 1]], *i8.gemm(a[[0, M - 1], :K], sa[[0, M - 1]], w[:, :K], ws), "bf16", "y")


@pytest.mark.parametrize("M", [3, 300])
def test_two_streams(M):
    """Calls on two streams at once, each with its own outputs."""
    x, *mats = layer_problem(M, 512, 640)
    mats = [tuple(map(dev, m)) for m in mats]
    xs = [x.to(DEV), (x * 3 + 1).to(DEV)]
    want = [layer(v, *mats) for v in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = layer(xs[i], *mats)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


def test_refusals():
    a, w, sa, sw = dev(codes(1, 4, 64)), dev(codes(2, 8, 64)), dev(scales(3, 4)), dev(scales(4, 8))
    with pytest.raises(ValueError):
        q4.gemm_i8(a, sa, w[:, :32], sw)                   # another K, not contiguous
    with pytest.raises(ValueError):
        q4.gemm_i8(a, sa[:3], w, sw)
    with pytest.raises(ValueError):
        q4.gemm_i8(a, sa, w, sw, bias=sw[:7])
    with pytest.raises(TypeError):
        q4.gemm_i8(a, sa, w, sw, dtype=torch.float64)
    with pytest.raises(TypeError):
        q4.gemm_i8(a, sa, w, sw, dtype=torch.float16, out=torch.empty(4, 8, device=DEV))
    with pytest.raises(ValueError):
        q4.gemm_i8(a, sa, w, sw, out=torch.empty(8, 4, device=DEV))
    with pytest.raises(q4.Q4Error):
        q4.gemm_i8(dev(codes(1, 4, 24)), sa, dev(codes(2, 8, 24)), sw)
    with pytest.raises(ValueError):
        q4.gemm_i8_swiglu(a, sa, (w, sw), (w[:7], sw[:7]))
    o = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        q4.gemm_i8_grouped(a, sa, w[None], sw[None], o.long())
    with pytest.raises(ValueError):
        q4.gemm_i8_grouped(a, sa, w[None], sw[None], torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        q4.gemm_i8_grouped(a, sa, w, sw, o)
    with pytest.raises(ValueError):
        q4.gemm_i8_grouped(a, sa, w[None].cpu(), sw[None], o)


def test_refusals_of_sizes_past_32_bits():
    """Row counts that an int of 32 bits would take for others."""
    M = 2**32 + 5
    a = torch.empty(1, 16, dtype=torch.int8, device=DEV).expand(M, 16)
    with pytest.raises(ValueError):
        q4.gemm_i8(a, torch.ones(1, device=DEV).expand(M), a[:4].contiguous(), torch.ones(4, device=DEV))
    a = torch.empty(2**31 + 5, 16, dtype=torch.int8, device=DEV)        # 34 GB, never touched
    with pytest.raises(q4.Q4Error):
        q4.gemm_i8(a[:4], torch.ones(4, device=DEV), a, torch.empty(2**31 + 5, device=DEV))
    with pytest.raises(q4.Q4Error):
        q4.gemm_i8(a, torch.empty(2**31 + 5, device=DEV), a[:4], torch.ones(4, device=DEV))


def test_refusals_of_the_quantiser():
    x = torch.randn(4, 64, device=DEV)
    c, s = q4.quant_i8(x)
    for bad in (x.double(), x.int()):
        with pytest.raises(TypeError):
            q4.quant_i8(bad)
    for bad in (x[0], x[None], x.t()):
        with pytest.raises(ValueError):
            q4.quant_i8(bad)
    with pytest.raises(q4.Q4Error):
        q4.quant_i8(x[:, :24].contiguous())
    for out in ((c[:3], s), (c, s[:3]), (c, s[:, None])):
        with pytest.raises(ValueError):
            q4.quant_i8(x, out=out)
    for out in ((c.float(), s), (c, s.half()), (None, s), (c, None)):
        with pytest.raises((TypeError, ValueError)):
            q4.quant_i8(x, out=out)


def test_refusals_name_the_argument():
    a, w, sa, sw = dev(codes(1, 4, 64)), dev(codes(2, 8, 64)), dev(scales(3, 4)), dev(scales(4, 8))
    o = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    cases = [(lambda: q4.gemm_i8(a, sa.double(), w, sw), "a_scales"),
             (lambda: q4.gemm_i8(a, sa, w, sw[:7]), "w_scales"),
             (lambda: q4.gemm_i8(a, sa, w.t(), sw), "w"), (lambda: q4.gemm_i8(a, sa, w, sw, bias=sw.half()), "bias"),
             (lambda: q4.gemm_i8_swiglu(a, sa, (w, sw), (w, sw[:7])), "w_scales"),
             (lambda: q4.gemm_i8_swiglu(a, sa, (w, sw), (w.float(), sw)), "w"),
             (lambda: q4.gemm_i8_swiglu(a, sa, (w, sw), (w, None)), "up"),
             (lambda: q4.gemm_i8_grouped(a, sa, w[None], sw[None], None), "offsets"),
             (lambda: q4.gemm_i8_grouped(a, sa, w[None], sw[None], o[None]), "offsets"),
             (lambda: q4.gemm_i8_grouped(a, sa, w[None], sw, o), "w_scales"),
             (lambda: q4.gemm_i8_grouped_swiglu(a, sa, (w[None], sw[None]), (w[None], sw[None]), None), "offsets"),
             (lambda: q4.gemm_i8_grouped_swiglu(a, sa, (w[None], sw[None]), (w[None], sw[None]), o, out=sw), "out")]
    for call, name in cases:
        with pytest.raises((TypeError, ValueError), match=name):
            call()


def test_calls_keep_nothing():
    """Outputs are freed with their last name, and a given output is returned itself."""
    a, w, sa, sw = dev(codes(1, 40, 64)), dev(codes(2, 80, 64)), dev(scales(3, 40)), dev(scales(4, 80))
    x, o = torch.randn(40, 64, device=DEV), torch.tensor([0, 9, 40], dtype=torch.int32, device=DEV)
    y = torch.empty(40, 80, device=DEV)
    two = torch.stack([w, w]), torch.stack([sw, sw])

    def calls():
        q4.quant_i8(x)
        assert q4.gemm_i8(a, sa, w, sw, out=y) is y
        assert q4.gemm_i8_swiglu(a, sa, (w, sw), (w, sw), out=y) is y
        q4.gemm_i8(a, sa, w, sw, bias=sw)
        q4.gemm_i8_grouped(a, sa, *two, o)
        q4.gemm_i8_grouped_swiglu(a, sa, two, two, o)

    calls()
    names = (a, w, sa, sw, x, o, y, two)
    before = torch.cuda.memory_allocated(), [sys.getrefcount(n) for n in names]
    for _ in range(50):
        calls()
    assert before == (torch.cuda.memory_allocated(), [sys.getrefcount(n) for n in names])


def test_threads():
    """Threads that call at once, each on a stream of its own."""
    x, *mats = layer_problem(70, 512, 640)
    mats = [tuple(map(dev, m)) for m in mats]
    xs = [(x * (i + 1)).to(DEV) for i in range(4)]
    want = [layer(v, *mats) for v in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(30):
                got[i] = layer(xs[i], *mats)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(4):
        assert all(torch.equal(p, q) for p, q in zip(got[i], want[i]))


# ---------------------------------------------------------------- far gates, other scales and operands, every launch

@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 12, 40, 300])
def test_swiglu_gates_far_below_zero(M, t):
    """Gates from 0 down to -170, whose silu is far below fp32's subnormal
    numbers at the end, with an up projection that brings the product back."""
    N, K = 260, 144
    a, wg, wu = (np.zeros((rows, K), dtype=np.int8) for rows in (M, N, N))
    a[:, 140], wg[:, 140] = 1, -(np.arange(N) % 129)
    wu[:, 140] = np.arange(N) % 50 - 75
    sa = np.resize(np.array([1, 0.71, 1.33, 0.69], dtype=np.float32), M)
    gate, up = (wg, np.ones(N, dtype=np.float32)), (wu, np.full(N, 2.0 ** 110, dtype=np.float32))
    y = q4.gemm_i8_swiglu(dev(a), dev(sa), tuple(map(dev, gate)), tuple(map(dev, up)), dtype=TYPES[t])
    check(y, *i8.swiglu(a, sa, gate, up), t, f"{M}")


def test_refusals_of_what_is_no_tensor():
    """An operand that is missing or no tensor is refused by its name, in every call."""
    a, w, sa, sw = dev(codes(1, 4, 64)), dev(codes(2, 8, 64)), dev(scales(3, 4)), dev(scales(4, 8))
    o = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    pair, pairs = (w, sw), (w[None], sw[None])
    for bad in (None, 3, [1.0]):
        cases = [(lambda: q4.gemm_i8(bad, sa, w, sw), "a "), (lambda: q4.gemm_i8(a, bad, w, sw), "a_scales "),
                 (lambda: q4.gemm_i8(a, sa, bad, sw), "w "), (lambda: q4.gemm_i8(a, sa, w, bad), "w_scales "),
                 (lambda: q4.gemm_i8_swiglu(bad, sa, pair, pair), "a "),
                 (lambda: q4.gemm_i8_swiglu(a, bad, pair, pair), "a_scales "),
                 (lambda: q4.gemm_i8_grouped(bad, sa, *pairs, o), "a "),
                 (lambda: q4.gemm_i8_grouped(a, sa, *pairs, bad), "offsets "),
                 (lambda: q4.gemm_i8_grouped_swiglu(bad, sa, pairs, pairs, o), "a "),
                 (lambda: q4.gemm_i8_grouped_swiglu(a, bad, pairs, pairs, o), "a_scales "),
                 (lambda: q4.gemm_i8_grouped_swiglu(a, sa, pairs, pairs, bad), "offsets "),
                 (lambda: q4.quant_i8(bad), "x "),
                 (lambda: q4.quant_i8(sa[None, :4].repeat(4, 16), out=(a, bad)), "scales "),
                 (lambda: q4.quant_i8(sa[None, :4].repeat(4, 16), out=(bad, sa)), "codes ")]
        for i, (call, name) in enumerate(cases):
            with pytest.raises(TypeError, match="^" + name):
                call()
                pytest.fail(f"case {i} with {bad} was taken")


# Rows and 16-byte vectors a row for each form of the quantiser: 64 threads a row
# take up to 4 vectors each (past one, only from 2048 rows on), 256 up to 8 (past
# one, only from 512 rows on), 1024 up to 8, and longer rows are read twice.
# Rows end inside the threads' last vectors and workgroups of four rows.
QUANT_FORMS = [(6, 4), (2051, 64), (2051, 68), (2050, 132), (2049, 252),
               (7, 68), (515, 256), (515, 260), (514, 516), (513, 1028), (515, 2044),
               (9, 260), (3, 1024), (3, 1028), (5, 2052), (3, 4100), (2, 8192), (3, 8196)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,vectors", QUANT_FORMS)
def test_quant_every_form(t, M, vectors):
    K = vectors * (4 if t == "f32" else 8)
    rng = np.random.default_rng(M * K)
    x = rng.standard_normal((M, K), dtype=np.float32) * rng.uniform(0.01, 30, (M, 1)).astype(np.float32)
    x[np.arange(M), rng.integers(0, K, M)] *= 9            # the largest one anywhere in a row
    x[M - 1, K - 1] = -200                                 # and in the last vector of the last
    x[M // 2] = 0
    if M > 2:
        x[1, K - 2] = np.inf
    xt = torch.from_numpy(x).to(TYPES[t])
    buf = torch.full((M * K + 32,), 77, dtype=torch.int8, device=DEV)
    ends = torch.full((M + 8,), 7.0, device=DEV)
    c, s = q4.quant_i8(xt.to(DEV), out=(buf[16:16 + M * K].view(M, K), ends[4:4 + M]))
    cw, sw = i8.quant(xt.double().numpy())
    assert np.array_equal(s.cpu().numpy(), sw, equal_nan=True)
    assert np.array_equal(c.cpu().numpy(), cw)
    assert (buf[:16] == 77).all() and (buf[16 + M * K:] == 77).all()
    assert (ends[:4] == 7).all() and (ends[4 + M:] == 7).all()


@pytest.mark.parametrize("M", [1, 9, 40, 100, 600])
def test_swiglu_rows_and_columns_do_not_mix(M):
    """Scales of NaN and Inf in either matrix and a zero row stay in their rows and columns."""
    N, K = 150, 400
    a, sa = codes(1, M, K), small_scales(3, K, M)
    gate, up = (codes(2, N, K), small_scales(4, K, N)), (codes(5, N, K), small_scales(6, K, N))
    a[M // 2] = 0
    sa[M - 1] = np.nan if M > 1 else 1
    gate[1][3], gate[1][70], up[1][5], up[1][149] = np.inf, np.nan, np.nan, np.inf
    with np.errstate(invalid="ignore"):
        want, bound = i8.swiglu(a, sa, gate, up)
    y = q4.gemm_i8_swiglu(dev(a), dev(sa), tuple(map(dev, gate)), tuple(map(dev, up))).cpu().numpy()
    fine = np.isfinite(want)
    assert fine[:, [0, 4, 6, 148]][:M - 1].all()
    assert np.array_equal(np.isnan(y), np.isnan(want)) and np.array_equal(np.isposinf(y), np.isposinf(want))
    assert np.array_equal(np.isneginf(y), np.isneginf(want))
    assert (np.abs(y[fine] - want[fine]) <= i8.tolerance(want, bound, "f32")[fine]).all()


# A bias in every tile: columns past the end, K inside a step, workgroups that go
# on to a next tile, and a last round in halves and in quarters.
BIAS = [(1, 896, 896), (12, 333, 4096), (36, 1373, 32), (24, 512, 2816), (64, 4090, 2064), (100, 896, 4864),
        (500, 2050, 2064), (330, 4870, 912), (1090, 5000, 528), (3775, 1827, 1056), (3984, 3781, 656),
        (5000, 300, 4112), (128, 3990, 4112), (56, 5099, 1984), (4209, 132, 400), (5511, 186, 8432),
        (2307, 3403, 256), (3099, 5093, 1328), (4300, 4100, 2064), (4096, 5300, 2000), (8200, 4097, 1040)]


@pytest.mark.parametrize("M,N,K", BIAS)
def test_bias_in_every_tile(M, N, K):
    a, w, sa, sw = codes(1, M, K), codes(2, N, K), small_scales(3, K, M), small_scales(4, K, N)
    b = np.random.default_rng(5).standard_normal(N).astype(np.float32) * 3
    y = q4.gemm_i8(dev(a), dev(sa), dev(w), dev(sw), bias=dev(b))
    want = exact_rows(a, sa, w, sw)
    bound = 3.1 * i8.U * want.abs()
    want = want + dev(b).double()
    bound = bound + 1.1 * i8.U * want.abs()                # as i8.gemm
    assert ((y.double() - want).abs() <= bound + i8.U * (want.abs() + bound)).all()


def test_bias_takes_every_tile():
    got = [q4.gemm_i8_geometry(1, *s) for s in BIAS]
    tiles = [(g["tile_rows"], g["tile_cols"]) for g in got]
    assert {8, 16, 32} <= {r for r, c in tiles}
    assert {(32, 32), (64, 32), (64, 64), (64, 128), (128, 128), (128, 256), (256, 256)} <= set(tiles)
    count = [-(-m // r) * -(-n // c) for (m, n, _), (r, c) in zip(BIAS, tiles)]
    # Workgroups that go through several tiles, with one matrix's bias past 512 scales and below.
    assert {(128, 128), (128, 256), (256, 256)} <= {t for t, n, g in zip(tiles, count, got) if g["grid"] < n}
    # More workgroups than the 256 that stay: the divided tiles' launch, as halves and as quarters.
    parts = {(g["grid"] - 256) // (n % 256) for t, n, g in zip(tiles, count, got)
             if t == (256, 256) and g["grid"] > 256}
    assert parts == {2, 4}


# Shapes of groups for every tile of 64 rows and more, with a workgroup for each
# tile and with workgroups that go through several.
GROUPED = [(1, 6615, 68, 400, 4), (1, 7191, 129, 144, 2), (1, 862, 1201, 272, 78), (1, 4301, 392, 128, 71),
           (1, 3698, 1170, 144, 49), (1, 1158, 7078, 128, 21), (1, 4051, 1805, 288, 66), (1, 7309, 2014, 416, 2),
           (1, 6435, 2432, 128, 2), (1, 2358, 6584, 144, 1), (2, 6222, 33, 144, 6), (2, 7043, 33, 144, 48),
           (2, 2457, 407, 272, 77), (2, 5320, 199, 128, 51), (2, 1461, 1344, 144, 28), (2, 989, 3873, 128, 20),
           (2, 3305, 1193, 272, 53), (2, 942, 7243, 416, 1), (2, 3696, 2272, 128, 2), (2, 4726, 1543, 144, 3)]


def test_grouped_shapes_take_every_tile():
    seen = set()
    for mats, M, N, K, E in GROUPED:
        g = q4.gemm_i8_geometry(mats, M, N, K, E)
        most = (M // g["tile_rows"] + E) * -(-N // g["tile_cols"])
        seen.add((mats, g["tile_rows"], g["tile_cols"] * mats, "each" if g["grid"] == most else
                  "several" if g["grid"] < most else "divided"))
    want = {(m, *t, k) for m in (1, 2) for t in ((64, 128), (128, 128), (128, 256)) for k in ("each", "several")}
    want |= {(m, *t) for m in (1, 2) for t in ((64, 64, "each"), (256, 256, "each"), (256, 256, "divided"))}
    assert want <= seen, want - seen


@pytest.mark.parametrize("mats,M,N,K,E", GROUPED)
def test_grouped_in_every_tile(mats, M, N, K, E):
    """Uneven groups, some empty, with rows before the first and behind the last."""
    rng = np.random.default_rng(M)
    share = rng.uniform(0.05, 1, E) ** 2
    share[rng.random(E) < 0.2] = 0
    share[E // 2] += 0.3
    off = 3 + np.concatenate([[0], np.cumsum(rng.multinomial(M - 8, share / share.sum()))])
    a, sa = codes(1, M, K), small_scales(3, K, M)
    gate, up = [(codes(s, E, N, K), small_scales(s + 1, K, E, N)) for s in (2, 5)]
    out = torch.full((M, N), 7.0, device=DEV)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    if mats == 2:
        q4.gemm_i8_grouped_swiglu(dev(a), dev(sa), tuple(map(dev, gate)), tuple(map(dev, up)), o, out=out)
    else:
        q4.gemm_i8_grouped(dev(a), dev(sa), *map(dev, gate), o, out=out)
    got = out.cpu().numpy().astype(np.float64)
    for e, lo, hi in i8.groups(off):
        g, u = (gate[0][e], gate[1][e]), (up[0][e], up[1][e])
        want, bound = i8.swiglu(a[lo:hi], sa[lo:hi], g, u) if mats == 2 else i8.gemm(a[lo:hi], sa[lo:hi], *g)
        assert (np.abs(got[lo:hi] - want) <= i8.tolerance(want, bound, "f32")).all(), f"expert {e}"
    assert (got[:off[0]] == 7).all() and (got[off[-1]:] == 7).all()
