"""GPU parity of the operators of 8-bit floating point against the 64-bit
oracle, through the Python binding.

Quantisers are compared exactly.  Products are compared in two ways: on codes
and scales whose every sum is a short binary number, where the result has to
be the rounded one exactly, at every size and tile; and on quantised normal
values, held to the bounds that include/q4f8.h gives plus half a step of the
output's type.
"""

import threading

import numpy as np
import pytest
import torch

import memory_bandwidth_amd as q4
from oracle import f8

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn


def dev(a):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t.view(F8) if t.dtype == torch.uint8 else t


def pair(m):
    return dev(m[0]), dev(m[1])


def by_block(scales):
    """Scales on the GPU as quant_f8 lays them out."""
    return dev(scales.T).t()


def bits(t):
    return t.view(torch.uint8).cpu().numpy() if t.dtype == F8 else t.cpu().numpy()


# ---------------------------------------------------------------- quantisers

def values_of(seed, M, K, t):
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal((M, K)).astype(np.float32))
    x[:, 5] *= 11
    return x.to(TYPES[t])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (65, 128), (7, 896), (33, 1040), (2, 4096), (17, 272), (5, 14336),
                                 (1, 131056), (1030, 272), (2100, 1936)])
def test_quant(t, M, K):
    x = values_of(M * K, M, K, t)
    c, s = q4.quant_f8(x.to(DEV))
    cw, sw = f8.quant(x.double().numpy())
    assert np.array_equal(bits(s), sw)
    assert np.array_equal(f8.decode(bits(c)), f8.decode(cw))
    assert s.t().is_contiguous()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("R,C", [(1, 16), (3, 48), (128, 128), (127, 144), (129, 896), (260, 272), (16, 4096), (1000, 400),
                                 (145, 1040), (2, 131056)])
@pytest.mark.parametrize("layout", ["rows", "columns", "both"])
def test_quant_block(t, R, C, layout):
    x = values_of(R * C, R, C, t)
    got = q4.quant_f8_block(x.to(DEV), layout=layout)
    cw, sw = f8.quant(x.double().numpy(), 128)
    want = {"rows": (cw, sw), "columns": f8.turned(cw, sw), "both": (cw, sw, *f8.turned(cw, sw))}[layout]
    assert len(got) == len(want)
    for g, w in zip(got, want):
        assert tuple(g.shape) == w.shape
        same = np.array_equal(f8.decode(bits(g)), f8.decode(w)) if g.dtype == F8 else np.array_equal(bits(g), w)
        assert same


def special(t):
    K = 400
    rng = np.random.default_rng(9)
    x = np.zeros((14, K), dtype=np.float32)
    x[0] = rng.choice(f8.MIDDLES, K)                       # scale 1 where a block holds 448: ties
    x[0, ::128] = 448
    x[1] = -rng.choice(f8.MIDDLES, K) * 0.75
    x[1, ::128] = 448 * 0.75
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
    x[11] = rng.standard_normal(K) * 2.0 ** rng.integers(-20, 3, K)
    x[12] = rng.choice([0.0, -0.0, 1.0], K)
    x[13] = rng.choice(f8.VALUES[:127], K)
    if t == "f32":
        x[6] = rng.integers(-9, 10, K) * 2.0 ** -149       # subnormal
        x[7] = rng.standard_normal(K) * 8e37
        x[8] = rng.choice(f8.MIDDLES, K) * 2.0 ** -126     # scale 2^-126, ties
        x[8, 1] = 448 * 2.0 ** -126
    return torch.from_numpy(x).to(TYPES[t])


@pytest.mark.parametrize("t", TYPES)
def test_quant_ties_and_special_blocks(t):
    x = special(t)
    c, s = q4.quant_f8(x.to(DEV))
    cw, sw = f8.quant(x.double().numpy())
    assert np.array_equal(bits(s), sw, equal_nan=True)
    assert np.array_equal(f8.decode(bits(c)), f8.decode(cw))
    c, s, ct, st = q4.quant_f8_block(x.to(DEV), layout="both")
    cw, sw = f8.quant(x.double().numpy(), 128)
    for g, w in zip((c, s, ct, st), (cw, sw, *f8.turned(cw, sw))):
        assert np.array_equal(f8.decode(bits(g)) if g.dtype == F8 else bits(g), f8.decode(w) if w.dtype == np.uint8 else w,
                              equal_nan=True)
    # Each special row as a block of its own.
    for r in range(x.shape[0]):
        c, s = q4.quant_f8_block(x[r:r + 1].to(DEV))
        cw, sw = f8.quant(x[r:r + 1].double().numpy(), 128)
        assert np.array_equal(bits(s), sw, equal_nan=True) and np.array_equal(f8.decode(bits(c)), f8.decode(cw)), r


def test_quant_near_ties():
    """Quotients within a few ulp of every middle, on both sides and on it, for many scales."""
    rng = np.random.default_rng(4)
    rows = []
    for _ in range(200):
        s = np.float32(rng.uniform(0.5, 1) * 2.0 ** rng.integers(-30, 30))
        x = (rng.choice(f8.MIDDLES, 128) * np.float64(s)).astype(np.float32)
        x = (x.view(np.int32) + rng.integers(-2, 3, 128).astype(np.int32)).view(np.float32) * rng.choice([-1, 1], 128)
        x[0] = np.float32(448) * s
        rows.append(x.astype(np.float32))
    x = np.stack(rows)
    c, got = q4.quant_f8(dev(x))
    cw, sw = f8.quant(x.astype(np.float64))
    assert np.array_equal(bits(got), sw) and np.array_equal(f8.decode(bits(c)), f8.decode(cw))


def test_quant_outputs_given():
    """Scales of any strides; codes and scales inside larger buffers, which keep what is around them."""
    M, K = 37, 400
    x = values_of(3, M, K, "bf16")
    cw, sw = f8.quant(x.double().numpy())
    codes = torch.zeros(M + 2, K, dtype=torch.uint8, device=DEV).view(F8)
    for scales in (torch.full((M, 4), 7.0, device=DEV), torch.full((M, 9), 7.0, device=DEV)[:, 2:6],
                   torch.full((4, 3 * M), 7.0, device=DEV).t()[::3]):
        c, s = q4.quant_f8(x.to(DEV), out=(codes[1:M + 1], scales))
        assert c.data_ptr() == codes[1].data_ptr() and s is scales
        assert np.array_equal(bits(s), sw) and np.array_equal(f8.decode(bits(c)), f8.decode(cw))
        assert not bits(codes)[[0, M + 1]].any()
    wide = torch.full((M, 9), 7.0, device=DEV)
    q4.quant_f8(x.to(DEV), out=(codes[1:M + 1], wide[:, 2:6]))
    assert (wide[:, :2] == 7).all() and (wide[:, 6:] == 7).all()
    cw, sw = f8.quant(x.double().numpy(), 128)
    out = (torch.empty(M, K, dtype=F8, device=DEV), torch.empty(1, 4, device=DEV), torch.empty(K, 48, dtype=F8, device=DEV),
           torch.empty(4, 1, device=DEV))
    got = q4.quant_f8_block(x.to(DEV), layout="both", out=out)
    assert all(g.data_ptr() == o.data_ptr() for g, o in zip(got, out))
    for g, w in zip(got, (cw, sw, *f8.turned(cw, sw))):
        assert np.array_equal(f8.decode(bits(g)) if g.dtype == F8 else bits(g), f8.decode(w) if w.dtype == np.uint8 else w)


def test_empty():
    z = lambda *s, **k: torch.zeros(*s, device=DEV, **k)                 # noqa: E731
    c, s = q4.quant_f8(z(0, 64))
    assert tuple(c.shape) == (0, 64) and tuple(s.shape) == (0, 1)
    got = q4.quant_f8_block(z(0, 64), layout="both")
    assert [tuple(t.shape) for t in got] == [(0, 64), (0, 1), (64, 0), (1, 0)]
    a, w, sw = z(0, 64).to(F8), z(5, 64).to(F8), z(1, 1)
    assert tuple(q4.gemm_f8(a, z(0, 1), w, sw).shape) == (0, 5)
    assert tuple(q4.gemm_f8_swiglu_backward(z(0, 5), a, z(0, 1), (w, sw), (w, sw)).shape) == (0, 10)


# ---------------------------------------------------------------- products, exactly
#
# Codes of 0, +-1, +-2, +-4 and scales that are one of two powers of two: products
# and their sums are whole multiples of one unit below 2^24 of it, and the
# products of eight are within 2^4 of each other, so that no step rounds.

SMALL = np.array([0x00, 0x38, 0xB8, 0x40, 0xC0, 0x48, 0xC8], dtype=np.uint8)


def short_codes(seed, *shape):
    return np.random.default_rng(seed).choice(SMALL, shape)


def short_scales(seed, rows, K, unit):
    return (np.random.default_rng(seed).choice([1.0, 2.0], (rows, f8.blocks(K))) * unit).astype(np.float32)


def unit(K):
    """A power of two that brings sums of K products near 1, from both scales."""
    return 2.0 ** -round(np.log2(K) / 4 + 1.5)


def short_problem(M, N, K, tall=1, mats=1, seed=1):
    u = unit(K)
    a = short_codes(seed, M, K), short_scales(seed + 1, M if tall == 1 else f8.blocks(M), K, u)
    return a, [(short_codes(seed + 2 + i, N, K), short_scales(seed + 5 + i, f8.blocks(N), K, u)) for i in range(mats)]


def spread_on_gpu(codes, scales, tall):
    s = scales.double().repeat_interleave(128, 1)[:, :codes.shape[1]].repeat_interleave(tall, 0)[:codes.shape[0]]
    return codes.double() * s


def exact_on_gpu(a, sa, w, sw):
    """P in float64, exact for these inputs."""
    tall = 1 if sa.shape[0] == a.shape[0] else 128
    return spread_on_gpu(a, sa, tall) @ spread_on_gpu(w, sw, 128).t()


def same(y, want, label):
    bad = (y != want.to(y.dtype)).nonzero()
    assert not len(bad), f"{label}: {len(bad)} of {y.numel()} differ, first at {bad[0].tolist()}"


GEMM = [(1, 1, 16), (1, 17, 48), (1, 896, 896), (1, 300, 4096), (2, 64, 128), (3, 129, 144), (8, 1000, 1040),
        (15, 33, 4096), (16, 16, 64), (17, 257, 272), (31, 130, 14336), (32, 512, 2816), (48, 100, 912),
        (64, 64, 128), (65, 127, 256), (100, 896, 4864), (128, 256, 1024), (129, 300, 1040), (200, 333, 2064),
        (256, 256, 256), (257, 511, 528), (300, 1024, 896), (511, 520, 4112), (700, 777, 1296), (1025, 1030, 400),
        (2049, 260, 144), (260, 4100, 208), (40, 70, 32)]
# Every kind of launch that the products choose from, for either way to multiply,
# with rows and columns that end inside tiles and K inside steps: one tile a
# workgroup and several, last rounds as they are, in halves and in quarters.
LARGE = [(64, 4100, 2064), (500, 2050, 2064), (3984, 3781, 656), (64, 3999, 4112), (36, 1373, 32), (126, 2093, 6016),
         (64, 4090, 14336), (128, 3990, 4112), (4300, 4100, 2064), (2304, 2560, 9216), (18, 9303, 800),
         (36, 8174, 1472), (38, 6292, 9520), (141, 5177, 800), (3065, 116, 1440), (4868, 387, 656), (5390, 659, 288),
         (7439, 1399, 272), (3692, 4667, 144), (4715, 1794, 304), (8655, 930, 272), (4771, 5846, 272),
         (5331, 4596, 656), (3083, 5219, 272), (4378, 345, 288), (7290, 193, 272), (6343, 103, 688),
         (1804, 4310, 1680), (2910, 2761, 400), (2755, 5834, 400), (789, 5441, 272), (198, 3608, 6208),
         (3630, 4229, 800), (5997, 33, 6976), (7171, 4233, 464), (1915, 8541, 912), (10, 1693, 976),
         (33, 7794, 4496)]


@pytest.mark.parametrize("M,N,K", GEMM + LARGE)
@pytest.mark.parametrize("t", TYPES)
def test_gemm_exact(M, N, K, t):
    (a, sa), [w] = short_problem(M, N, K)
    args = dev(a), by_block(sa), *pair(w)
    same(q4.gemm_f8(*args, dtype=TYPES[t]), exact_on_gpu(*args), f"{M} {N} {K}")


@pytest.mark.parametrize("M,N,K", [(1, 77, 256), (5, 64, 400), (40, 520, 144), (130, 64, 1024), (257, 300, 656),
                                   (600, 515, 400), (1300, 2100, 272), (4300, 4100, 528)])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_gemm_scales_of_row_blocks_and_bias(M, N, K, t):
    (a, sa), [w] = short_problem(M, N, K, tall=128)
    b = (np.random.default_rng(5).integers(-64, 65, N) / 16).astype(np.float32)
    args = dev(a), dev(sa), *pair(w)
    same(q4.gemm_f8(*args, bias=dev(b), dtype=TYPES[t]), exact_on_gpu(*args) + dev(b).double(), f"{M} {N} {K}")


@pytest.mark.parametrize("M,N,K", [(3, 40, 656), (40, 200, 656), (70, 520, 272), (600, 515, 400)])
def test_gemm_strides_of_scales(M, N, K):
    (a, sa), [w] = short_problem(M, N, K)
    KB = sa.shape[1]
    want = exact_on_gpu(dev(a), dev(sa), *pair(w))
    wide = torch.full((M, KB + 5), float("nan"), device=DEV)
    wide[:, 2:2 + KB] = dev(sa)
    apart = torch.full((3 * KB, 2 * M), float("nan"), device=DEV)
    apart[1::3, ::2] = dev(sa).t()
    one = torch.full((KB,), 0.5, device=DEV).expand(M, KB)
    for s in (dev(sa), wide[:, 2:2 + KB], apart[1::3, ::2].t()):
        same(q4.gemm_f8(dev(a), s, *pair(w)), want, str(s.stride()))
        same(q4.gemm_f8(dev(a), s, *pair(w), dtype=torch.bfloat16), want, str(s.stride()))
    same(q4.gemm_f8(dev(a), one, *pair(w)), exact_on_gpu(dev(a), one.contiguous(), *pair(w)), "one row for all")


@pytest.mark.parametrize("M,N", [(1, 5), (20, 18), (70, 70), (300, 260)])
@pytest.mark.parametrize("t", ["f32", "f16"])
def test_gemm_longest(M, N, t):
    K = 131056
    (a, sa), [w] = short_problem(M, N, K)
    args = dev(a), by_block(sa), *pair(w)
    same(q4.gemm_f8(*args, dtype=TYPES[t]), exact_on_gpu(*args), f"{M} {N}")


def launches(mats, M, N, K, t):
    """What a call's launches are: the tile, and whether workgroups go through several, or tiles are left and divided."""
    g = q4.gemm_f8_geometry(mats, M, N, K, dtype=t)
    r, wide = g["tile_rows"], g["tile_cols"] * mats
    tiles = -(-M // r) * -(-N // g["tile_cols"])
    if r <= 32 or (r, wide) == (64, 32):
        return r, g["block"]
    left = tiles % 256
    name = "one each"
    if r == wide == 256 and tiles > 256 and 0 < left <= 128:
        name = "halves" if left > 64 else "quarters"
    return r, wide, "several" if name == "one each" and g["grid"] < tiles else name


def test_sizes_take_every_launch():
    common = {(8, 256), (8, 512), (16, 256), (16, 512), (32, 256), (32, 512), (64, 64, "one each"), (64, 128, "one each"),
              (128, 128, "one each"), (128, 128, "several"), (128, 256, "one each")}
    f32 = common | {(128, 256, "several")}
    f16 = common | {(256, 256, "one each"), (256, 256, "several"), (256, 256, "halves"), (256, 256, "quarters")}
    for mats, shapes, more in ((1, GEMM + LARGE, {(64, 256)}), (2, GATED, set())):
        for t, want in ((torch.float32, f32), (torch.bfloat16, f16)):
            seen = {launches(mats, *s, t) for s in shapes}
            assert want | more <= seen, (mats, t, (want | more) - seen)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,N", [(1, 40), (5, 64), (70, 72), (300, 264)])
@pytest.mark.parametrize("skew", [0, 1])
def test_gemm_out_in_a_larger_buffer(t, M, N, skew):
    """Outputs that start off a 16-byte border, with guards on both sides."""
    (a, sa), [w] = short_problem(M, N, 160)
    args = dev(a), by_block(sa), *pair(w)
    buf = torch.full((M * N + 32,), 7.0, dtype=TYPES[t], device=DEV)
    out = buf[8 + skew:8 + skew + M * N].view(M, N)
    y = q4.gemm_f8(*args, dtype=TYPES[t], out=out)
    assert y.data_ptr() == out.data_ptr()
    same(y, exact_on_gpu(*args), f"{M} {N}")
    assert (buf[:8 + skew] == 7).all() and (buf[8 + skew + M * N:] == 7).all()


def bias_of(N, seed=5):
    """Whole sixteenths, other ones in every column tile."""
    return (np.random.default_rng(seed).integers(-64, 65, N) / 16).astype(np.float32)


# Stages that a workgroup keeps on their way, by tile, where it goes through several tiles.
STAGES = {(128, 128): 2, (128, 256): 3}


@pytest.mark.parametrize("t,M,N,K", [("bf16", 8192, 4096, 256), ("f16", 8192, 4096, 256), ("bf16", 32, 132383, 208),
                                     ("f32", 8192, 8192, 272), ("f32", 4096, 8192, 384), ("f32", 99, 134948, 192)])
def test_gemm_bias_of_tiles_in_turn(t, M, N, K):
    """Three tiles or more a workgroup, and as many blocks of K as stages: the loads of a tile's first step are then
    followed by the next one's bias, in the place of the one before."""
    g = q4.gemm_f8_geometry(1, M, N, K, dtype=TYPES[t])
    tile = g["tile_rows"], g["tile_cols"]
    assert -(-M // tile[0]) * -(-N // tile[1]) > 2 * g["grid"] and f8.blocks(K) == STAGES[tile]
    (a, sa), [w] = short_problem(M, N, K)
    args, b = (dev(a), by_block(sa), *pair(w)), dev(bias_of(N))
    want = (exact_on_gpu(*args) + b.double()).to(TYPES[t])
    for i in range(5):
        same(q4.gemm_f8(*args, bias=b, dtype=TYPES[t]), want, f"{M} {N} {K}, call {i}")


# A bias in every kind of launch, whose tiles each bring it in a way of their own: few rows from memory (8, 16, 32
# and 64 rows, four and eight wavefronts), tiles through LDS (64 x 64, 64 x 128, 128 x 128, 128 x 256 and 256 x 256,
# one and several a workgroup, in halves and in quarters).  Columns end inside a tile in all of them.
BIASED = [(1, 300, 4096), (3, 129, 144), (10, 1693, 976), (65, 127, 256), (16, 45, 64), (40, 70, 32), (100, 890, 4864),
          (141, 5177, 800), (33, 7794, 4496), (198, 3608, 6208), (333, 4864, 896), (500, 2050, 2064), (4868, 387, 656),
          (5390, 659, 288), (8655, 930, 272), (2910, 2761, 400), (1804, 4310, 1680), (2755, 5834, 400),
          (1915, 8541, 912), (7171, 4233, 464), (5331, 4596, 656), (4300, 4100, 2064)]


def test_biased_sizes_take_every_launch():
    both = {(8, 256), (8, 512), (16, 256), (16, 512), (32, 256), (32, 512), (64, 256), (64, 64, "one each"),
            (64, 128, "one each"), (128, 128, "one each"), (128, 128, "several"), (128, 256, "one each"),
            (128, 256, "several")}
    largest = {(256, 256, k) for k in ("one each", "several", "halves", "quarters")}
    for t, want in (("f32", both), ("f16", both | largest), ("bf16", both | largest)):
        seen = {launches(1, *s, TYPES[t]) for s in BIASED}
        assert want <= seen, (t, want - seen)


@pytest.mark.parametrize("M,N,K", BIASED)
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("tall", [1, 128])
def test_gemm_bias(M, N, K, t, tall):
    (a, sa), [w] = short_problem(M, N, K, tall=tall)
    args, b = (dev(a), by_block(sa) if tall == 1 else dev(sa), *pair(w)), dev(bias_of(N))
    same(q4.gemm_f8(*args, bias=b, dtype=TYPES[t]), exact_on_gpu(*args) + b.double(), f"{M} {N} {K}")


# ---------------------------------------------------------------- gates, on exact products

GATED = [(1, 1, 16), (1, 896, 896), (4, 300, 4096), (16, 65, 144), (30, 1000, 1040), (64, 32, 128), (100, 130, 2816),
         (257, 200, 528), (520, 515, 1296), (64, 2100, 2064), (1500, 4100, 400), (96, 999, 4112), (40, 499, 8208),
         (40, 1373, 48), (100, 1789, 6160), (4300, 2050, 2064), (9, 10, 16), (9, 9, 1056), (17, 9, 16), (4189, 9, 16),
         (19, 2724, 1040), (33, 6864, 1104), (35, 8135, 5824), (8550, 92, 784), (5390, 330, 288), (7439, 700, 272),
         (7056, 1172, 144), (4715, 897, 304), (8655, 465, 272), (4771, 2923, 272), (5331, 2298, 656), (3083, 2610, 272),
         (5470, 151, 320), (1804, 2155, 1680), (2910, 1381, 400), (2755, 2917, 400),
         (1033, 2083, 288), (44, 7211, 7504), (1968, 4020, 784), (3992, 4079, 480), (806, 8365, 1440),
         (9, 4168, 400), (4186, 174, 192)]


def gated_problem(M, N, K, size=4.0):
    """a, gate, up and their exact products g (some beyond +-8 * size) and u, float64 on the host."""
    (a, sa), [gate, up] = short_problem(M, N, K, mats=2)
    gate = gate[0], gate[1] * np.float32(size)
    g, u = (exact_on_gpu(dev(a), dev(sa), *pair(m)).cpu().numpy() for m in (gate, up))
    return (dev(a), by_block(sa)), pair(gate), pair(up), g, u


def check(y, want, bound, t, label):
    got = y.float().cpu().numpy().astype(np.float64)
    tol = f8.tolerance(want, bound, t)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{label}: {int(bad.sum())} of {bad.size} outside, first at {np.argwhere(bad)[0]}, worst "
                           f"{np.nanmax(np.abs(got - want) / tol):.3g} of the tolerance")


@pytest.mark.parametrize("M,N,K", GATED)
@pytest.mark.parametrize("t", TYPES)
def test_swiglu(M, N, K, t):
    a, gate, up, g, u = gated_problem(M, N, K)
    check(q4.gemm_f8_swiglu(*a, gate, up, dtype=TYPES[t]), *f8.gated(g, 0, u, 0), t, f"{M} {N} {K}")


@pytest.mark.parametrize("M,N,K", GATED)
@pytest.mark.parametrize("t,td", [("f32", "bf16"), ("f16", "f32"), ("bf16", "f16"), ("bf16", "bf16")])
def test_swiglu_backward(M, N, K, t, td):
    a, gate, up, g, u = gated_problem(M, N, K)
    dh = torch.from_numpy(np.random.default_rng(3).standard_normal((M, N)).astype(np.float32)).to(TYPES[td])
    d = q4.gemm_f8_swiglu_backward(dh.to(DEV), *a, gate, up, dtype=TYPES[t])
    check(d, *f8.gradient(dh.double().numpy(), g, 0, u, 0), t, f"{M} {N} {K}")


@pytest.mark.parametrize("M,N,K", [(3, 40, 64), (70, 150, 256)])
def test_far_gates(M, N, K):
    """Gates far to both sides: silu(g) -> g and -> 0 with its small values, no NaN."""
    a, gate, up, g, u = gated_problem(M, N, K, size=64.0)
    assert (g < -87).any() and (g < -174).any() and (g > 100).any()
    up = up[0], up[1] * 2.0 ** 60
    u = u * 2.0 ** 60
    check(q4.gemm_f8_swiglu(*a, gate, up), *f8.gated(g, 0, u, 0), "f32", "forward")
    dh = np.random.default_rng(3).standard_normal((M, N)).astype(np.float32)
    check(q4.gemm_f8_swiglu_backward(dev(dh), *a, gate, up), *f8.gradient(dh.astype(np.float64), g, 0, u, 0), "f32",
          "backward")


@pytest.mark.parametrize("M,N", [(3, 40), (70, 72), (300, 264)])
@pytest.mark.parametrize("skew", [0, 1])
def test_swiglu_backward_in_larger_buffers(M, N, skew):
    """dh and d that start off a 16-byte border, with guards around d."""
    a, gate, up, g, u = gated_problem(M, N, 160)
    dh = torch.from_numpy(np.random.default_rng(3).standard_normal(M * N + 1).astype(np.float32)).bfloat16().to(DEV)
    dh = dh[skew:skew + M * N].view(M, N)
    buf = torch.full((2 * M * N + 32,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[8 + skew:8 + skew + 2 * M * N].view(M, 2 * N)
    d = q4.gemm_f8_swiglu_backward(dh, *a, gate, up, dtype=torch.bfloat16, out=out)
    assert d.data_ptr() == out.data_ptr()
    check(d, *f8.gradient(dh.double().cpu().numpy(), g, 0, u, 0), "bf16", f"{M} {N}")
    assert (buf[:8 + skew] == 7).all() and (buf[8 + skew + 2 * M * N:] == 7).all()


# ---------------------------------------------------------------- quantised values

REAL = [(1, 300, 4096), (7, 129, 144), (33, 520, 912), (100, 896, 2816), (200, 333, 2064), (300, 1024, 896),
        (600, 515, 1296), (1500, 1100, 528)]


def real_problem(M, N, K, mats=1, tall=1):
    rng = np.random.default_rng(M + N + K)
    x = rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.02, 8, 1)
    return f8.quant(x, tall), [f8.quant(rng.standard_normal((N, K)) * K ** -0.5, 128) for _ in range(mats)]


@pytest.mark.parametrize("M,N,K", REAL)
@pytest.mark.parametrize("t", TYPES)
def test_gemm_of_quantised_values(M, N, K, t):
    (a, sa), [w] = real_problem(M, N, K)
    y = q4.gemm_f8(dev(a), by_block(sa), *pair(w), dtype=TYPES[t])
    check(y, *f8.product(a, sa, *w, t == "f32"), t, f"{M} {N} {K}")
    # Few steps of the type in all: a mistake that the bound of single values
    # would let pass shows in their mean square.  Rounding to a type is off by
    # 0.3 steps in this mean, a step half an epsilon to one; the 8-bit unit by less than
    # 2^-13 of the largest of eight for each product, which for normal codes is 2^-15.
    want = f8.product(a, sa, *w, True)[0]
    off = y.double().cpu().numpy() - want
    rms = np.sqrt((off ** 2).mean() / (want ** 2).mean())
    assert rms < 0.5 * torch.finfo(TYPES[t]).eps + (2.0 ** -20 if t == "f32" else 2.0 ** -14)


@pytest.mark.parametrize("M,N", [(1, 17), (40, 70), (300, 264), (700, 777)])
@pytest.mark.parametrize("t", TYPES)
def test_small_products_beside_large_ones(M, N, t):
    """One product of 1 among seven of 1.875 * 2^-14, which the 8-bit unit may drop and float32 outputs may not."""
    K = 272
    a, w = np.full((M, K), 0x0F, dtype=np.uint8), np.full((N, K), 0x02, dtype=np.uint8)        # 1.875 * 2^-6, 2^-8
    a[:, 3::8] = w[:, 3::8] = 0x38                                                              # 1
    sa, sw = (np.ones((n, 3), dtype=np.float32) for n in (M, f8.blocks(N)))
    want, bound = f8.product(a, sa, w, sw, t == "f32")
    assert want[0, 0] == 34 * (1 + 7 * 1.875 * 2.0 ** -14)
    y = q4.gemm_f8(dev(a), by_block(sa), dev(w), dev(sw), dtype=TYPES[t])
    check(y, want, bound, t, f"{M} {N}")
    if t == "f32":
        same(y, torch.full((M, N), want[0, 0], dtype=torch.float64, device=DEV), f"{M} {N}")


@pytest.mark.parametrize("M,N,K", REAL)
@pytest.mark.parametrize("t", TYPES)
def test_gates_of_quantised_values(M, N, K, t):
    (a, sa), [gate, up] = real_problem(M, N, K, 2)
    g, eg = f8.product(a, sa, *gate, t == "f32")
    u, eu = f8.product(a, sa, *up, t == "f32")
    args = dev(a), by_block(sa), pair(gate), pair(up)
    check(q4.gemm_f8_swiglu(*args, dtype=TYPES[t]), *f8.gated(g, eg, u, eu), t, "forward")
    dh = np.random.default_rng(3).standard_normal((M, N)).astype(np.float32)
    check(q4.gemm_f8_swiglu_backward(dev(dh), *args, dtype=TYPES[t]),
          *f8.gradient(dh.astype(np.float64), g, eg, u, eu), t, "backward")


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 9, 40, 100, 600])
def test_rows_do_not_mix(M, t):
    """NaN and infinite scales and NaN codes stay in their rows and columns, and zero rows are zero."""
    N, K = 150, 400
    (a, sa), [w] = short_problem(M, N, K)
    a, w0 = a.copy(), w[0].copy()
    a[M // 2] = 0
    w0[3, 7] = 0x7F
    sa = sa.copy()
    sa[M - 1, 2] = np.nan
    y = q4.gemm_f8(dev(a), by_block(sa), dev(w0), dev(w[1]), dtype=TYPES[t]).float().cpu().numpy()
    with np.errstate(invalid="ignore"):
        want = f8.values(a, sa) @ f8.values(w0, w[1]).T
    assert np.array_equal(np.isnan(y), np.isnan(want))
    assert np.isnan(y[M - 1]).all() and np.isnan(y[:, 3]).all()
    if M > 1:
        assert not y[M // 2][np.arange(N) != 3].any()
    # The last, short block's scale infinite in a row.
    sa[M - 1, 2] = 1
    sa[M - 1, 3] = np.inf
    y = q4.gemm_f8(dev(a), by_block(sa), dev(w[0]), dev(w[1]), dtype=TYPES[t]).float().cpu().numpy()
    last = f8.decode(a)[M - 1, 384:] @ f8.decode(w[0])[:, 384:].T          # its sums: infinite, or 0 * Inf
    assert np.array_equal(np.isinf(y[M - 1]), last != 0) and np.array_equal(np.isnan(y[M - 1]), last == 0)
    assert np.isfinite(y[:M - 1]).all()


@pytest.mark.parametrize("M,N,K", [(1, 300, 400), (9, 300, 400), (40, 300, 656), (141, 5177, 800), (130, 300, 912),
                                   (600, 515, 400), (3083, 5219, 272)])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_infinite_scales(M, N, K, t):
    """A block's sum times an infinite scale, whichever operand has it: infinite, or NaN where the sum is zero."""
    (a, sa), [w] = short_problem(M, N, K)
    a, sa, (w, sw) = dev(a), by_block(sa).clone(), pair(w)
    sw[0, 1] = sw[-1, -1] = np.inf
    sa[M // 2, 0] = -np.inf
    y = q4.gemm_f8(a, sa, w, sw, dtype=TYPES[t])
    want = torch.zeros(M, N, dtype=torch.float64, device=DEV)
    for b in range(sa.shape[1]):
        k = slice(128 * b, 128 * b + 128)
        by = sa[:, b, None].double() * sw[:, b].double().repeat_interleave(128)[:N]
        want += (a[:, k].double() @ w[:, k].double().t()) * by
    assert torch.equal(y.isnan(), want.isnan())
    same(torch.where(y.isnan(), 0, y), torch.where(want.isnan(), 0, want), f"{M} {N} {K}")


# ---------------------------------------------------------------- past 32 bits

def test_arrays_past_32_bits():
    """Operands, scales' blocks and outputs whose last parts lie beyond 4 GiB."""
    K, N = 131056, 33_000                                  # 4.3 GB of weights
    w = torch.zeros(N, K, dtype=torch.uint8, device=DEV)
    w[:] = dev(short_codes(2, K)).view(torch.uint8)
    w[:, 5] = dev(short_codes(3, N)).view(torch.uint8)
    w = w.view(F8)
    sw = dev(short_scales(4, f8.blocks(N), K, unit(K)))
    at = slice(N - 300, N)
    for M in (3, 70):
        a, sa = dev(short_codes(1, M, K)), by_block(short_scales(5, M, K, unit(K)))
        nb = f8.blocks(N - 300) - 1
        first = N - 300 - 128 * nb
        want = exact_on_gpu(a, sa, w[128 * nb:], sw[nb:])[:, first:]
        same(q4.gemm_f8(a, sa, w, sw)[:, at], want, f"{M} rows")
        same(q4.gemm_f8_swiglu(a, sa, (w, sw), (w, sw))[:, at].float().isfinite(), torch.ones(M, 300, device=DEV), "gated")
    del w
    M, N, K = 70_000, 32_768, 272                          # 4.6 GB of outputs, twice that of gradients
    (a, sa), [g, u] = short_problem(M, N, K, mats=2)
    args = dev(a), by_block(sa), *pair(g)
    rows = [0, M // 2 + 1, M - 1]
    y = q4.gemm_f8(*args, dtype=torch.bfloat16)
    same(y[rows], exact_on_gpu(args[0][rows], args[1][rows], *pair(g)), "y")
    dh = y.clamp_(-4, 4)
    d = q4.gemm_f8_swiglu_backward(dh, args[0], args[1], pair(g), pair(u), dtype=torch.bfloat16)
    gate, up = (exact_on_gpu(args[0][rows], args[1][rows], *pair(m)).cpu().numpy() for m in (g, u))
    check(d[rows], *f8.gradient(dh[rows].double().cpu().numpy(), gate, 0, up, 0), "bf16", "d")
    del d, y, dh
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(70_000, 32_768, device=DEV, dtype=torch.float16, generator=g)
    c, s, ct, st = q4.quant_f8_block(x, layout="both")
    cr, sr = q4.quant_f8(x)
    last = x[-(70_000 % 128):].double().cpu().numpy()      # the last blocks' rows
    cw, sw = f8.quant(last[:, -256:], 128)
    n = last.shape[0]
    assert np.array_equal(f8.decode(bits(c[-n:, -256:])), f8.decode(cw)) and np.array_equal(bits(s[-1:, -2:]), sw)
    assert np.array_equal(f8.decode(bits(ct[-256:, -n:])), f8.decode(cw.T)) and np.array_equal(bits(st[-2:, -1:]), sw.T)
    cw, sw = f8.quant(last[:, -256:])
    assert np.array_equal(f8.decode(bits(cr[-n:, -256:])), f8.decode(cw)) and np.array_equal(bits(sr[-n:, -2:]), sw)


@pytest.mark.parametrize("M,N", [(3, 40), (40, 200), (300, 264), (700, 777)])
@pytest.mark.parametrize("strides", [(2 ** 20, 1), (1, 2 ** 31), (2 ** 20, 3)])
@pytest.mark.parametrize("tall", [1, 128])
def test_scales_as_far_apart_as_may_be(M, N, strides, tall):
    """Scales of the largest strides, as quant_f8 writes them and as the products read them."""
    K = 272
    rows, KB = M if tall == 1 else f8.blocks(M), f8.blocks(K)
    place = torch.zeros((rows - 1) * strides[0] + (KB - 1) * strides[1] + 1, device=DEV)
    apart = place.as_strided((rows, KB), strides)
    if tall == 1:
        x = values_of(M, M, K, "bf16")
        codes = torch.empty(M, K, dtype=F8, device=DEV)
        q4.quant_f8(x.to(DEV), out=(codes, apart))
        cw, sw = f8.quant(x.double().numpy())
        assert np.array_equal(bits(apart), sw) and np.array_equal(f8.decode(bits(codes)), f8.decode(cw))
        assert int((place != 0).sum()) == rows * KB
    (a, sa), [w] = short_problem(M, N, K, tall=tall)
    apart.copy_(dev(sa))
    want = exact_on_gpu(dev(a), dev(sa), *pair(w))
    for t in (torch.float32, torch.bfloat16):
        same(q4.gemm_f8(dev(a), apart, *pair(w), dtype=t), want, f"{M} {N} {strides}")


# ---------------------------------------------------------------- a layer's step

def step(x, dy, gate, up, down):
    """A feed-forward layer's training step as a program writes it; gate, up [F, D] and down [D, F] in bf16."""
    w13 = torch.cat([gate, up])
    F, D = gate.shape
    FB = F // 128
    w, sw, wt, swt = q4.quant_f8_block(w13, layout="both")
    w2, s2, w2t, s2t = q4.quant_f8_block(down, layout="both")
    a, sa = q4.quant_f8(x)
    pairs = (w[:F], sw[:FB]), (w[F:], sw[FB:])
    h = q4.gemm_f8_swiglu(a, sa, *pairs, dtype=torch.bfloat16)
    y = q4.gemm_f8(*q4.quant_f8(h), w2, s2, dtype=torch.bfloat16)
    dh = q4.gemm_f8(*q4.quant_f8(dy), w2t, s2t, dtype=torch.bfloat16)
    d = q4.gemm_f8_swiglu_backward(dh, a, sa, *pairs, dtype=torch.bfloat16)
    dx = q4.gemm_f8(*q4.quant_f8(d), wt, swt, dtype=torch.bfloat16)
    turn = lambda v: q4.quant_f8_block(v, layout="columns")              # noqa: E731
    dw13 = q4.gemm_f8(*turn(d), *turn(x))
    dw2 = q4.gemm_f8(*turn(dy), *turn(h))
    return y, dx, dw13, dw2


def step_problem(T, D, F, seed=1):
    rng = np.random.default_rng(seed)
    make = lambda *s, size=1.0: torch.from_numpy((rng.standard_normal(s) * size).astype(np.float32)).bfloat16()  # noqa: E731
    return (make(T, D), make(T, D, size=0.01), make(F, D, size=D ** -0.5), make(F, D, size=D ** -0.5),
            make(D, F, size=F ** -0.5))


@pytest.mark.parametrize("T,D,F", [(1, 128, 128), (77, 256, 384), (600, 896, 640)])
def test_training_step(T, D, F):
    """Against autograd in float64.  Each e4m3 rounding is off by 2^-4 of a value at most, 2^-5.8 in the mean
    square; a gradient is reached through six of them, none enlarged much: below 0.1 of its size."""
    tensors = step_problem(T, D, F)
    got = step(*(t.to(DEV) for t in tensors))
    x, dy, gate, up, down = (t.double() for t in tensors)
    for t in (x, gate, up, down):
        t.requires_grad_()
    g = x @ gate.t()
    y = (g * torch.sigmoid(g) * (x @ up.t())) @ down.t()
    y.backward(dy)
    for name, v, want in (("y", got[0], y.detach()), ("dx", got[1], x.grad), ("dw13", got[2], torch.cat([gate.grad, up.grad])),
                          ("dw2", got[3], down.grad)):
        assert tuple(v.shape) == tuple(want.shape)
        assert ((v.double().cpu() - want).norm() / want.norm()).item() < 0.1, name


def test_gradient_against_differences():
    """d is the slope of sum(dh y) in the products' results: by differences of the library's own forward pass along
    up's scales and gate's, which scale u and g."""
    M, N, K = 40, 60, 272
    a, gate, up, g, u = gated_problem(M, N, K, 1.0)
    dh = np.random.default_rng(3).standard_normal((M, N)).astype(np.float32)
    d = q4.gemm_f8_swiglu_backward(dev(dh), *a, gate, up).double().cpu().numpy()
    h = 2.0 ** -9                                   # scales times 1 +- h are exact; g and u move by h of themselves
    for i, v in ((0, g), (1, u)):
        ys = []
        for f in (1 + h, 1 - h):
            pairs = (gate[0], gate[1] * f) if i == 0 else gate, (up[0], up[1] * f) if i == 1 else up
            ys.append(q4.gemm_f8_swiglu(*a, *pairs).double().cpu().numpy())
        slope = (ys[0] - ys[1]) * dh / (2 * h)
        # Differences: third derivatives of silu are below 0.6, so that h^2 g^3 |u dh| / 6 is left out and the
        # two values' own errors, 17 + 5 |g| steps of 2^-24 each, are divided by h.
        tol = h * h * np.abs(g ** 3 * u * dh) * (i == 0) + (40 + 12 * np.abs(g)) * f8.U * np.abs(dh * (np.abs(ys[0]) + 1e-30)) / h
        tol += 2.0 ** -18 * np.abs(d[:, N * i:N * i + N] * v) + 1e-30
        assert (np.abs(slope - d[:, N * i:N * i + N] * v) <= tol).all()


def test_results_do_not_require_grad():
    """As the docstrings say: autograd does not see the calls, and a Function of a program's own makes a step of them."""
    x = torch.randn(40, 256, device=DEV, requires_grad=True)
    w = torch.randn(384, 256, device=DEV, requires_grad=True)
    codes, scales, codes_t, scales_t = q4.quant_f8_block(w, layout="both")
    a, sa = q4.quant_f8(x)
    y = q4.gemm_f8(a, sa.requires_grad_(), codes, scales)
    assert not any(t.requires_grad for t in (a, codes, scales, codes_t, scales_t, y))
    sa = sa.detach()

    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, v):
            return q4.gemm_f8(*q4.quant_f8(v), codes, scales)

        @staticmethod
        def backward(ctx, dy):
            return q4.gemm_f8(*q4.quant_f8(dy), codes_t, scales_t)

    got = Product.apply(x)
    assert got.requires_grad and torch.equal(got, y)
    dy = torch.randn(40, 384, device=DEV)
    got.backward(dy)
    want = q4.gemm_f8(*q4.quant_f8(dy), codes_t, scales_t)
    assert torch.equal(x.grad, want) and w.grad is None


# ---------------------------------------------------------------- streams, graphs, threads

@pytest.mark.parametrize("T", [1, 20, 300])
def test_captured_step_is_the_eager_one(T):
    D, F = 256, 384
    problems = [[t.to(DEV) for t in step_problem(T, D, F, seed)] for seed in (1, 2, 3)]
    eager = [[t.clone() for t in step(*p)] for p in problems]
    held = [t.clone() for t in problems[0]]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*held)
    for i in (0, 1, 2, 0):
        for h, p in zip(held, problems[i]):
            h.copy_(p)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, e) for g, e in zip(got, eager[i]))
        step(*problems[(i + 1) % 3])


def test_two_graphs_and_streams_at_once():
    """Two captured products replayed on two streams, neither of which has a workspace to share."""
    cases = []
    for seed in (1, 2):
        (a, sa), [w] = short_problem(100, 700, 912, seed=seed)
        args = dev(a), by_block(sa), *pair(w)
        want = exact_on_gpu(*args)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            y = q4.gemm_f8(*args, dtype=torch.bfloat16)
        cases.append((torch.cuda.Stream(), graph, y, want, args))
    for _ in range(3):
        for stream, graph, *_ in cases:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, y, want, _ in cases:
            same(y, want, "graph")
            y.zero_()
        torch.cuda.synchronize()


def test_calls_from_threads():
    problems = [short_problem(m, 300, 400, seed=m) for m in (1, 20, 90, 300)]
    args = [(dev(a), by_block(sa), *pair(w)) for (a, sa), [w] in problems]
    want = [exact_on_gpu(*p) for p in args]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                y = q4.gemm_f8(*args[i])
                torch.cuda.current_stream().synchronize()
                if not torch.equal(y, want[i].float()):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_refusals_on_the_device():
    (a, sa), [w] = short_problem(4, 40, 64)
    a, sa, (wc, ws) = dev(a), dev(sa), pair(w)
    dh = torch.zeros(4, 40, device=DEV)
    bad = [(ValueError, lambda: q4.gemm_f8(a, sa[:3], wc, ws)), (ValueError, lambda: q4.gemm_f8(a, sa, wc, ws[:, :0])),
           (ValueError, lambda: q4.gemm_f8(a[:, ::2], sa, wc, ws)), (ValueError, lambda: q4.gemm_f8(a, sa, wc[:, :48], ws)),
           (ValueError, lambda: q4.gemm_f8(a, sa, wc, ws, bias=dh[0, :3])), (TypeError, lambda: q4.gemm_f8(a, sa.half(), wc, ws)),
           (ValueError, lambda: q4.gemm_f8(a, sa.cpu(), wc, ws)), (ValueError, lambda: q4.gemm_f8(a, sa, wc, ws, out=dh[:, :3])),
           (TypeError, lambda: q4.gemm_f8(a, sa, wc, ws, dtype=torch.float16, out=dh)),
           (ValueError, lambda: q4.gemm_f8_swiglu(a, sa, (wc, ws), (wc[:20], ws))),
           (ValueError, lambda: q4.gemm_f8_swiglu_backward(dh[:3], a, sa, (wc, ws), (wc, ws))),
           (ValueError, lambda: q4.gemm_f8_swiglu_backward(dh, a, sa, (wc, ws), (wc, ws), out=dh)),
           (TypeError, lambda: q4.gemm_f8_swiglu_backward(None, a, sa, (wc, ws), (wc, ws))),
           (TypeError, lambda: q4.gemm_f8_swiglu_backward(dh.double(), a, sa, (wc, ws), (wc, ws))),
           (ValueError, lambda: q4.quant_f8(dh[:, ::2])), (ValueError, lambda: q4.quant_f8(dh[0])),
           (ValueError, lambda: q4.quant_f8(dh[:, :16].contiguous(), out=(a[:, :16], sa))),
           (ValueError, lambda: q4.quant_f8_block(dh[:, :16].contiguous(), out=(a,))),
           (q4.Q4Error, lambda: q4.quant_f8(dh)), (q4.Q4Error, lambda: q4.quant_f8_block(dh))]      # 40 columns
    for i, (kind, fn) in enumerate(bad):
        with pytest.raises(kind):
            fn()
            print("not refused:", i)
