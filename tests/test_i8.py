"""8-bit operators: what can be checked without a GPU.  The library exports
what include/q4i8.h declares, refuses bad arguments before it touches the
device, and the oracle agrees with integer arithmetic and worked values."""

import os
import re
import subprocess

import numpy as np
import pytest
import torch

import memory_bandwidth_amd as q4
from oracle import i8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000          # fake, aligned, never dereferenced device address


@pytest.fixture(scope="module")
def L():
    from memory_bandwidth_amd import build
    if not os.path.exists(q4.LIB_PATH) or not os.path.exists(build.BIND):
        build.build()
    return q4.lib()


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "q4i8.h")).read(), flags=re.S)
    return re.findall(r"^int\s+([a-z_0-9]+)\s*\(", text, flags=re.M)


def test_header_and_exports_agree(L):
    assert tuple(declared()) == q4.EXPORTS_I8
    out = subprocess.run(["nm", "-D", "--defined-only", q4.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert set(declared()) <= exported


def call(L, fn, M, N, K, t=q4.I8_F32, E=2, p=None, at=()):
    """Calls fn with fake pointers; `at` overrides pointers by position."""
    n = {"quant_i8": 3, "gemm_i8": 6, "gemm_i8_swiglu": 7, "gemm_i8_grouped": 6, "gemm_i8_grouped_swiglu": 8}[fn]
    ptr = [A] * n
    for i, v in at:
        ptr[i] = v
    if fn == "quant_i8":
        return L.quant_i8(ptr[0], t, ptr[1], ptr[2], M, K, None)
    sizes = [M, E, N, K] if "grouped" in fn else [M, N, K]
    return getattr(L, fn)(*ptr, t, *sizes, None)


CALLS = [f for f in q4.EXPORTS_I8 if f != "gemm_i8_geometry"]
GEMMS = [f for f in CALLS if f != "quant_i8"]


@pytest.mark.parametrize("fn", GEMMS)
@pytest.mark.parametrize("M,N,K,want", [
    (-1, 8, 64, q4.Q4_EINVAL), (1, -1, 64, q4.Q4_EINVAL), (1, 8, 0, q4.Q4_EINVAL), (1, 8, 24, q4.Q4_EINVAL),
    (1, 8, 8, q4.Q4_EINVAL), (1, 8, 131072, q4.Q4_EINVAL), (2**24 + 1, 8, 64, q4.Q4_EINVAL),
    (1, 2**24 + 1, 64, q4.Q4_EINVAL), (2**24, 2**24, 64, q4.Q4_EINVAL),
    (0, 8, 64, q4.Q4_OK), (4, 0, 64, q4.Q4_OK), (0, 8, 131056, q4.Q4_OK),
])
def test_gemm_sizes(L, fn, M, N, K, want):
    assert call(L, fn, M, N, K) == want


@pytest.mark.parametrize("fn", CALLS)
@pytest.mark.parametrize("t", [-1, 3])
def test_types(L, fn, t):
    assert call(L, fn, 4, 8, 64, t=t) == q4.Q4_EINVAL


@pytest.mark.parametrize("fn", [f for f in GEMMS if "grouped" in f])
def test_group_counts(L, fn):
    assert call(L, fn, 4, 8, 64, E=0) == q4.Q4_EINVAL
    assert call(L, fn, 4, 8, 64, E=65537) == q4.Q4_EINVAL
    assert call(L, fn, 4, 2**24, 64, E=256) == q4.Q4_EINVAL


@pytest.mark.parametrize("fn", CALLS)
def test_pointers(L, fn):
    n = {"quant_i8": 3, "gemm_i8": 6, "gemm_i8_swiglu": 7, "gemm_i8_grouped": 6, "gemm_i8_grouped_swiglu": 8}[fn]
    for i in range(n):
        if fn == "gemm_i8" and i == 4:                 # bias may be NULL
            continue
        assert call(L, fn, 4, 8, 64, at=[(i, None)]) == q4.Q4_ENULL, i
        assert call(L, fn, 4, 8, 64, at=[(i, A + 1)]) == q4.Q4_EALIGN, i
    for i in {"quant_i8": (0, 1), "gemm_i8": (0, 2), "gemm_i8_swiglu": (0, 2, 4), "gemm_i8_grouped": (0, 2),
              "gemm_i8_grouped_swiglu": (0, 2, 4)}[fn]:
        assert call(L, fn, 4, 8, 64, at=[(i, A + 8)]) == q4.Q4_EALIGN, i


@pytest.mark.parametrize("M,K,want", [(-1, 64, q4.Q4_EINVAL), (1, 0, q4.Q4_EINVAL), (1, 40, q4.Q4_EINVAL),
                                      (1, 131072, q4.Q4_EINVAL), (0, 64, q4.Q4_OK)])
def test_quant_sizes(L, M, K, want):
    assert call(L, "quant_i8", M, 8, K) == want


@pytest.mark.skipif(torch.cuda.is_available(), reason="a GPU would be given fake addresses")
@pytest.mark.parametrize("fn", CALLS)
def test_no_device(L, fn):
    assert call(L, fn, 4, 8, 64) == q4.Q4_EDEVICE


def test_binding_refuses_host_tensors_and_wrong_types(L):
    a, s = torch.zeros(2, 32, dtype=torch.int8), torch.ones(2)
    w, sw = torch.zeros(4, 32, dtype=torch.int8), torch.ones(4)
    with pytest.raises(ValueError):
        q4.gemm_i8(a, s, w, sw)
    with pytest.raises(TypeError):
        q4.gemm_i8(a.float(), s, w, sw)
    with pytest.raises(TypeError):
        q4.quant_i8(a)
    with pytest.raises(ValueError):
        q4.quant_i8(a.float())


def test_module_returns_none_for_what_it_cannot_take(L):
    m = q4._load_bind()
    a, s = torch.zeros(2, 32, dtype=torch.int8), torch.ones(2)
    w, sw = torch.zeros(4, 32, dtype=torch.int8), torch.ones(4)
    good = [a, s, w, sw, None, None, torch.float32, None]
    assert m.gemm(*good) is None                           # on the host
    for i in range(8):
        assert m.gemm(*good[:i], "no", *good[i + 1:]) is None
    assert m.swiglu(a, s, w, sw, w, sw, None, torch.float32, None) is None
    assert m.quant(a.float(), None, None) is None and m.quant(None, None, None) is None
    for fn in (m.gemm, m.swiglu, m.quant):
        with pytest.raises(TypeError):
            fn(a)


@pytest.mark.parametrize("bad", [None, 3, [1.0]])
def test_binding_refuses_what_is_no_tensor(L, bad):
    s, w, sw = torch.ones(2), torch.zeros(4, 32, dtype=torch.int8), torch.ones(4)
    off = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: q4.gemm_i8(bad, s, w, sw), lambda: q4.gemm_i8_swiglu(bad, s, (w, sw), (w, sw)),
                 lambda: q4.gemm_i8_grouped(bad, s, w[None], sw[None], off),
                 lambda: q4.gemm_i8_grouped_swiglu(bad, s, (w[None], sw[None]), (w[None], sw[None]), off)):
        with pytest.raises(TypeError, match="^a must be a torch.Tensor"):
            call()
    with pytest.raises(TypeError, match="^x must be a torch.Tensor"):
        q4.quant_i8(bad)


# Shapes (matrices, M, N, K, groups) and the tile of y that they take.
PLANS = [((1, 1, 14336, 4096, 0), (8, 64)), ((1, 12, 4096, 4096, 0), (16, 16)), ((1, 24, 4096, 14336, 0), (32, 16)),
         ((1, 64, 4096, 14336, 0), (32, 32)), ((1, 64, 1024, 4096, 0), (16, 16)),
         ((1, 512, 2048, 2048, 0), (64, 64)), ((1, 333, 4864, 896, 0), (64, 128)),
         ((1, 1024, 14336, 512, 0), (128, 128)), ((1, 3775, 1826, 1056, 0), (128, 256)),
         ((1, 8192, 14336, 4096, 0), (256, 256)), ((2, 8192, 14336, 4096, 0), (256, 128)),
         ((2, 200, 2816, 1024, 64), (16, 64)), ((2, 900, 2816, 1024, 64), (64, 64)),
         ((2, 8000, 2816, 1024, 64), (128, 128))]


@pytest.mark.parametrize("shape,tile", PLANS)
def test_geometry(L, shape, tile):
    mats, M, N, K, E = shape
    g = q4.gemm_i8_geometry(mats, M, N, K, E)
    assert (g["tile_rows"], g["tile_cols"]) == tile
    assert g["block"] in (256, 512)
    tiles = -(-M // tile[0]) * -(-N // tile[1])
    # One workgroup a tile, or a chip full of them that go through the tiles;
    # groups may end inside a tile.
    assert g["grid"] == tiles or g["grid"] in (256, 512) and g["grid"] < tiles or E and tiles < g["grid"]


# Shapes of the largest tiles, the workgroups of their whole rounds (256 that
# stay, or one a tile from 65 steps on), and of what is left: tiles x 2 halves
# or 4 quarters.
LAST_ROUNDS = [((1, 8192, 14336, 4096), 256, 0), ((1, 4300, 4100, 2064), 256, 33 * 4),
               ((1, 4096, 5300, 2000), 256, 80 * 2), ((1, 8200, 4097, 1040), 256, 49 * 4),
               ((1, 4352, 8192, 9216), 512, 32 * 4), ((1, 4300, 2050, 2064), 153, 0),
               ((2, 4300, 4100, 2064), 256, 49 * 4), ((2, 4096, 5300, 2000), 256, 0),
               ((2, 8200, 4097, 1040), 256, 65 * 2), ((2, 4352, 8192, 9216), 1024, 64 * 4),
               ((2, 4096, 4700, 9216), 512, 80 * 2)]


@pytest.mark.parametrize("shape,whole,divided", LAST_ROUNDS)
def test_geometry_counts_every_launch(L, shape, whole, divided):
    assert q4.gemm_i8_geometry(*shape) == {"tile_rows": 256, "tile_cols": 256 // shape[0], "grid": whole + divided,
                                           "block": 512}


@pytest.mark.parametrize("mats", [1, 2])
def test_geometry_of_groups_counts_every_launch(L, mats):
    """With groups the GPU counts the tiles: a launch for each way they may be left."""
    g = q4.gemm_i8_geometry(mats, 8190, 4096 // mats, 14336, 8)
    tiles = (8190 // 256 + 8) * (4096 // 256)
    assert g == {"tile_rows": 256, "tile_cols": 256 // mats, "grid": tiles + 2 * 128 + 4 * 64, "block": 512}


def test_geometry_refusals(L):
    for shape in ((0, 4, 8, 64), (3, 4, 8, 64), (1, 4, 8, 24), (1, -1, 8, 64), (1, 4, 8, 64, -1),
                  (1, 2**24, 2**24, 64)):
        with pytest.raises(q4.Q4Error):
            q4.gemm_i8_geometry(*shape)
    assert q4.gemm_i8_geometry(1, 0, 8, 64)["grid"] == 0


# ---------------------------------------------------------------- the oracle

def test_oracle_quant_worked_values():
    # Row 0: scale exactly 1, ties at .5 go to the even integer.  Row 1: zeros.  Row 2: an infinity.
    x = np.array([[127, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5], [0] * 8, [1, np.inf, 0, 0, 0, 0, 0, 0]])
    c, s = i8.quant(x)
    assert c[0].tolist() == [127, 0, 2, 2, 0, -2, -2, 126]
    assert s[0] == 1 and s[1] == np.float32(2.0 ** -126) and not c[1].any()
    assert np.isnan(s[2]) and not c[2].any()


def test_oracle_product_is_integer_arithmetic():
    rng = np.random.default_rng(3)
    a = rng.integers(-128, 128, (5, 4096), dtype=np.int8)
    w = rng.integers(-128, 128, (7, 4096), dtype=np.int8)
    a[0], w[0] = -128, -128
    one = np.ones(7, dtype=np.float32)
    assert np.array_equal(i8.product(a, one[:5], w, one), a.astype(np.int64) @ w.astype(np.int64).T)


def test_oracle_swiglu_and_bias_worked_values():
    a = np.array([[2, 0]], dtype=np.int8)
    g = (np.array([[3, 9]], dtype=np.int8), np.array([0.5], dtype=np.float32))
    u = (np.array([[-4, 9]], dtype=np.int8), np.array([0.25], dtype=np.float32))
    sa = np.array([1.0], dtype=np.float32)
    y, _ = i8.swiglu(a, sa, g, u)                  # g = 3, u = -2
    assert y[0, 0] == pytest.approx(-2 * 3 / (1 + np.exp(-3.0)), rel=1e-15)
    y, _ = i8.gemm(a, sa, *g, bias=np.array([10], dtype=np.float32))
    assert y[0, 0] == 13
    assert i8.groups([0, 2, 2, 5]) == [(0, 0, 2), (2, 2, 5)]


# ---------------------------------------------------------------- the bounds, against fp32 arithmetic

F = np.float32


def fp32_product(a, sa, w, sw):
    """The steps of include/q4i8.h: the exact sum, converted, times a_scales, times w_scales."""
    acc = (a.astype(np.int64) @ w.astype(np.int64).T).astype(F)
    return acc * sa[:, None] * sw[None, :]


def fp32_swiglu(g, u):
    """silu(g) * u in fp32 as the header defines it, far gates through e^g in two halves."""
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        near = g * (F(1) / (F(1) + np.exp2(-g * F(np.log2(np.e))))) * u
        half = np.exp2(g * F(np.log2(np.e) / 2))
        return np.where(g < F(-87), g * half * u * half, near)


def inside(got, want, bound, t="f32"):
    """Whether each value is inside what the GPU's are held to."""
    return np.abs(got.astype(np.float64) - want) <= i8.tolerance(want, bound, t)


def bound_problem(seed=1, M=9, N=200, K=912):
    rng = np.random.default_rng(seed)
    a, wg, wu = (rng.integers(-128, 128, (r, K), dtype=np.int8) for r in (M, N, N))
    sa, sg, su = ((rng.uniform(0.5, 2, r) / (74 * K ** 0.25)).astype(F) for r in (M, N, N))
    return a, sa, (wg, sg * F(4)), (wu, su), (rng.standard_normal(N) * 3).astype(F)


def test_bounds_hold_fp32_steps_and_little_more():
    a, sa, gate, up, bias = bound_problem()
    p = fp32_product(a, sa, *gate)
    want, bound = i8.gemm(a, sa, *gate)
    assert inside(p, want, bound).all()
    assert np.max(np.abs(p - want) / bound) > 0.1
    want, bound = i8.gemm(a, sa, *gate, bias=bias)
    assert inside(p + bias, want, bound).all()
    # One rounding fewer: the last product and the addition in one step.
    one = ((a.astype(np.int64) @ gate[0].astype(np.int64).T).astype(F) * sa[:, None]).astype(np.float64)
    assert inside((one * gate[1].astype(np.float64) + bias).astype(F), want, bound).all()
    want, bound = i8.swiglu(a, sa, gate, up)
    y = fp32_swiglu(p, fp32_product(a, sa, *up))
    assert inside(y, want, bound).all()
    assert np.max(np.abs(y - want) / bound) > 0.1


def test_bounds_refuse_mistakes():
    """What is computed a little wrongly is outside, in most places and not only in one."""
    a, sa, gate, up, bias = bound_problem()
    p, u = fp32_product(a, sa, *gate), fp32_product(a, sa, *up)
    want, bound = i8.gemm(a, sa, *gate, bias=bias)
    for name, y in {"P in fp16": p.astype(np.float16).astype(F) + bias, "no bias": p,
                    "the next column's bias": p + np.roll(bias, 1),
                    "the next row's scale": fp32_product(a, np.roll(sa, 1), *gate) + bias,
                    "the next column's scale": fp32_product(a, sa, gate[0], np.roll(gate[1], 1)) + bias,
                    "one product less": fp32_product(a[:, :-1], sa, gate[0][:, :-1], gate[1]) + bias,
                    "scales in fp16": fp32_product(a, sa.astype(np.float16).astype(F), *gate) + bias}.items():
        assert inside(y, want, bound).mean() < 0.1, name
    want, bound = i8.swiglu(a, sa, gate, up)
    for name, y in {"gate and up exchanged": fp32_swiglu(u, p),
                    "g in fp16": fp32_swiglu(p.astype(np.float16).astype(F), u),
                    "u in fp16": fp32_swiglu(p, u.astype(np.float16).astype(F)),
                    "no silu": p * u, "sigmoid": p / (F(1) + np.exp(-F(1.702) * p)) * u}.items():
        assert inside(y, want, bound).mean() < 0.1, name
    # The exponential, where it has a say: its half step of 2^-12 or more times its weight 1 / (1 + e^g) > 0.1.
    near = np.abs(p + 1) < 3
    y = p * (F(1) / (F(1) + np.exp(np.where(near, -p, 0)).astype(np.float16).astype(F))) * u
    assert inside(y, want, bound)[near].mean() < 0.1


@pytest.mark.parametrize("size", [2.0 ** 110, 1e-3])
def test_bounds_of_far_gates(size):
    """Gates from -174 to 174, with up products that bring silu's small values back or do not."""
    g = np.linspace(-128, 127, 256).astype(np.int8)[:, None]
    one, scale = np.ones((1, 1), dtype=np.int8), np.array([1.36], dtype=F)
    sa, up = np.ones(256, dtype=F), (one, np.array([size], dtype=F))
    a = np.concatenate([g, np.ones_like(g)], axis=1)
    gate, up = (np.array([[1, 0]], dtype=np.int8), scale), (np.array([[0, 1]], dtype=np.int8), up[1])
    want, bound = i8.swiglu(a, sa, gate, up)
    v, u = fp32_product(a, sa, *gate), fp32_product(a, sa, *up)
    y = fp32_swiglu(v, u)
    assert inside(y, want, bound).all()
    # The bound that q4i8.h gives.
    rel = np.where(v < 0, 5.2 * np.abs(v) + 17, 17).astype(np.float64) * i8.U * np.abs(want)
    assert (bound <= rel + np.abs(u.astype(np.float64)) * (v < -174) * 2.0 ** -244 + 2.0 ** -149).all()
    if size > 1:
        with np.errstate(over="ignore", under="ignore"):
            lost = v * np.where(F(1) + np.exp(-v) < 2.0 ** 126, F(1) / (F(1) + np.exp(-v)), F(0)) * u
        far = (v < -87.4)[:, 0]
        assert not inside(lost, want, bound)[far].any() and inside(lost, want, bound)[~far].all()
