"""Operators of 8-bit floating point: what can be checked without a GPU.  The
library exports what include/q4f8.h declares, refuses bad arguments before it
touches the device, and the oracle agrees with worked values, with exact
arithmetic and, for gradients, with differences."""

import importlib.util
import os
import random
import re
import subprocess
from fractions import Fraction

import numpy as np
import pytest
import torch

import memory_bandwidth_amd as q4
from oracle import f8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000          # fake, aligned, never dereferenced device address
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def L():
    from memory_bandwidth_amd import build
    if not os.path.exists(q4.LIB_PATH) or not os.path.exists(build.BIND):
        build.build()
    return q4.lib()


def test_header_and_exports_agree(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "q4f8.h")).read(), flags=re.S)
    declared = re.findall(r"^int\s+([a-z_0-9]+)\s*\(", text, flags=re.M)
    assert tuple(declared) == q4.EXPORTS_F8
    out = subprocess.run(["nm", "-D", "--defined-only", q4.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert set(declared) <= {ln.split()[-1] for ln in out.splitlines() if " T " in ln}


# Pointers of each call, in order, and those that need 16 bytes.
POINTERS = {"quant_f8": 3, "quant_f8_block": 5, "gemm_f8": 6, "gemm_f8_swiglu": 7, "gemm_f8_swiglu_backward": 8}
WIDE = {"quant_f8": (0, 1), "quant_f8_block": (0, 1, 3), "gemm_f8": (0, 2), "gemm_f8_swiglu": (0, 2, 4),
        "gemm_f8_swiglu_backward": (1, 3, 5)}
CALLS = list(POINTERS)
GEMMS = CALLS[2:]


def call(L, fn, M, N, K, t=q4.I8_F32, td=q4.I8_F16, at=(), sm=1, sk=4, block=1):
    """Calls fn with fake pointers; `at` overrides pointers by position."""
    p = [A] * POINTERS[fn]
    for i, v in at:
        p[i] = v
    if fn == "quant_f8":
        return L.quant_f8(p[0], t, p[1], p[2], sm, sk, M, K, None)
    if fn == "quant_f8_block":
        return L.quant_f8_block(p[0], t, p[1], p[2], p[3], p[4], M, K, None)
    if fn == "gemm_f8_swiglu_backward":
        return L.gemm_f8_swiglu_backward(p[0], td, p[1], p[2], sm, sk, block, *p[3:], t, M, N, K, None)
    return getattr(L, fn)(p[0], p[1], sm, sk, block, *p[2:], t, M, N, K, None)


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


@pytest.mark.parametrize("t", [-1, 3])
def test_type_of_the_gradient(L, t):
    assert call(L, "gemm_f8_swiglu_backward", 4, 8, 64, td=t) == q4.Q4_EINVAL


@pytest.mark.parametrize("fn", GEMMS)
def test_scale_layouts(L, fn):
    for bad in ({"sm": -1}, {"sk": -1}, {"sm": 2**20 + 1}, {"sk": 2**31 + 1}, {"block": 0}, {"block": 2},
                {"block": 64}):
        assert call(L, fn, 4, 8, 64, **bad) == q4.Q4_EINVAL, bad


def test_quant_strides(L):
    for bad in ({"sm": 0}, {"sm": -1}, {"sk": 0}, {"sm": 2**20 + 1}, {"sk": 2**31 + 1}):
        assert call(L, "quant_f8", 4, 8, 256, **bad) == q4.Q4_EINVAL, bad
    assert call(L, "quant_f8", 0, 8, 256) == q4.Q4_OK


@pytest.mark.parametrize("M,K,sm,sk,fine", [
    (4, 256, 1, 4, True), (4, 256, 1, 3, False), (4, 256, 1, 1, False), (4, 256, 2, 1, True), (4, 256, 2, 2, False),
    (4, 384, 3, 1, True), (4, 384, 2, 1, False), (1, 256, 0, 1, True), (1, 256, 0, 0, False), (4, 128, 1, 0, True),
    (4, 128, 0, 1, False), (1, 128, 0, 0, True), (0, 256, 0, 1, True)])
def test_quant_scales_have_places_of_their_own(L, M, K, sm, sk, fine):
    want = q4.Q4_EINVAL if not fine else q4.Q4_OK if M == 0 else q4.Q4_ENULL
    assert call(L, "quant_f8", M, 8, K, sm=sm, sk=sk, at=[(0, None)]) == want


@pytest.mark.parametrize("fn", CALLS)
def test_pointers(L, fn):
    for i in range(POINTERS[fn]):
        if fn == "gemm_f8" and i == 4:                 # bias may be NULL
            continue
        assert call(L, fn, 4, 8, 64, at=[(i, None)]) == q4.Q4_ENULL, i
        assert call(L, fn, 4, 8, 64, at=[(i, A + 1)]) == q4.Q4_EALIGN, i
    assert call(L, "gemm_f8", 4, 8, 64, at=[(4, A + 2)]) == q4.Q4_EALIGN
    for i in WIDE[fn]:
        assert call(L, fn, 4, 8, 64, at=[(i, A + 8)]) == q4.Q4_EALIGN, i


def test_quant_block_needs_an_output(L):
    assert call(L, "quant_f8_block", 4, 8, 64, at=[(i, None) for i in (1, 2, 3, 4)]) == q4.Q4_ENULL


@pytest.mark.parametrize("fn", ["quant_f8", "quant_f8_block"])
@pytest.mark.parametrize("M,K,want", [(-1, 64, q4.Q4_EINVAL), (1, 0, q4.Q4_EINVAL), (1, 40, q4.Q4_EINVAL),
                                      (1, 131072, q4.Q4_EINVAL), (2**22, 64, q4.Q4_EINVAL), (0, 64, q4.Q4_OK)])
def test_quant_sizes(L, fn, M, K, want):
    assert call(L, fn, M, 8, K) == want


@pytest.mark.skipif(torch.cuda.is_available(), reason="a GPU would be given fake addresses")
@pytest.mark.parametrize("fn", CALLS)
def test_no_device(L, fn):
    assert call(L, fn, 4, 8, 64) == q4.Q4_EDEVICE


def operands(M=2, N=4, K=32):
    return (torch.zeros(M, K).to(F8), torch.ones(M, 1), torch.zeros(N, K).to(F8), torch.ones(1, 1))


def test_binding_refuses_host_tensors_and_wrong_types(L):
    a, s, w, sw = operands()
    x = torch.zeros(2, 32)
    for bad in (lambda: q4.gemm_f8(a, s, w, sw), lambda: q4.gemm_f8_swiglu(a, s, (w, sw), (w, sw)),
                lambda: q4.gemm_f8_swiglu_backward(x, a, s, (w, sw), (w, sw)), lambda: q4.quant_f8(x),
                lambda: q4.quant_f8_block(x), lambda: q4.quant_f8_block(x, layout="turned")):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q4.gemm_f8(x, s, w, sw), lambda: q4.gemm_f8(a, s, w, sw, dtype=torch.float64),
                lambda: q4.gemm_f8_swiglu(a, s, (w, None), (w, sw)), lambda: q4.quant_f8(a),
                lambda: q4.quant_f8_block(a), lambda: q4.gemm_f8_geometry(1, 4, 8, 64, dtype=torch.int8)):
        with pytest.raises(TypeError):
            bad()


@pytest.mark.parametrize("bad", [None, 3, [1.0]])
def test_binding_refuses_what_is_no_tensor(L, bad):
    a, s, w, sw = operands()
    for fn in (lambda: q4.gemm_f8(bad, s, w, sw), lambda: q4.gemm_f8_swiglu(bad, s, (w, sw), (w, sw)),
               lambda: q4.gemm_f8_swiglu_backward(torch.zeros(2, 4), bad, s, (w, sw), (w, sw))):
        with pytest.raises(TypeError, match="^a must be a torch.Tensor"):
            fn()
    for fn in (q4.quant_f8, q4.quant_f8_block):
        with pytest.raises(TypeError, match="^x must be a torch.Tensor"):
            fn(bad)


def test_module_returns_none_for_what_it_cannot_take(L):
    m = q4._load_bind()
    a, s, w, sw = operands()
    for fn, good in ((m.gemm_f8, [a, s, w, sw, None, torch.float32, None]),
                     (m.swiglu_f8, [a, s, w, sw, w, sw, torch.float32, None]),
                     (m.swiglu_backward_f8, [torch.zeros(2, 4), a, s, w, sw, w, sw, torch.float32, None])):
        assert fn(*good) is None                           # on the host
        for i in range(len(good)):
            assert fn(*good[:i], "no", *good[i + 1:]) is None
        with pytest.raises(TypeError):
            fn(a)
    assert m.quant_f8(torch.zeros(2, 32), None, None) is None and m.quant_f8(None, None, None) is None
    assert m.quant_block_f8(torch.zeros(2, 32), True, False, None, None, None, None) is None


# Shapes (matrices, type, M, N, K) and the tile of y that they take.
PLANS = [((1, torch.bfloat16, 1, 14336, 4096), 8), ((1, torch.bfloat16, 8192, 14336, 4096), 256),
         ((2, torch.bfloat16, 8192, 14336, 4096), 256), ((1, torch.float32, 8192, 14336, 4096), 128)]


@pytest.mark.parametrize("shape,rows", PLANS)
def test_geometry(L, shape, rows):
    mats, t, M, N, K = shape
    g = q4.gemm_f8_geometry(mats, M, N, K, t)
    assert g["tile_rows"] == rows and g["block"] in (256, 512) and g["grid"] > 0


def test_geometry_refusals(L):
    for shape in ((0, 4, 8, 64), (3, 4, 8, 64), (1, 4, 8, 24), (1, -1, 8, 64), (1, 2**24, 2**24, 64)):
        with pytest.raises(q4.Q4Error):
            q4.gemm_f8_geometry(*shape)
    assert q4.gemm_f8_geometry(1, 0, 8, 64)["grid"] == 0


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_fit_script_has_the_librarys_choice(L, t):
    """perf/fit_gemm_f8.py, which fits the constants of the choice, estimates as the library does."""
    spec = importlib.util.spec_from_file_location("fit_gemm_f8", os.path.join(ROOT, "perf", "fit_gemm_f8.py"))
    fit = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fit)
    rng = random.Random(3)
    shapes = [fit.draw(rng)[:4] for _ in range(1000)]
    shapes += [[rng.randint(1, 200), rng.randint(1, 5000), 16 * rng.randint(1, 20), rng.choice([1, 2])]
               for _ in range(500)]
    calls = fit.Calls(t, shapes)
    for i, ((M, N, K, mats), kernel) in enumerate(zip(shapes, calls.choose(fit.constants(t)))):
        g = q4.gemm_f8_geometry(mats, M, N, K, torch.float32 if t == "f32" else torch.bfloat16)
        assert (g["tile_rows"], g["tile_cols"]) == calls.tile(i, kernel), (M, N, K, mats)


# ---------------------------------------------------------------- the oracle

def test_oracle_codes_are_torchs():
    """All 256 codes against torch's e4m3 type, and encoding them gives them back."""
    codes = np.arange(256, dtype=np.uint8)
    assert np.array_equal(f8.decode(codes), torch.from_numpy(codes).view(F8).double().numpy(), equal_nan=True)
    finite = codes[~np.isnan(f8.decode(codes))]
    assert np.array_equal(f8.encode(f8.decode(finite)), finite)


def test_oracle_encode_worked_values():
    # 1 = 0x38, 1.125 = 0x39: between them 1.0625 goes to the even code; 2^-10 to 0, 1.5 * 2^-9 to 2.
    q = np.array([1.0625, 1.0624, 1.0626, -1.0625, 1.1875, 2.0 ** -10, 2.0 ** -10 * 1.0001, 1.5 * 2.0 ** -9, 448, 460,
                  1e9, 0.0])
    assert f8.encode(q).tolist() == [0x38, 0x38, 0x39, 0xB8, 0x3A, 0, 1, 2, 0x7E, 0x7E, 0x7E, 0]


def test_oracle_quant_worked_values():
    x = np.zeros((3, 200))
    x[0, :4] = [448, 1.0625, -448, 2.0 ** -10]
    x[0, 130:132] = [-896, 2.125]                    # second block, 72 long: scale 2
    x[2, 5] = np.inf
    c, s = f8.quant(x)
    assert s[0].tolist() == [1, 2] and s[1].tolist() == [2.0 ** -126] * 2
    assert c[0, :4].tolist() == [0x7E, 0x38, 0xFE, 0] and c[0, 130:132].tolist() == [0xFE, 0x38]
    assert np.isnan(s[2, 0]) and s[2, 1] == np.float32(2.0 ** -126) and not c[2].any()
    x[2, 5] = 4480
    c, s = f8.quant(x, 128)
    assert s.shape == (1, 2) and s[0].tolist() == [10, 2] and c[2, 5] == 0x7E
    ct, st = f8.turned(c, s)
    assert ct.shape == (200, 16) and st.shape == (2, 1) and np.array_equal(ct[:, :3], c.T) and not ct[:, 3:].any()


def small_problem(seed=1, M=5, N=140, K=272):
    rng = np.random.default_rng(seed)
    a, sa = f8.quant(rng.standard_normal((M, K)))
    w, sw = f8.quant(rng.standard_normal((N, K)) * 0.2, 128)
    return a, sa, w, sw


def test_oracle_product_is_exact_arithmetic():
    a, sa, w, sw = small_problem()
    p, _ = f8.product(a, sa, w, sw, True)
    for m, n in ((0, 0), (4, 139), (2, 130)):
        want = sum(Fraction(f8.VALUES[a[m, k]]) * Fraction(float(sa[m, k // 128])) * Fraction(f8.VALUES[w[n, k]]) *
                   Fraction(float(sw[n // 128, k // 128])) for k in range(a.shape[1]))
        assert p[m, n] == pytest.approx(float(want), rel=1e-13)
    # Scales for blocks of rows.
    b, sb = f8.quant(np.random.default_rng(2).standard_normal((130, 272)), 128)
    p, _ = f8.product(b, sb, w, sw, True)
    assert p[129, 7] == pytest.approx(float((f8.decode(b)[129] * np.repeat(sb[1], 128)[:272]) @
                                            (f8.decode(w)[7] * np.repeat(sw[0], 128)[:272])), rel=1e-12)


def test_oracle_gated_and_gradient_worked_values():
    g, u, dh = np.array([[3.0, 0.0, -1.0]]), np.array([[-2.0, 5.0, 4.0]]), np.array([[1.0, 2.0, -1.0]])
    y, _ = f8.gated(g, 0, u, 0)
    assert y[0, 0] == pytest.approx(-6 / (1 + np.exp(-3.0)), rel=1e-15) and y[0, 1] == 0
    d, _ = f8.gradient(dh, g, 0, u, 0)
    s = 1 / (1 + np.exp(1.0))
    assert d[0].tolist() == pytest.approx([-2 * (1 / (1 + np.exp(-3.0))) * (1 + 3 / (1 + np.exp(3.0))), 5.0,
                                           -4 * s * (1 - (1 - s)), 3 / (1 + np.exp(-3.0)), 0.0, s])


def test_oracle_gradient_is_the_slope():
    """Against central differences of the forward oracle, step 1e-5: its error is 1e-10 of third derivatives below 1."""
    rng = np.random.default_rng(5)
    g, u, dh = (rng.standard_normal((4, 50)) * 3 for _ in range(3))
    d, _ = f8.gradient(dh, g, 0, u, 0)
    h = 1e-5
    for i, slope in ((0, (f8.gated(g + h, 0, u, 0)[0] - f8.gated(g - h, 0, u, 0)[0]) / (2 * h)),
                     (1, (f8.gated(g, 0, u + h, 0)[0] - f8.gated(g, 0, u - h, 0)[0]) / (2 * h))):
        assert np.allclose(d[:, 50 * i:50 * i + 50], dh * slope, rtol=1e-7, atol=1e-8)


# ---------------------------------------------------------------- the bounds, against fp32 arithmetic

F = np.float32


def fp32_product(a, sa, w, sw, drop=False):
    """The steps of include/q4f8.h in fp32; with drop, the products of eight aligned to the largest."""
    x, y = f8.decode(a), f8.decode(w)
    acc = np.zeros((a.shape[0], w.shape[0]), dtype=F)
    for b in range(f8.blocks(a.shape[1])):
        total = np.zeros_like(acc)
        for k in range(128 * b, min(128 * b + 128, a.shape[1]), 8):
            p = x[:, None, k:k + 8] * y[None, :, k:k + 8]
            if drop:
                _, e = np.frexp(np.abs(x[:, None, k:k + 8]))
                _, f = np.frexp(np.abs(y[None, :, k:k + 8]))
                top = np.where(p != 0, e + f - 2, -99).max(2, keepdims=True)
                step = 2.0 ** (top - 13.0)
                p = np.trunc(p / step) * step
            total = (total + p.sum(2)).astype(F)
        scale = (sa[:, b, None] * np.repeat(sw[:, b], 128)[None, :w.shape[0]]).astype(F)
        acc = (acc.astype(np.float64) + total.astype(np.float64) * scale).astype(F)
    return acc


def inside(got, want, bound, t="f32"):
    return np.abs(got.astype(np.float64) - want) <= f8.tolerance(want, bound, t)


@pytest.mark.parametrize("drop", [False, True])
def test_bounds_hold_the_products_steps(drop):
    a, sa, w, sw = small_problem(3, 7, 150, 912)
    want, bound = f8.product(a, sa, w, sw, not drop)
    got = fp32_product(a, sa, w, sw, drop)
    assert inside(got, want, bound).all()
    if drop:
        assert not inside(got, *f8.product(a, sa, w, sw, True)).all()


def fp32_gradient(dh, g, u):
    e = np.exp2(-np.abs(g) * F(np.log2(np.e)))
    big = F(1) / (F(1) + e)
    small = e * big
    s, r = np.where(g < 0, small, big), np.where(g < 0, big, small)
    near = dh * (u * (s * (F(1) + g * r))), dh * (g * s)
    half = np.exp2(g * F(np.log2(np.e) / 2))
    far = (F(1) + g) * half * u * (half * dh), g * half * (half * dh)
    return np.concatenate([np.where(g < -87, f, n) for f, n in zip(far, near)], 1)


@pytest.mark.parametrize("size", [1, 40, 170])
def test_bounds_hold_the_gates_steps_and_refuse_mistakes(size):
    rng = np.random.default_rng(size)
    g, u, dh = ((rng.standard_normal((20, 60)) * s).astype(F) for s in (size, 2, 0.01))
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        got = fp32_gradient(dh, g, u)
    want, bound = f8.gradient(*(v.astype(np.float64) for v in (dh, g)), 0, u.astype(np.float64), 0)
    assert inside(got, want, bound).all()
    assert np.max(np.abs(got - want) / bound) > 0.02
    if size > 1:
        return
    s = 1 / (1 + np.exp(-g.astype(np.float64)))
    for name, d in {"no slope of the gate": dh * u * s, "1 + g s": dh * u * s * (1 + g * s),
                    "gradients exchanged": dh * g * s, "s in fp16": dh * u * (s.astype(np.float16) * (1 + g * (1 - s)))}.items():
        assert inside(d.astype(F), want[:, :60], bound[:, :60]).mean() < 0.1, name
    y, bound = f8.gated(g.astype(np.float64), 0, u.astype(np.float64), 0)
    with np.errstate(over="ignore"):
        silu = g * (F(1) / (F(1) + np.exp2(-g * F(np.log2(np.e)))))
    assert inside(silu * u, y, bound).all()
    assert inside(silu.astype(np.float16).astype(F) * u, y, bound).mean() < 0.1


def test_bounds_refuse_mistakes_of_products():
    """At small K, in most places: exact products first, then the 8-bit unit's."""
    a, sa, w, sw = small_problem(4, 9, 200, 400)
    p = fp32_product(a, sa, w, sw)
    want, bound = f8.product(a, sa, w, sw, True)
    cut_a = a.copy()
    cut_a[:, -1] = 0
    moved = np.roll(sa, 1, 1)
    for name, y in {"P in fp16": p.astype(np.float16), "one product less": fp32_product(cut_a, sa, w, sw),
                    "the next block's scale": fp32_product(a, moved, w, sw),
                    "the next row's scale": fp32_product(a, np.roll(sa, 1, 0), w, sw),
                    "the other block of rows": fp32_product(a, sa, w, sw[::-1].copy()),
                    "scales in fp16": fp32_product(a, sa.astype(np.float16).astype(F), w, sw)}.items():
        assert inside(y.astype(F), want, bound).mean() < 0.5, name
    want, bound = f8.product(a, sa, w, sw, False)
    for name, y in {"the next block's scale": fp32_product(a, moved, w, sw),
                    "the other block of rows": fp32_product(a, sa, w, sw[::-1].copy())}.items():
        assert inside(y.astype(F), want, bound, "bf16").mean() < 0.5, name
