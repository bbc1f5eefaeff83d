"""The operators of 8-bit floating point, as cases to be timed and compared.

`own` chooses what `run` does: False computes an operator from elementary
torch operations, True calls memory_bandwidth_amd.  `exact` gives the results
in 64 bits, from the definitions.  Codes are e4m3; blocks are 128 long, the
last of a row as long as what is left; b(k) is the block of k:

  rows      s[m, b] = max(fp32(max over the block of |x[m, k]| / 448), 2^-126)
            c[m, k] = the e4m3 value nearest to x[m, k] / s[m, b(k)], ties to even
  blocks    the same with one s for each 128 x 128 block of x [R, C]; codes as x
            lies, transposed ([C, R up to a multiple of 16], zeros behind), or both
  gemm      y[m, n] = sum_k a[m, k] sa[m, b(k)] w[n, k] sw[b(n), b(k)] (+ bias[n]),
            or with sa[b(m), b(k)]
  swiglu    y = silu(g) u, silu(v) = v / (1 + e^-v), with g and u products as
            above of the same rows with two matrices
  backward  the gradients of sum(dh * silu(g) u) for g and u, side by side:
            [dh u s (1 + g (1 - s)), dh g s], s = 1 / (1 + e^-g)
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
F8 = torch.float8_e4m3fn


def listed():
    return [
        # One token's activations before a projection: latency.
        {"name": "rows one token", "op": "rows", "M": 1, "K": 4096, "t": "bf16"},
        # A prompt's activations before the down projection: a stream.
        {"name": "rows prompt", "op": "rows", "M": 4099, "K": 14336, "t": "f32"},
        # A projection's weights in a training step: codes for the forward and for the backward product.
        {"name": "blocks weights", "op": "blocks", "R": 14336, "C": 4096, "t": "bf16", "layout": "both"},
        # A small model's activations for its weight gradient, an odd number of tokens.
        {"name": "blocks activations", "op": "blocks", "R": 1999, "C": 896, "t": "f16", "layout": "columns"},
        # One token through the up projection: the weights are streamed once.
        {"name": "gemm one token", "op": "gemm", "M": 1, "N": 14336, "K": 4096, "t": "bf16", "bias": False,
         "a": "rows"},
        # A short prompt on a small model, ragged, with a bias.
        {"name": "gemm short prompt", "op": "gemm", "M": 333, "N": 4864, "K": 896, "t": "f16", "bias": True,
         "a": "rows"},
        # A long prompt, up projection: bound by the matrix cores.
        {"name": "gemm long prompt", "op": "gemm", "M": 8192, "N": 14336, "K": 4096, "t": "bf16", "bias": False,
         "a": "rows"},
        # The weight gradient of a small model's gate and up projections over 4099 tokens.
        {"name": "gemm weight gradient", "op": "gemm", "M": 9728, "N": 896, "K": 4112, "t": "f32", "bias": False,
         "a": "blocks"},
        # Four sequences decoding, gate and up projections.
        {"name": "swiglu 4 sequences", "op": "swiglu", "M": 4, "N": 14336, "K": 4096, "t": "f32"},
        # A prompt of odd length, gate and up projections.
        {"name": "swiglu prompt", "op": "swiglu", "M": 1999, "N": 14336, "K": 4096, "t": "bf16"},
        # A short text in a small model's training step.
        {"name": "backward short", "op": "backward", "M": 333, "N": 4864, "K": 896, "t": "f16"},
        # A longer one in a large model's.
        {"name": "backward prompt", "op": "backward", "M": 1999, "N": 14336, "K": 4096, "t": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "blocks", "gemm", "gemm", "swiglu", "backward"])
    t = rng.choice(["f32", "f16", "bf16"])
    k = 16 * _log(rng, 16, 896)
    if op == "rows":
        return {"op": op, "M": min(_log(rng, 1, 8192), 58_000_000 // k), "K": k, "t": t}
    if op == "blocks":
        return {"op": op, "R": min(_log(rng, 16, 14336), 58_000_000 // k), "C": k, "t": t,
                "layout": rng.choice(["rows", "columns", "both"])}
    n = _log(rng, 64, 14336)
    mats = 1 if op == "gemm" else 2
    rows = min(_log(rng, 1, 8192), 400_000_000_000 // (mats * n * k))
    case = {"op": op, "M": rows, "N": n, "K": k, "t": t}
    if op == "gemm":
        case["bias"] = rng.random() < 0.5
        case["a"] = rng.choice(["rows", "rows", "blocks"])
    return case


def _up(n, to):
    return -(-n // to)


def _activations(g, rows, k):
    """Activations of a layer's input: normal, a few channels much larger than the others."""
    x = torch.randn(rows, k, generator=g, device="cuda")
    big = torch.rand(k, generator=g, device="cuda") < 0.01
    return x * torch.where(big, 8.0, 1.0)


def _largest(x, rows):
    """The largest magnitude of each block of `rows` x 128."""
    r, c = x.shape
    padded = torch.zeros(_up(r, rows) * rows, _up(c, 128) * 128, device=x.device, dtype=x.dtype)
    padded[:r, :c] = x.abs()
    return padded.reshape(_up(r, rows), rows, _up(c, 128), 128).amax((1, 3))


def _spread(s, rows, r, c):
    """A scale for each value of [r, c] from those of its blocks of `rows` x 128."""
    s = s.repeat_interleave(128, 1)[:, :c]
    return s if rows == 1 else s.repeat_interleave(rows, 0)[:r]


def _held(x, rows):
    """x as a program holds it: codes, and scales of blocks of `rows` x 128."""
    s = (_largest(x, rows) / 448).clamp_min(2.0**-126)
    return (x / _spread(s, rows, *x.shape)).clamp(-448, 448).to(F8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, t = case["op"], DTYPES[case["t"]]
    state = {"op": op, "t": t}
    if op == "rows":
        state["x"] = _activations(g, case["M"], case["K"]).to(t)
        return state
    if op == "blocks":
        state["x"], state["layout"] = _activations(g, case["R"], case["C"]).to(t), case["layout"]
        return state
    m, n, k = case["M"], case["N"], case["K"]
    if case.get("a") == "blocks":
        state["a"], state["sa"] = _held(_activations(g, m, k), 128)
    else:
        state["a"], sa = _held(_activations(g, m, k), 1)
        state["sa"] = sa.t().contiguous().t()         # as quant_f8 lays them out: rows run fastest
    for name in ("w",) if op == "gemm" else ("wg", "wu"):
        w = torch.randn(n, k, generator=g, device="cuda").mul_(k**-0.5)
        state[name], state["s" + name] = _held(w, 128)
    if op == "gemm":
        state["bias"] = torch.randn(n, generator=g, device="cuda") if case["bias"] else None
    if op == "backward":
        state["dh"] = (torch.randn(m, n, generator=g, device="cuda") * 0.01).to(t)
    return state


def _codes(x, s):
    """The e4m3 values nearest to x / s.  The quotients are taken in 64 bits, where none that is no tie becomes one."""
    q = x.double() / s.double()
    step = torch.exp2((torch.frexp(q).exponent - 1).clamp_min(-6).double() - 3)
    return (torch.round(q / step) * step).clamp(-448, 448).to(F8)


def _product(s, name):
    a, w = s["a"], s[name]
    rows = 1 if s["sa"].shape[0] == a.shape[0] else 128
    left = a.float() * _spread(s["sa"], rows, *a.shape)
    right = w.float() * _spread(s["s" + name], 128, *w.shape)
    return left @ right.t()


def _plain(s):
    op = s["op"]
    if op in ("rows", "blocks"):
        x, rows = s["x"], 1 if op == "rows" else 128
        scales = (_largest(x, rows).double() / 448).float().clamp_min(2.0**-126)
        codes = _codes(x, _spread(scales, rows, *x.shape))
        if op == "rows":
            return {"codes": codes, "scales": scales}
        out = {}
        if s["layout"] != "columns":
            out.update(codes=codes, scales=scales)
        if s["layout"] != "rows":
            r, c = x.shape
            turned = torch.zeros(c, _up(r, 16) * 16, device=x.device, dtype=F8)
            turned[:, :r] = codes.t()
            out.update(codes_t=turned, scales_t=scales.t().contiguous())
        return out
    if op == "gemm":
        y = _product(s, "w")
        return {"y": (y if s["bias"] is None else y + s["bias"]).to(s["t"])}
    g, u = _product(s, "wg"), _product(s, "wu")
    sig = 1 / (1 + torch.exp(-g))
    if op == "swiglu":
        return {"y": (g * sig * u).to(s["t"])}
    dh = s["dh"].float()
    return {"d": torch.cat([dh * u * (sig * (1 + g * (1 - sig))), dh * (g * sig)], 1).to(s["t"])}


def _called(s):
    import memory_bandwidth_amd as q4

    op = s["op"]
    if op == "rows":
        codes, scales = q4.quant_f8(s["x"])
        return {"codes": codes, "scales": scales}
    if op == "blocks":
        got = q4.quant_f8_block(s["x"], layout=s["layout"])
        names = {"rows": ("codes", "scales"), "columns": ("codes_t", "scales_t"),
                 "both": ("codes", "scales", "codes_t", "scales_t")}[s["layout"]]
        return dict(zip(names, got))
    if op == "gemm":
        return {"y": q4.gemm_f8(s["a"], s["sa"], s["w"], s["sw"], bias=s["bias"], dtype=s["t"])}
    gate, up = (s["wg"], s["swg"]), (s["wu"], s["swu"])
    if op == "swiglu":
        return {"y": q4.gemm_f8_swiglu(s["a"], s["sa"], gate, up, dtype=s["t"])}
    return {"d": q4.gemm_f8_swiglu_backward(s["dh"], s["a"], s["sa"], gate, up, dtype=s["t"])}


def run(state):
    if own:
        return _called(state)
    return _plain(state)


def work(case):
    op, e = case["op"], SIZE[case["t"]]
    if op == "rows":
        m, k = case["M"], case["K"]
        return {"bytes": m * k * (e + 1) + 4 * m * _up(k, 128), "flops": 4 * m * k}
    if op == "blocks":
        r, c, layout = case["R"], case["C"], case["layout"]
        moved = r * c * e
        moved += r * c + 4 * _up(r, 128) * _up(c, 128) if layout != "columns" else 0
        moved += c * 16 * _up(r, 16) + 4 * _up(r, 128) * _up(c, 128) if layout != "rows" else 0
        return {"bytes": moved, "flops": 4 * r * c}
    m, n, k = case["M"], case["N"], case["K"]
    mats, kb = 1 if op == "gemm" else 2, _up(k, 128)
    moved = m * k + 4 * kb * (_up(m, 128) if case.get("a") == "blocks" else m)
    moved += mats * (n * k + 4 * _up(n, 128) * kb) + m * n * e
    moved += 4 * n if case.get("bias") else 0
    moved += 2 * m * n * e if op == "backward" else 0
    return {"bytes": moved, "flops": 2.0 * mats * m * n * k}


def _nearest(q):
    """Of all e4m3 values the one nearest to q (float64); of two, the one with the even code."""
    values = [c / 512 if c < 8 else (1 + c % 8 / 8) * 2.0 ** (c // 8 - 7) for c in range(127)]
    values = torch.tensor(values, dtype=torch.float64, device=q.device)
    middle = (values[1:] + values[:-1]) / 2
    out = torch.empty_like(q)
    for part, to in zip(q.reshape(-1).split(1 << 24), out.view(-1).split(1 << 24)):
        i = torch.searchsorted(middle, part.abs())
        tie = (i < 126) & (middle[i.clamp_max(125)] == part.abs()) & (i % 2 == 1)
        to.copy_(torch.copysign(values[i + tie.long()], part))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rows", "blocks"):
        x = s["x"].double()
        r, c = x.shape
        tall = 1 if op == "rows" else 128
        scale = torch.empty(_up(r, tall), _up(c, 128), dtype=torch.float64, device=x.device)
        q = torch.empty_like(x)
        for j in range(scale.shape[1]):
            cols = slice(128 * j, 128 * j + 128)
            most = x[:, cols].abs().max(1).values
            if tall == 128:
                most = torch.stack([part.max() for part in most.split(128)])
            scale[:, j] = most / 448
            used = scale[:, j].float().double().clamp_min(2.0**-126)
            q[:, cols] = x[:, cols] / used.repeat_interleave(tall)[:r, None]
        codes = _nearest(q)
        out = {}
        if op == "rows" or case["layout"] != "columns":
            out.update(codes=codes, scales=scale)
        if op == "blocks" and case["layout"] != "rows":
            out["codes_t"] = torch.nn.functional.pad(codes.t(), (0, -r % 16))
            out["scales_t"] = scale.t()
        return out
    m, n, k = case["M"], case["N"], case["K"]
    blocks = range(_up(k, 128))
    left = s["a"].double()
    for b in blocks:
        of = s["sa"][:, b].double()
        if case.get("a") == "blocks":
            of = of.repeat_interleave(128)[:m]
        left[:, 128 * b:128 * b + 128] *= of[:, None]
    sums = []
    for name in ("w",) if op == "gemm" else ("wg", "wu"):
        y = torch.empty(m, n, dtype=torch.float64, device="cuda")
        for lo in range(0, n, 128):
            w = s[name][lo:lo + 128].double()
            for b in blocks:
                w[:, 128 * b:128 * b + 128] *= s["s" + name][lo // 128, b].double()
            y[:, lo:lo + 128] = torch.mm(left, w.t())
        sums.append(y)
    if op == "gemm":
        y = sums[0]
        return {"y": y if s["bias"] is None else y + s["bias"].double()}
    g, u = sums
    if op == "swiglu":
        return {"y": g * torch.sigmoid(g) * u}
    dh, sig = s["dh"].double(), torch.sigmoid(g)
    return {"d": torch.cat([dh * u * sig * (1 + g * torch.sigmoid(-g)), dh * g * sig], 1)}
