"""The 8-bit integer operators, as cases to be timed and compared.

`own` chooses what `run` does: False computes an operator from elementary
torch operations, True calls memory_bandwidth_amd.  `exact` gives the results
in 64 bits, from the definitions:

  quant           s[m] = max(fp32(max_k |x[m, k]| / 127), 2^-126)
                  c[m, k] = the integer nearest to x[m, k] / s[m], ties to even
  gemm            y[m, n] = sa[m] sw[n] sum_k a[m, k] w[n, k] (+ bias[n])
  swiglu          y = silu(g) u, silu(v) = v / (1 + e^-v), with g and u products
                  as above of the same rows with two matrices
  grouped         the gemm of rows offsets[e] .. offsets[e+1] with matrix e
  grouped_swiglu  the swiglu of rows offsets[e] .. offsets[e+1] with matrices e
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # One token's activations before a projection: latency.
        {"name": "quant one token", "op": "quant", "M": 1, "K": 4096, "t": "bf16"},
        # A prompt's activations before the down projection: a stream.
        {"name": "quant prompt", "op": "quant", "M": 4099, "K": 14336, "t": "f32"},
        # One token through the up projection: the weights are streamed once.
        {"name": "gemm one token", "op": "gemm", "M": 1, "N": 14336, "K": 4096, "t": "bf16", "bias": False},
        # A batch of sequences decoding, down projection.
        {"name": "gemm 24 sequences", "op": "gemm", "M": 24, "N": 4096, "K": 14336, "t": "f32", "bias": False},
        # A short prompt on a small model, ragged, with a bias.
        {"name": "gemm short prompt", "op": "gemm", "M": 333, "N": 4864, "K": 896, "t": "f16", "bias": True},
        # A long prompt, up projection: bound by the matrix cores.
        {"name": "gemm long prompt", "op": "gemm", "M": 8192, "N": 14336, "K": 4096, "t": "bf16", "bias": False},
        # Four sequences decoding, gate and up projections.
        {"name": "swiglu 4 sequences", "op": "swiglu", "M": 4, "N": 14336, "K": 4096, "t": "f32"},
        # A prompt of odd length, gate and up projections.
        {"name": "swiglu prompt", "op": "swiglu", "M": 1999, "N": 14336, "K": 4096, "t": "bf16"},
        # Eight sequences decoding with two experts each, down projection.
        {"name": "grouped 8 sequences", "op": "grouped", "T": 16, "E": 8, "N": 4096, "K": 14336, "t": "bf16"},
        # A prompt over eight experts, down projection.
        {"name": "grouped prompt", "op": "grouped", "T": 8190, "E": 8, "N": 4096, "K": 14336, "t": "bf16"},
        # A decoding batch over many small experts, gate and up projections.
        {"name": "grouped swiglu batch", "op": "grouped_swiglu", "T": 96, "E": 64, "N": 2816, "K": 1024, "t": "f16"},
        # A prompt over many small experts, gate and up projections.
        {"name": "grouped swiglu prompt", "op": "grouped_swiglu", "T": 8000, "E": 64, "N": 2816, "K": 1024, "t": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "swiglu", "grouped", "grouped_swiglu"])
    t = rng.choice(["f32", "f16", "bf16"])
    k = 16 * _log(rng, 16, 896)
    if op == "quant":
        return {"op": op, "M": min(_log(rng, 1, 8192), 58_000_000 // k), "K": k, "t": t}
    n = _log(rng, 64, 14336)
    rows = min(_log(rng, 1, 8192), 200_000_000_000 // (n * k))      # no larger than the largest listed
    if op in ("gemm", "swiglu"):
        case = {"op": op, "M": rows, "N": n, "K": k, "t": t}
        if op == "gemm":
            case["bias"] = rng.random() < 0.5
        return case
    e = _log(rng, 2, 64)
    k = min(k, max(256, 250_000_000 // (e * n) // 16 * 16))
    return {"op": op, "T": rows, "E": e, "N": n, "K": k, "t": t}


def _rows(case):
    return case["T"] if "T" in case else case["M"]


def _activations(g, rows, k):
    """Activations of a layer's input: normal, a few channels much larger than the others."""
    x = torch.randn(rows, k, generator=g, device="cuda")
    big = torch.rand(k, generator=g, device="cuda") < 0.01
    return x * torch.where(big, 8.0, 1.0)


def _token_codes(g, rows, k):
    x = _activations(g, rows, k)
    s = x.abs().amax(1) / 127
    return torch.round(x / s[:, None]).to(torch.int8), s


def _weights(g, *shape):
    """Normal weights that a per-channel quantiser left between -127 and 127, and their scales."""
    w = torch.empty(shape, dtype=torch.int8, device="cuda")
    for part in w.reshape(-1).split(1 << 26):
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(34).round_().clamp_(-127, 127))
    s = torch.rand(shape[:-1], generator=g, device="cuda") * 0.0004 + 0.0002
    return w, s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, rows, k = case["op"], _rows(case), case["K"]
    state = {"op": op, "t": DTYPES[case["t"]]}
    if op == "quant":
        state["x"] = _activations(g, rows, k).to(state["t"])
        return state
    state["a"], state["sa"] = _token_codes(g, rows, k)
    lead = (case["E"],) if "E" in case else ()
    if op in ("gemm", "grouped"):
        state["w"], state["sw"] = _weights(g, *lead, case["N"], k)
    else:
        state["wg"], state["sg"] = _weights(g, *lead, case["N"], k)
        state["wu"], state["su"] = _weights(g, *lead, case["N"], k)
    if op == "gemm":
        state["bias"] = torch.randn(case["N"], generator=g, device="cuda") if case["bias"] else None
    if lead:
        # A router's choice: some experts are liked far more than others.
        liked = torch.randn(case["E"], generator=g, device="cuda").mul(0.7).exp()
        chosen = torch.multinomial(liked, rows, replacement=True, generator=g)
        count = torch.bincount(chosen, minlength=case["E"])
        state["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
        state["most"] = int(count.max())
    return state


def _product(a, sa, w, sw):
    return (a.float() @ w.float().t()) * sa[:, None] * sw


def _grouped_product(a, sa, w, sw, offsets, most):
    """The groups' rows laid out as [E, most, K], one batched product, the rows taken back."""
    rows = torch.arange(a.shape[0], device=a.device)
    of = torch.searchsorted(offsets[1:].long(), rows, right=True)
    place = rows - offsets[of]
    laid = torch.zeros(w.shape[0], most, a.shape[1], device=a.device)
    laid[of, place] = a.float()
    y = torch.bmm(w.float(), laid.transpose(1, 2).contiguous())[of, :, place]
    return y * sa[:, None] * sw[of]


def _silu(v):
    return v / (1 + torch.exp(-v))


def _plain(s):
    op = s["op"]
    if op == "quant":
        x = s["x"]
        scales = (x.float().abs().amax(1).double() / 127).float().clamp_min(2.0**-126)
        codes = torch.round(x.double() / scales.double()[:, None]).to(torch.int8)
        return {"codes": codes, "scales": scales}
    if op == "gemm":
        y = _product(s["a"], s["sa"], s["w"], s["sw"])
        if s["bias"] is not None:
            y = y + s["bias"]
    elif op == "swiglu":
        y = _silu(_product(s["a"], s["sa"], s["wg"], s["sg"])) * _product(s["a"], s["sa"], s["wu"], s["su"])
    elif op == "grouped":
        y = _grouped_product(s["a"], s["sa"], s["w"], s["sw"], s["offsets"], s["most"])
    else:
        y = _silu(_grouped_product(s["a"], s["sa"], s["wg"], s["sg"], s["offsets"], s["most"]))
        y = y * _grouped_product(s["a"], s["sa"], s["wu"], s["su"], s["offsets"], s["most"])
    return {"y": y.to(s["t"])}


def _called(s):
    import memory_bandwidth_amd as q4

    op = s["op"]
    if op == "quant":
        codes, scales = q4.quant_i8(s["x"])
        return {"codes": codes, "scales": scales}
    if op == "gemm":
        y = q4.gemm_i8(s["a"], s["sa"], s["w"], s["sw"], bias=s["bias"], dtype=s["t"])
    elif op == "swiglu":
        y = q4.gemm_i8_swiglu(s["a"], s["sa"], (s["wg"], s["sg"]), (s["wu"], s["su"]), dtype=s["t"])
    elif op == "grouped":
        y = q4.gemm_i8_grouped(s["a"], s["sa"], s["w"], s["sw"], s["offsets"], dtype=s["t"])
    else:
        y = q4.gemm_i8_grouped_swiglu(s["a"], s["sa"], (s["wg"], s["sg"]), (s["wu"], s["su"]), s["offsets"],
                                      dtype=s["t"])
    return {"y": y}


def run(state):
    if own:
        return _called(state)
    return _plain(state)


def work(case):
    op, rows, k, e = case["op"], _rows(case), case["K"], SIZE[case["t"]]
    if op == "quant":
        return {"bytes": rows * k * (e + 1) + 4 * rows, "flops": 4 * rows * k}
    n, mats = case["N"], 2 if op in ("swiglu", "grouped_swiglu") else 1
    # With groups: the matrices of the experts that have rows, taken as drawn evenly.
    groups = case["E"] * (1 - (1 - 1 / case["E"]) ** rows) if "E" in case else 1
    moved = rows * k + 4 * rows + mats * groups * n * (k + 4) + rows * n * e
    moved += 4 * n if case.get("bias") else 0
    moved += 4 * (case["E"] + 1) if "E" in case else 0
    return {"bytes": moved, "flops": 2.0 * mats * rows * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        x = s["x"].to(torch.float64)
        scale = torch.maximum(x.max(1).values, -x.min(1).values) / 127
        used = scale.to(torch.float32).to(torch.float64).clamp_min(2.0**-126)
        below = torch.floor(x / used[:, None])
        part = x / used[:, None] - below
        up = (part > 0.5) | ((part == 0.5) & (below % 2 != 0))
        return {"codes": (below + up).to(torch.int8), "scales": scale}
    pairs = [("w", "sw")] if "w" in s else [("wg", "sg"), ("wu", "su")]
    limits = s["offsets"].tolist() if "offsets" in s else [0, _rows(case)]
    parts = []
    for e, (lo, hi) in enumerate(zip(limits[:-1], limits[1:])):
        if hi == lo:
            continue
        a = s["a"][lo:hi].to(torch.float64)
        sums = []
        for w, sw in pairs:
            wm, wv = (s[w][e], s[sw][e]) if "offsets" in s else (s[w], s[sw])
            wm = wm.to(torch.float64) * wv.to(torch.float64)[:, None]
            sums.append(torch.mm(a, wm.t()) * s["sa"][lo:hi].to(torch.float64)[:, None])
        parts.append(sums[0] if len(sums) == 1 else sums[0] * torch.sigmoid(sums[0]) * sums[1])
    y = torch.cat(parts)
    if s.get("bias") is not None:
        y = y + s["bias"].to(torch.float64)
    return {"y": y}
