"""How gemm_f8's choice among its kernels compares with the best of them, and its constants fitted anew.

csrc/gemm_f8.hip chooses a kernel by estimated times, whose constants (kCosts16 for 16-bit outputs, kCosts32 for
float32) were fitted to measured calls.  After a change to a kernel:

  python perf/fit_gemm_f8.py build LIB         the library with a switch that forces a kernel (needs hipcc, no GPU)
  python perf/fit_gemm_f8.py sweep LIB FILE    times every kernel at random sizes, a JSON line a call appended (GPU)
  python perf/fit_gemm_f8.py fit FILE ...      how far the constants as they are lie behind the best kernel of each
                                               call, the same for constants fitted anew (--only: some of them), and
                                               those as source

A line is [[M, N, K, matrices, type], {kernel: us, .., "chosen": us}].  `choose` here is that of gemm_f8.hip over
arrays of calls; tests/test_f8.py holds the two to each other.
"""

import argparse
import ctypes
import json
import math
import os
import random
import re
import subprocess
import sys
import time

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
SOURCE = os.path.join(ROOT, "memory_bandwidth_amd", "csrc", "gemm_f8.hip")

CUS = 256
KERNELS = ("few8", "few16", "few32", "few32x32", "few64", "tile64", "tile128", "tile_wide", "tile256", "tile_deep")
# Rows, columns and most wavefronts of a few-rows kernel; rows of y and of weights of a tile.
FEW = {"few8": (8, 16, 8), "few16": (16, 16, 8), "few32": (32, 16, 8), "few32x32": (32, 32, 8), "few64": (64, 32, 4)}
TILES = {"tile64": (64, 128), "tile128": (128, 128), "tile_wide": (128, 256), "tile256": (256, 256),
         "tile_deep": (64, 64)}
# In the order in which the source tries them: of equal times the first one's.
ORDER = ("few8", "few16", "few32", "few32x32", "few64", "tile_deep", "tile64", "tile128", "tile_wide", "tile256")
# The constants of a table in the order of struct Costs.
FIELDS = (("few8", 5), ("few16", 5), ("few32", 5), ("few32x32", 5), ("few64", 5), ("mb", 1), ("again", 1), ("off", 1),
          ("deep", 2), ("stretch", 1), ("tile64", 2), ("tile128", 2), ("tile128_many", 2), ("wide", 2), ("tile256", 2))
NEVER = 1e30


def constants(t: str) -> dict:
    """The table of a type (bf16, f32) in the source."""
    name = "kCosts32" if t == "f32" else "kCosts16"
    body = re.search(r"constexpr Costs %s = (\{.*?\});" % name, open(SOURCE).read(), re.S).group(1)
    values = [float(v) for v in re.findall(r"-?\d+\.\d*", body)]
    assert len(values) == sum(n for _, n in FIELDS)
    out = {}
    for field, n in FIELDS:
        out[field], values = values[:n], values[n:]
    return out


def as_source(t: str, c: dict) -> str:
    parts = [("{%s}" if n > 1 else "%s") % ", ".join("%.3f" % v for v in c[f]) for f, n in FIELDS]
    return "constexpr Costs %s = {%s};" % ("kCosts32" if t == "f32" else "kCosts16", ", ".join(parts))


def up(a, b):
    return -(-a // b)


class Calls:
    """Sizes of calls of one type, as arrays, and what the estimates need of them."""

    def __init__(self, t: str, shapes):
        self.t = t
        self.M, self.N, self.K, self.mats = (np.array([s[i] for s in shapes], dtype=np.int64) for i in range(4))
        self.steps, self.mb = up(self.K, 128), self.mats * self.N * self.K * 1e-6
        self.few = {k: self._split(*FEW[k]) for k in FEW}
        self.tiles = {k: up(self.M, bm) * up(self.N, bw // self.mats) for k, (bm, bw) in TILES.items()}

    def _split(self, bm, cols, most):
        """Row tiles, log2 of the wavefronts on a strip, of a workgroup, wavefronts of a CU and a wavefront's blocks."""
        tiles, strips = up(self.M, bm), up(self.N, cols)
        log2 = np.zeros_like(tiles)
        for _ in range(3):
            more = (2 << log2 <= most) & (self.steps >> log2 > 1) & (tiles * strips << log2 < 1536)
            log2 += more
        eights = tiles * up(strips, 8 >> log2) if most == 8 else 0 * tiles
        waves = np.where((log2 < 3) & ((eights < CUS // 2) | (eights > CUS)), 4, most)
        groups = tiles * up(strips, waves >> log2)
        return tiles, log2, waves, (up(groups, CUS) * waves).astype(float), up(self.steps, 1 << log2)

    def costs(self, c: dict) -> np.ndarray:
        """Estimated times [call, kernel of ORDER]."""
        s, two, out = self.steps, self.mats == 2, {}
        for k in FEW:
            start, block, shared, shared_two, first = c[k]
            tiles, _, _, waves, blocks = self.few[k]
            each = np.maximum(block, np.where(two, shared_two, shared) * waves)
            read = c["mb"][0] * self.mb * (1 + c["again"][0] * (tiles - 1)) - c["off"][0]
            out[k] = np.maximum(start + each * (first + blocks), read)
        for k in ("few32x32", "few64"):
            out[k] = np.where(two, NEVER, out[k])
        at = lambda f: c[f][0] + c[f][1] * s                                                 # noqa: E731
        t = self.tiles
        out["tile_deep"] = np.where(t["tile_deep"] <= CUS, at("deep"), NEVER)
        out["tile64"] = np.maximum(1, t["tile64"] / CUS * c["stretch"][0]) * at("tile64")
        out["tile128"] = np.where(t["tile128"] <= CUS, at("tile128"), t["tile128"] / CUS * at("tile128_many"))
        out["tile_wide"] = up(t["tile_wide"], CUS) * at("wide")
        left = t["tile256"] % CUS
        divided = np.where(left > 64, at("wide"), np.where(left > 0, at("tile128"), 0.0))
        whole = (t["tile256"] < CUS) | (left > 128)
        out["tile256"] = np.where(whole, up(t["tile256"], CUS) * at("tile256"), t["tile256"] // CUS * at("tile256") + divided)
        if self.t == "f32":
            out["tile256"] = np.full(len(s), NEVER)
        return np.stack([out[k] for k in ORDER], 1)

    def choose(self, c: dict) -> list:
        best = [ORDER[i] for i in self.costs(c).argmin(1)]
        small = lambda m: "few16" if m <= 16 else "few32"                                     # noqa: E731
        return ["few8" if m <= 8 else small(m) if k < 128 else b for m, k, b in zip(self.M, self.K, best)]

    def tile(self, i: int, kernel: str) -> tuple:
        """Rows and columns of y that a workgroup of a kernel makes at a time, for call i."""
        if kernel in FEW:
            bm, cols, _ = FEW[kernel]
            _, log2, waves, _, _ = self.few[kernel]
            return bm, int(waves[i] >> log2[i]) * cols
        bm, bw = TILES[kernel]
        return bm, int(bw // self.mats[i])


# ---------------------------------------------------------------- build

def build(out: str) -> None:
    """The library from its sources, with gemm_f8_forced in gemm_f8.hip: below 0 the choice is as it is."""
    from memory_bandwidth_amd import build as b
    folder = os.path.splitext(os.path.abspath(out))[0] + "_objects"
    os.makedirs(folder, exist_ok=True)
    text = open(SOURCE).read()
    for old, new in (("namespace {\n", 'extern "C" { int gemm_f8_forced = -1; }\n\nnamespace {\n'),
                     ("Kernel choose(const Args &p, int mats) {\n", "Kernel choose(const Args &p, int mats) {\n"
                      "    if (gemm_f8_forced >= 0) return (Kernel)gemm_f8_forced;\n")):
        assert text.count(old) == 1
        text = text.replace(old, new)
    forced = os.path.join(folder, "gemm_f8.hip")
    with open(forced, "w") as f:
        f.write(text)
    objects, running = [], []
    for s in b.SOURCES:
        src = forced if s == "gemm_f8.hip" else os.path.join(b.CSRC, s)
        objects.append(os.path.join(folder, os.path.splitext(s)[0] + ".o"))
        running.append(subprocess.Popen([b.hipcc(), *b.HIP_FLAGS, "-c", src, "-o", objects[-1]]))
    if any([p.wait() for p in running]):
        raise SystemExit("hipcc failed")
    subprocess.run([b.hipcc(), f"--offload-arch={b.ARCH}", "-shared", "-fPIC", "-o", out, *objects], check=True)


# ---------------------------------------------------------------- sweep

def draw(rng: random.Random) -> list:
    """Sizes of a call: 9 to 8192 rows, N 64 to 14336, K 128 to 14336, at most 300 GFLOP."""
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))        # noqa: E731
    while True:
        M, N, K, mats = log(9, 8192), log(64, 14336), 16 * log(8, 896), rng.choice([1, 1, 2])
        if 2e-9 * M * N * K * mats <= 300:
            return [M, N, K, mats, rng.choice(["bf16", "f32"])]


def candidates(M: int, N: int, K: int, mats: int, t: str) -> list:
    """Kernels that a call can take and that are not hopeless: few rows a tile are read again for every tile."""
    assert M > 8 and K >= 128
    out = []
    for k in KERNELS:
        if (k == "tile256" and (t == "f32" or M < 100)) or (k in ("few32x32", "few64") and mats == 2):
            continue
        if k in FEW and M > 1300 and M * N > 1_500_000:
            continue
        if k in TILES and M <= 16:
            continue
        out.append(k)
    return out


def sweep(lib_path: str, file: str, calls: int, seed: int) -> None:
    import torch

    import memory_bandwidth_amd as q4
    q4.LIB_PATH = os.path.abspath(lib_path)
    forced = ctypes.c_int.in_dll(q4.lib(), "gemm_f8_forced")
    types = {"bf16": torch.bfloat16, "f32": torch.float32}
    rng = random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def codes(*shape):
        return (torch.randn(*shape, device="cuda", generator=g) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)

    def scales(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    for _ in range(calls):
        M, N, K, mats, t = shape = draw(rng)
        # Up to six sets of operands in turn, so that they come from memory as a model's do.
        sets = max(1, min(6, int(1.5e9 // ((M + mats * N) * K + 4 * M * N))))
        KB, dtype = up(K, 128), types[t]
        data = [(codes(M, K), scales(KB, M).t(), [(codes(N, K), scales(up(N, 128), KB)) for _ in range(mats)])
                for _ in range(sets)]
        y = torch.empty(M, N, dtype=dtype, device="cuda")

        def run(d):
            a, sa, w = d
            if mats == 1:
                q4.gemm_f8(a, sa, *w[0], dtype=dtype, out=y)
            else:
                q4.gemm_f8_swiglu(a, sa, *w, dtype=dtype, out=y)

        def timed() -> float:
            """us of a call, the least of three replays of a graph of some 3 ms."""
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            run(data[0])
            torch.cuda.synchronize()
            start.record()
            for d in data:
                run(d)
            end.record()
            end.synchronize()
            n = max(sets, min(60, int(3.0 / max(start.elapsed_time(end) / sets, 1e-3))))
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                for i in range(n):
                    run(data[i % sets])
            took = []
            for _ in range(4):
                start.record()
                graph.replay()
                end.record()
                end.synchronize()
                took.append(start.elapsed_time(end) / n * 1e3)
            return round(min(took[1:]), 2)

        row = {}
        for k in candidates(*shape):
            forced.value = KERNELS.index(k)
            row[k] = timed()
        forced.value = -1
        row["chosen"] = timed()
        line = json.dumps([shape, row])
        print(line, flush=True)
        with open(file, "a") as f:
            f.write(line + "\n")


# ---------------------------------------------------------------- fit

class Measured(Calls):
    def __init__(self, t: str, rows: list):
        super().__init__(t, [r[0] for r in rows])
        self.times = np.array([[r[1].get(k, np.nan) for k in ORDER] for r in rows])
        self.behind = self.times / np.nanmin(self.times, 1, keepdims=True)
        self.behind[np.isnan(self.behind)] = 2.5                      # not timed: hopeless

    def behind_best(self, c: dict) -> np.ndarray:
        return self.behind[np.arange(len(self.M)), self.costs(c).argmin(1)]

    def score(self, c: dict) -> float:
        """What the chosen kernel lies behind the best, more so beyond 12%, and how far the estimates of those near are off."""
        costs = self.costs(c)
        r = self.behind[np.arange(len(self.M)), costs.argmin(1)]
        near = (self.behind < 1.8) & ~np.isnan(self.times) & (costs < NEVER)
        off = np.abs(np.log(np.maximum(costs, 0.1) / np.where(near, self.times, 1)))[near]
        return float(np.log(r).mean() + 2 * np.maximum(0, r - 1.12).mean() + 0.1 * off.mean())


def report(what: str, r: np.ndarray) -> None:
    print(f"  {what}: {100 * (r.mean() - 1):.1f}% behind the best on average, {100 * (np.percentile(r, 95) - 1):.0f}% or "
          f"more in one of twenty, {100 * (r.max() - 1):.0f}% at most", flush=True)


def fit(files: list, only: str, seconds: float, seed: int) -> None:
    rows = [json.loads(line) for f in files for line in open(f)]
    rng = np.random.default_rng(seed)
    for t in ("bf16", "f32"):
        of = [r for r in rows if r[0][4] == t]
        if len(of) < 8:
            continue
        fitted, held = Measured(t, of[: len(of) * 3 // 4]), Measured(t, of[len(of) * 3 // 4:])
        best = constants(t)
        print(f"{t}: {len(of)} calls, of which the last {len(held.M)} are not fitted to")
        report("as they are, all", Measured(t, of).behind_best(best))
        report("as they are, those not fitted to", held.behind_best(best))
        # Few constants at a time, kept where the score falls.
        places = [(f, i) for f, n in FIELDS for i in range(n) if not only or f in only.split(",")]
        score, end = fitted.score(best), time.time() + seconds
        while time.time() < end:
            c = {f: list(v) for f, v in best.items()}
            for _ in range(rng.integers(1, 4)):
                f, i = places[rng.integers(len(places))]
                c[f][i] = c[f][i] * math.exp(rng.normal() * 0.2) + rng.normal() * 0.02
            new = fitted.score(c)
            if new < score - 1e-7:
                score, best = new, c
        report("fitted anew, those not fitted to", held.behind_best(best))
        print(as_source(t, best), flush=True)


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    sub = p.add_subparsers(dest="do", required=True)
    b = sub.add_parser("build")
    b.add_argument("lib")
    s = sub.add_parser("sweep")
    s.add_argument("lib")
    s.add_argument("file")
    s.add_argument("--calls", type=int, default=300)
    s.add_argument("--seed", type=int, default=1)
    f = sub.add_parser("fit")
    f.add_argument("files", nargs="+")
    f.add_argument("--only", default="", help="fields of struct Costs to fit, by commas; the others stay")
    f.add_argument("--seconds", type=float, default=60)
    f.add_argument("--seed", type=int, default=1)
    a = p.parse_args()
    if a.do == "build":
        build(a.lib)
    elif a.do == "sweep":
        sweep(a.lib, a.file, a.calls, a.seed)
    else:
        fit(a.files, a.only, a.seconds, a.seed)


if __name__ == "__main__":
    main()
