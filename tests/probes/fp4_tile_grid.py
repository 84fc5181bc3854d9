"""Every tile of fp4_scaled_mm timed on a grid of layer shapes, next to the tile
the library picks by itself, and the costs of that choice fitted to the times.
Measurement infrastructure, not a test.

    python3 tests/probes/fp4_tile_grid.py > grid.jsonl        # on the GPU
    python3 tests/probes/fp4_tile_grid.py --fit grid.jsonl    # on any machine

Shapes: M 8 to 8192 against N 512 to 12288 and K 512 to 12288 (up to 4.6e11
products), random codes and scale bytes from seeded generators, two to eight
weights in turn so that they come from HBM where they are large, bf16 output,
no bias. A time is the median of three replays of a graph of ten calls. Tiles
that cannot be near the best are left out: small-M tiles beyond 256 rows, tiles
of 256 rows up to 64. One JSON line per shape.

--fit prints, for each tile, the constants of the cost model of
csrc/scaled_mm_fp4.hip that fit these times best (non-negative least squares of
relative errors), and what the choice costs over the best tile: the library's
(as recorded) and that of the fitted constants.
"""
from __future__ import annotations

import json
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, ROOT)

ROWS = (8, 16, 24, 32, 48, 64, 96, 128, 192, 256, 384, 512, 768, 1024, 1536, 2048, 4096, 8192)
CHANNELS = (512, 1024, 2560, 4096, 8192, 12288)
DEPTHS = (512, 1024, 2048, 4096, 8192, 12288)
MAX_WORK = 4.6e11
SMALL_ROWS = 256


def tile_dims(name: str):
    """(small-M, rows, columns) of a tile's name."""
    rows, columns = name.lstrip("s").split("/")[0].split("x")
    return name.startswith("s"), int(rows), int(columns)


def measure() -> int:
    import torch
    if not torch.cuda.is_available():
        print("no GPU", file=sys.stderr)
        return 2
    from w8a8_int8_dynamic_amd import ops
    tiles = {t: ops.fp4_tile_name(t) for t in range(ops.fp4_tile_count())}
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def codes(rows, k):
        scales = torch.randint(120, 127, (rows, -(-k // 512) * 16), dtype=torch.uint8, device="cuda", generator=g)
        return (torch.randint(0, 256, (rows, k // 2), dtype=torch.uint8, device="cuda", generator=g),
                scales[:, :k // 32])

    def time_us(call, sets):
        for i in range(2):
            call(i % sets)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in range(10):
                call(i % sets)
        graph.replay()
        times = []
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 100)
        return sorted(times)[1]

    for n in CHANNELS:
        for k in DEPTHS:
            sets = max(2, min(8, int(400e6 / (n * k * 17 / 32))))
            weights = [ops.fp4_prepack_weight(*codes(n, k)) for _ in range(sets)]
            for m in ROWS:
                if m * n * k > MAX_WORK:
                    continue
                x = [codes(m, k) for _ in range(sets)]
                out = [torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
                us = {}
                for t, name in tiles.items():
                    small, rows, _ = tile_dims(name)
                    if (small and m > SMALL_ROWS) or (rows >= 256 and m <= 64):
                        continue
                    us[name] = round(time_us(
                        lambda i: ops.fp4_scaled_mm(*x[i], *weights[i], n, out=out[i & 1], tile=t), sets), 2)
                print(json.dumps({"M": m, "N": n, "K": k, "auto": tiles[ops.fp4_tile_auto(m, n, k)], "us": us}),
                      flush=True)
    return 0


def terms(name: str, m: int, n: int, k: int):
    small, rows, columns = tile_dims(name)
    tiles, kblocks = -(-m // rows) * -(-n // columns), -(-k // 128)
    if small:
        return [1.0, tiles * kblocks, np.ceil(-(-k // 512) / 8.0)]              # fixed, work, chain
    rounds = np.ceil(tiles / 256)
    return [1.0, rounds * kblocks, rounds, n * k * 17 / 32e6, m * n * 2e-6]     # fixed, kblock, round, weight, out


def fit(path: str) -> int:
    from scipy.optimize import nnls
    grid = [json.loads(line) for line in open(path) if line.startswith("{")]
    names = list(dict.fromkeys(name for r in grid for name in r["us"]))
    cost = {}
    for name in names:
        at = [(terms(name, r["M"], r["N"], r["K"]), r["us"][name]) for r in grid if name in r["us"]]
        a = np.array([[v / us for v in t] for t, us in at])
        cost[name] = nnls(a, np.ones(len(a)))[0]
        print(name, " ".join(f"{v:.4g}" for v in cost[name]), f"rms error {np.sqrt(np.mean((a @ cost[name] - 1) ** 2)):.3f}")
    for what, choose in (("library", lambda r: r["auto"]),
                         ("fitted", lambda r: min(r["us"], key=lambda t: np.dot(terms(t, r["M"], r["N"], r["K"]), cost[t])))):
        over = np.array([r["us"][choose(r)] / min(r["us"].values()) for r in grid])
        print(f"{what} choice over the best of {len(grid)} shapes: mean {over.mean():.4f}, largest {over.max():.3f}, "
              f"over 1.05 on {(over > 1.05).sum()}")
    return 0


if __name__ == "__main__":
    sys.exit(fit(sys.argv[2]) if sys.argv[1:2] == ["--fit"] else measure())
