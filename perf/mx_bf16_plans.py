"""Times of every plan of the products of bf16 rows with MXFP4 weights, and the costs fitted to them.

A plan is a tile and the number of parts that its sums are cut into ("3x1": three
parts on tile 1; "+3x1": only the tiles behind the last whole round of the GPU).  The
library chooses one by the costs in ``csrc/w4_mx_bf16_gemm.hip``; the table of times
that they are fitted to is ``profiles/mx_bf16_plans.txt``.

  python perf/mx_bf16_plans.py sweep forward|gated|backward|many   # times, on an MI355X: one product a line
  python perf/mx_bf16_plans.py check profiles/mx_bf16_plans.txt    # the chosen plans against the best ones
  python perf/mx_bf16_plans.py fit profiles/mx_bf16_plans.txt      # costs for kCosts, and their error (scipy)

A line: kind (0 forward, 1 gated, 2 backward), rows, outputs, sum's other size as the
calls name them (m, n, k), and microseconds of each plan (median of five runs of graph
replays over two sets of operands in turn).
"""

import ctypes
import json
import math
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

FORWARD, GATED, BACKWARD = 0, 1, 2
#: rows, columns and groups of waves of the tiles; of each kind, whether a tile's blocks share a CU in pairs
TILES = ((256, 256, 1), (128, 256, 1), (128, 128, 1), (64, 128, 2), (32, 64, 4))
PAIRS = ((0, 0, 1, 1, 1), (0, 0, 1, 1, 1), (0, 0, 1, 0, 1))
CUS = 256


def geometry(kind, m, n, k, plan):
    """(tile, parts, steps of the sum, tiles, tiles that are whole)."""
    tail = plan[0] == "+"
    parts, tile = map(int, plan.lstrip("+").split("x"))
    rows, cols, _ = TILES[tile]
    out = k if kind == BACKWARD else n
    cols = cols // 2 if kind == GATED else cols
    tiles = -(-m // rows) * -(-out // cols)
    whole = tiles // CUS * CUS if tail else tiles if parts == 1 else 0
    return tile, parts, -(-(n if kind == BACKWARD else k) // 64), tiles, whole


def plans(kind, m, n, k, many):
    """The plans that are timed: many=True few parts, for products of many tiles."""
    few = [(1, 0), (2, 0), (3, 0), (1, 1), (2, 1), (1, 2), (1, 3)] if many else None
    for tile in range(5):
        if not many and tile not in ((3, 4) if m <= 32 else (2, 3, 4) if m <= 64 else range(4) if m >= 1500 else range(5)):
            continue
        for parts in (1, 2, 3, 4, 6, 8, 12, 16):
            if few is not None and (parts, tile) not in few:
                continue
            name = f"{parts}x{tile}"
            _, _, steps, tiles, _ = geometry(kind, m, n, k, name)
            if parts <= steps and (tiles <= 6000 if parts == 1 else tiles * parts <= (1024 if many else 600)):
                yield name
        for parts in (2, 3, 4):
            name = f"+{parts}x{tile}"
            _, _, _, tiles, whole = geometry(kind, m, n, k, name)
            if tiles > CUS and tiles > whole and not (kind == BACKWARD and tile == 4):
                yield name


def products(which):
    if which == "many":
        for kind in (FORWARD, GATED, BACKWARD):
            for m in (1024, 2048, 4096, 8192):
                for n, k in ((4096, 11008), (11008, 4096), (5632, 2048), (2048, 5632), (4096, 4096), (22016, 4096)):
                    if 2e10 <= m * n * k * (2 if kind == GATED else 1) <= 1e12:
                        yield kind, m, n, k
        return
    kind = ("forward", "gated", "backward").index(which)
    rows = (1, 16, 64, 130, 333, 700, 1500) if kind == BACKWARD else (24, 64, 130, 333, 700, 1500)
    outs = (304, 1000, 2728, 5504, 11008, 22016) if kind == BACKWARD else (300, 1000, 2730, 5500, 11008)
    for m in rows:
        for n in outs:
            for k in (512, 2080, 4096, 11008):
                if m * n * k * (2 if kind == GATED else 1) <= 4.5e10:
                    yield kind, m, n, k


# ------------------------------------------------------------------ times (GPU)
def library():
    import weight_only_bit_unpack_amd as w4
    i, j, p = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    w4._lib.w4_mx_bf16_kernel_of.argtypes = [i, j, j, j]
    w4._lib.w4_mx_bf16_product_on.argtypes = [i, i, i, j, j, p, p, p, j, p, p, i, p]
    return w4


def operands(w4, kind, m, n, k):
    import torch
    gen = torch.Generator("cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")
    sets = []
    for _ in range(2):
        wq, ws = w4.w4_mx_quantize(rand(2 * n if kind == GATED else n, k) * 0.02, w4.W4_MXFP4)
        x = rand(m, n if kind == BACKWARD else k).to(torch.bfloat16)
        y = torch.empty((m, k if kind == BACKWARD else n), dtype=torch.bfloat16, device="cuda")
        gu = torch.empty((m, 2 * n), dtype=torch.bfloat16, device="cuda") if kind == GATED and m > 64 else None
        sets.append((wq, ws, x, gu, y))
    return sets


def replays(call, sets, seconds):
    """us a call, of a captured row of twelve."""
    import torch
    side, reps = torch.cuda.Stream(), 12
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sets:
            call(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for i in range(reps):
            call(sets[i % len(sets)])
    graph.replay()
    torch.cuda.synchronize()
    start = time.perf_counter()
    graph.replay()
    torch.cuda.synchronize()
    rounds = max(1, min(50, int(seconds / (time.perf_counter() - start))))
    times = []
    for _ in range(5):
        a, b = torch.cuda.Event(True), torch.cuda.Event(True)
        a.record()
        for _ in range(rounds):
            graph.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3 / (rounds * reps))
    return sorted(times)[2]


def sweep(which):
    import torch
    w4 = library()
    for kind, m, n, k in products(which):
        sets, times = operands(w4, kind, m, n, k), {}
        for plan in plans(kind, m, n, k, which == "many"):
            tile, parts, *_ = geometry(kind, m, n, k, plan)
            kernel = 16 * parts + tile + (1024 if plan[0] == "+" else 0)

            def call(s):
                wq, ws, x, gu, y = s
                status = w4._lib.w4_mx_bf16_product_on(
                    kernel, kind, w4.W4_SILU, n, k, wq.data_ptr(), ws.data_ptr(), x.data_ptr(), m,
                    None if gu is None else gu.data_ptr(), y.data_ptr(), 1, torch.cuda.current_stream().cuda_stream)
                if status:
                    raise ValueError(f"{plan} does not fit: {status}")

            times[plan] = round(replays(call, sets, 0.006 if which == "many" else 0.003), 1)
        print(json.dumps([kind, m, n, k, times]), flush=True)


# ------------------------------------------------------------------ the chosen plans
def table(path):
    with open(path) as f:
        return [json.loads(line) for line in f if line.startswith("[")]


def chosen(w4, kind, m, n, k):
    code = w4._lib.w4_mx_bf16_kernel_of(kind, n, k, m)
    return ("+" if code >= 1024 else "") + f"{code % 1024 // 16}x{code % 16}"


def losses(rows):
    """(time of the chosen plan / the best one's, product, chosen, best) of each product
    whose chosen plan was timed (few rows forward have a kernel of their own)."""
    w4, out = library(), []
    for kind, m, n, k, times in rows:
        if kind != BACKWARD and m <= 16:
            continue
        own = chosen(w4, kind, m, n, k)
        if own in times:
            best = min(times, key=times.get)
            out.append((times[own] / times[best], (kind, m, n, k), own, times[own], best, times[best]))
    return sorted(out, reverse=True)


def check(path):
    rows = table(path)
    found = losses(rows)
    print(f"{len(rows)} products, {sum(len(r[4]) for r in rows)} times; the chosen plan timed for {len(found)}")
    print(f"mean {math.exp(sum(math.log(f[0]) for f in found) / len(found)):.4f} of the best")
    for ratio, product, own, t, best, b in found[:8]:
        print(f"  {ratio:.2f} {product}: {own} {t} us, {best} {b} us")


# ------------------------------------------------------------------ the costs
def predicted(p, kind, plan):
    """us by costs p: first, step, first2, step2 of each tile, launch, join, copy, part, rates."""
    tile, parts, steps, tiles, whole = plan
    rows, cols, groups = TILES[tile]
    first, step, first2, step2 = p[4 * tile:4 * tile + 4]
    launch, join, copy, part, *rates = p[20:]
    power = rows * cols * groups * 128e-9 / rates[tile > 0]
    pairs = PAIRS[kind][tile]

    def rounds(blocks, count):
        per = CUS * (2 if pairs else 1)
        full, rest = divmod(blocks, per)
        f, s = (first2, step2) if pairs else (first, step)
        us = full * (f + count * max(s, per * power))
        if rest:
            f, s = (first2, step2) if rest > CUS else (first, step)
            us += f + count * max(s, rest * power)
        return us

    us = launch + rounds(whole, -(-steps // groups))
    if parts > 1:
        count, blocks = -(-(-(-steps // parts)) // groups), (tiles - whole) * parts
        if pairs and whole // CUS % 2 == 1:
            us += count * max(step2 - step, min(blocks, CUS) * power) + rounds(max(blocks - CUS, 0), count)
        else:
            us += rounds(blocks, count)
        us += join + parts * (part + copy * rows * cols / 16384)
    return us


START = [7, 1.5, 7, 2, 4, .9, 5, 1.5, 3, .55, 4, .9, 2.5, .7, 4, 1.2, 2, .5, 3, .8, 3.5, 1.5, .25, .1, 1.35, 1.24]


def fit(path):
    import numpy as np
    from scipy.optimize import least_squares
    rows = table(path)
    for kind, name in enumerate(("forward", "gated", "backward")):
        data = [(geometry(*r[:4], plan), us) for r in rows if r[0] == kind for plan, us in r[4].items()]
        error = lambda x: [math.log(predicted(np.exp(x), kind, plan) / us) for plan, us in data]
        x = least_squares(error, np.log(START), loss="soft_l1", f_scale=0.1).x
        p, rms = np.exp(x), float(np.sqrt(np.mean(np.square(error(x)))))
        print(f"{name}: {len(data)} times, root mean square of the error {100 * rms:.1f}%")
        for tile in range(5):
            print("  tile", tile, [round(float(v), 2) for v in p[4 * tile:4 * tile + (4 if PAIRS[kind][tile] else 2)]])
        print("  launch, join, copy, part, rates", [round(float(v), 2) for v in p[20:]])


if __name__ == "__main__":
    {"sweep": sweep, "check": check, "fit": fit}[sys.argv[1]](sys.argv[2])
