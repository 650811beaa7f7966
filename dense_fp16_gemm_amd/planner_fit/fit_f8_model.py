"""Fit of the time model of the 8-bit products' tile and ring kernels (model() and
kKernels in csrc/f8.hip) to measured times.  Host only: reads the kernel table from
the source and the measurements in f8_timings.jsonl, runs no GPU code.

f8_timings.jsonl: one MI355X (256 CUs), every tile and ring kernel on shapes drawn from 1
to 8192 rows and sizes of 64 to 16384, one record per call and shape, entries
[kernel, ranges of K, us]; times of calls captured in a row, best of three replays,
operands quantised before and read from HBM.

  call       shape                what is timed
  product    M, N, K              gemm_nt_f8 of an A in F8
  experts    T, E, top, N, K      gemm_nt_f8_experts of gathered tokens in F8, random routings
  gradients  T, E, top, M, N      gemm_nt_f8_experts_grad

The model, in us, of `wgs` workgroups of `steps` groups of 128 columns each:
  rounds  = whole rounds x (full x steps + start x slots)
            + the last: step x steps + start for at most a workgroup a CU, else a whole one
  t       = (rounds^4 + (bytes / memory)^4 + (multiplications / matrix)^4)^(1/4) + launch
            + [ranges] join + 2 x 4 bytes of each range's sums / partial
with start, step and full for each kernel (full = step where one workgroup fits on a
CU) and the rest shared.  The fit minimises a robust squared error of the logarithm;
experts and gradients count 1.5 times.

usage: python3 fit_f8_model.py
"""
from __future__ import annotations

import json
import math
import os
import re

import numpy as np
from scipy.optimize import least_squares

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(os.path.dirname(HERE), "csrc", "f8.hip")
TIMINGS = os.path.join(HERE, "f8_timings.jsonl")
CUS, GROUP = 256, 128
SHARED = ("memory", "join", "partial", "launch", "matrix")


def cdiv(a, b):
    return -(-a // b)


def kernel_table():
    """[(block_m, block_n, slots, (start, step, full))] of the tile and ring kernels."""
    src = open(SOURCE).read()
    tab = src[src.index("static const Kernel kKernels[] = {"):]
    out = []
    for name, args in re.findall(r"\b(TILE|RING)\(([^)]*)\)", tab[:tab.index("};")]):
        v = [float(x) for x in args.split(",")]
        slots = int(v[4]) if name == "TILE" else 2
        out.append((int(v[0] * v[2]) * 32, int(v[1] * v[3]) * 32, slots, tuple(v[5:])))
    return out


def source_constants():
    """The shared constants as model() has them."""
    src = open(SOURCE).read()
    body = src[src.index("static double model("):]
    body = body[:body.index("\n}\n")]
    num = r"([0-9.e+]+)"
    return {"memory": float(re.search(r"bytes / " + num, body)[1]),
            "matrix": float(re.search(r"GROUP / " + num, body)[1]),
            "launch": float(re.search(r"return us \+ " + num, body)[1]),
            "join": float(re.search(r"splits > 1 \? " + num, body)[1]),
            "partial": float(re.search(r"wgs \* tile / " + num, body)[1])}


def features(call, shape, kernel, ranges):
    """(workgroups, groups of each, bytes of the ranges' sums, bytes, multiplications)
    as search() in the source counts them."""
    bm, bn, _, _ = kernel
    if call == "product":
        m, n, k = shape
        kb, tiles = cdiv(k, GROUP), cdiv(m, bm) * cdiv(n, bn)
        per = cdiv(kb, ranges)
        wgs = tiles * cdiv(kb, per)
        sums = 4 * wgs * bm * bn if ranges > 1 else 0
        return wgs, per, sums, n * k + m * k + 2 * m * n, tiles * bm * bn * kb * GROUP
    t, e, top, n, k = shape
    slots = t * top
    if call == "experts":
        used = e * (1 - (1 - 1 / e) ** slots)
        most = 2 * slots / (used * bm)
        whole = math.floor(most)
        down = used * (1 if most <= 1 else (0.5 * whole + most - whole) * (whole + 1) / most)
        wgs = math.ceil(cdiv(n, bn) * down)
        return wgs, cdiv(k, GROUP), 0, used * n * k + slots * k + 2 * slots * n, wgs * bm * bn * k
    wgs = e * cdiv(n, bm) * cdiv(k, bn)
    per = slots / e / GROUP + 0.5 if slots > 64 * e else 1
    return wgs, per, 0, slots * (n + k) + 2 * e * n * k, wgs * bm * bn * per * GROUP


def model(slots, own, shared, wgs, per, sums, read, volume, ranges):
    start, step, full = own
    if slots == 1:
        full = step
    rounds, rest = divmod(wgs, CUS * slots)
    taken = full * per + start * slots
    us = rounds * taken
    if rest:
        us += step * per + start if rest <= CUS else taken
    us = (us ** 4 + (read / shared["memory"]) ** 4 + (volume / shared["matrix"]) ** 4) ** 0.25
    return us + shared["launch"] + (shared["join"] + sums / shared["partial"] if ranges > 1 else 0)


def load_rows(table):
    rows = []
    for line in open(TIMINGS):
        r = json.loads(line)
        for i, ranges, us in r["entries"]:
            rows.append((r["call"], tuple(r["shape"]), i, ranges, us,
                         features(r["call"], r["shape"], table[i], ranges)))
    return rows


def fit(table, rows):
    count = len(table)

    def unpack(x):
        return np.exp(x[:3 * count]).reshape(count, 3), dict(zip(SHARED, np.exp(x[3 * count:])))

    def residuals(x):
        own, shared = unpack(x)
        return np.array([(1.0 if call == "product" else 1.5) *
                         math.log(model(table[i][2], own[i], shared, *f, ranges) / us)
                         for call, _, i, ranges, us, f in rows])

    x0 = []
    for bm, bn, _, _ in table:
        step = bm * bn / 65536 * 1.2 + 0.15
        x0 += [0.0, math.log(step), math.log(1.6 * step)]
    x0 += [math.log(v) for v in (5e6, 2.5, 4e6, 3.0, 1.35e9)]
    return unpack(least_squares(residuals, x0, loss="soft_l1", f_scale=0.1).x)


def main():
    table = kernel_table()
    rows = load_rows(table)
    own, shared = fit(table, rows)
    for name in SHARED:
        print(f"{name} = {shared[name]:.6g}")
    for i, (bm, bn, slots, _) in enumerate(table):
        start, step, full = own[i]
        errors = []
        for call in ("product", "experts", "gradients"):
            logs = [math.log(model(slots, own[i], shared, *f, ranges) / us)
                    for c, _, j, ranges, us, f in rows if c == call and j == i]
            errors.append("%s %.3f" % (call, math.sqrt(np.mean(np.square(logs)))))
        print(f"  {bm}x{bn} {start:.3f} {step:.4f} {full if slots > 1 else step:.4f}  error: " + ", ".join(errors))
    shapes: dict = {}
    for call, shape, i, ranges, us, f in rows:
        t = model(table[i][2], own[i], shared, *f, ranges)
        shapes.setdefault((call, shape), []).append((t, us))
    for call in ("product", "experts", "gradients"):
        picks = sorted((min(v)[1] / min(us for _, us in v), shape) for (c, shape), v in shapes.items() if c == call)
        print(f"{call}: {len(picks)} shapes, the model's choice over the best: mean "
              f"{np.mean([p[0] for p in picks]):.3f}, worst {picks[-1][0]:.3f} at {picks[-1][1]}")


if __name__ == "__main__":
    main()
