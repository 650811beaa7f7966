"""The constants by which the 8-bit products' kernels are chosen are the output of
the committed fit.

dense_fp16_gemm_amd/planner_fit/fit_f8_model.py fits the time model of csrc/f8.hip to
the committed timings (host only); its shared constants and each kernel's must be the
ones that the source carries.
"""
import io
import os
import re
import sys
from contextlib import redirect_stdout

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FIT_DIR = os.path.join(ROOT, "dense_fp16_gemm_amd", "planner_fit")


def test_fit_reproduces_the_source_constants():
    sys.path.insert(0, FIT_DIR)
    try:
        import fit_f8_model
    finally:
        sys.path.pop(0)
    buf = io.StringIO()
    with redirect_stdout(buf):
        fit_f8_model.main()
    out = buf.getvalue()
    source = fit_f8_model.source_constants()
    assert set(source) == set(fit_f8_model.SHARED)
    for name, value in source.items():
        fitted = float(re.search(rf"^{name} = ([0-9.e+]+)$", out, re.M)[1])
        assert abs(fitted / value - 1) < 0.01, (name, fitted, value)
    table = fit_f8_model.kernel_table()
    lines = re.findall(r"^  (\d+)x(\d+) ([0-9.]+) ([0-9.]+) ([0-9.]+)", out, re.M)
    assert len(lines) == len(table) == 6
    for (bm, bn, *fitted), (m, n, _, own) in zip(lines, table):
        assert (int(bm), int(bn)) == (m, n)
        for f, s in zip(fitted, own):
            assert abs(float(f) / s - 1) < 0.01, (bm, bn, fitted, own)


def test_choices_are_near_the_best():
    """What the model chooses of the timed kernels: in the mean 3% behind each shape's
    best, and the worst as the source's comment says."""
    sys.path.insert(0, FIT_DIR)
    try:
        import fit_f8_model as fit
    finally:
        sys.path.pop(0)
    table, shared = fit.kernel_table(), fit.source_constants()
    shapes = {}
    for call, shape, i, ranges, us, f in fit.load_rows(table):
        t = fit.model(table[i][2], table[i][3], shared, *f, ranges)
        shapes.setdefault((call, shape), []).append((t, us))
    assert len(shapes) == 142
    for call, worst in (("product", 1.14), ("experts", 1.41), ("gradients", 1.13)):
        over = [min(v)[1] / min(us for _, us in v) for (c, _), v in shapes.items() if c == call]
        assert sum(over) / len(over) < 1.03 and max(over) < worst
