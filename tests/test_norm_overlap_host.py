"""Norms: outputs or a workspace that lie on weights, positions, frequencies or each other are refused (no kernel runs)."""
import random

import pytest

from sparse_compressed_attention_gb300 import _lib as L
from tests.test_cache_host import lib, norm, part, refused          # noqa: F401  (lib is the fixture)

BASE, DY, OUT = 1 << 24, (1 << 24) + (1 << 20), (1 << 24) + (2 << 20)      # part()'s x, dy and out: 4 rows of 2 heads of 64 bf16
WS = 1 << 40


def clean(**over):
    return part(BASE, **dict(dict(w=1 << 32, dw=1 << 33), **over))


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("at", [OUT, OUT - 240, OUT + 512, OUT + 1008])
def test_outputs_on_what_all_blocks_read(lib, grad, at):                   # noqa: F811
    text = "weights, positions or frequencies"
    kw = dict(pos=1 << 34, f=1 << 35, ws=(WS, 1 << 30))
    refused(lib, norm(lib, grad, q=clean(w=at), **kw), L.V4_ERR_INVALID_ARG, text)
    kw = dict(ws=(WS, 1 << 30), q=clean())
    if at >= OUT:
        refused(lib, norm(lib, grad, pos=at, f=1 << 35, **kw), L.V4_ERR_INVALID_ARG, text)
        refused(lib, norm(lib, grad, pos=1 << 34, f=at, **kw), L.V4_ERR_INVALID_ARG, text)


@pytest.mark.parametrize("over,ws,text", [
    (dict(dw=OUT + 16), WS, "overlaps a weight gradient"), (dict(), OUT - 1024 * 1024, "workspace overlaps an input"),
    (dict(dw=WS + 4096), WS, "workspace overlaps a weight gradient"), (dict(w=WS + 256), WS, "workspace overlaps an input"),
    (dict(), BASE, "workspace overlaps an input"), (dict(out=1 << 50), BASE, "workspace overlaps an input"),
    (dict(x=1 << 50, dy=1 << 51), OUT, "workspace overlaps an output")])
def test_gradient_outputs_and_workspace(lib, over, ws, text):              # noqa: F811
    kw = dict(pos=1 << 34, f=1 << 35)
    refused(lib, norm(lib, True, q=clean(**over), ws=(ws, 1 << 30), **kw), L.V4_ERR_INVALID_ARG, text)
    for where in ("pos", "f"):
        refused(lib, norm(lib, True, q=clean(), ws=(1 << 34, 1 << 30), **dict(kw, **{where: (1 << 34) + 512})),
                L.V4_ERR_INVALID_ARG, "workspace overlaps an input")


def test_every_run_of_a_strided_output_is_looked_at(lib):                  # noqa: F811
    """Weights that have a byte in common with some run of the output, by enumeration: heads within rows and rows within heads."""
    rng = random.Random(1)
    for _ in range(300):
        rows, heads, dim = rng.randint(1, 5), rng.randint(1, 4), 8 * rng.randint(1, 6)
        inner, outer = (heads, rows) if rng.random() < 0.5 else (rows, heads)
        si = dim + 8 * rng.randint(0, 12)
        so = (inner - 1) * si + dim + 8 * rng.randint(0, 40)
        rs, hs = (so, si) if inner is heads else (si, so)
        runs = [2 * (t * rs + h * hs) for t in range(rows) for h in range(heads)]
        run = rng.choice(runs)
        at = run + 16 * rng.randint(-(4 * dim // 16) + 1, 2 * dim // 16 - 1)
        if not any(at < r + 2 * dim and r < at + 4 * dim for r in runs):
            continue
        p = part(BASE, x=1 << 50, heads=heads, out=1 << 30, out_row_stride=rs, out_head_stride=hs, w=(1 << 30) + at,
                 x_row_stride=1 << 12, x_head_stride=1 << 8)
        refused(lib, norm(lib, False, q=p, rows=rows, dim=dim, R=0, begin=0), L.V4_ERR_INVALID_ARG, "weights, positions")
