"""The digits that stand for a bf16 row under 4-bit weights, over whole rows: the
scale of a block reaches only so far below that of the row's largest value (60
binary places, MX; 17, NV), so small blocks are off by a share of the row's largest.
The shares are those include/moe.h promises; modelled in numpy (no GPU)."""
import os
import re

import numpy as np
import pytest

from .test_fp4_digits import DIGITS, bf16, digits

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")
# columns of a block, and how far its scale goes below the largest one's
FORMATS = {"mx": (32, 60), "nv": (16, 17)}


def promised(fmt):
    text = re.sub(r"\s*\n \*\s*", " ", open(HEADER).read())
    m = re.search(r"none by more than 2\^-(\d+), MX, or 2\^-(\d+), NV, of the row's largest", text)
    return int(m.group(1 if fmt == "mx" else 2))


def error(x, fmt):
    """Largest error of a row's digits (x: float64 bf16 values)."""
    block, reach = FORMATS[fmt]
    exponent = lambda v: int(np.floor(np.log2(np.abs(v).max())))       # noqa: E731
    top, worst = exponent(x), 0.0
    for b in x.reshape(-1, block):
        if not b.any():
            continue
        u = 2.0 ** (top + max(exponent(b) - top, -reach) - 1)
        d = digits((b / u).astype(np.float32))
        back = u * (d.astype(np.float64) * 8.0 ** -np.arange(DIGITS)[:, None]).sum(axis=0)
        worst = max(worst, np.abs(back - b).max())
    return worst


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_blocks_below_the_reach_of_the_scales(fmt):
    block, reach = FORMATS[fmt]
    bound, seen = 2.0 ** -promised(fmt), 0.0
    rng = np.random.default_rng(1)
    m = np.arange(128, 256) / 128.0
    for below in range(0, reach + 50):
        x = np.zeros((m.size // block + 1, block))
        x[0, 0] = 1.0                                    # a row's largest, a power of two
        x[1:] = (m * rng.choice([-1.0, 1.0], m.size) * 2.0 ** -below).reshape(-1, block)
        assert (bf16(x) == x).all()
        if below == 0:
            x[1:] /= 2
        err = error(x.reshape(-1), fmt)
        assert err <= bound, below
        seen = max(seen, err)
    assert seen == bound                                 # no smaller power of two would do


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_rows_of_blocks_of_all_magnitudes(fmt):
    block, reach = FORMATS[fmt]
    rng = np.random.default_rng(2)
    for _ in range(50):
        x = rng.standard_normal((24, block)) * 2.0 ** rng.uniform(-reach - 40, 0, (24, 1))
        x = bf16(x).astype(np.float64).reshape(-1)
        assert error(x, fmt) <= 2.0 ** -promised(fmt) * np.abs(x).max()
