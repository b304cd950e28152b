"""The digits that stand for a bf16 row under 4-bit weights, modelled in numpy
(no GPU): twelve base-8 digits of -4..4 per value, taken in fp32 as the kernel
takes them, all of them e2m1 values; exact down to 2^-27 of a block's largest
value, off by at most 2^-35 of it below; and the lower six found without the
upper ones."""
import numpy as np
import pytest

DIGITS = 12
E2M1 = {0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0}


def bf16(x):
    """Nearest bf16 of fp32 values (ties to even)."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16
    return b.astype(np.uint32).view(np.float32)


def digits(t, n=DIGITS):
    """n digits of fp32 t, |t| < 4, every step in fp32."""
    out = []
    t = np.asarray(t, np.float32)
    for _ in range(n):
        r = np.rint(t)
        out.append(r)
        t = (t - r) * np.float32(8)
    return np.stack(out)


def blocks(seed, spread):
    rng = np.random.default_rng(seed)
    x = bf16(rng.standard_normal((400, 32)) * 2.0 ** rng.uniform(-spread, 0, (400, 32)))
    e = np.floor(np.log2(np.abs(x).max(axis=1, keepdims=True).astype(np.float64)))
    return x.astype(np.float64), 2.0 ** (e - 1)              # values, unit


@pytest.mark.parametrize("spread", [0, 10, 26, 60])
def test_digits_hold_the_values(spread):
    x, u = blocks(spread, spread)
    t = (x / u).astype(np.float32)
    assert (np.abs(t) < 4).all()
    d = digits(t)
    assert set(np.abs(d).reshape(-1).tolist()) <= E2M1 and np.abs(d).max() <= 4
    back = u * (d.astype(np.float64) * 8.0 ** -np.arange(DIGITS)[:, None, None]).sum(axis=0)
    top = np.abs(x).max(axis=1, keepdims=True)
    err = np.abs(back - x)
    assert (err <= 2.0 ** -35 * top).all()
    assert (err[np.abs(x) >= 2.0 ** -27 * top] == 0).all()


def test_every_bf16_significand():
    """All significands at the top of a block, and ties of the sixth digit."""
    m = np.concatenate([np.arange(128, 256) / 64.0, -np.arange(128, 256) / 64.0])
    for shift in range(0, 30):
        t = (m * 2.0 ** -shift).astype(np.float32)
        d = digits(t)
        back = (d.astype(np.float64) * 8.0 ** -np.arange(DIGITS)[:, None]).sum(axis=0)
        if shift <= 26:
            assert (back == t).all(), shift
        assert (np.abs(back - t) <= 0.5 * 8.0 ** -(DIGITS - 1)).all()


def test_lower_digits_alone():
    """What is left after the sixth digit, from one rounding to its unit."""
    m = np.arange(128, 256) / 64.0
    t = np.concatenate([s * m * 2.0 ** -k for s in (1, -1) for k in range(40)]).astype(np.float32)
    s = t * np.float32(8.0 ** 5)
    low = (s - np.rint(s)) * np.float32(8)
    assert (digits(t)[6:] == digits(low, 6)).all()


def test_epilogue_sum_is_exact_for_one_value():
    """The digits' weighted sum from the lowest up, in fp32, gives the value."""
    m = np.arange(128, 256) / 64.0
    for shift in (0, 7, 20, 26):
        t = (m * 2.0 ** -shift).astype(np.float32)
        d = digits(t)
        acc = d[-1].astype(np.float32)
        for k in range(DIGITS - 2, -1, -1):
            acc = np.float32(acc * np.float32(0.125)) + d[k].astype(np.float32)
        assert (acc == t).all()
