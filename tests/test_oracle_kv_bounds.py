"""The attention bounds' figures for rounding, against roundings done one by one."""

import numpy as np
import pytest

from oracle import kv, mxfp4


def bf16(x):
    return mxfp4.bf16_bits_to_f64(mxfp4.round_to_bf16_bits(x))


def two_bf16(x):
    hi = bf16(x)
    return hi + bf16(x - hi)


def fp16(x):
    """As the kernel for few rows has it: times 2^6, rounded, times a factor of down to 2^-1, in FP16."""
    y = (x * 64).astype(np.float16)
    return (y * np.float16(0.5)).astype(np.float64) / 32


@pytest.mark.parametrize("rounded,bound,least", [(bf16, kv.P_ONE_BF16, 0.99), (two_bf16, kv.P_TWO_BF16, 0.1), (fp16, kv.P_FP16, 0.5)])
def test_a_probability_is_off_by_no_more(rounded, bound, least):
    p = np.concatenate([np.linspace(0.5, 1, 20001), 2.0 ** -np.linspace(0, 20, 20001)])
    err = np.abs(rounded(p) - p) / p
    assert least * bound < err.max() <= bound


def rows_of_two_keys(rounded):
    """Rows whose second key alone has a value, 1: out = p / (1 + p), the sum taken before the rounding, as the kernels
    do.  Returns what they answer, and their bound's terms without the keys' sums, which two keys do not use."""
    p = np.linspace(0.5, 1, 20001)[:, None, None]
    o = p / (1 + p)
    flat = np.zeros(o.shape[:2])
    got = bf16(rounded(p) / (1 + p))
    return got, o, lambda p_round: kv.attention_bounds(o, flat, o, flat, p_round=p_round)[0] - 2.0 ** -10 * o


def test_one_term_needs_its_own_bound():
    got, o, bound = rows_of_two_keys(bf16)
    assert (np.abs(got - o) <= bound(kv.P_ONE_BF16)).all()
    assert (np.abs(got - o) > bound(2.0 ** -9)).any()


@pytest.mark.parametrize("rounded", [two_bf16, fp16])
def test_finer_roundings_hold_the_default(rounded):
    got, o, bound = rows_of_two_keys(rounded)
    assert (np.abs(got - o) <= bound(2.0 ** -9)).all()
