"""The plain references of the new operators against brute force and differences
(no GPU)."""

import numpy as np
import pytest

import operator_reference as ref


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gates_gradient_against_differences(score, renorm):
    """Central differences of the gates, step h: error O(h^2) + 2^-53 / h, about 1e-9."""
    rng = np.random.default_rng(7)
    l = rng.normal(size=11)
    l[3] = -np.inf
    ids = np.array([5, 0, 9, 3])
    dg = rng.normal(size=4)
    lowest = ref.LOWEST["f32"]
    got, _ = ref.gates_backward(l, ids, dg, score, renorm, 2.5, lowest)
    h = 1e-5
    for i in range(11):
        hi, lo = l.copy(), l.copy()
        hi[i] += h
        lo[i] -= h
        diff = (ref.gates_of(hi, ids, score, renorm, 2.5, lowest) -
                ref.gates_of(lo, ids, score, renorm, 2.5, lowest)) / (2 * h)
        assert abs(got[i] - (diff * dg).sum()) < 1e-8, i


def test_choice_ties_and_masks():
    l = np.array([1.0, 3, -np.inf, 3, 1, 3])
    m = np.isneginf(l)
    assert ref.chosen(l, m, "sigmoid", None, 4).tolist() == [1, 3, 5, 0]
    assert ref.chosen(l, m, "softmax", None, 6).tolist() == [1, 3, 5, 0, 4, 2]
    # two groups of three: 3 + 1 against 3 + 3; the masked expert only fills up
    assert ref.chosen(l, m, "sigmoid", None, 2, 2, 1, 2).tolist() == [3, 5]
    assert ref.chosen(l, m, "sigmoid", None, 3, 2, 1, 1).tolist() == [1, 0, 2]
    gone = np.full(6, -np.inf)
    assert ref.chosen(gone, gone < 0, "softmax", None, 3).tolist() == [0, 1, 2]
    assert (ref.gates_of(gone, [0, 1, 2], "softmax", True, 1.0, ref.LOWEST["f32"]) == 0).all()


def test_e2m1_table():
    """sign, two exponent bits (bias 1), one mantissa bit; exponent 0 is subnormal."""
    for q in range(16):
        e, m = q >> 1 & 3, q & 1
        v = (1 + m / 2) * 2.0 ** (e - 1) if e else m / 2
        assert ref.E2M1[q] == (-v if q & 8 else v)


def test_w4_dequant_order():
    packed = np.array([[0x21, 0x43]], np.uint8)  # columns 0..3 hold codes 1, 2, 3, 4
    s = np.array([[1.0, 2.0]])
    np.testing.assert_array_equal(ref.w4_dequant(packed, s, None, "int4", 2),
                                  [[-7, -6, -10, -8]])
    np.testing.assert_array_equal(
        ref.w4_dequant(packed, np.array([[127, 128]]), None, "e2m1", 2), [[.5, 1, 3, 4]])
