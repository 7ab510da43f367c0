"""Pins of the mixture-of-experts oracle: hand-worked choices and rows, and every
gradient against central differences of its forward function."""
import numpy as np
import pytest

from oracle import moe, quant


def test_hand_worked_choice():
    x = np.array([[0.0, 2.0, 2.0, -1.0, 1.0, -np.inf]])
    idx, w, _ = moe.route(x, 3, renormalize=False)
    assert idx.tolist() == [[1, 2, 4]]                       # the tie of 1 and 2 goes to 1
    s = 1 / (1 + np.exp(-np.array([2.0, 2.0, 1.0])))
    assert np.allclose(w, s)
    # groups {0, 1}, {2, 3}, {4, 5}: the best by one score are 0 and 1 (tie of experts 1 and 2)
    assert moe.route(x, 2, n_groups=3, topk_groups=1)[0].tolist() == [[1, 0]]
    # by two scores group 0 has 0.5 + 0.88, group 1 0.88 + 0.27, group 2 0.73 alone
    assert moe.route(x, 4, n_groups=3, topk_groups=2, group_top=2)[0].tolist() == [[1, 2, 0, 3]]
    # a bias moves the choice but not the weight
    idx, w, _ = moe.route(x, 1, bias=[0, 0, 0, 5, 0, 5], renormalize=False)
    assert idx.tolist() == [[3]] and np.allclose(w, 1 / (1 + np.e))


def test_masked_rows():
    x = np.full((2, 4), -np.inf)
    x[1, 2] = -30.0
    for score in (moe.SOFTMAX, moe.SIGMOID):
        idx, w, _ = moe.route(x, 2, score=score)
        assert idx.tolist() == [[-1, -1], [2, -1]]
        assert w[0].tolist() == [0, 0] and w[1, 0] == 1.0 and w[1, 1] == 0


@pytest.mark.parametrize("score", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((3, 7))
    g = rng.standard_normal((3, 3))
    idx = moe.route(x, 3, score=score)[0]
    idx[2, 2] = -1                                            # a missing choice

    def loss(v):
        s = moe.scores(v, score)
        total = 0.0
        for t in range(3):
            live = [j for j in range(3) if idx[t, j] >= 0]
            z = sum(s[t, idx[t, j]] for j in live) if renorm else 1.0
            total += sum(g[t, j] * 2.5 * s[t, idx[t, j]] / z for j in live)
        return total

    at = [(t, e) for t in range(3) for e in range(7)]
    num = moe.finite_difference(loss, x, at).reshape(3, 7)
    dx = moe.route_backward(x, idx, g, score, renorm, 2.5)
    assert np.max(np.abs(num - dx)) < 1e-8


def test_rows_by_hand():
    idx = np.array([[4, 5], [5, -1], [9, 5], [4, 7]])
    row, off, cnt = moe.rows_contiguous(idx, 4, 3)            # experts 4, 5, 6
    assert cnt.tolist() == [2, 3, 0] and off.tolist() == [0, 128, 256, 256]
    assert row.tolist() == [[0, 128], [129, -1], [-1, 130], [1, -1]]
    row, m = moe.rows_masked(idx, 4, 3, 2)
    assert m.tolist() == [2, 2, 0]
    assert row.tolist() == [[0, 2], [3, -1], [-1, -1], [1, -1]]


def test_combine_and_its_gradients():
    rng = np.random.default_rng(5)
    y, w = rng.standard_normal((4, 6)), rng.standard_normal((3, 2))
    row = np.array([[0, 3], [2, -1], [1, 1]])
    out, _ = moe.combine(y, row, w)
    assert np.allclose(out[0], w[0, 0] * y[0] + w[0, 1] * y[3]) and np.allclose(out[1], w[1, 0] * y[2])
    d = rng.standard_normal((3, 6))
    dw, _ = moe.combine_dw(d, y, row)
    num = moe.finite_difference(lambda v: np.sum(d * moe.combine(y, row, v)[0]), w, [(t, j) for t in range(3) for j in range(2)])
    assert np.max(np.abs(num.reshape(3, 2) - dw)) < 1e-8
    assert dw[1, 1] == 0.0


def test_gate_gradient_against_differences():
    rng = np.random.default_rng(7)
    g, u, dh = rng.standard_normal((3, 2, 5)) * 3
    (dg, _), (du, _) = moe.gate_backward(g, u, dh)
    at = [(i, j) for i in range(2) for j in range(5)]
    num = moe.finite_difference(lambda v: np.sum(dh * moe.gate(v, u)), g, at).reshape(2, 5)
    assert np.max(np.abs(num - dg)) < 1e-7
    num = moe.finite_difference(lambda v: np.sum(dh * moe.gate(g, v)), u, at).reshape(2, 5)
    assert np.max(np.abs(num - du)) < 1e-7
    assert np.allclose(moe.gate(np.array([0.0, 1.0]), np.array([3.0, 2.0])), [0.0, 2.0 / (1 + np.exp(-1.0))])


def test_quantized_check_tells_a_wrong_step():
    rng = np.random.default_rng(9)
    v = rng.standard_normal((3, 160))
    q, s = quant.quant_act_1x128(v.astype(np.float32))
    moe.check_quantized(q, s, v, 2.0 ** -23 * np.abs(v), "right")
    for q2, s2 in ((q ^ np.uint8(0x80), s), (q + np.uint8(1), s), (q, s * np.float32(1.001))):
        with pytest.raises(AssertionError):
            moe.check_quantized(q2, s2, v, 2.0 ** -23 * np.abs(v), "wrong")


def test_decoded_rows():
    rng = np.random.default_rng(11)
    q, s = quant.quant_act_1x128(rng.standard_normal((4, 144)).astype(np.float32))
    assert np.array_equal(moe.decode_rows(q, s), quant.dequant_act(q, s).astype(np.float32))
