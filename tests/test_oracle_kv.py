"""Pins of the key/value cache's oracle: hand-worked pages, turns and scales, the gradient of the
rotation against differences, and attention against a direct softmax."""
import numpy as np
import pytest

from oracle import e4m3, kv


def test_pages_by_hand():
    table = np.full((4, 3), -1)
    table[0, 0] = 7                                            # 10 of 16 tokens
    table[2, :2] = [3, 4]
    free = [11, 12, 13, 99]
    t, lens, cu, pos, slots, left = kv.assign([10, 0, 32, 5], [8, 0, 1, 0], table, free, 3, 16, 12)
    assert t[0].tolist() == [7, 13, -1] and t[2].tolist() == [3, 4, 12]
    assert lens.tolist() == [18, 0, 33, 5] and cu.tolist() == [0, 8, 8, 9, 9]
    assert pos.tolist() == [10, 11, 12, 13, 14, 15, 16, 17, 32, -1, -1, -1]
    assert slots.tolist() == [7 * 16 + 10 + i for i in range(6)] + [208, 209, 192, -1, -1, -1] and left.tolist() == [1, 0]
    # two pages for three requests that need one each, the second two: it is refused, and all that need one behind it
    t, lens, cu, pos, slots, left = kv.assign([0, 0, 0, 3], [1, 17, 1, 1], np.full((4, 3), 5), free, 2, 16, 20)
    assert lens.tolist() == [1, 0, 0, 4] and left.tolist() == [1, 2] and t[0, 0] == 12 and t[1:].min() == 5
    assert slots[0] == 192 and np.all(slots[1:19] == -1) and slots[19] == 83
    # more rows than there are, and a row of the table that is too short
    t, lens, cu, pos, slots, left = kv.assign([0, 47], [5, 9], np.full((2, 3), -1), free, 4, 16, 7)
    assert cu.tolist() == [0, 5, 7] and lens.tolist() == [5, 47] and left.tolist() == [3, 0]
    lens, free2, n = kv.release([1, 0, 1], [17, 40, 16], np.array([[1, 2, 3], [4, 5, 6], [7, 8, 9]]), [50, 51, 0, 0, 0], 2, 16)
    assert lens.tolist() == [0, 40, 0] and free2.tolist() == [50, 51, 1, 2, 7] and n == 5


def test_turns_by_hand():
    x = np.arange(8.0)[None, None] + 1
    y = kv.rope(x, [1], [np.pi / 2, 0.0])
    assert np.allclose(y[0, 0], [-3, 2, 1, 4, 5, 6, 7, 8])
    y = kv.rope(x, [1], [np.pi / 2, np.pi], interleaved=True, scale=2.0)
    assert np.allclose(y[0, 0], [-4, 2, -6, -8, 5, 6, 7, 8])
    assert np.allclose(kv.rope(kv.rope(x, [9], [0.3, 0.7]), [9], [0.3, 0.7], inverse=True), x)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotations_gradient_against_differences(interleaved):
    rng = np.random.default_rng(1)
    x, g = rng.standard_normal((2, 1, 10)), rng.standard_normal((2, 1, 10))
    args = ([3, 1000], [1.0, 0.3, 0.001, 0.2], interleaved, 1.3)
    back = kv.rope(g, *args, inverse=True)
    back[..., 8:] = g[..., 8:]
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = 1e-5
        num = (np.sum(g * kv.rope(x + d, *args)) - np.sum(g * kv.rope(x - d, *args))) / 2e-5
        assert abs(num - back[i]) < 1e-8


def test_scales_and_codes_by_hand():
    assert kv.page_scale(0.0) == 0 and kv.page_scale(448.0) == 1 and kv.page_scale(448.5) == 2 and kv.page_scale(224.0) == 0.5
    assert kv.page_scale(1e-40) == 2.0 ** -126
    codes, scale = np.zeros((2, 1, 16, 64), np.uint8), np.zeros((2, 1))
    x = np.zeros((3, 1, 64))
    x[0, 0, 0], x[1, 0, 1], x[2, 0, 2] = 7.0, 3.0, 8.0
    codes, scale = kv.append(x[:2], [16, 17], codes, scale, 16)
    assert scale.tolist() == [[0.0], [2.0 ** -6]] and e4m3.decode(codes[1, 0, :2, :2]).tolist() == [[448, 0], [0, 192]]
    codes, scale = kv.append(x[2:], [18], codes, scale, 16)
    assert scale[1, 0] == 2.0 ** -5 and e4m3.decode(codes[1, 0, :3, :3]).tolist() == [[224, 0, 0], [0, 96, 0], [0, 0, 256]]


def test_attention_by_hand():
    rng = np.random.default_rng(2)
    page, D = 16, 64
    kc = e4m3.encode(rng.standard_normal((3, 1, page, D)).astype(np.float32))
    vc = e4m3.encode(rng.standard_normal((3, 1, D, page)).astype(np.float32))
    ks, vs = np.array([[1.0], [0.5], [2.0]]), np.array([[1.0], [4.0], [0.25]])
    q = rng.standard_normal((3, 2, D))
    out, lse, size, _ = kv.attention(q, kc, ks, vc, vs, np.array([[2, 0], [1, 9]]), [0, 2, 3], [18, 20], 0.1)
    k = np.concatenate([e4m3.decode(kc[2, 0]) * 2, e4m3.decode(kc[0, 0])])
    v = np.concatenate([e4m3.decode(vc[2, 0]).T * 0.25, e4m3.decode(vc[0, 0]).T])
    for i, m in ((0, 17), (1, 18)):
        for h in range(2):
            x = np.exp(0.1 * k[:m] @ q[i, h])
            assert np.allclose(out[i, h], (x / x.sum()) @ v[:m]) and np.isclose(lse[i, h], np.log(x.sum()))
    x = np.exp(0.1 * (e4m3.decode(kc[1, 0]) * 0.5) @ q[2, 0])  # the second page does not exist
    assert np.allclose(out[2, 0], (x / x.sum()) @ (e4m3.decode(vc[1, 0]).T * 4))
    assert np.all(size + 1e-12 >= np.abs(out))
    out, lse, _, _ = kv.attention(q, kc, ks, vc, vs, np.array([[2, 0]]), [0, 3], [2], 0.1)
    assert np.all(out[0] == 0) and np.all(np.isneginf(lse[0])) and np.all(out[1] != 0)
