"""The oracle of the linear-attention operators against facts that do not come
from it: hand-worked values, explicit sums, differences, invariants, torch's
float8 type.  A mistake planted in the oracle must break one of them."""
import numpy as np
import pytest
import torch

from oracle import linattn_oracle as R


def draw(rng, B, T, H, K, V):
    q, k = (rng.normal(size=(B, T, H, K)) for _ in range(2))
    return q, k, rng.normal(size=(B, T, H, V))


def test_hand_worked_tokens():
    # K = V = 1, a = 1/2, s_in = 4: S = 4/2 + 1*2 = 4, o = 3*4 = 12; S = 4/2 + 2*1 = 4, o = -4
    q, k, v = (np.array(x, float).reshape(1, 2, 1, 1) for x in ([3, -1], [1, 2], [2, 1]))
    o, S = R.linattn_ref(q, k, v, [np.log(0.5)], s_in=np.full((1, 1, 1, 1), 4.0))
    np.testing.assert_allclose(o.ravel(), [12.0, -4.0])
    np.testing.assert_allclose(S.ravel(), [4.0])


@pytest.mark.parametrize("lengths", [None, [7, 0], [3, 5]])
def test_recurrence_equals_the_sums(lengths):
    rng = np.random.default_rng(1)
    q, k, v = draw(rng, 2, 7, 3, 4, 5)
    g = np.array([0.0, -0.3, -np.inf])
    s0 = rng.normal(size=(2, 3, 4, 5))
    o, _ = R.linattn_ref(q, k, v, g, 0.7, lengths, s0)
    np.testing.assert_allclose(o, R.linattn_bruteforce(q, k, v, g, 0.7, lengths, s0), rtol=1e-12, atol=1e-12)


def test_a_sequence_in_pieces_is_the_sequence():
    rng = np.random.default_rng(2)
    q, k, v = draw(rng, 1, 9, 2, 3, 4)
    g = [-0.1, -1.0]
    o, S = R.linattn_ref(q, k, v, g)
    o1, S1 = R.linattn_ref(q[:, :4], k[:, :4], v[:, :4], g)
    o2, S2 = R.linattn_ref(q[:, 4:], k[:, 4:], v[:, 4:], g, s_in=S1)
    np.testing.assert_allclose(np.concatenate([o1, o2], 1), o, rtol=1e-12)
    np.testing.assert_allclose(S2, S, rtol=1e-12)


@pytest.mark.parametrize("lengths", [None, [5, 2]])
def test_gradients_equal_differences(lengths):
    rng = np.random.default_rng(3)
    q, k, v = draw(rng, 2, 5, 2, 3, 2)
    g = [-0.2, -1.5]
    s0, do, ds = rng.normal(size=(2, 2, 3, 2)), rng.normal(size=v.shape), rng.normal(size=(2, 2, 3, 2))

    def loss(q, k, v, s0):
        o, S = R.linattn_ref(q, k, v, g, 1.3, lengths, s0)
        return float(np.sum(o * do) + np.sum(S * ds))

    grads = R.linattn_ref_backward(q, k, v, g, do, 1.3, lengths, s0, ds)
    x = {"q": q, "k": k, "v": v, "s_in": s0}
    for name in x:
        for _ in range(12):
            at = tuple(rng.integers(n) for n in x[name].shape)
            d = np.zeros_like(x[name])
            d[at] = 1e-5
            up, down = (loss(*[x[m] + (s * d if m == name else 0.0) for m in x]) for s in (1.0, -1.0))
            assert abs((up - down) / 2e-5 - grads[name][at]) < 1e-7 * (1 + abs(grads[name][at])), (name, at)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation(layout):
    rng = np.random.default_rng(4)
    x = rng.normal(size=(2, 3, 2, 10))
    pos = rng.integers(0, 2 ** 31, size=(2, 3))
    f = np.array([1.0, 0.1, 1e-4])
    y = R.rope_ref(x, pos, f, layout)
    np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
    np.testing.assert_allclose(R.rope_ref(y, pos, f, layout, inverse=True), x, atol=1e-12)
    # a quarter turn sends the first of a pair to the second
    one = np.zeros((1, 1, 1, 4))
    one[..., 0] = 1.0
    z = R.rope_ref(one, [[1]], np.array([np.pi / 2, 0.0]), layout)
    np.testing.assert_allclose(z.ravel(), np.eye(4)[1 if layout == "interleaved" else 2], atol=1e-15)
    # products of turned rows depend on the distance alone
    a, b = rng.normal(size=(2, 1, 1, 1, 6))
    near = np.sum(R.rope_ref(a, [[5]], f, layout) * R.rope_ref(b, [[2]], f, layout))
    far = np.sum(R.rope_ref(a, [[1000005]], f, layout) * R.rope_ref(b, [[1000002]], f, layout))
    assert abs(near - far) < 1e-9


def test_norm_and_its_gradients():
    rng = np.random.default_rng(5)
    h, w, dy, dh = rng.normal(size=(3, 8)), rng.normal(size=8), rng.normal(size=(3, 8)), rng.normal(size=(3, 8))
    np.testing.assert_allclose(R.rms_norm_ref(np.array([[3.0, 4.0]]), [1.0, 2.0], 0.0), [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    g = R.rms_norm_ref_backward(dy, h, w, 0.01, dh)
    loss = lambda h, w: float(np.sum(R.rms_norm_ref(h, w, 0.01) * dy) + np.sum(h * dh))  # noqa: E731
    for at in np.ndindex(h.shape):
        d = np.zeros_like(h)
        d[at] = 1e-6
        assert abs((loss(h + d, w) - loss(h - d, w)) / 2e-6 - g["x"][at]) < 1e-7
    for c in range(8):
        d = np.zeros(8)
        d[c] = 1e-6
        assert abs((loss(h, w + d) - loss(h, w - d)) / 2e-6 - g["weight"][c]) < 1e-7


def test_e4m3_rounding_is_torchs():
    assert len(R.E4M3) == 127 and R.E4M3[-1] == 448.0 and R.E4M3[1] == 2.0 ** -9
    rng = np.random.default_rng(6)
    mid = (R.E4M3[1:] + R.E4M3[:-1]) / 2   # ties
    x = np.concatenate([R.E4M3, mid, -mid, rng.uniform(-448, 448, 500), rng.normal(size=500) * 0.01]).astype(np.float32)
    np.testing.assert_array_equal(R.e4m3_nearest(x), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())


def test_scales():
    y = np.zeros((2, 300))
    y[0, 5], y[0, 299] = -896.0, 44.8
    np.testing.assert_allclose(R.scales_ref(y, 128), [[2.0, 1.0, 0.1], [1.0, 1.0, 1.0]])
    np.testing.assert_allclose(R.scales_ref(y, 0), [[2.0], [1.0]])


@pytest.mark.parametrize("mistake", ["decay before the token", "no decay of s_in", "adjoint decays late", "pairs swapped"])
def test_planted_mistakes_are_found(mistake, monkeypatch):
    """Each mistake, planted in the oracle, breaks one of the facts above."""
    if mistake == "pairs swapped":
        true = R.rope_ref
        monkeypatch.setattr(R, "rope_ref", lambda x, p, f, layout="half", inverse=False: true(
            x, p, f, "half" if layout == "interleaved" else "interleaved", inverse))
        with pytest.raises(AssertionError):
            test_rotation("half")
        return
    if mistake == "adjoint decays late":
        true = R.linattn_ref_backward

        def wrong(q, k, v, g, do, scale=1.0, lengths=None, s_in=None, ds_out=None):
            out = true(q, k, v, g, do, scale, lengths, s_in, ds_out)
            out["s_in"] = out["s_in"] / np.exp(np.asarray(g))[:, None, None]
            return out

        monkeypatch.setattr(R, "linattn_ref_backward", wrong)
        with pytest.raises(AssertionError):
            test_gradients_equal_differences(None)
        return
    true = R.linattn_ref

    def wrong(q, k, v, g, scale=1.0, lengths=None, s_in=None):
        if mistake == "no decay of s_in" and s_in is not None:
            s_in = np.asarray(s_in) / np.exp(np.maximum(g, -50.0))[:, None, None]
        if mistake == "decay before the token":
            k = np.asarray(k) * np.exp(np.maximum(g, -50.0))[:, None]
        return true(q, k, v, g, scale, lengths, s_in)

    monkeypatch.setattr(R, "linattn_ref", wrong)
    with pytest.raises(AssertionError):
        test_hand_worked_tokens()
