"""The oracle of the selective state space layer's operators, pinned without
itself: explicit sums, closed forms, pieces of a sequence, central
differences, and planted mistakes that the checks have to notice."""
import numpy as np
import pytest

from oracle import ssm_oracle as R


def draw(seed, B=2, T=6, D=8, N=3, G=2):
    r = np.random.default_rng(seed)
    return {"x": r.normal(size=(B, T, D)), "dt": r.normal(size=(B, T, D)), "A": -np.exp(r.normal(size=(D, N))),
            "Bm": r.normal(size=(B, T, G, N)), "Cm": r.normal(size=(B, T, G, N)), "D": r.normal(size=D),
            "z": r.normal(size=(B, T, D)), "dt_bias": r.normal(size=D), "s_in": r.normal(size=(B, D, N))}


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("lengths", [None, [6, 2], [0, 9]])
def test_scan_is_the_explicit_sum(softplus, lengths):
    p = draw(1)
    y, _ = R.scan_ref(**p, softplus=softplus, lengths=lengths)
    np.testing.assert_allclose(y, R.scan_bruteforce(**p, softplus=softplus, lengths=lengths), rtol=1e-12, atol=1e-12)


def test_scan_closed_form():
    """A constant step and input: a geometric sum."""
    T, D, N = 7, 2, 1
    A = np.array([[-0.5], [-2.0]])
    one = np.ones((1, T, D))
    y, s = R.scan_ref(one, 0.25 * one, A, np.ones((1, T, 1, N)), np.ones((1, T, 1, N)), softplus=False)
    e = np.exp(0.25 * A[:, 0])
    np.testing.assert_allclose(y[0], 0.25 * (1 - e ** np.arange(1, T + 1)[:, None]) / (1 - e), rtol=1e-13)
    np.testing.assert_allclose(s[0, :, 0], y[0, -1], rtol=1e-13)


def test_pieces_of_a_sequence():
    p = draw(2, T=9)
    y, s = R.scan_ref(**p)
    cut = lambda a, b: {n: v[:, a:b] if n in ("x", "dt", "Bm", "Cm", "z") else v for n, v in p.items()}  # noqa: E731
    y0, s0 = R.scan_ref(**cut(0, 4))
    y1, s1 = R.scan_ref(**dict(cut(4, 9), s_in=s0))
    np.testing.assert_allclose(np.concatenate((y0, y1), 1), y, rtol=1e-12)
    np.testing.assert_allclose(s1, s, rtol=1e-12)
    w = np.random.default_rng(3).normal(size=(8, 4))
    c, k = R.conv_ref(p["x"], w)
    c0, k0 = R.conv_ref(p["x"][:, :2], w)
    c1, k1 = R.conv_ref(p["x"][:, 2:], w, s_in=k0)
    np.testing.assert_allclose(np.concatenate((c0, c1), 1), c, rtol=1e-12)
    np.testing.assert_array_equal(k1, k)
    np.testing.assert_array_equal(k, p["x"][:, -3:])


def test_conv_by_hand():
    x = np.array([1.0, 2.0, 4.0]).reshape(1, 3, 1)
    y, s = R.conv_ref(x, np.array([[10.0, 1.0]]), bias=[0.5], activation=None, s_in=np.full((1, 1, 1), 3.0))
    assert y.ravel().tolist() == [31.5, 12.5, 24.5] and s.ravel().tolist() == [4.0]
    y, s = R.conv_ref(x, np.array([[10.0, 1.0]]), activation=None, lengths=[1], s_in=np.full((1, 1, 1), 3.0))
    assert y.ravel().tolist() == [31.0, 0.0, 0.0] and s.ravel().tolist() == [1.0]


def differences(f, p, names, got, step=1e-6):
    """The loss's own rounding, a hundred operations of 2^-53 of its size, divided by the step: 1e-8 of the loss.
    (Steps without softplus may be negative: states grow, and the loss is far above its slope.)"""
    for n in names:
        d = np.random.default_rng(len(n)).normal(size=p[n].shape)
        up, down = f({**p, n: p[n] + step * d}), f({**p, n: p[n] - step * d})
        slope, want = (up - down) / (2 * step), float((got[n] * d).sum())
        assert abs(slope - want) <= 1e-6 * max(1.0, abs(want)) + 1e-8 * abs(up), (n, slope, want)


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("lengths", [None, [6, 3]])
def test_scan_gradients_are_differences(softplus, lengths):
    p = draw(4)
    r = np.random.default_rng(5)
    dy, ds = r.normal(size=p["x"].shape), r.normal(size=p["s_in"].shape)

    def loss(q):
        y, s = R.scan_ref(**q, softplus=softplus, lengths=lengths)
        return float((y * dy).sum() + (s * ds).sum())

    g = R.scan_ref_backward(**p, dy=dy, ds_out=ds, softplus=softplus, lengths=lengths)
    g["Bm"], g["Cm"] = g["B"], g["C"]
    differences(loss, p, list(p), g)
    g["A"] = 2 * g["A"]   # a planted mistake
    with pytest.raises(AssertionError):
        differences(loss, p, ["A"], g)


@pytest.mark.parametrize("activation", [None, "silu"])
@pytest.mark.parametrize("lengths", [None, [5, 1], [0, 5]])
def test_conv_gradients_are_differences(activation, lengths):
    r = np.random.default_rng(6)
    p = {"x": r.normal(size=(2, 5, 3)), "weight": r.normal(size=(3, 4)), "bias": r.normal(size=3),
         "s_in": r.normal(size=(2, 3, 3))}
    dy, ds = r.normal(size=(2, 5, 3)), r.normal(size=(2, 3, 3))

    def loss(q):
        y, s = R.conv_ref(**q, activation=activation, lengths=lengths)
        return float((y * dy).sum() + (s * ds).sum())

    differences(loss, p, list(p), R.conv_ref_backward(**p, dy=dy, ds_out=ds, activation=activation, lengths=lengths))


@pytest.mark.parametrize("activation", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("gates", [1, 2, 6])
def test_block_norm_gradients_are_differences(activation, gates):
    r = np.random.default_rng(7)
    p = {"x": r.normal(size=(6, 5)), "residual": r.normal(size=(6, 5)), "gate": r.normal(size=(gates, 5)),
         "post": r.normal(size=5), "pre": r.normal(size=5)}
    dy, dh = r.normal(size=(6, 5)), r.normal(size=(6, 5))

    def loss(q):
        q = dict(q)
        pre = q.pop("pre")
        h = R.block_h_ref(**q, scale=0.5, activation=activation, eps=1e-3)
        return float((R.block_norm_ref(h, pre, 1e-3) * dy).sum() + (h * dh).sum())

    h = R.block_h_ref(**{n: v for n, v in p.items() if n != "pre"}, scale=0.5, activation=activation, eps=1e-3)
    g = R.block_norm_ref_backward(p["x"], h, dy, dh, p["gate"], p["post"], p["pre"], 0.5, activation, 1e-3)
    g["post"], g["pre"] = g["post_weight"], g["pre_weight"]
    differences(loss, p, list(p), g)


def test_block_norm_by_hand():
    h = R.block_h_ref(np.array([[3.0, 4.0]]), residual=np.array([[1.0, 1.0]]), gate=np.array([[2.0, 0.0]]), scale=0.5)
    assert h.tolist() == [[4.0, 1.0]]
    n = R.block_norm_ref(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0)
    np.testing.assert_allclose(n, np.array([[3.0, 8.0]]) / np.sqrt(12.5), rtol=1e-15)
