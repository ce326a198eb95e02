"""Pins of the fp64 restatement of the node-level operators (oracle/layers.py):
gradients against differences, norms against their definition, rotations
against the block norm."""
import numpy as np
import pytest

from oracle import layers as ol


def test_embedding_gradient_is_the_adjoint():
    rng = np.random.default_rng(1)
    ids = rng.integers(-1, 6, 40)
    T, gy = rng.standard_normal((5, 7)), rng.standard_normal((40, 7))
    lhs = (ol.embedding(ids, T, 1.7) * gy).sum()
    assert np.isclose(lhs, (T * ol.embedding_grad(ids, gy, 5, 1.7)).sum(), rtol=1e-13)
    d = ol.embedding_grad(ids, gy, 5, 1.7, padding=3)
    assert not d[3].any() and np.array_equal(np.delete(d, 3, 0), np.delete(ol.embedding_grad(ids, gy, 5, 1.7), 3, 0))


@pytest.mark.parametrize("kind", ["none", "sigmoid", "silu", "tanh"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
def test_block_norm_gradient_matches_differences(kind, post, pre):
    rng = np.random.default_rng(2)
    N, L, C, eps, scale = 3, 2, 4, 1e-3, 0.6
    if not post:
        kind = "none"
    x, gx, gh = (rng.standard_normal((N, 9, C)) for _ in range(3))
    b = rng.standard_normal((N, 9, C)) if post else None
    gate = rng.standard_normal((N, L + 1, C)) if post and kind != "none" else None
    wo = rng.standard_normal((L + 1, C)) if post else None
    wi = rng.standard_normal((L + 1, C)) if pre else None
    gx = gx if post else None
    gh = gh if pre else None

    def value(args):
        y, h = ol.block_norm(*args, scale, eps, kind)
        return (0.0 if gx is None else (y * gx).sum()) + (0.0 if gh is None else (h * gh).sum())

    args = [x, b, gate, wo, wi]
    grads = ol.block_norm_grad(*args, gx, gh, scale, eps, kind)
    step = 1e-6
    for k, (a, g) in enumerate(zip(args, grads)):
        assert (a is None) == (g is None)
        if a is None:
            continue
        for i in rng.choice(a.size, 12, replace=False):
            hi, lo = a.copy(), a.copy()
            hi.flat[i] += step
            lo.flat[i] -= step
            d = (value(args[:k] + [hi] + args[k + 1:]) - value(args[:k] + [lo] + args[k + 1:])) / (2 * step)
            # central differences: step^2 f''' / 6 and rounding 1e-16 |f| / step, |f| < 100
            assert abs(d - g.flat[i]) < 1e-7


def test_block_norm_commutes_with_rotations():
    """Rotating the l = 1 rows of x and b rotates x_out and h."""
    rng = np.random.default_rng(3)
    Q = np.linalg.qr(rng.standard_normal((3, 3)))[0]
    x, b = rng.standard_normal((2, 5, 4, 6))
    gate, wo, wi = rng.standard_normal((5, 2, 6)), rng.standard_normal((2, 6)), rng.standard_normal((2, 6))

    def rot(v):
        v = v.copy()
        v[:, 1:4] = np.einsum("ij,njc->nic", Q, v[:, 1:4])
        return v

    for p, q in zip(ol.block_norm(x, b, gate, wo, wi, 0.5, 1e-6, "silu"),
                    ol.block_norm(rot(x), rot(b), gate, wo, wi, 0.5, 1e-6, "silu")):
        assert np.allclose(rot(p), q, atol=1e-13)


def test_clip():
    ts = [np.array([3.0]), np.array([[0.0, 4.0]])]
    n, out = ol.clip(ts, 1.0, eps=1e-6)
    assert n == 5.0 and np.isclose(ol.gradient_norm(out), 1.0, rtol=1e-6)
    assert all(np.array_equal(a, b) for a, b in zip(ol.clip(ts, 10.0)[1], ts))
