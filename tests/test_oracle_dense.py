"""The oracle of the norm and of the 16-bit products: sums written out, and gradients against differences."""
import numpy as np
import pytest

from oracle import dense


def test_norm_by_hand():
    y, r = dense.rms_norm([[3.0, 4.0], [0.0, 0.0]], [1.0, 0.5], 12.5)
    assert np.allclose(r, [0.2, 12.5 ** -0.5], rtol=1e-15) and np.allclose(y[0], [0.6, 0.4], rtol=1e-15)
    assert np.all(y[1] == 0)


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (2, 17)])
def test_norm_gradient_against_differences(rows, cols):
    rng = np.random.default_rng(rows * cols)
    h, w, g, gh = rng.standard_normal((rows, cols)), rng.standard_normal(cols), rng.standard_normal((rows, cols)), \
        rng.standard_normal((rows, cols))
    eps, d = 1e-2, 1e-5

    def loss(h, w):
        return (dense.rms_norm(h, w, eps)[0] * g).sum() + (h * gh).sum()

    gx, gw = dense.rms_norm_backward(g, h, w, dense.rms_norm(h, w, eps)[1], gh)
    # central differences: the third derivative over 6, times d^2, and 1e-16 of the loss over d
    for i in np.ndindex(h.shape):
        e = np.zeros_like(h)
        e[i] = d
        assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * d) - gx[i]) < 1e-7
    for c in range(cols):
        e = np.zeros_like(w)
        e[c] = d
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * d) - gw[c]) < 1e-8


def test_products_by_loops():
    rng = np.random.default_rng(0)
    x, w, g = rng.standard_normal((6, 3)), rng.standard_normal((3, 4, 3)), rng.standard_normal((6, 4))
    off = [1, 3, 3, 5]
    out, mag = dense.grouped_matmul(x, w, off)
    back, _ = dense.grouped_matmul(g, w, off, transpose_w=True)
    gw, _ = dense.grouped_matmul_wgrad(g, x, off)
    assert np.isnan(out[0]).all() and np.isnan(out[5]).all() and np.all(gw[1] == 0)
    want = np.zeros_like(gw)
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        for r in range(lo, hi):
            for j in range(4):
                assert np.isclose(out[r, j], sum(x[r, i] * w[e, j, i] for i in range(3)))
                assert np.isclose(mag[r, j], sum(abs(x[r, i] * w[e, j, i]) for i in range(3)))
                for i in range(3):
                    want[e, j, i] += g[r, j] * x[r, i]
            for i in range(3):
                assert np.isclose(back[r, i], sum(g[r, j] * w[e, j, i] for j in range(4)))
    assert np.allclose(gw, want)


def test_product_gradients_against_differences():
    """The loss sum(out g) is linear in x and in w: differences of any size give the gradients."""
    rng = np.random.default_rng(1)
    x, w, g = rng.standard_normal((5, 2)), rng.standard_normal((2, 3, 2)), rng.standard_normal((5, 3))
    off = [0, 2, 5]
    loss = lambda x, w: (dense.grouped_matmul(x, w, off)[0] * g).sum()  # noqa: E731
    gx, gw = dense.grouped_matmul(g, w, off, transpose_w=True)[0], dense.grouped_matmul_wgrad(g, x, off)[0]
    for a, grad, f in ((x, gx, lambda e: loss(x + e, w)), (w, gw, lambda e: loss(x, w + e))):
        for i in np.ndindex(a.shape):
            e = np.zeros_like(a)
            e[i] = 1.0
            assert np.isclose((f(e) - f(-e)) / 2, grad[i], atol=1e-12)
