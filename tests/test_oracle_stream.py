"""The oracle's residual norm and sorted rows: closed forms, and gradients
against differences."""
import numpy as np

from oracle import stream as S


def test_norm_closed_forms():
    g = np.random.default_rng(0)
    s = g.standard_normal((5, 12)) * 3
    y, rstd = S.norm_forward(s, np.ones(12), 1e-12)
    assert np.allclose((y ** 2).mean(1), 1, rtol=1e-11)
    y, rstd = S.norm_forward(np.zeros((2, 4)), np.ones(4), 0.25)
    assert (y == 0).all() and (rstd == 2).all()


def test_norm_gradient_is_the_difference_quotient():
    g = np.random.default_rng(1)
    s, w, dy, d_next = g.standard_normal((4, 9)), g.standard_normal(9), g.standard_normal((4, 9)), g.standard_normal((4, 9))
    eps = 0.3

    def value(s, w):
        return (S.norm_forward(s, w, eps)[0] * dy).sum() + (s * d_next).sum()

    rstd = S.norm_forward(s, w, eps)[1]
    d, dw = S.norm_backward(dy, s, w, rstd, d_next)
    h = 1e-6
    for a, grad in ((s, d), (w, dw)):
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = value(s, w)
            a[i] = keep - h
            down = value(s, w)
            a[i] = keep
            assert abs((up - down) / (2 * h) - grad[i]) <= 1e-8


def test_rows_there_and_back():
    g = np.random.default_rng(2)
    T, k, c, M = 6, 3, 5, 14
    pos = np.full(T * k, -1)
    pos[g.permutation(T * k)[:M]] = g.permutation(M)
    pos = pos.reshape(T, k)
    x, y, w, d = g.standard_normal((T, c)), g.standard_normal((M, c)), g.random((T, k)), g.standard_normal((T, c))
    rows = S.sort_rows(x, pos, np.full((M, c), np.nan))
    assert not np.isnan(rows).any()
    # the weights of a token summed over its local slots come back with its row
    back = S.combine_rows(rows, pos, w)
    assert np.allclose(back, x * np.where(pos >= 0, w, 0).sum(1)[:, None], rtol=1e-14)
    dy, dw = S.combine_rows_backward(d, y, pos, w, np.full((M, c), np.nan))
    h = 1e-6
    value = lambda y, w: (S.combine_rows(y, pos, w) * d).sum()  # noqa: E731
    for a, grad in ((y, dy), (w, dw)):
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = value(y, w)
            a[i] = keep - h
            down = value(y, w)
            a[i] = keep
            assert abs((up - down) / (2 * h) - grad[i]) <= 1e-8
    # the sort's gradient: its transpose
    u = g.standard_normal((M, c))
    assert np.isclose((rows * u).sum(), (x * S.combine_rows(u, pos, None)).sum(), rtol=1e-13)
