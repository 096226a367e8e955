"""The oracle of the model's ends against closed forms and differences."""

import numpy as np
import pytest

from oracle import model, step


def test_embedding_is_a_product_with_one_hot_rows():
    rng = np.random.default_rng(0)
    table, tokens = rng.standard_normal((11, 5)), rng.integers(0, 11, 20)
    hot = np.eye(11)[tokens]
    assert np.allclose(model.embedding(tokens, table, 3.0), 3 * hot @ table, rtol=1e-15)
    dy = rng.standard_normal((20, 5))
    got, size, terms = model.embedding_backward(dy, tokens, 11, 3.0)
    assert np.allclose(got, 3 * hot.T @ dy, rtol=1e-13) and (size >= np.abs(got) - 1e-12).all()
    assert (terms == np.bincount(tokens, minlength=11)).all()


def test_embedding_outside_and_padding():
    table = np.ones((4, 2))
    got = model.embedding([0, -1, 4, 3], table)
    assert np.isnan(got[1]).all() and np.isnan(got[2]).all() and (got[[0, 3]] == 1).all()
    dy = np.ones((5, 2))
    got, _, terms = model.embedding_backward(dy, [0, -1, 4, 3, 3], 4, padding=0)
    assert (got[:3] == 0).all() and (got[3] == 2).all() and terms.tolist() == [0, 0, 0, 2]
    got, _, _ = model.embedding_backward(dy, [0, -1, 4, 3, 3], 4, held=np.full((4, 2), 10.0))
    assert got[:, 0].tolist() == [11, 10, 10, 12]


def test_packed_values_are_within_half_a_scale():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((9, 100)) * np.exp2(rng.integers(-20, 20, (9, 100)))).astype(np.float32)
    codes, scales = model.pack_activations(x)
    assert codes.shape == (9, 100) and scales.shape == (9, 4)
    back = model.unpack_activations(codes, scales)
    step_of = np.exp2(np.repeat(scales.astype(float), 32, axis=1)[:, :100] - 133)
    assert (np.abs(back - x) <= step_of / 2).all()
    for r in range(9):
        for b in range(4):
            top = np.abs(x[r, 32 * b:32 * b + 32].astype(float)).max()
            s = 2.0 ** (float(scales[r, b]) - 133)
            assert 127 * s >= top and 127 * s / 2 < top


@pytest.mark.parametrize("top,e", [(0.0, 1), (127 * 2.0 ** -132, 1), (127.5 * 2.0 ** -132, 2), (127.0, 133), (128.0, 134),
                                   (1.0, 127), (127 / 64, 127), (2.0, 128), (127 * 2.0 ** 121, 254),
                                   (2.0 ** 127 * 1.99, 255), (np.inf, 255), (np.nan, 255), (2.0 ** -149, 1)])
def test_packed_scales(top, e):
    codes, scales = model.pack_activations(np.array([[top, 0.0]]))
    assert scales[0, 0] == e and codes[0, 1] == 0
    back = model.unpack_activations(codes, scales)
    assert np.isnan(back).all() if e == 255 else abs(back[0, 0] - top) <= 2.0 ** (e - 134)


def test_packed_ties_go_to_even():
    codes, _ = model.pack_activations(np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5]]))
    assert codes[0].tolist() == [127, 0, 2, 2, 0, -2, -2]


def test_layer_norm_gradient_holds_for_the_packed_input():
    """The gradient from packed values is the exact one at the unpacked values, whose statistics it is given."""
    rng = np.random.default_rng(2)
    x, dy, h = rng.standard_normal((3, 40)), rng.standard_normal((3, 40)), 1e-6
    x = model.unpack_activations(*model.pack_activations(x))
    _, mean, rstd = step.layer_norm(x)
    dx, _, _ = step.layer_norm_backward(dy, x, None, mean, rstd)
    for at in [(0, 0), (1, 39), (2, 7)]:
        d = np.zeros_like(x)
        d[at] = h
        slope = ((step.layer_norm(x + d)[0] - step.layer_norm(x - d)[0]) * dy).sum() / (2 * h)
        # the difference's own rounding: 2^-52 of terms of order one over 2h, and its h^2 term
        assert abs(slope - dx[at]) < 1e-8


def test_cross_entropy_of_known_logits():
    x = np.array([[1.0, 0.0], [0.0, 0.0], [0.0, 2.0]])
    w = np.array([[np.log(3.0), 0.0], [0.0, 1.0], [0.0, 1.0]])
    loss, lse = model.cross_entropy(x, w, [0, 1, -100])
    assert np.allclose(lse, [np.log(5), np.log(3), np.log(1 + 2 * np.e ** 2)])
    assert np.allclose(loss, [np.log(5 / 3), np.log(3), 0])
    assert np.isnan(model.cross_entropy(x, w, [3, -1, 0])[0][:2]).all()


def test_cross_entropy_gradient_against_differences():
    rng = np.random.default_rng(3)
    x, w, t = rng.standard_normal((5, 4)), rng.standard_normal((7, 4)), [0, 6, -100, 3, 3]
    g, h = rng.standard_normal(5), 1e-6
    lse = model.cross_entropy(x, w, t)[1]
    dx, dw, dz = model.cross_entropy_backward(g, x, w, t, lse)
    assert (dx[2] == 0).all() and np.allclose(dz.sum(1), 0)

    def value(x, w):
        return (g * model.cross_entropy(x, w, t)[0]).sum()

    for at in [(0, 0), (1, 3), (2, 1), (4, 2)]:
        d = np.zeros_like(x)
        d[at] = h
        assert abs((value(x + d, w) - value(x - d, w)) / (2 * h) - dx[at]) < 1e-8
    for at in [(0, 0), (6, 1), (3, 3), (2, 2)]:
        d = np.zeros_like(w)
        d[at] = h
        assert abs((value(x, w + d) - value(x, w - d)) / (2 * h) - dw[at]) < 1e-8


def test_cross_entropy_rows_that_take_no_part():
    x = np.array([[1.0, 2.0], [np.nan, np.inf], [3.0, 1.0]])
    w = np.ones((3, 2))
    dx, dw, _ = model.cross_entropy_backward([1.0, 5.0, 0.0], x, w, [1, -100, 2], [3 + np.log(3), 0, 0])
    assert np.isfinite(dw).all() and (dx[1:] == 0).all() and np.isfinite(dx[0]).all()
