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
