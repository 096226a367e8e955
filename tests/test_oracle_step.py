"""The training-step oracle against the mathematics: the gradient norm, AdamW,
the packed states' format and rounding, layer norm's gradient against
differences."""

import math

import numpy as np
import pytest

from oracle import step


def test_grad_norm_values():
    assert step.grad_norm([]) == 0.0
    assert step.grad_norm([[3.0], [4.0]]) == 5.0
    assert step.grad_norm([np.full(4, 1e300)]) == pytest.approx(2e300, rel=1e-15)
    assert math.isnan(step.grad_norm([[1.0, math.nan, math.inf]]))
    assert step.grad_norm([[1.0, -math.inf]]) == math.inf


def test_first_step_moves_by_lr_against_the_sign():
    """With zero states the first step's update is lr * g / (|g| + eps)."""
    g = np.array([1e-3, -2.0, 5e4])
    p, m, v = step.adamw(np.ones(3), g, np.zeros(3), np.zeros(3), step=1, lr=0.1, eps=0.0)
    assert np.allclose(p, 1 - 0.1 * np.sign(g), rtol=0, atol=1e-15)
    assert np.allclose(m, 0.1 * g) and np.allclose(v, 0.001 * g * g)


def test_constant_gradient_states_have_closed_forms():
    p, m, v = np.zeros(1), np.zeros(1), np.zeros(1)
    for t in range(1, 51):
        p, m, v = step.adamw(p, [0.25], m, v, step=t, lr=0.0)
    assert m[0] == pytest.approx(0.25 * (1 - 0.9 ** 50), rel=1e-13)
    assert v[0] == pytest.approx(0.0625 * (1 - 0.999 ** 50), rel=1e-13)


def test_weight_decay_is_decoupled():
    p, _, _ = step.adamw([2.0], [0.0], [0.0], [0.0], step=1, lr=0.1, weight_decay=0.5, eps=1e-8)
    assert p[0] == pytest.approx(2.0 * (1 - 0.05), rel=1e-15)


def test_clip_factor():
    assert step.factor_f32(10.0, 1.0) == np.float32(1) / (np.float32(10) + np.float32(1e-6))
    assert step.factor_f32(0.1, 1.0) == 1
    assert step.factor_f32(8.0, 1.0, 0.25) == np.float32(0.25) * (np.float32(1) / np.float32(2.000001))
    assert np.isnan(step.factor_f32(math.nan, 1.0))


@pytest.mark.parametrize("kind", ["exp_avg", "exp_avg_sq"])
def test_codes_are_ordered_and_distinct(kind):
    v = step.code_values(kind)
    up = v[:128] if kind == "exp_avg" else v
    assert (np.diff(up) > 0).all() and up[0] == 0
    assert up[-1] == 1.875
    if kind == "exp_avg":
        assert (v[128:] == -up).all()
    # neighbours are at most an eighth apart once the exponent is not the smallest
    assert (np.diff(up[8:]) / up[8:-1]).max() <= 0.125


@pytest.mark.parametrize("kind", ["exp_avg", "exp_avg_sq"])
@pytest.mark.parametrize("e", [1, 2, 100, 127, 200, 254])
def test_every_code_round_trips(kind, e):
    """A value that a code stands for comes back as that code, whatever the noise."""
    values = step.code_values(kind)
    codes = np.arange(256, dtype=np.uint8)
    if kind == "exp_avg":
        codes[128] = 0           # the code of -0 is +0's but for its sign
    x = values[codes] * 2.0 ** (e - 127)
    x32 = x.astype(np.float32)
    exact = x32.astype(np.float64) == x      # e = 1 reaches below float32's subnormals
    for seed in (0, 1, 2):
        got, scales = step.pack(x32, step.random_bits(seed, 0, 256), kind)
        assert scales.tolist() == [e]
        assert (got == codes)[exact].all()
    assert exact.all() or e < 3


@pytest.mark.parametrize("kind", ["exp_avg", "exp_avg_sq"])
def test_rounding_goes_to_a_neighbour_and_is_unbiased(kind):
    rng = np.random.default_rng(5)
    x = (rng.standard_normal(STATE := 256) * 10.0 ** rng.uniform(-4, 0, 256)).astype(np.float32)
    x = np.abs(x) if kind == "exp_avg_sq" else x
    total, seeds = np.zeros(STATE), 400
    for seed in range(seeds):
        codes, scales = step.pack(x, step.random_bits(seed, 3, STATE), kind)
        got = step.unpack(codes, scales, kind)
        scale = 2.0 ** (int(scales[0]) - 127)
        gap = np.maximum(np.abs(x) / 8, scale * 2.0 ** (-17 if kind == "exp_avg" else -33))
        assert (np.abs(got - x) <= gap).all()
        total += got
    # a mean of `seeds` roundings, each off by at most a gap: six standard deviations of half a gap
    assert (np.abs(total / seeds - x) <= 6 * 0.5 * gap / math.sqrt(seeds) + 1e-12).all()


def test_positive_second_moments_never_vanish():
    x = np.zeros(256, np.float32)
    x[0], x[1], x[2] = 1.0, 1e-30, 0.0
    for seed in range(20):
        codes, scales = step.pack(x, step.random_bits(seed, 0, 256), "exp_avg_sq")
        assert codes[1] == 1 and codes[2] == 0


def test_blocks_without_a_finite_value_are_nan():
    for bad in (math.nan, math.inf, -math.inf, 3.3e38):
        x = np.ones(300, np.float32)
        x[299] = bad
        codes, scales = step.pack(x, step.random_bits(0, 0, 300), "exp_avg")
        assert scales[0] == 127 and scales[1] == 255
        got = step.unpack(codes, scales, "exp_avg")
        assert np.isfinite(got[:256]).all() and np.isnan(got[256:]).all()


def test_random_bits_are_spread():
    bits = step.random_bits(7, 2, 1 << 16)
    for k in range(32):
        assert abs(((bits >> np.uint64(k)) & np.uint64(1)).mean() - 0.5) < 6 * 0.5 / 256
    a, b = step.random_bits(7, 3, 1 << 12), step.random_bits(8, 2, 1 << 12)
    assert (a != bits[:1 << 12]).mean() > 0.99 and (b != bits[:1 << 12]).mean() > 0.99


def test_layer_norm_rows_have_mean_beta_and_unit_scale():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((7, 33)) * 3 + 5
    y, mean, rstd = step.layer_norm(x, eps=0.0)
    assert np.allclose(y.mean(1), 0, atol=1e-14) and np.allclose((y * y).mean(1), 1)
    assert np.allclose(mean, x.mean(1)) and np.allclose(1 / rstd ** 2, x.var(1))


@pytest.mark.parametrize("affine", [True, False])
def test_layer_norm_gradient_against_differences(affine):
    """Every partial derivative of sum(dy * y) by central differences, statistics included."""
    rng = np.random.default_rng(2)
    rows, cols, eps = 3, 6, 1e-3
    x, dy = rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols))
    gamma = rng.standard_normal(cols) if affine else None
    beta = rng.standard_normal(cols) if affine else None
    _, mean, rstd = step.layer_norm(x, gamma, beta, eps)
    dx, dgamma, dbeta = step.layer_norm_backward(dy, x, gamma, mean, rstd)

    def loss(x, gamma, beta):
        return float((dy * step.layer_norm(x, gamma, beta, eps)[0]).sum())

    def slope(array, at, **kw):
        h, vals = 1e-6, []
        for s in (h, -h):
            moved = array.copy()
            moved[at] += s
            vals.append(loss(**{**dict(x=x, gamma=gamma, beta=beta), **{kw["name"]: moved}}))
        return (vals[0] - vals[1]) / (2 * h)

    for at in np.ndindex(rows, cols):
        assert slope(x, at, name="x") == pytest.approx(dx[at], abs=1e-7)
    if affine:
        for c in range(cols):
            assert slope(gamma, c, name="gamma") == pytest.approx(dgamma[c], abs=1e-7)
            assert slope(beta, c, name="beta") == pytest.approx(dbeta[c], abs=1e-7)


@pytest.mark.parametrize("kind", ["exp_avg", "exp_avg_sq"])
@pytest.mark.parametrize("e", [1, 2, 5, 10, 11, 12, 30])
def test_written_codes_are_exact_in_float32(kind, e):
    """Down to float32's subnormals, whose spacing some codes undercut: a state that was rounded from a float32
    value reads back exactly, and a positive second moment not as 0."""
    rng = np.random.default_rng(e)
    for seed in range(4):
        x = (np.exp2(rng.uniform(-149, e - 127, 256))).astype(np.float32)
        x[0], x[1], x[2] = 1.5 * 2.0 ** (e - 127), 2.0 ** -149, 3 * 2.0 ** -149
        codes, scales = step.pack(x, step.random_bits(seed, 0, 256), kind)
        got = step.unpack(codes, scales, kind)
        assert scales.tolist() == [e]
        assert np.array_equal(got.astype(np.float32).astype(np.float64), got)
        assert (got > 0).all() or kind == "exp_avg"
