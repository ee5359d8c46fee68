"""The fp64 definitions of the operators on 4-bit weights: against plain loops, and
each gradient against central differences of its own forward (CPU)."""
import numpy as np
import pytest

from minimax_scale_search_b200 import synth
from oracle import gptq, w4


def _layer(R, K, seed):
    qw, qz, _, gi = synth.make_gptq_tensors(R, K, seed=seed)
    s = np.random.default_rng(seed).uniform(0.01, 0.05, (K // 128, R)).astype(np.float16).view(np.uint16)
    return (qw, qz, s, gi), w4.layer(qw, qz, s)


def test_layer_is_the_dequantised_weight():
    (qw, qz, s, gi), (n, sc) = _layer(24, 384, 3)
    assert np.array_equal(w4.weight(n, sc), gptq.dequantize_v1(qw, qz, s, gi))
    assert n.min() >= -16 and n.max() <= 14


@pytest.mark.parametrize("act", w4.ACTIVATIONS)
def test_slopes_are_the_activations_derivatives(act):
    z = np.concatenate([np.linspace(-9, 9, 181) + 0.013, [30.0, -30.0]])  # no point at relu's corner
    h = 1e-5
    d = (w4.activation(z + h, act) - w4.activation(z - h, act)) / (2 * h)
    # central differences: h^2/6 |f'''| (f''' < 3 here) + rounding 2^-53 |f| / h, |f| <= 30
    assert np.max(np.abs(d - w4.slope(z, act))) < 0.5 * 3 * h * h + 30 * 2.0 ** -52 / h


@pytest.mark.parametrize("act", ["gelu", "silu", "gelu_tanh"])
def test_layer_gradients_are_differences(act):
    rng = np.random.default_rng(5)
    _, (n, s) = _layer(8, 256, 5)
    x, b, c = rng.normal(size=(3, 256)), rng.normal(size=8), rng.normal(size=(3, 8))

    def loss(x, s, b):
        return float((c * w4.linear(x, n, s, b, act)[0]).sum())

    pre = w4.linear(x, n, s, b, act)[1]
    dz, db = w4.activation_backward(c, pre, act)
    dx, ds = w4.linear_backward(dz, x, n, s)
    h = 1e-6
    for (arr, grad) in ((x, dx), (s, ds.T), (b, db)):
        flat = arr.reshape(-1)
        for i in rng.choice(flat.size, min(12, flat.size), replace=False):
            keep = flat[i]
            flat[i] = keep + h
            up = loss(x, s, b)
            flat[i] = keep - h
            down = loss(x, s, b)
            flat[i] = keep
            g = grad.reshape(-1)[i]
            # z moves by up to h * |dz/dp| (< 300 for a scale): third-order term and rounding of the loss
            assert abs((up - down) / (2 * h) - g) < 1e-4 * (1 + np.abs(grad).max()), (arr.shape, i)


def test_table_gradient_is_a_difference_and_skips_other_ids():
    rng = np.random.default_rng(6)
    scales, codes = synth.make_codes(5 * 2, seed=6)
    q, _ = w4.table(scales, codes, 256)
    s = rng.uniform(0.01, 0.1, (5, 2))
    ids = [3, -1, 0, 3, 9, 3]
    d = rng.normal(size=(6, 256))
    out = w4.embedding(ids, q, s, 4.0)
    assert not out[1].any() and not out[4].any() and np.array_equal(out[0], out[3])
    g = w4.embedding_backward(d, ids, q, 4.0)
    assert not g[[1, 2, 4]].any()
    for v in range(5):
        for j in range(2):
            up = s.copy()
            up[v, j] += 1.0  # linear in the scales: a difference is the derivative
            diff = ((w4.embedding(ids, q, up, 4.0) - out) * d).sum()
            assert abs(diff - g[v, j]) < 1e-9 * (1 + np.abs(g).max())
