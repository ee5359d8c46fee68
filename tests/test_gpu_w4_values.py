"""The operators on 4-bit weights at the ends of their types' ranges: every finite
16-bit argument of the activations and of their slopes.

The fp32 arithmetic behind a result of 16 bits is counted as follows, u = 2^-24 a rounding:
exp(x) by the fast instruction is within (2 + 1.173 |x|) 2^-23 of its value (the CUDA guide's bound), its
argument's own roundings, five at most, add 5 |x| u; a quotient with a divisor between 1 and 2 adds 2^-22, the
ratio of Mills 2^-22 and its evaluation 2^-21 (eight steps, terms of at most twice the result), the few products after them 2^-22.  Values below
2^-126 carry 2^-149 of absolute error, times factors of at most 300."""
import math

import numpy as np
import pytest

from minimax_scale_search_b200 import synth  # noqa: F401  (the package, before any GPU work)

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -134 + 2.0 ** -140, "fp16": 2.0 ** -25}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
C = math.sqrt(2 / math.pi)


def every_finite(dt):
    """[T, 128] of every finite value of the type, T = 510 or 496."""
    import torch
    bits = np.arange(1 << 16, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view({"bf16": torch.bfloat16, "fp16": torch.float16}[dt])
    return x[torch.isfinite(x.float())].view(-1, 128).cuda()


def f64(t):
    return t.double().cpu().numpy()


def sigmoid(a):
    """(p, 1 - p), each to its own last digits."""
    e = np.exp(-np.minimum(np.abs(a), 1000.0))
    big, small = 1 / (1 + e), e / (1 + e)
    return np.where(a < 0, small, big), np.where(a < 0, big, small)


def parts(z, act):
    """The argument of the activation's exponential, the activation, and the two terms of its slope."""
    if act == "none":
        return 0 * z, z, 0 * z + 1, 0 * z
    if act == "relu":
        return 0 * z, np.maximum(z, 0), (z > 0).astype(np.float64), 0 * z
    if act == "gelu":
        p = 0.5 * np.vectorize(math.erfc, otypes=[np.float64])(-z / math.sqrt(2))
        a = -np.minimum(z * z / 2, 1000.0)
        return a, z * p, p, z * np.exp(a) / math.sqrt(2 * math.pi)
    a = z if act == "silu" else 2 * C * (z + 0.044715 * z ** 3)
    p, q = sigmoid(a)
    return a, z * p, p, z * p * q * (1.0 if act == "silu" else 2 * C * (1 + 3 * 0.044715 * z * z))


def arithmetic(a):
    """Relative error of the fp32 arithmetic around exp(a); beyond 110 the exponential has left fp32."""
    a = np.minimum(np.abs(a), 110.0)
    return (2 + 1.173 * a) * 2.0 ** -23 + 5 * a * 2.0 ** -24 + 2.0 ** -20


def identity():
    """A layer of 128 x 128 whose weights are 1 on the diagonal and 0 beside it."""
    import torch
    from minimax_scale_search_b200 import cq
    u = np.full((128, 128), 8, dtype=np.uint32)
    np.fill_diagonal(u, 9)
    words = np.zeros((16, 128), dtype=np.uint32)
    for j in range(8):
        words |= u[:, j::8].T << np.uint32(4 * j)
    return cq.w4_weights(cq.GPTQTensors(torch.from_numpy(words.view(np.int32)).cuda(),
                                        torch.full((1, 16), 0x77777777, dtype=torch.int32, device="cuda"),
                                        torch.ones((1, 128), dtype=torch.float16, device="cuda"),
                                        torch.zeros(128, dtype=torch.int32, device="cuda")))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ACTIVATIONS)
@pytest.mark.parametrize("rows", [8, 510])
def test_activation_of_every_finite_value(act, dt, rows):
    """Through the few-row kernel and through the tensor-core kernel; small results of large negative arguments keep
    their digits down to the type's smallest."""
    from minimax_scale_search_b200 import cq
    import torch
    x, w = every_finite(dt), identity()
    got = [cq.w4_linear(x[i:i + rows], w, activation=act, want_pre=True) for i in range(0, x.shape[0], rows)]
    y, pre = (torch.cat([g[k] for g in got]) for k in (0, 1))
    z = f64(x)
    assert np.array_equal(f64(pre), z)  # one product with 1 and 127 with 0
    a, e, _, _ = parts(z, act)
    assert np.all(np.abs(f64(y) - e) <= (U[dt] + arithmetic(a)) * np.abs(e) + TINY[dt])


def check_slopes(act, dt, keep):
    import torch
    from minimax_scale_search_b200 import cq
    pre = torch.where(keep(every_finite(dt)), every_finite(dt), 0)
    dz, db = cq.activation_backward(torch.ones_like(pre), pre, act)
    a, _, p, q = parts(f64(pre), act)
    off = arithmetic(a) * (np.abs(p) + np.abs(q))  # before the result's rounding
    assert np.all(np.abs(f64(dz) - (p + q)) <= U[dt] * np.abs(p + q) + off + TINY[dt])
    sums = (pre.shape[0] + 8) * 2.0 ** -24 * np.abs(p + q).sum(0)
    assert np.all(np.abs(f64(db) - (p + q).sum(0)) <= off.sum(0) + sums + pre.shape[0] * 2.0 ** -140)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ACTIVATIONS)
def test_slope_of_every_value_up_to_1e19(act, dt):
    check_slopes(act, dt, lambda z: z.float().abs() <= 1e19)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ACTIVATIONS)
def test_slope_of_every_finite_value(act, dt):
    """Beyond 1.8e19 the argument's square leaves fp32; the slope there is 0 or 1."""
    check_slopes(act, dt, lambda z: z == z)


@pytest.mark.parametrize("act", ACTIVATIONS)
def test_slope_of_what_is_not_finite(act):
    """inf and NaN as the formulas have them: relu's slope is a comparison, the others multiply."""
    import torch
    from minimax_scale_search_b200 import cq
    z = torch.tensor([[math.nan, math.inf, -math.inf, 0.0] * 2], dtype=torch.bfloat16, device="cuda")
    got = cq.activation_backward(torch.ones_like(z), z, act)[0][0, :3].float().tolist()
    if act == "none":
        assert got == [1, 1, 1]
    elif act == "relu":
        assert got == [0, 1, 0]
    else:
        assert all(math.isnan(v) for v in got)


def layer_of(u, scale, R=8, K=256):
    """A layer whose every code is u with a zero point of 8 (weights scale * (u - 8)), its scales all `scale`."""
    import torch
    from minimax_scale_search_b200 import cq
    word = int(np.array([u * 0x11111111], dtype=np.uint32).view(np.int32)[0])
    full = lambda *s, v: torch.full(s, v, dtype=torch.int32, device="cuda")  # noqa: E731
    return cq.w4_weights(cq.GPTQTensors(full(K // 8, R, v=word), full(K // 128, R // 8, v=0x77777777),
                                        torch.full((K // 128, R), scale, dtype=torch.float16, device="cuda"),
                                        torch.arange(K, dtype=torch.int32, device="cuda") // 128))


@pytest.mark.parametrize("T", [1, 13, 40])
def test_large_inputs_with_small_scales(T):
    """Inputs whose sums with the integer codes alone would leave fp32 (128 x 7 x 2^120), where the result does not."""
    import torch
    from minimax_scale_search_b200 import cq
    x = torch.full((T, 256), 2.0 ** 120, dtype=torch.bfloat16, device="cuda")
    x[:, 1::2] *= 0.75
    got = f64(cq.w4_linear(x, layer_of(15, 2.0 ** -14)))
    assert np.all(got == 256 * 7 * 0.875 * 2.0 ** 120 * 2.0 ** -14)  # 7 x 7 x 2^k: exact


@pytest.mark.parametrize("T", [1, 13, 40])
@pytest.mark.parametrize("power", [-126, -130, -133])
def test_smallest_inputs(T, power):
    """Inputs down to bfloat16's smallest value keep their digits: each sum below is 7 x 2^k, a bfloat16 value."""
    import torch
    from minimax_scale_search_b200 import cq
    x = torch.full((T, 256), 2.0 ** power, dtype=torch.bfloat16, device="cuda")
    got = f64(cq.w4_linear(x, layer_of(15, 1.0)))
    assert np.all(got == 256 * 7 * 2.0 ** power)
    one = torch.zeros_like(x)
    one[:, 37] = 2.0 ** power
    assert np.all(f64(cq.w4_linear(one, layer_of(15, 1.0))) == 7 * 2.0 ** power)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 13, 40])
def test_infinite_and_missing_scales(T, dt):
    """Infinite weights of one sign times positive inputs are infinite, not NaN; a scale of NaN is NaN; neither
    leaves its output (layer) or its group's inputs (input gradient)."""
    import torch
    from minimax_scale_search_b200 import cq
    torch_dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dt]
    w = layer_of(9, 0.5, R=16, K=384)
    w.scales[1, 3], w.scales[1, 5], w.scales[2, 8] = math.inf, -math.inf, math.nan
    y = cq.w4_linear(torch.ones((T, 384), dtype=torch_dt, device="cuda"), w).float()
    expect = torch.full((T, 16), 192.0, device="cuda")
    expect[:, 3], expect[:, 5], expect[:, 8] = math.inf, -math.inf, math.nan
    assert torch.equal(y.nan_to_num(7.0), expect.nan_to_num(7.0))
    dz = torch.ones((T, 16), dtype=torch_dt, device="cuda")
    dz[:, 5] = 2.0
    w.scales[1, 5] = 0.5
    dx = cq.w4_linear_backward(dz, None, w, want_dscales=False)[0].float()
    assert bool((dx[:, :128] == 8.5).all() and torch.isposinf(dx[:, 128:256]).all() and torch.isnan(dx[:, 256:]).all())
