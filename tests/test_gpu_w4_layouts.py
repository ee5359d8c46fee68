"""Operands that lie beside each other in one buffer: the operators on 4-bit weights give what
they give on operands in memory of their own, and write nothing else."""
import numpy as np
import pytest

from minimax_scale_search_b200 import synth

pytestmark = pytest.mark.gpu

R = K = 256


def layer(seed):
    import torch
    from minimax_scale_search_b200 import cq
    qw, qz, _, gi = synth.make_gptq_tensors(R, K, seed=seed)
    s = (0.02 * np.random.default_rng(seed).lognormal(0, 0.5, (K // 128, R))).astype(np.float16)
    on = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int32)).cuda()  # noqa: E731
    return cq.w4_weights(cq.GPTQTensors(on(qw), on(qz), torch.from_numpy(s).cuda(), on(gi)))


@pytest.mark.parametrize("dt", ["bfloat16", "float16"])
@pytest.mark.parametrize("T", [1, 7, 16, 33, 300])
@pytest.mark.parametrize("step", [1, 2])
def test_columns_of_one_buffer(T, dt, step):
    import torch
    from minimax_scale_search_b200 import cq
    torch.manual_seed(T)
    w = layer(T)
    first = torch.randn((T * step, 5 * R), device="cuda").to(getattr(torch, dt))
    buf = first.clone()
    a, b, c, d, e = (buf[::step, i * R:(i + 1) * R] for i in range(5))
    x, res = a.contiguous(), b.contiguous()
    y, pre = cq.w4_linear(x, w, activation="silu", residual=res, want_pre=True)
    cq.w4_linear(a, w, activation="silu", residual=b, want_pre=True, pre=c, out=d)
    assert torch.equal(c, pre) and torch.equal(d, y)
    dz, db = cq.activation_backward(y, pre, "silu")
    assert torch.equal(cq.activation_backward(d, c, "silu", out=e)[1], db) and torch.equal(e, dz)
    dx, ds = cq.w4_linear_backward(dz, x, w)
    assert torch.equal(cq.w4_linear_backward(e, a, w, dx=d)[1], ds) and torch.equal(d, dx)
    # the inputs' columns and, where every other row was used, the rows between
    assert torch.equal(buf[:, :2 * R], first[:, :2 * R])
    if step == 2:
        assert torch.equal(buf[1::2], first[1::2])
    assert cq.w4_status() == cq.CQ_OK
