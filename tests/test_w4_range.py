"""Layers whose weights pass float16's range, on the CPU: fp16 calls that would round a weight to inf are refused."""
import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def cq():
    from minimax_scale_search_b200 import build
    build.build()
    from minimax_scale_search_b200 import cq as binding
    return binding


class Cuda(torch.Tensor):
    """A host tensor that the binding takes for a CUDA tensor."""
    is_cuda = property(lambda self: True)


R, K = 64, 256


def make(cq, scale, zeros=0x77777777, at=(1, 5)):
    t = lambda v: torch.as_tensor(v).as_subclass(Cuda)  # noqa: E731
    s = torch.full((2, R), 0.01, dtype=torch.float16)
    s[at] = scale
    qzeros = torch.from_numpy(np.full((2, R // 8), zeros, dtype=np.uint32).view(np.int32).copy())
    return cq.w4_weights(cq.GPTQTensors(t(torch.zeros((K // 8, R), dtype=torch.int32)), t(qzeros), t(s),
                                        t(torch.arange(K, dtype=torch.int32) // 128)))


@pytest.fixture
def launches(cq, monkeypatch):
    made = []
    monkeypatch.setattr(cq, "_place", lambda dev, stream: (0, None))
    monkeypatch.setattr(cq, "_call", lambda context, function, *args: made.append(function))
    return made


def operands(T, dtype):
    return (torch.zeros((T, n), dtype=dtype).as_subclass(Cuda) for n in (K, R))


# with a zero point of 7 the weights are scale * (-8 .. 7), with 15 scale * (-16 .. -1), with 0 scale * (-1 .. 14)
@pytest.mark.parametrize("scale,zeros,fits", [(8184.0, 0x77777777, True), (8192.0, 0x77777777, False), (-8192.0, 0x77777777, False),
                                              (4092.0, 0xFFFFFFFF, True), (4096.0, 0xFFFFFFFF, False), (4676.0, 0, True),
                                              (4684.0, 0, False), (float("inf"), 0x77777777, True), (float("nan"), 0, True)])
def test_fp16_products_with_weights_beyond_its_range_are_refused(cq, launches, scale, zeros, fits):
    w = make(cq, scale, zeros)
    x, dz = operands(17, torch.float16)
    if fits:
        cq.w4_linear(x, w)
        cq.w4_linear_backward(dz, x, w)
        assert len(launches) == 2
    else:
        with pytest.raises(ValueError, match="float16's range"):
            cq.w4_linear(x, w)
        with pytest.raises(ValueError, match="float16's range"):
            cq.w4_linear_backward(dz, x, w)
        assert not launches
    # few rows, the scale gradient and bfloat16 have no such limit
    x, dz = operands(16, torch.float16)
    cq.w4_linear(x, w)
    cq.w4_linear_backward(dz, x, w, want_dx=False)
    x, dz = operands(17, torch.bfloat16)
    cq.w4_linear(x, w)
    cq.w4_linear_backward(dz, x, w)
