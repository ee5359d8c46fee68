"""Calls of the layer's operators at the limits of their sizes and without an operand, on the CPU."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)
NONE = ctypes.c_void_p(None)


@pytest.fixture(scope="module")
def cq():
    from minimax_scale_search_b200 import build
    build.build()
    from minimax_scale_search_b200 import cq as binding
    return binding


@pytest.mark.parametrize("R", [(1 << 31) - 8, (1 << 31) - 120])
def test_outputs_whose_last_tile_passes_31_bits_are_refused(cq, R):
    """The last tile of 128 outputs would end at 2^31, which 32-bit tile coordinates do not reach."""
    assert cq.lib.cq_w4_linear_backward(FAKE, R, FAKE, 128, 0, 4, FAKE, FAKE, FAKE, R, 128, FAKE, 128, FAKE, NONE) == \
        cq.CQ_ERR_UNSUPPORTED
    assert cq.lib.cq_w4_linear(FAKE, 128, 0, 40, FAKE, FAKE, FAKE, R, 128, NONE, 0, NONE, 0, FAKE, R, NONE, 0, NONE) == \
        cq.CQ_ERR_UNSUPPORTED


class Cuda(torch.Tensor):
    """A host tensor that the binding takes for a CUDA tensor."""
    is_cuda = property(lambda self: True)


def test_scale_gradient_asks_for_the_input(cq, monkeypatch):
    monkeypatch.setattr(cq, "_place", lambda dev, stream: (0, None))
    monkeypatch.setattr(cq, "_call", lambda *a: pytest.fail("launched"))
    made = lambda *s, dtype=torch.float16: torch.zeros(s, dtype=dtype).as_subclass(Cuda)  # noqa: E731
    w = cq.W4Weights(made(32, 64, dtype=torch.int32), made(2, 8, dtype=torch.int32), made(2, 64), 64, 256)
    dz = made(4, 64)
    for kw in ({}, dict(want_dx=False), dict(dx=made(4, 256))):
        with pytest.raises(ValueError, match="dscales needs x"):
            cq.w4_linear_backward(dz, None, w, **kw)
        with pytest.raises(ValueError, match=r"x must be \[4, 256\]"):
            cq.w4_linear_backward(dz, made(4, 128), w, **kw)


def test_table_of_other_types_is_refused(cq, monkeypatch):
    """Patterns of binary16 and words of codes: bfloat16 scales or float codes would be read as something else."""
    monkeypatch.setattr(cq, "_place", lambda dev, stream: (0, None))
    made = []
    monkeypatch.setattr(cq, "_call", lambda *a: made.append(a))
    new = lambda *s, dtype: torch.zeros(s, dtype=dtype).as_subclass(Cuda)  # noqa: E731
    ids, K, V = new(3, dtype=torch.int64), 256, 5
    for scales in (torch.int16, torch.uint16, torch.float16):
        for codes in (torch.int32, torch.uint32):
            cq.w4_embedding(ids, new(V * 2, dtype=scales), new(V * 2, 16, dtype=codes), K)
            cq.w4_embedding_backward(new(3, K, dtype=torch.float32), ids, new(V * 2, 16, dtype=codes))
    assert len(made) == 12
    with pytest.raises(ValueError, match="scales"):
        cq.w4_embedding(ids, new(V * 2, dtype=torch.bfloat16), new(V * 2, 16, dtype=torch.int32), K)
    with pytest.raises(ValueError, match="codes"):
        cq.w4_embedding(ids, new(V * 2, dtype=torch.float16), new(V * 2, 16, dtype=torch.float32), K)
    with pytest.raises(ValueError, match="codes"):
        cq.w4_embedding_backward(new(3, K, dtype=torch.float32), ids, new(V * 2, 16, dtype=torch.float32))
    assert len(made) == 12


def test_status_is_that_of_the_streams_device(cq, monkeypatch):
    """The report lies on the device of the stream, which need not be the current one."""
    import contextlib
    from types import SimpleNamespace
    current, asked = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(cq, "lib", SimpleNamespace(cq_w4_status=lambda s: asked.append((current[0], s.value)) or 0))
    assert cq.w4_status(SimpleNamespace(device=3, cuda_stream=77)) == cq.CQ_OK
    assert asked == [(3, 77)] and current == [0]
