"""Which operands' memory may overlap, on the CPU: the binding's own check against the sets
of bytes that two operands have, and each operator's refusals, with the launch
itself replaced (host tensors that say they are CUDA tensors)."""
import itertools

import pytest
import torch


@pytest.fixture(scope="module")
def cq():
    from minimax_scale_search_b200 import build
    build.build()
    from minimax_scale_search_b200 import cq as binding
    return binding


def bytes_of(t):
    at = torch.zeros(t.shape, dtype=torch.int64)
    for d, (n, s) in enumerate(zip(t.shape, t.stride())):
        at += (torch.arange(n) * s).view([-1 if i == d else 1 for i in range(t.dim())])
    at = t.data_ptr() + at.reshape(-1) * t.element_size()
    return set((at[:, None] + torch.arange(t.element_size())).reshape(-1).tolist())


def test_overlap_is_that_of_the_bytes(cq):
    """Slices of one buffer: whole, by columns, by rows, every other row, of one row, of other widths and types."""
    buf = torch.zeros(40 * 24, dtype=torch.float16)
    wide, narrow = buf.view(40, 24), buf[8:8 + 44 * 16].view(44, 16)
    views = [buf, buf[100:100], buf[:100], buf[90:200], buf[23:24], wide[3:9], wide[8:20], wide[20:21],
             buf[:480].view(torch.float32), buf[480:520].view(torch.float32), narrow[::3, :8], narrow[1::3, 8:], narrow[5:6, 3:9]]
    views += [wide[r0:r1:step, c0:c1] for r0, r1 in ((0, 40), (0, 4), (4, 8), (5, 6)) for step in (1, 2, 3)
              for c0, c1 in ((0, 8), (8, 24), (4, 12), (0, 24), (23, 24))]
    views += [buf[16 + k:16 + k + 30 * 24].view(30, 24)[:, :w] for k in (0, 8, 16, 23) for w in (1, 8, 9, 16)]  # rows that wrap around
    sets = [bytes_of(v) for v in views]
    for (a, sa), (b, sb) in itertools.product(zip(views, sets), repeat=2):
        assert cq._overlap(a, b) == bool(sa & sb), (a.shape, a.stride(), a.storage_offset(), b.shape, b.stride(), b.storage_offset())


# ---- the operators -----------------------------------------------------------------------------------


class Cuda(torch.Tensor):
    """A host tensor that the binding takes for a CUDA tensor."""
    is_cuda = property(lambda self: True)


def cuda(t):
    return t.as_subclass(Cuda)


R, K, T, V = 256, 256, 8, 40


class Job:
    """The operands of every operator, each in memory of its own, and a list of the launches made."""

    def __init__(self, cq):
        self.cq, self.made = cq, []
        half = lambda *s: cuda(torch.zeros(s, dtype=torch.float16))  # noqa: E731
        word = lambda *s: cuda(torch.zeros(s, dtype=torch.int32))  # noqa: E731
        self.w = cq.W4Weights(word(K // 8, R), word(K // 128, R // 8), half(K // 128, R), R, K)
        self.x, self.y, self.pre, self.res, self.dz, self.bias = half(T, K), half(T, R), half(T, R), half(T, R), half(T, R), half(R)
        self.ids, self.codes, self.scales = cuda(torch.zeros(T, dtype=torch.int64)), word(V * K // 128, 16), half(V * K // 128)
        self.dout, self.rows = half(T, K), half(T, K)
        self.ws = cuda(torch.zeros(cq.w4_embedding_workspace_bytes(T, K), dtype=torch.uint8))

    def linear(self, **kw):
        return self.cq.w4_linear(self.x, self.w, **kw)

    def backward(self, **kw):
        return self.cq.w4_linear_backward(self.dz, self.x, self.w, **kw)

    def activation(self, **kw):
        return self.cq.activation_backward(self.dz, self.pre, "silu", **kw)

    def lookup(self, **kw):
        return self.cq.w4_embedding(self.ids, self.scales, self.codes, K, **kw)

    def table(self, **kw):
        return self.cq.w4_embedding_backward(self.dout, self.ids, self.codes, **kw)


@pytest.fixture
def job(cq, monkeypatch):
    job = Job(cq)
    monkeypatch.setattr(cq, "_place", lambda dev, stream: (0, None))
    monkeypatch.setattr(cq, "_call", lambda context, function, *args: job.made.append(function))
    return job


def over(t, shape, dtype, tail=False):
    """An operand of this shape and type over the first (or last) bytes of t."""
    words = t.reshape(-1).view(torch.uint8)
    n = torch.zeros(shape, dtype=dtype).numel() * torch.empty(0, dtype=dtype).element_size()
    return words[words.numel() - n if tail else 0:][:n].view(dtype).view(shape)


HALF = torch.float16


def big(n):
    return cuda(torch.zeros(n, dtype=HALF))


def refused(job, call, name, target, others):
    """`call(**{name: memory})` is refused where that memory has the first or the last bytes of an operand."""
    for other in others:
        for tail in (False, True):
            memory = over(other, *target, tail=tail)
            with pytest.raises(ValueError, match="overlap"):
                call(**{name: memory})
    assert not job.made


def test_halves_of_one_buffer_are_taken(job):
    """Columns of one buffer, side by side, share no memory: every operator takes them."""
    cq = job.cq
    buf = cuda(torch.zeros((T, 4 * R), dtype=torch.float16))
    a, b, c, d = (buf[:, i * R:(i + 1) * R] for i in range(4))
    cq.w4_linear(a, job.w, residual=b, want_pre=True, pre=c, out=d)
    cq.w4_linear(a, job.w, residual=b, out=b)
    cq.w4_linear_backward(a, b, job.w, dx=c)
    cq.activation_backward(a, b, "gelu", out=c)
    rows = cuda(torch.zeros((2 * T, K), dtype=torch.float16))
    cq.w4_linear(rows[::2], job.w, out=rows[1::2])  # every other row
    assert len(job.made) == 5


def test_layer_refuses_an_output_over_any_operand(job):
    job.w = job.cq.W4Weights(over(big(64 * R), (K // 8, R), torch.int32), job.w.qzeros, job.w.scales, R, K)
    words = job.w.qweight
    refused(job, job.linear, "out", ((T, R), HALF), [job.x, words])
    refused(job, lambda **kw: job.linear(want_pre=True, **kw), "pre", ((T, R), HALF), [job.x, words])
    # the smaller operands lie within the output's memory
    for small in ("bias", "qzeros", "scales"):
        for name in ("out", "pre"):
            memory = big(T * R).view(T, R)
            flat, w, bias = memory.view(-1), job.w, None
            if small == "bias":
                bias = flat[512:512 + R]
            elif small == "qzeros":
                w = job.cq.W4Weights(w.qweight, over(flat, (K // 128, R // 8), torch.int32, tail=True), w.scales, R, K)
            else:
                w = job.cq.W4Weights(w.qweight, w.qzeros, over(flat, (K // 128, R), HALF, tail=True), R, K)
            with pytest.raises(ValueError, match="overlap"):
                job.cq.w4_linear(job.x, w, bias=bias, want_pre=name == "pre", **{name: memory})
    assert not job.made


def test_layer_gradients_refuse_outputs_over_any_operand(job):
    refused(job, job.backward, "dx", ((T, K), HALF), [job.dz, job.x, job.w.qweight])
    refused(job, lambda **kw: job.backward(want_dscales=False, **kw), "dx", ((T, K), HALF), [job.dz, job.w.qweight])
    for small in ("qzeros", "scales"):
        memory = big(T * K).view(T, K)
        zeros = over(memory, (K // 128, R // 8), torch.int32) if small == "qzeros" else job.w.qzeros
        scales = over(memory, (K // 128, R), HALF) if small == "scales" else job.w.scales
        with pytest.raises(ValueError, match="overlap"):
            job.cq.w4_linear_backward(job.dz, None, job.cq.W4Weights(job.w.qweight, zeros, scales, R, K), want_dscales=False, dx=memory)
    refused(job, job.backward, "dscales", ((K // 128, R), torch.float32), [job.dz, job.x, job.w.qweight])
    assert not job.made


def test_activation_gradient_refuses_a_bias_gradient_over_any_operand(job):
    refused(job, job.activation, "dbias", ((R,), torch.float32), [job.dz, job.pre])
    refused(job, lambda **kw: job.activation(out=job.y, **kw), "dbias", ((R,), torch.float32), [job.y])
    job.activation(out=job.dz)
    job.activation(out=job.pre)
    assert len(job.made) == 2


def test_lookup_refuses_an_output_over_any_operand(job):
    refused(job, job.lookup, "out", ((T, K), HALF), [job.codes])
    for small in ("ids", "scales"):
        memory = big(T * K).view(T, K)
        for tail in (False, True):
            ids = over(memory, (T,), torch.int64, tail) if small == "ids" else job.ids
            scales = over(memory, (V * K // 128,), HALF, tail) if small == "scales" else job.scales
            with pytest.raises(ValueError, match="overlap"):
                job.cq.w4_embedding(ids, scales, job.codes, K, out=memory)
    assert not job.made
    job.lookup(out=job.rows)
    assert len(job.made) == 1


def test_table_gradient_refuses_outputs_over_any_operand(job):
    refused(job, job.table, "out", ((V, K // 128), torch.float32), [job.dout, job.codes])
    refused(job, lambda **kw: job.table(workspace=job.ws, **kw), "out", ((V, K // 128), torch.float32), [job.ws])
    assert not job.made
    job.table(out=cuda(torch.zeros((V, K // 128))), workspace=job.ws)
    assert len(job.made) == 1
