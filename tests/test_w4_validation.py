"""Refusals of the operators on 4-bit weights, on the CPU: the C entry points return
an argument error before anything is enqueued (fake addresses are never
dereferenced), the binding raises ValueError."""
import ctypes

import pytest
import torch

FAKE = 0x10000


@pytest.fixture(scope="module")
def cq():
    from minimax_scale_search_b200 import build
    build.build()
    from minimax_scale_search_b200 import cq as binding
    return binding


def vp(p):
    return ctypes.c_void_p(p)


def linear(cq, x=FAKE, ldx=256, dt=0, T=4, qw=FAKE, qz=FAKE, sc=FAKE, R=64, K=256, b=0, act=0, res=0, ldres=64, y=FAKE,
           ldy=64, pre=0, ldpre=64):
    return cq.lib.cq_w4_linear(vp(x), ldx, dt, T, vp(qw), vp(qz), vp(sc), R, K, vp(b), act, vp(res), ldres, vp(y), ldy,
                               vp(pre), ldpre, vp(None))


@pytest.mark.parametrize("bad", [dict(dt=2), dict(dt=-1), dict(T=-1), dict(R=-8), dict(R=60), dict(K=0), dict(K=-128),
                                 dict(K=200), dict(x=0), dict(x=FAKE + 8), dict(ldx=248), dict(ldx=260), dict(qw=0),
                                 dict(qw=FAKE + 4), dict(qz=0), dict(qz=FAKE + 2), dict(sc=0), dict(sc=FAKE + 2),
                                 dict(b=FAKE + 1), dict(act=-1), dict(act=5), dict(res=FAKE, ldres=56),
                                 dict(res=FAKE + 2), dict(res=FAKE, ldres=65), dict(y=0), dict(y=FAKE + 4),
                                 dict(ldy=56), dict(ldy=68), dict(pre=FAKE + 2), dict(pre=FAKE, ldpre=8)])
def test_linear_refuses(cq, bad):
    assert linear(cq, **bad) == cq.CQ_ERR_INVALID_ARG


def test_linear_limits_and_empty_calls(cq):
    assert linear(cq, T=1 << 31) == cq.CQ_ERR_UNSUPPORTED
    assert linear(cq, R=1 << 31) == cq.CQ_ERR_UNSUPPORTED
    assert linear(cq, K=1 << 31) == cq.CQ_ERR_UNSUPPORTED
    assert linear(cq, T=0, x=0, y=0) == cq.CQ_OK
    assert linear(cq, R=0, qw=0, qz=0, sc=0, y=0) == cq.CQ_OK


def backward(cq, dz=FAKE, lddz=64, x=FAKE, ldx=256, dt=0, T=4, qw=FAKE, R=64, K=256, dx=FAKE, lddx=256, ds=FAKE):
    return cq.lib.cq_w4_linear_backward(vp(dz), lddz, vp(x), ldx, dt, T, vp(qw), vp(FAKE), vp(FAKE), R, K, vp(dx), lddx,
                                        vp(ds), vp(None))


@pytest.mark.parametrize("bad", [dict(dt=2), dict(T=-1), dict(R=12), dict(K=0), dict(K=64), dict(dz=0), dict(dz=FAKE + 2),
                                 dict(lddz=56), dict(lddz=67), dict(x=0), dict(x=FAKE + 2), dict(ldx=128),
                                 dict(dx=FAKE + 8), dict(lddx=128), dict(lddx=257), dict(ds=FAKE + 4), dict(qw=FAKE + 8)])
def test_linear_backward_refuses(cq, bad):
    assert backward(cq, **bad) == cq.CQ_ERR_INVALID_ARG


def test_linear_backward_asks_only_for_what_it_reads(cq):
    assert backward(cq, x=0, ds=0, dx=0) == cq.CQ_OK           # nothing wanted
    assert backward(cq, T=0, dz=0, x=0, ds=0) == cq.CQ_OK      # no rows
    assert backward(cq, T=1 << 31) == cq.CQ_ERR_UNSUPPORTED


def test_activation_backward_refuses(cq):
    def call(dy=FAKE, lddy=64, pre=FAKE, ldpre=64, dt=0, T=4, R=64, act=2, dz=FAKE, lddz=64, db=FAKE):
        return cq.lib.cq_activation_backward(vp(dy), lddy, vp(pre), ldpre, dt, T, R, act, vp(dz), lddz, vp(db), vp(None))
    for bad in (dict(dt=2), dict(T=-1), dict(R=4), dict(act=5), dict(act=-1), dict(dy=0), dict(pre=0), dict(dz=0),
                dict(dy=FAKE + 2), dict(lddy=56), dict(ldpre=66), dict(lddz=8), dict(db=FAKE + 2)):
        assert call(**bad) == cq.CQ_ERR_INVALID_ARG, bad
    assert call(R=1 << 31, lddy=1 << 31, ldpre=1 << 31, lddz=1 << 31) == cq.CQ_ERR_UNSUPPORTED
    assert call(R=0, dy=0, pre=0, dz=0) == cq.CQ_OK


def test_embedding_refuses(cq):
    def call(ids=FAKE, wide=1, T=4, sc=FAKE, codes=FAKE, V=10, K=256, m=1.0, dt=0, out=FAKE):
        return cq.lib.cq_w4_embedding(vp(ids), wide, T, vp(sc), vp(codes), V, K, m, dt, vp(out), vp(None))
    for bad in (dict(ids=0), dict(ids=FAKE + 4), dict(wide=2), dict(wide=0, ids=FAKE + 2), dict(T=-1), dict(sc=0),
                dict(sc=FAKE + 1), dict(codes=0), dict(codes=FAKE + 2), dict(V=-1), dict(K=0), dict(K=100), dict(dt=3),
                dict(out=0), dict(out=FAKE + 8), dict(m=float("nan")), dict(m=float("inf"))):
        assert call(**bad) == cq.CQ_ERR_INVALID_ARG, bad
    assert call(T=1 << 31) == cq.CQ_ERR_UNSUPPORTED
    assert call(V=1 << 31) == cq.CQ_ERR_UNSUPPORTED
    assert call(T=0, ids=0, out=0, sc=0, codes=0) == cq.CQ_OK


def test_embedding_backward_refuses(cq):
    size = cq.w4_embedding_workspace_bytes(4, 256)
    assert size % 256 == 0 and cq.w4_embedding_workspace_bytes(0, 256) == 256

    def call(d=FAKE, dt=0, ids=FAKE, wide=1, T=4, codes=FAKE, V=10, K=256, m=1.0, out=FAKE, ws=FAKE, wsb=size):
        return cq.lib.cq_w4_embedding_backward(vp(d), dt, vp(ids), wide, T, vp(codes), V, K, m, vp(out), vp(ws), wsb,
                                               vp(None))
    for bad in (dict(d=0), dict(d=FAKE + 8), dict(dt=3), dict(ids=0), dict(ids=FAKE + 4), dict(T=-1), dict(codes=0),
                dict(V=-1), dict(K=0), dict(K=130), dict(out=0), dict(out=FAKE + 2), dict(m=float("inf"))):
        assert call(**bad) == cq.CQ_ERR_INVALID_ARG, bad
    for bad in (dict(ws=0), dict(ws=FAKE + 16), dict(wsb=size - 1)):
        assert call(**bad) == cq.CQ_ERR_WORKSPACE, bad
    assert call(T=1 << 31) == cq.CQ_ERR_UNSUPPORTED
    assert call(V=0, codes=0, out=0, d=0) == cq.CQ_OK


def test_binding_refuses_host_tensors_and_bad_types(cq):
    t = cq.GPTQTensors(torch.zeros((16, 8), dtype=torch.int32), torch.zeros((1, 1), dtype=torch.int32),
                       torch.zeros((1, 8), dtype=torch.float16), torch.zeros(128, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        cq.w4_weights(t)
    t.scales = t.scales.float()
    with pytest.raises(ValueError, match="scales"):
        cq.w4_weights(t)
    with pytest.raises(ValueError, match="multiple of 128"):
        cq.w4_weights(cq.GPTQTensors(torch.zeros((8, 8), dtype=torch.int32), None, None, None))
    w = cq.W4Weights(t.qweight, t.qzeros, t.scales, 8, 128)
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        cq.w4_linear(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        cq.w4_linear_backward(x, x, w)
    with pytest.raises(ValueError, match="CUDA"):
        cq.activation_backward(x, x, "gelu")
    with pytest.raises(ValueError, match="CUDA"):
        cq.w4_embedding(torch.zeros(3, dtype=torch.int64), t.scales, t.qweight, 128)
    with pytest.raises(ValueError, match="CUDA"):
        cq.w4_embedding_backward(x, torch.zeros(2, dtype=torch.int64), t.qweight)
    with pytest.raises(ValueError, match="unknown activation"):
        cq._activation("tanh")


def test_row_strides(cq):
    """The binding's own check of a [rows, cols] operand, which needs no device."""
    x = torch.zeros((6, 80), dtype=torch.float16)
    assert cq._rows16("x", x[:, :64], 6, 64, x) == 80
    assert cq._rows16("x", x[::2, :64], 3, 64, x) == 160
    assert cq._rows16("x", x[:1, :64], 1, 64, x) == 80
    odd = torch.zeros((1, 67), dtype=torch.float16)
    assert cq._rows16("x", odd[:, :64], 1, 64, x) == 64      # one row: its stride does not matter
    assert cq._rows16("x", x[:0], 0, 80, x) == 80
    for bad in (x[:, 4:68], torch.zeros((64, 6), dtype=torch.float16).t(), torch.zeros((6, 65), dtype=torch.float16)[:, :64],
                x[:1, :64].expand(6, 64)):
        with pytest.raises(ValueError, match="16-byte"):
            cq._rows16("x", bad, 6, 64, x)
    with pytest.raises(ValueError, match=r"\[6, 64\]"):
        cq._rows16("x", x, 6, 64, x)
    with pytest.raises(ValueError, match="float16"):
        cq._rows16("x", x.float(), 6, 80, x)
