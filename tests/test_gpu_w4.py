"""The operators on 4-bit weights (csrc/cq_linear.cu, csrc/cq_embedding.cu)
against their fp64 definitions (oracle/w4.py).

Tolerances count the roundings, each at most half a step u (bf16 2^-8, fp16
2^-11, fp32 2^-24) of the value rounded, or a whole step where the hardware may
truncate (sums on the tensor cores).  With A = sum of the magnitudes of a
product's terms, the sum of n terms is off by at most n 2^-23 A, weights that
are rounded to the operands' type add u A, and an activation (slope at most
1.2) multiplies that by 1.2; the result's own rounding adds u |y|."""
import numpy as np
import pytest

from minimax_scale_search_b200 import synth
from oracle import w4

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -149}  # half a step of the smallest values
SLOPE = 1.2


def dtype_of(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def device(a):
    import torch
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    elif a.dtype == np.uint32:
        a = a.view(np.int32)
    return torch.from_numpy(a).cuda()


def values(rng, shape, dt, std=1.0, pad=0):
    """(tensor of the type whose rows lie `pad` elements apart, its values in fp64)."""
    import torch
    a = torch.from_numpy(rng.normal(0, std, (shape[0], shape[1] + pad))).to(dtype_of(dt)).cuda()
    a = a[:, :shape[1]]
    return a, a.double().cpu().numpy()


def f64(t):
    return t.double().cpu().numpy()


def make_layer(R, K, seed, scale=0.02):
    """(cq.W4Weights, n, s): any codes and zero points, scales around `scale`."""
    import torch
    from minimax_scale_search_b200 import cq
    qw, qz, _, gi = synth.make_gptq_tensors(R, K, seed=seed)
    s = (scale * np.random.default_rng(seed).lognormal(0, 0.5, (K // 128, R))).astype(np.float16)
    t = cq.GPTQTensors(device(qw), device(qz), torch.from_numpy(s).cuda(), device(gi))
    n, sc = w4.layer(qw, qz, s.view(np.uint16))
    return cq.w4_weights(t), n, sc


def linear_bound(x, n, s, bias, pre, out, dt, res=None, slope=1.0):
    K = n.shape[1]
    A = np.abs(x) @ np.abs(w4.weight(n, s)).T + (0 if bias is None else np.abs(bias))
    fp32 = 8 * 2.0 ** -23 * (np.abs(pre) + np.abs(out) + (0 if res is None else np.abs(res)))  # the epilogue's arithmetic
    return slope * A * (U[dt] + (K + 8) * 2.0 ** -23) + fp32 + U[dt] * np.abs(out) + TINY[dt]


# rows of x: one token, tiles of 8 and 16 with one more or less, 128- and 256-row tiles, several tiles;
# R and K: the smallest, no multiple of a tile, several tiles, long K
SHAPES = [(1, 8, 128), (1, 1024, 1024), (2, 40, 384), (7, 264, 1024), (8, 136, 2176), (9, 40, 128), (15, 1032, 256),
          (16, 8, 4096), (17, 8, 128), (17, 136, 384), (31, 264, 640), (33, 40, 1152), (64, 1032, 256), (65, 128, 128),
          (127, 520, 384), (129, 136, 512), (255, 264, 128), (256, 256, 256), (257, 8, 640), (300, 392, 1152),
          (515, 1096, 384), (1025, 136, 256)]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T,R,K", SHAPES)
def test_linear(T, R, K, dt):
    from minimax_scale_search_b200 import cq
    rng = np.random.default_rng(T * 7 + R + K)
    act = w4.ACTIVATIONS[(T + R // 8 + K // 128) % 5]
    w, n, s = make_layer(R, K, T + R + K)
    x, x64 = values(rng, (T, K), dt, pad=8 * (T % 3))
    b, b64 = values(rng, (1, R), dt, 0.2)
    res, r64 = values(rng, (T, R), dt, pad=8 * (R // 8 % 2))
    y, pre = cq.w4_linear(x, w, bias=b[0], activation=act, residual=res, want_pre=True)
    ey, ez = w4.linear(x64, n, s, b64[0], act, r64)
    assert np.all(np.abs(f64(pre) - ez) <= linear_bound(x64, n, s, b64[0], ez, ez, dt))
    assert np.all(np.abs(f64(y) - ey) <= linear_bound(x64, n, s, b64[0], ez, ey, dt, r64, SLOPE))
    # without an epilogue: the product alone
    y0 = cq.w4_linear(x, w)
    e0 = w4.linear(x64, n, s)[0]
    assert np.all(np.abs(f64(y0) - e0) <= linear_bound(x64, n, s, None, e0, e0, dt))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_many_full_tiles(dt):
    """Enough rows and outputs that every SM has several tiles of 256 tokens, with shared memory busy."""
    from minimax_scale_search_b200 import cq
    T, R, K = 4000, 4104, 2048
    rng = np.random.default_rng(17)
    w, n, s = make_layer(R, K, 17)
    x, x64 = values(rng, (T, K), dt)
    e = w4.linear(x64, n, s)[0]
    bound = linear_bound(x64, n, s, None, e, e, dt)
    for _ in range(3):
        assert np.all(np.abs(f64(cq.w4_linear(x, w)) - e) <= bound)
    dz, d64 = values(rng, (T, R), dt, 0.1)
    edx, _ = w4.linear_backward(d64, x64, n, s)
    A = np.abs(d64) @ np.abs(w4.weight(n, s))
    bound = A * (U[dt] + (R + 8) * 2.0 ** -23) + U[dt] * np.abs(edx) + TINY[dt]
    for _ in range(3):
        assert np.all(np.abs(f64(cq.w4_linear_backward(dz, None, w, want_dscales=False)[0]) - edx) <= bound)


@pytest.mark.parametrize("act", w4.ACTIVATIONS)
@pytest.mark.parametrize("T", [3, 40])
def test_activations_over_their_range(act, T):
    """One weight of 1 per output: z runs over every part of the activation."""
    import torch
    from minimax_scale_search_b200 import cq
    R = K = 128
    qw = np.zeros((K // 8, R), dtype=np.uint32)
    for r in range(R):
        qw[:, r] = 0x88888888
        qw[r // 8, r] = (0x88888888 & ~(0xF << (4 * (r % 8)))) | (0x9 << (4 * (r % 8)))
    t = cq.GPTQTensors(device(qw), device(np.full((1, R // 8), 0x77777777, np.uint32)),
                       torch.ones((1, R), dtype=torch.float16, device="cuda"),
                       torch.zeros(K, dtype=torch.int32, device="cuda"))
    z = np.linspace(-12, 12, T * K).reshape(T, K)
    x = torch.from_numpy(z).to(torch.float16).cuda()
    z = f64(x)
    y, pre = cq.w4_linear(x, cq.w4_weights(t), activation=act, want_pre=True)
    assert np.array_equal(f64(pre), z)  # a single exact product
    e = w4.activation(z, act)
    # arguments of erfc, exp and tanh are rounded: relative 2^-24 of an exponent up to 72 (gelu at -12), 2^-17 in all
    assert np.all(np.abs(f64(y) - e) <= (U["fp16"] + 2.0 ** -17) * np.abs(e) + TINY["fp16"] + 2.0 ** -22 * (act == "gelu_tanh") * np.abs(z))


def test_exact_rows_use_exact_weights():
    """Up to 16 rows the weights are not rounded: a scale whose products need more bits
    than bfloat16 has gives fp32-exact sums."""
    import torch
    from minimax_scale_search_b200 import cq
    w, n, s = make_layer(64, 256, 4)
    x = torch.zeros((16, 256), dtype=torch.bfloat16, device="cuda")
    for t in range(16):
        x[t, 17 * t % 256] = 1.0
    y = cq.w4_linear(x, w)
    e = w4.linear(f64(x), n, s)[0]
    assert torch.equal(y.cpu(), torch.from_numpy(e).to(torch.bfloat16))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [16, 40, 300])
def test_rows_do_not_touch_each_other(T, dt):
    """Inf and NaN in one row of x reach only that row; rows behind the last one and
    columns beside the outputs are left as they were."""
    import torch
    from minimax_scale_search_b200 import cq
    R, K = 136, 384
    w, n, s = make_layer(R, K, 8)
    x, x64 = values(np.random.default_rng(T), (T, K), dt)
    clean = cq.w4_linear(x, w)
    bad = x.clone()
    bad[5, 3], bad[T - 1, K - 1] = float("inf"), float("nan")
    buf = torch.full((T + 9, R + 24), 7.0, dtype=dtype_of(dt), device="cuda")
    cq.w4_linear(bad, w, out=buf[:T, 8:R + 8])
    keep = [t for t in range(T) if t not in (5, T - 1)]
    assert torch.equal(buf[keep, 8:R + 8], clean[keep])
    assert torch.isnan(buf[T - 1, 8:R + 8].float()).all() and not torch.isfinite(buf[5, 8:R + 8].float()).all()
    assert (buf[T:] == 7.0).all() and (buf[:, :8] == 7.0).all() and (buf[:, R + 8:] == 7.0).all()
    dz, _ = values(np.random.default_rng(T + 1), (T, R), dt)
    dx = cq.w4_linear_backward(dz, None, w, want_dscales=False)[0]
    dbad = dz.clone()
    dbad[2, 4] = float("nan")
    gbuf = torch.full((T + 5, K + 16), 7.0, dtype=dtype_of(dt), device="cuda")
    cq.w4_linear_backward(dbad, None, w, want_dscales=False, dx=gbuf[:T, :K])
    keep = [t for t in range(T) if t != 2]
    assert torch.equal(gbuf[keep, :K], dx[keep]) and torch.isnan(gbuf[2, :K].float()).all()
    assert (gbuf[T:] == 7.0).all() and (gbuf[:, K:] == 7.0).all()


def test_residual_may_be_the_output():
    import torch
    from minimax_scale_search_b200 import cq
    for T in (4, 200):
        w, _, _ = make_layer(264, 1024, 9)
        x, _ = values(np.random.default_rng(T), (T, 1024), "bf16")
        res, _ = values(np.random.default_rng(T + 1), (T, 264), "bf16", pad=8)
        ref = cq.w4_linear(x, w, activation="silu", residual=res)
        out = cq.w4_linear(x, w, activation="silu", residual=res, out=res)
        assert out.data_ptr() == res.data_ptr() and torch.equal(out, ref)


BACKWARD = [(1, 8, 128), (5, 40, 384), (16, 136, 256), (33, 264, 640), (64, 64, 128), (100, 1032, 256), (129, 136, 1152),
            (256, 256, 256), (300, 520, 384), (777, 72, 640), (1500, 136, 256)]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T,R,K", BACKWARD)
def test_linear_backward(T, R, K, dt):
    from minimax_scale_search_b200 import cq
    rng = np.random.default_rng(T + R * 3 + K)
    w, n, s = make_layer(R, K, T + K)
    dz, d64 = values(rng, (T, R), dt, 0.1, pad=8 * (T % 2))
    x, x64 = values(rng, (T, K), dt, pad=8 * (K // 128 % 3))
    dx, ds = cq.w4_linear_backward(dz, x, w)
    edx, eds = w4.linear_backward(d64, x64, n, s)
    A = np.abs(d64) @ np.abs(w4.weight(n, s))
    assert np.all(np.abs(f64(dx) - edx) <= A * (U[dt] + (R + 8) * 2.0 ** -23) + U[dt] * np.abs(edx) + TINY[dt])
    # sums over T, then over the group's 128 inputs, in fp32 of exact products
    A = w4.linear_backward(np.abs(d64), np.abs(x64), np.abs(n), s)[1]
    assert np.all(np.abs(f64(ds) - eds) <= A * (T + 128 + 8) * 2.0 ** -23)
    # each alone gives the same bytes
    assert (cq.w4_linear_backward(dz, x, w, want_dscales=False)[0] == dx).all()
    assert (cq.w4_linear_backward(dz, x, w, want_dx=False)[1] == ds).all()


def test_empty_calls():
    import torch
    from minimax_scale_search_b200 import cq
    w, _, _ = make_layer(64, 256, 3)
    x, dz = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert cq.w4_linear(x, w).shape == (0, 64)
    old = torch.full((2, 64), 3.0, device="cuda")
    dx, ds = cq.w4_linear_backward(dz, x, w, dscales=old)
    assert dx.shape == (0, 256) and not ds.any()
    dz2, db = cq.activation_backward(dz, dz, "gelu", dbias=torch.full((64,), 3.0, device="cuda"))
    assert dz2.shape == (0, 64) and not db.any()
    scales, codes = (device(a) for a in synth.make_codes(6, seed=1))
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    assert cq.w4_embedding(ids, scales, codes, 256).shape == (0, 256)
    g = cq.w4_embedding_backward(torch.empty((0, 256), device="cuda"), ids, codes, out=torch.full((3, 2), 5.0, device="cuda"))
    assert not g.any()


def test_a_layer_without_outputs():
    import torch
    from minimax_scale_search_b200 import cq
    z = lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    w = cq.w4_weights(cq.GPTQTensors(z(32, 0), z(2, 0), z(2, 0, dtype=torch.float16), torch.arange(256, dtype=torch.int32, device="cuda") // 128))
    x = torch.ones((5, 256), dtype=torch.bfloat16, device="cuda")
    assert cq.w4_linear(x, w).shape == (5, 0)
    dx, ds = cq.w4_linear_backward(x[:, :0], x, w, dx=torch.ones_like(x))
    assert not dx.any() and ds.shape == (2, 0)


def test_operands_that_overlap_are_refused():
    import torch
    from minimax_scale_search_b200 import cq
    w, _, _ = make_layer(256, 256, 1)
    buf = torch.zeros((20, 256), dtype=torch.float16, device="cuda")
    x = torch.zeros((8, 256), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="overlap x"):
        cq.w4_linear(buf[:8], w, out=buf[4:12])
    with pytest.raises(ValueError, match="residual itself"):
        cq.w4_linear(x, w, residual=buf[:8], out=buf[1:9])
    with pytest.raises(ValueError, match="pre must not overlap"):
        cq.w4_linear(x, w, out=buf[:8], want_pre=True, pre=buf[7:15])
    with pytest.raises(ValueError, match="only with want_pre"):
        cq.w4_linear(x, w, pre=buf[:8])
    with pytest.raises(ValueError, match="dx must not overlap"):
        cq.w4_linear_backward(buf[:8], x, w, dx=buf[2:10])
    with pytest.raises(ValueError, match="dy or pre itself"):
        cq.activation_backward(buf[:8], x, "silu", out=buf[1:9])


def test_act_order_is_refused():
    import torch
    from minimax_scale_search_b200 import cq
    qw, qz, gs, gi = synth.make_gptq_tensors(16, 256, seed=2, act_order=True)
    with pytest.raises(ValueError, match="act-order"):
        cq.w4_weights(cq.GPTQTensors(device(qw), device(qz), device(gs).view(torch.float16), device(gi)))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("act", w4.ACTIVATIONS)
@pytest.mark.parametrize("T,R", [(1, 8), (3, 72), (255, 64), (300, 1032), (2000, 136)])
def test_activation_backward(T, R, act, dt):
    from minimax_scale_search_b200 import cq
    rng = np.random.default_rng(T + R)
    dy, y64 = values(rng, (T, R), dt, 0.1, pad=8)
    pre, p64 = values(rng, (T, R), dt, 3.0, pad=8 * (T % 2))
    dz, db = cq.activation_backward(dy, pre, act)
    edz, edb = w4.activation_backward(y64, p64, act)
    # the slope is a sum of terms of at most 2.2 |z| + 1 in magnitude, each a few fp32 roundings off
    err = np.abs(y64) * (2.2 * np.abs(p64) + 1) * 16 * 2.0 ** -23 * (act not in ("none", "relu"))
    assert np.all(np.abs(f64(dz) - edz) <= err + U[dt] * np.abs(edz) + TINY[dt])
    assert np.all(np.abs(f64(db) - edb) <= err.sum(0) + np.abs(edz).sum(0) * (T + 8) * 2.0 ** -24)
    again = dy.clone()
    assert (cq.activation_backward(again, pre, act, out=again, want_dbias=False)[0] == dz).all()  # in place


def make_table(V, K, seed):
    import torch
    scales, codes = synth.make_codes(V * K // 128, seed=seed)
    scales = (0.02 * np.random.default_rng(seed).lognormal(0, 0.5, scales.size)).astype(np.float16).view(np.uint16)
    return device(scales), device(codes), *w4.table(scales, codes, K)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,V,K,wide", [(1, 1, 128, True), (5, 7, 384, False), (16, 300, 1024, True), (333, 50, 640, True),
                                        (1000, 1000, 256, False)])
def test_embedding_and_its_gradient(T, V, K, wide, dt):
    import torch
    from minimax_scale_search_b200 import cq
    rng = np.random.default_rng(T + V)
    scales, codes, q, s = make_table(V, K, T + K)
    ids = rng.integers(-1, V + 1, T)  # -1 and V name no row
    it = torch.from_numpy(ids).to(torch.int64 if wide else torch.int32).cuda()
    m = 1.0 if T % 2 else 11.3
    out = cq.w4_embedding(it, scales, codes, K, multiplier=m, dtype=dtype_of(dt))
    e = w4.embedding(ids, q, s, np.float64(np.float32(m)))
    assert np.all(np.abs(f64(out) - e) <= (U[dt] + 2.0 ** -24) * np.abs(e) + TINY[dt])
    d, d64 = values(rng, (T, K), dt, 0.1)
    g = cq.w4_embedding_backward(d, it, codes, multiplier=m)
    eg = w4.embedding_backward(d64, ids, q, np.float64(np.float32(m)))
    A = w4.embedding_backward(np.abs(d64), ids, np.abs(q), m)
    assert np.all(np.abs(f64(g) - eg) <= A * (128 + 2) * 2.0 ** -24)  # 128 terms in fp32, tokens in fp64, two roundings


@pytest.mark.parametrize("T", [1, 31, 32, 33, 255, 256, 257, 1023, 4097, 20000])
@pytest.mark.parametrize("kind", ["same", "ascending", "descending", "few", "none"])
def test_embedding_gradient_of_every_order_of_tokens(T, kind):
    """One row for all tokens, a row for each, a few rows in runs that end at and
    beside the kernels' tile edges, and no row at all."""
    import torch
    from minimax_scale_search_b200 import cq
    V, K = T + 1, 128
    rng = np.random.default_rng(T)
    ids = {"same": np.full(T, V - 1), "ascending": np.arange(T), "descending": np.arange(T)[::-1],
           "few": np.sort(rng.integers(0, min(V, 5), T))[rng.permutation(T)], "none": np.full(T, -7)}[kind]
    scales, codes, q, s = make_table(V, K, 5)
    d, d64 = values(rng, (T, K), "fp32", 0.1)
    g = cq.w4_embedding_backward(d, torch.from_numpy(ids.copy()).cuda(), codes)
    p = (d64 * q[np.clip(ids, 0, V - 1)]) * ((ids >= 0) & (ids < V))[:, None]
    e, A = np.zeros(V), np.zeros(V)
    np.add.at(e, np.clip(ids, 0, V - 1), p.sum(1))
    np.add.at(A, np.clip(ids, 0, V - 1), np.abs(p).sum(1))
    assert np.all(np.abs(f64(g)[:, 0] - e) <= A * (128 + 2) * 2.0 ** -24)


@pytest.mark.parametrize("T", [5, 700])
def test_a_table_of_more_rows_than_fp32_counts(T):
    """2^24 + 3 rows: neighbouring row numbers that fp32 does not tell apart stay apart."""
    import torch
    from minimax_scale_search_b200 import cq
    V, K = (1 << 24) + 3, 128
    codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (V, 16), dtype=torch.int32, device="cuda")
    ids = V - 1 - torch.arange(T, device="cuda") % 4
    d = torch.randn((T, K), device="cuda")
    g = cq.w4_embedding_backward(d, ids, codes)
    few = codes[V - 4:].cpu().numpy().view(np.uint32)
    q = w4.table(np.ones(4, np.uint16), few, K)[0]
    e = w4.embedding_backward(f64(d), (ids - (V - 4)).cpu().numpy(), q)
    A = w4.embedding_backward(np.abs(f64(d)), (ids - (V - 4)).cpu().numpy(), np.abs(q))
    assert np.all(np.abs(f64(g[V - 4:]) - e) <= A * (128 + 2) * 2.0 ** -24)
    assert int((g != 0).sum()) <= 4


def test_ids_of_any_shape_and_a_shared_workspace():
    import torch
    from minimax_scale_search_b200 import cq
    scales, codes, q, s = make_table(40, 256, 2)
    ids = torch.randint(0, 40, (3, 5, 2), device="cuda")
    out = cq.w4_embedding(ids, scales, codes, 256, dtype=torch.bfloat16)
    assert out.shape == (3, 5, 2, 256)
    assert torch.equal(out.view(-1, 256), cq.w4_embedding(ids.view(-1), scales, codes, 256, dtype=torch.bfloat16))
    ws = torch.empty(cq.w4_embedding_workspace_bytes(30, 256), dtype=torch.uint8, device="cuda")
    d = torch.randn((3, 5, 2, 256), device="cuda")
    a = cq.w4_embedding_backward(d, ids, codes, workspace=ws)
    b = cq.w4_embedding_backward(2 * d, ids, codes, workspace=ws)
    assert torch.equal(b, 2 * a)
    with pytest.raises(ValueError, match="workspace"):
        cq.w4_embedding_backward(d, ids, codes, workspace=ws[:-256])


def test_calls_are_deterministic():
    import torch
    from minimax_scale_search_b200 import cq
    rng = np.random.default_rng(1)
    w, _, _ = make_layer(520, 2176, 1)
    for T in (5, 16, 100, 700):
        x, _ = values(rng, (T, 2176), "bf16")
        dz, _ = values(rng, (T, 520), "bf16")
        runs = [(cq.w4_linear(x, w), *cq.w4_linear_backward(dz, x, w), *cq.activation_backward(dz, dz, "silu"))
                for _ in range(3)]
        for r in runs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def _model(V, H, F):
    """A quantised table, a layer, and the table as a layer, by the framework's own selection and export."""
    import torch
    from minimax_scale_search_b200 import cq
    gen = torch.Generator(device="cuda").manual_seed(0)
    made = []
    for R, K in ((V, H), (F, H)):
        W = (0.05 * torch.randn((R, K), generator=gen, device="cuda")).half()
        D = torch.rand((2, K), generator=gen, device="cuda") + 0.1
        made.append(cq.select_scales(W, D))
    up = cq.w4_weights(cq.gptq_export(made[1].scales, made[1].codes, F, H))
    head = cq.w4_weights(cq.gptq_export(made[0].scales, made[0].codes, V, H))
    return made[0], up, head


def test_a_run_together_with_its_gradients():
    """Lookup, a layer with its activation, the table again as the output layer; then the
    gradients back to the table's and the layer's scales, against the same chain in fp64
    on the values that each operator handed on, and against differences of the whole."""
    import torch
    from minimax_scale_search_b200 import cq
    V, H, F, T = 304, 256, 256, 37
    table, up, head = _model(V, H, F)
    ids = torch.randint(0, V, (T,), device="cuda")
    e = cq.w4_embedding(ids, table.scales, table.codes, H, multiplier=16.0, dtype=torch.bfloat16)
    h, pre = cq.w4_linear(e, up, activation="gelu", residual=e, want_pre=True)
    logits = cq.w4_linear(h, head)
    c = torch.randn_like(logits) * 0.1
    dh, ds_head = cq.w4_linear_backward(c, h, head)
    dpre, _ = cq.activation_backward(dh, pre, "gelu")
    de, ds_up = cq.w4_linear_backward(dpre, e, up)
    dtotal = (de.float() + dh.float()).bfloat16()
    ds_table = cq.w4_embedding_backward(dtotal, ids, table.codes, multiplier=16.0)

    sn, cn = cq.to_numpy_bits(table)
    q, s = w4.table(sn, cn, H)
    n_up, s_up = w4.layer(*(t.cpu().numpy() for t in (up.qweight, up.qzeros)), up.scales.cpu().numpy().view(np.uint16))
    i = ids.cpu().numpy()
    c64 = f64(c)

    def loss(s_table, s_layer, s_out):
        e = w4.embedding(i, q, s_table, 16.0)
        h = w4.linear(e, n_up, s_layer, None, "gelu", e)[0]
        return (c64 * w4.linear(h, q, s_out)[0]).sum()

    # every tensor handed on is rounded to bfloat16 (2^-8 of it): gradients agree to a few such roundings of
    # the largest; a difference of the fp64 loss is exact to 1e-6 of that
    rng = np.random.default_rng(3)
    used = i[:6]
    for which, grad, pick in ((0, f64(ds_table), [(v, g) for v in used for g in (0, 1)]),
                              (1, f64(ds_up).T, [(r, r % 2) for r in rng.integers(0, F, 8)]),
                              (2, f64(ds_head).T, [(r, r % 2) for r in rng.integers(0, V, 8)])):
        for at in pick:
            diff = []
            for h in (1e-6, -1e-6):
                args = [s.copy(), s_up.copy(), s.copy()]
                args[which][at] += h
                diff.append(loss(*args))
            d = (diff[0] - diff[1]) / 2e-6
            assert abs(grad[at] - d) <= 6 * 2.0 ** -8 * np.abs(grad).max(), (which, at)


def test_captured_graphs_replay_on_new_inputs():
    """Two graphs that hold the whole chain, replayed in turn on new contents of the same buffers."""
    import torch
    from minimax_scale_search_b200 import cq
    w, _, _ = make_layer(264, 384, 12)
    scales, codes, _, _ = make_table(50, 384, 3)

    def chain(ids, c):
        e = cq.w4_embedding(ids, scales, codes, 384, dtype=torch.bfloat16)
        h, pre = cq.w4_linear(e, w, activation="silu", want_pre=True)
        dz, db = cq.activation_backward(c, pre, "silu")
        dx, ds = cq.w4_linear_backward(dz, e, w)
        return h, db, dx, ds, cq.w4_embedding_backward(dx, ids, codes)

    made = []
    for T in (6, 150):
        ids, c = torch.randint(0, 50, (T,), device="cuda"), torch.randn((T, 264), device="cuda").bfloat16()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            chain(ids, c)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = chain(ids, c)
        made.append((g, ids, c, outs))
    for seed in range(3):
        torch.manual_seed(seed)
        for g, ids, c, outs in made:
            ids.copy_(torch.randint(-1, 51, ids.shape, device="cuda"))
            c.copy_(torch.randn(c.shape, device="cuda"))
            g.replay()
        for g, ids, c, outs in made:
            ref = chain(ids, c)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_a_side_stream():
    """Given a stream, a call runs on it (after work already there), with outputs from its pool."""
    import torch
    from minimax_scale_search_b200 import cq
    w, _, _ = make_layer(264, 1024, 6)
    x, _ = values(np.random.default_rng(0), (50, 1024), "fp16")
    late = torch.zeros_like(x)
    ref, ref_ds = cq.w4_linear(x, w), cq.w4_linear_backward(cq.w4_linear(x, w), x, w)[1]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
    y = cq.w4_linear(late, w, stream=s)
    ds = cq.w4_linear_backward(y, late, w, stream=s)[1]
    s.synchronize()
    assert torch.equal(y, ref) and torch.equal(ds, ref_ds)


def test_offsets_beyond_32_bits():
    """Outputs of more than 2^31 elements: the rows at and behind the border against a small call of the same rows."""
    import torch
    from minimax_scale_search_b200 import cq
    T, R, K = 70001, 32768, 128
    w, _, _ = make_layer(R, K, 21)
    x = torch.randn((T, K), device="cuda").half()
    rows = torch.tensor([0, 1, 65535, 65536, 65537, *range(T - 60, T)], device="cuda")
    y, pre = cq.w4_linear(x, w, activation="silu", want_pre=True)
    y2, pre2 = cq.w4_linear(x[rows], w, activation="silu", want_pre=True)
    assert torch.equal(y[rows], y2) and torch.equal(pre[rows], pre2)
    dz, db = cq.activation_backward(y, pre, "silu", out=y)  # in place
    dz2, _ = cq.activation_backward(y2, pre2, "silu")
    assert torch.equal(dz[rows], dz2) and torch.isfinite(db).all()
    del pre
    dx, ds = cq.w4_linear_backward(dz, x, w)
    dx2, _ = cq.w4_linear_backward(dz2, None, w, want_dscales=False)
    # the small call shares the contraction of R among CTAs: each side's sum is off by at most R 2^-23 of its terms' sum
    terms = (dz2.double().abs() @ torch.from_numpy(np.abs(w4.weight(*make_layer(R, K, 21)[1:]))).cuda())
    assert bool(((dx[rows].double() - dx2.double()).abs() <= terms * 2 * (R * 2.0 ** -23) + 2 * U["fp16"] * dx2.double().abs() + TINY["fp16"]).all())
    half = 35008
    parts = sum(cq.w4_linear_backward(d, v, w, want_dx=False)[1].double() for d, v in ((dz[:half], x[:half]), (dz[half:], x[half:])))
    assert bool(((ds.double() - parts).norm() <= 1e-5 * parts.norm()))  # 136 spans of 512 tokens added in fp32, each 2^-24 off
    assert cq.w4_status() == cq.CQ_OK


def test_table_offsets_beyond_32_bits():
    import torch
    from minimax_scale_search_b200 import cq
    T, V, K = 20001, 64, 131072
    scales, codes = (device(a) for a in synth.make_codes(V * K // 128, seed=9))
    scales = torch.full_like(scales, 0x2000)
    ids = torch.randint(-1, V + 1, (T,), device="cuda")
    out = cq.w4_embedding(ids, scales, codes, K)
    rows = torch.tensor([0, 16383, 16384, 16385, *range(T - 5, T)], device="cuda")
    assert torch.equal(out[rows], cq.w4_embedding(ids[rows], scales, codes, K))
    g = cq.w4_embedding_backward(out, ids, codes)
    few = cq.w4_embedding_backward(out[-300:].contiguous(), ids[-300:].contiguous(), codes)
    count = torch.bincount(ids[(ids >= 0) & (ids < V)], minlength=V)
    late = torch.bincount(ids[-300:][(ids[-300:] >= 0) & (ids[-300:] < V)], minlength=V)
    # every token of a row has the same dots: a row's sum is its count of them (fp64 sums, rounded once)
    expect = few.double() / late.clamp(min=1)[:, None] * count[:, None]
    named = late > 0
    assert bool(((g.double() - expect)[named].abs() <= 3 * 2.0 ** -24 * expect[named].abs()).all())


def test_concurrent_calls_on_two_streams():
    """No state is shared between calls: two streams with calls of every kind at once."""
    import torch
    from minimax_scale_search_b200 import cq
    w, _, _ = make_layer(1032, 1152, 5)
    scales, codes, _, _ = make_table(500, 1152, 5)
    work = []
    for T in (9, 700):
        x, _ = values(np.random.default_rng(T), (T, 1152), "bf16")
        dz, _ = values(np.random.default_rng(T + 1), (T, 1032), "bf16")
        work.append((x, dz, torch.randint(-1, 500, (T,), device="cuda")))

    def all_of(x, dz, ids, stream):
        return (cq.w4_linear(x, w, stream=stream), *cq.w4_linear_backward(dz, x, w, stream=stream),
                *cq.activation_backward(dz, dz, "gelu", stream=stream),
                cq.w4_embedding(ids, scales, codes, 1152, stream=stream),
                cq.w4_embedding_backward(x, ids, codes, stream=stream))

    refs = [all_of(*v, None) for v in work]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[all_of(*v, s) for v, s in zip(work, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for run in got:
        for a, b in zip(run, refs):
            assert all(torch.equal(i, j) for i, j in zip(a, b))


@pytest.mark.parametrize("T,R,K", [(777, 1032, 2176), (40, 4096, 256), (2000, 136, 128)])
def test_gradients_in_a_row_over_the_same_buffers(T, R, K):
    """The launches of a call may overlap each other, but nothing before or after the call: inputs are
    written right before it and cleared right after it, with nothing waited for."""
    import torch
    from minimax_scale_search_b200 import cq
    rng = np.random.default_rng(T)
    w, _, _ = make_layer(R, K, T)
    inputs = [(values(rng, (T, R), "bf16")[0], values(rng, (T, K), "bf16")[0]) for _ in range(6)]
    want = []
    for dz, x in inputs:
        want.append(cq.w4_linear_backward(dz, x, w))
        torch.cuda.synchronize()
    dz, x, dx = torch.empty_like(inputs[0][0]), torch.empty_like(inputs[0][1]), torch.empty_like(inputs[0][1])
    ds = torch.empty_like(want[0][1])
    got = []
    torch.cuda.synchronize()
    for a, b in inputs:
        dz.copy_(a)
        x.copy_(b)
        cq.w4_linear_backward(dz, x, w, dx=dx, dscales=ds)
        dz.zero_()
        x.zero_()
        got.append((dx.clone(), ds.clone()))
        dx.fill_(-1)
        ds.fill_(-1)
    for (a, b), (c, d) in zip(got, want):
        assert torch.equal(a, c) and torch.equal(b, d)


@pytest.mark.parametrize("T,V,K", [(5, 40, 256), (1001, 300, 1152), (9000, 50, 384)])
def test_table_gradients_in_a_row_over_the_same_buffers(T, V, K):
    import torch
    from minimax_scale_search_b200 import cq
    rng = np.random.default_rng(T)
    codes = device(rng.integers(0, 2 ** 32, (V * (K // 128), 16), dtype=np.uint32))
    inputs = [(values(rng, (T, K), "bf16")[0], device(rng.integers(0, V, T))) for _ in range(6)]
    want = []
    for dout, ids in inputs:
        want.append(cq.w4_embedding_backward(dout, ids, codes))
        torch.cuda.synchronize()
    dout, ids, out = torch.empty_like(inputs[0][0]), torch.empty_like(inputs[0][1]), torch.empty_like(want[0])
    ws = torch.empty(cq.w4_embedding_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")
    got = []
    torch.cuda.synchronize()
    for a, b in inputs:
        dout.copy_(a)
        ids.copy_(b)
        cq.w4_embedding_backward(dout, ids, codes, out=out, workspace=ws)
        dout.zero_()
        ids.zero_()
        ws.zero_()
        got.append(out.clone())
        out.fill_(-1)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_gradients_that_overlap_their_operands_are_refused():
    import torch
    from minimax_scale_search_b200 import cq
    w, _, _ = make_layer(256, 256, 1)
    buf = torch.zeros(64 * 256, dtype=torch.float16, device="cuda")
    x, dz = buf[:8 * 256].view(8, 256), torch.zeros((8, 256), dtype=torch.float16, device="cuda")
    spare = buf[2048:2048 + 1024].view(torch.float32).view(2, 256)
    cq.w4_linear_backward(dz, x, w, dscales=spare)  # right behind x
    with pytest.raises(ValueError, match="dscales must not overlap"):
        cq.w4_linear_backward(dz, x, w, dscales=buf[2040:2040 + 1024].view(torch.float32).view(2, 256))
    with pytest.raises(ValueError, match="dscales must not overlap"):
        cq.w4_linear_backward(dz, dz, w, dx=buf[512:512 + 2048].view(8, 256), dscales=spare)
    codes = torch.zeros((40 * 2, 16), dtype=torch.int32, device="cuda")
    ids = torch.zeros(8, dtype=torch.int64, device="cuda")
    dout = torch.zeros((8, 256), dtype=torch.float32, device="cuda")
    with pytest.raises(ValueError, match="out must not overlap"):
        cq.w4_embedding_backward(dout, ids, codes, out=dout.view(-1)[:80].view(40, 2))
    with pytest.raises(ValueError, match="workspace must not overlap"):
        cq.w4_embedding_backward(dout, ids, torch.zeros_like(codes), workspace=dout)
    cq.w4_status()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_activation_gradient_in_place_over_many_rows(dt):
    """Rows are read ahead of those that are written: dz over dy or pre gives the same."""
    import torch
    from minimax_scale_search_b200 import cq
    rng = np.random.default_rng(8)
    dy, pre = values(rng, (5003, 136), dt, pad=8)[0], values(rng, (5003, 136), dt, 2.0, pad=8)[0]
    want, db = cq.activation_backward(dy, pre, "silu")
    for which in (0, 1):
        a = [torch.cat([t, t[:, :8]], 1)[:, :136] for t in (dy, pre)]
        got, b = cq.activation_backward(*a, "silu", out=a[which])
        assert got is a[which] and torch.equal(got, want) and torch.equal(b, db)
