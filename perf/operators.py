"""Operators on 4-bit weights in groups of 128, as measured cases.

Each case is one call that a program makes with the framework's quantised tensors:

* ``linear``: y = act(x W^T + b) + residual from the GPTQ v1 tensors of a layer;
* ``linear_backward``: the gradients of that layer's input and of its group scales;
* ``activation_backward``: the gradient at the activation's argument, and the bias' gradient;
* ``embedding``: rows of a quantised table, scaled;
* ``embedding_backward``: the gradient of the table's group scales, summed by token.

``run`` computes them in plain torch where ``own`` is false, and through the framework where it is true.
"""
import math

import torch

own = False

GROUP = 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # one new token through a small projection: nothing but latency
        dict(name="linear_token", op="linear", dtype="bf16", T=1, R=1024, K=1024, act="none", bias=True, residual=False,
             pre=False, symmetric=True, wide=False),
        # thirteen sequences, one new token each, through the sweep's layer: the weights' bytes
        dict(name="linear_batch", op="linear", dtype="fp16", T=13, R=30336, K=16384, act="none", bias=True,
             residual=True, pre=False, symmetric=True, wide=False),
        # a short ragged prompt through a layer whose sizes fill no tile, zero points of their own, strided rows
        dict(name="linear_ragged", op="linear", dtype="fp16", T=333, R=4104, K=1152, act="gelu", bias=True,
             residual=False, pre=True, symmetric=False, wide=True),
        # a training step's tokens through the large workload's layer: tensor throughput
        dict(name="linear_prompt", op="linear", dtype="bf16", T=4096, R=14336, K=4096, act="silu", bias=True,
             residual=True, pre=True, symmetric=True, wide=False),
        # a small fine-tuning batch of odd sizes, backwards
        dict(name="grad_ragged", op="linear_backward", dtype="fp16", T=777, R=1032, K=2176, symmetric=False, wide=True),
        # the training step's layer, backwards
        dict(name="grad_prompt", op="linear_backward", dtype="bf16", T=4096, R=14336, K=4096, symmetric=True,
             wide=False),
        # the activation of a small odd layer, backwards
        dict(name="act_ragged", op="activation_backward", dtype="fp16", T=333, R=1032, act="gelu"),
        # the training step's activation, backwards
        dict(name="act_prompt", op="activation_backward", dtype="bf16", T=4096, R=14336, act="silu"),
        # the new tokens of a decode batch
        dict(name="embed_batch", op="embedding", dtype="bf16", T=16, V=30336, K=1024, multiplier=1.0),
        # the tokens of a long prompt, scaled by the square root of the width
        dict(name="embed_prompt", op="embedding", dtype="fp16", T=8192, V=30336, K=4096, multiplier=64.0),
        # a small odd batch, gradients kept in 32 bits
        dict(name="embed_grad_ragged", op="embedding_backward", dtype="fp32", T=1001, V=8192, K=1152, multiplier=1.0),
        # a training step's tokens
        dict(name="embed_grad_prompt", op="embedding_backward", dtype="bf16", T=8192, V=30336, K=4096, multiplier=64.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_backward", "activation_backward", "embedding", "embedding_backward"))
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("linear", "linear_backward"):
        while True:
            T, R, K = _log_int(rng, 1, 4096), 8 * _log_int(rng, 1, 3792), GROUP * _log_int(rng, 1, 128)
            if T * R * K <= 4096 * 14336 * 4096 and T * max(R, K) <= 4096 * 14336 and R * K >= 1 << 16:
                break
        case = dict(op=op, dtype=rng.choice(("bf16", "fp16")), T=T, R=R, K=K, symmetric=flag(), wide=flag())
        if op == "linear":
            case.update(act=rng.choice(ACTIVATIONS), bias=flag(), residual=flag(), pre=flag())
        return case
    if op == "activation_backward":
        return dict(op=op, dtype=rng.choice(("bf16", "fp16")), T=_log_int(rng, 1, 4096), R=8 * _log_int(rng, 1, 1792),
                    act=rng.choice(ACTIVATIONS[1:]))
    T, V, K = _log_int(rng, 1, 8192), _log_int(rng, 16, 30336), GROUP * _log_int(rng, 1, 32)
    return dict(op=op, dtype=rng.choice(("bf16", "fp16", "fp32")), T=T, V=V, K=K,
                multiplier=rng.choice((1.0, math.sqrt(K))))


# ---- inputs ---------------------------------------------------------------------------------------------------------


def _normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda") * std


def _nibbles(gen, shape):
    """Codes 0..15 of normally distributed weights under the scale that the selection gives them."""
    return (torch.randn(shape, generator=gen, device="cuda") * 2.6).round_().add_(8).clamp_(0, 15).to(torch.int32)


def _words(gen, shape):
    """int32 words of eight nibbles, low nibble first."""
    w = _nibbles(gen, shape)
    for j in range(1, 8):
        w |= _nibbles(gen, shape) << (4 * j)
    return w


def _scales(gen, shape):
    return (0.02 / 2.6 * torch.exp(_normal(gen, shape, 0.3))).to(torch.float16)


def _rows(gen, T, n, dtype, std, wide):
    """[T, n] values with a few large columns; where `wide`, the first n columns of a wider buffer."""
    ld = n + 64 if wide else n
    gain = torch.where(torch.rand(ld, generator=gen, device="cuda") < 0.005, 8.0, 1.0)
    return (_normal(gen, (T, ld), std) * gain).to(dtype)[:, :n]


def _ids(gen, T, V):
    """Token numbers, the low ones far more frequent; one in 64 is padding (-1)."""
    ids = (V * torch.rand(T, generator=gen, device="cuda", dtype=torch.float64) ** 3).to(torch.int64)
    return torch.where(torch.rand(T, generator=gen, device="cuda") < 1 / 64, -1, ids)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s, op, dt = dict(case), case["op"], DTYPES[case["dtype"]]
    T, R, K, V = (case.get(k) for k in ("T", "R", "K", "V"))
    if op in ("linear", "linear_backward"):
        s["qweight"], s["scales"] = _words(gen, (K // 8, R)), _scales(gen, (K // GROUP, R))
        if case["symmetric"]:
            s["qzeros"] = torch.full((K // GROUP, R // 8), 0x77777777, dtype=torch.int32, device="cuda")
        else:
            s["qzeros"] = _words(gen, (K // GROUP, R // 8))
        s["g_idx"] = torch.arange(K, dtype=torch.int32, device="cuda") // GROUP
        s["x"] = _rows(gen, T, K, dt, 1.0, case["wide"])
        if op == "linear":
            s["b"] = _normal(gen, (R,), 0.1).to(dt) if case["bias"] else None
            s["res"] = _normal(gen, (T, R)).to(dt) if case["residual"] else None
        else:
            s["dz"] = _rows(gen, T, R, dt, 0.05, case["wide"])
        if own:
            from minimax_scale_search_b200 import cq
            s["weights"] = cq.w4_weights(cq.GPTQTensors(s["qweight"], s["qzeros"], s["scales"], s["g_idx"]))
    elif op == "activation_backward":
        s["z"], s["dy"] = _normal(gen, (T, R), 1.5).to(dt), _normal(gen, (T, R), 0.05).to(dt)
    else:
        s["codes"], s["scales"] = _words(gen, (V * K // GROUP, 16)), _scales(gen, (V * K // GROUP,))
        s["ids"] = _ids(gen, T, V)
        if op == "embedding_backward":
            s["dout"] = _rows(gen, T, K, dt, 0.05, False)
    return s


# ---- one pass -------------------------------------------------------------------------------------------------------


def _nibble_shifts():
    return torch.arange(0, 32, 4, dtype=torch.int32, device="cuda")


def _layer_codes(s):
    """u - (z + 1) of every weight, float32 [K/128, 128, R]."""
    K, R, sh = s["K"], s["R"], _nibble_shifts()
    u = ((s["qweight"][:, None, :] >> sh[None, :, None]) & 15).view(K // GROUP, GROUP, R)
    z = ((s["qzeros"][:, :, None] >> sh) & 15).view(K // GROUP, 1, R)
    return (u - (z + 1)).float()


def _activation(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z / (1 + torch.exp(-z))


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def _run_own(s):
    from minimax_scale_search_b200 import cq
    op, dt = s["op"], DTYPES[s["dtype"]]
    if op == "linear":
        got = cq.w4_linear(s["x"], s["weights"], bias=s["b"], activation=s["act"], residual=s["res"],
                           want_pre=s["pre"])
        return {"y": got[0], "pre": got[1]} if s["pre"] else {"y": got}
    if op == "linear_backward":
        dx, dscales = cq.w4_linear_backward(s["dz"], s["x"], s["weights"])
        return {"dx": dx, "dscales": dscales}
    if op == "activation_backward":
        dz, dbias = cq.activation_backward(s["dy"], s["z"], s["act"])
        return {"dz": dz, "dbias": dbias}
    if op == "embedding":
        return {"out": cq.w4_embedding(s["ids"], s["scales"], s["codes"], s["K"], multiplier=s["multiplier"], dtype=dt)}
    return {"dscales": cq.w4_embedding_backward(s["dout"], s["ids"], s["codes"], multiplier=s["multiplier"])}


def run(s):
    if own:
        return _run_own(s)
    op, dt = s["op"], DTYPES[s["dtype"]]
    T, R, K, V = (s.get(k) for k in ("T", "R", "K", "V"))
    if op == "linear":
        w = (_layer_codes(s) * s["scales"].float()[:, None, :]).view(K, R)
        z = s["x"].float() @ w
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _activation(z, s["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"y": y.to(dt), "pre": z.to(dt)} if s["pre"] else {"y": y.to(dt)}
    if op == "linear_backward":
        n, dz = _layer_codes(s), s["dz"].float()
        dx = dz @ (n * s["scales"].float()[:, None, :]).view(K, R).t()
        dw = (s["x"].float().t() @ dz).view(K // GROUP, GROUP, R)
        return {"dx": dx.to(dt), "dscales": (dw * n).sum(1)}
    if op == "activation_backward":
        dz = s["dy"].float() * _slope(s["z"].float(), s["act"])
        return {"dz": dz.to(dt), "dbias": dz.sum(0)}
    ng, ids = K // GROUP, s["ids"]
    fine = (ids >= 0) & (ids < V)
    at = torch.where(fine, ids, 0)
    q = ((s["codes"].view(V, ng, 16)[at][..., None] >> _nibble_shifts()) & 15).view(T, ng, GROUP).float() - 8
    if op == "embedding":
        out = q * s["scales"].view(V, ng)[at].float()[..., None] * s["multiplier"]
        return {"out": torch.where(fine[:, None], out.view(T, K), 0.0).to(dt)}
    p = (s["dout"].float().view(T, ng, GROUP) * q).sum(-1) * fine[:, None]
    total = torch.zeros((V, ng), dtype=torch.float64, device="cuda").index_add_(0, at, p.double())
    return {"dscales": (total * s["multiplier"]).float()}


# ---- what a pass cannot do without -----------------------------------------------------------------------------------


def _distinct(T, V):
    """Expected number of distinct tokens among T of _ids()."""
    edge = torch.arange(V + 1, dtype=torch.float64) / V
    p = (edge ** (1 / 3)).diff() * (63 / 64)
    return float((1 - (1 - p) ** T).sum())


def work(case):
    op, e = case["op"], {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    T, R, K, V = (case.get(k, 0) for k in ("T", "R", "K", "V"))
    layer = R * K / 2 + R * K / GROUP * 2 + R * K / GROUP / 2
    if op == "linear":
        outs = 1 + bool(case["residual"]) + bool(case["pre"])
        return {"bytes": layer + e * (T * K + outs * T * R + R * bool(case["bias"])), "flops": 2.0 * T * R * K}
    if op == "linear_backward":
        return {"bytes": layer + e * (2 * T * K + T * R) + 4 * R * K / GROUP, "flops": 4.0 * T * R * K}
    if op == "activation_backward":
        return {"bytes": 3.0 * e * T * R + 4 * R, "flops": 10.0 * T * R}
    rows = _distinct(T, V)
    if op == "embedding":
        return {"bytes": 8 * T + rows * (K / 2 + K / GROUP * 2) + e * T * K, "flops": 2.0 * T * K}
    return {"bytes": 8 * T + rows * K / 2 + e * T * K + 4 * V * K / GROUP, "flops": 2.0 * T * K}


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------------


def _bytes_to_codes(words):
    """The eight nibbles of each word in a new last dimension, by the bytes of the words."""
    b = words.contiguous().view(torch.uint8).view(*words.shape, 4)
    return torch.stack((b % 16, b // 16), dim=-1).flatten(-2)


def _exact_layer(s):
    """(n, scale) of a layer as float64: n [R, K] and the scale of every weight [R, K/128]."""
    R, K = s["R"], s["K"]
    u = _bytes_to_codes(s["qweight"].t()).view(R, K // GROUP, GROUP)
    z = _bytes_to_codes(s["qzeros"]).view(K // GROUP, R).t()
    return u.double().sub_(z.double()[:, :, None] + 1), s["scales"].t().double()


def _exact_activation(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _exact_slope(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    if act == "gelu_tanh":
        p, inner = torch.sigmoid(2 * c * (z + 0.044715 * z * z * z)), c * (1 + 0.134145 * z * z)
        return p + z * 2 * p * (1 - p) * inner
    p = torch.sigmoid(z)
    return p + z * p * (1 - p)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    T, R, K, V = (case.get(k) for k in ("T", "R", "K", "V"))
    if op == "linear":
        n, scale = _exact_layer(s)
        z = torch.einsum("tk,rk->tr", s["x"].double(), n.mul_(scale[:, :, None]).view(R, K))
        z = z + (0 if s["b"] is None else s["b"].double())
        y = _exact_activation(z, case["act"]) + (0 if s["res"] is None else s["res"].double())
        return {"y": y, "pre": z} if case["pre"] else {"y": y}
    if op == "linear_backward":
        n, scale = _exact_layer(s)
        dw = torch.einsum("tr,tk->rk", s["dz"].double(), s["x"].double()).view(R, K // GROUP, GROUP)
        dscales = torch.einsum("rgi,rgi->gr", dw, n)
        dx = torch.einsum("tr,rk->tk", s["dz"].double(), n.mul_(scale[:, :, None]).view(R, K))
        return {"dx": dx, "dscales": dscales}
    if op == "activation_backward":
        dz = s["dy"].double() * _exact_slope(s["z"].double(), case["act"])
        return {"dz": dz, "dbias": dz.sum(0)}
    ng, ids = K // GROUP, s["ids"]
    rows = _bytes_to_codes(s["codes"].view(V, K // 8)[ids.clamp(0, V - 1)]).view(T, ng, GROUP).double() - 8
    rows[(ids < 0) | (ids >= V)] = 0
    if op == "embedding":
        scale = s["scales"].double().view(V, ng)[ids.clamp(0, V - 1)]
        return {"out": (rows * (scale * case["multiplier"])[:, :, None]).view(T, K)}
    dots = torch.einsum("tgi,tgi->tg", s["dout"].double().view(T, ng, GROUP), rows) * case["multiplier"]
    total = torch.zeros((V, ng), dtype=torch.float64, device="cuda")
    return {"dscales": total.index_put_((ids.clamp(0, V - 1),), dots, accumulate=True)}
