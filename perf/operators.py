"""Timed cases of the operators around a quantized layer and its training loss.

Three operators, each in its forms for training and for serving:

  layer norm      forward, backward (with the reduction of the weight's and the
                  bias's gradient), and the forward fused with the per-token
                  s8 quantizer that feeds the W8A8 product;
  W8A8 product    with bias, activation and residual in its epilogue, from one
                  token to thousands, and the backward of that epilogue;
  distillation    a student's logits against a teacher's top logits: loss,
                  gradient, and both in one call.

``listed()`` gives the cases, ``draw(rng)`` one more of the same ranges,
``prepare(case, seed)`` the inputs on the GPU and ``run(state)`` one pass.
With ``own`` false a pass is the operator written in elementary torch
operations in 32 bits; with ``own`` true it is the call of the library.
``exact(case, seed)`` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
ACT_FLOPS = {"none": 0, "relu": 1, "silu": 4, "gelu": 8, "gelu_tanh": 9}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the norm of one token in decoding: latency only
        {"name": "norm 1x4096 bf16", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "wdtype": "bf16"},
        # a training step's or a prompt's tokens, the size of the per-token quantizer's workload
        {"name": "norm 8192x4096 bf16", "op": "norm", "rows": 8192, "cols": 4096, "dtype": "bf16", "wdtype": "f32"},
        # the same tokens on the way back
        {"name": "norm backward 8192x4096 bf16", "op": "norm_backward", "rows": 8192, "cols": 4096, "dtype": "bf16",
         "wdtype": "f32"},
        # an odd width, whose rows start at any alignment, in full precision
        {"name": "norm backward 1021x5003 f32", "op": "norm_backward", "rows": 1021, "cols": 5003, "dtype": "f32",
         "wdtype": "f32"},
        # one token through norm, quantizer and the up projection: the decoding step of a W8A8 block
        {"name": "norm+product 1x4096x11008", "op": "norm_product", "m": 1, "n": 11008, "k": 4096, "dtype": "bf16",
         "act": "gelu_tanh", "bias": True, "residual": False},
        # sixteen sequences decoding together, the down projection with the residual added
        {"name": "product 16x4096x11008", "op": "product", "m": 16, "n": 4096, "k": 11008, "dtype": "bf16",
         "act": "none", "bias": True, "residual": True},
        # a prompt of ragged length
        {"name": "product 777x4096x4096 f16", "op": "product", "m": 777, "n": 4096, "k": 4096, "dtype": "f16",
         "act": "silu", "bias": True, "residual": True},
        # the W8A8 product of the library's own benchmark, now with its epilogue
        {"name": "product 8192x11008x4096", "op": "product", "m": 8192, "n": 11008, "k": 4096, "dtype": "bf16",
         "act": "gelu_tanh", "bias": True, "residual": False},
        # the way back through that epilogue
        {"name": "epilogue backward 8192x11008", "op": "epilogue_backward", "m": 8192, "n": 11008, "dtype": "bf16",
         "act": "gelu_tanh"},
        # loss, then gradient, as a program with automatic differentiation calls them
        {"name": "distill 512x32000 f32", "op": "distill", "rows": 512, "vocab": 32000, "k": 64, "dtype": "f32",
         "temperature": 2.0, "rest": False, "padded": False},
        # a training step's tokens over a large vocabulary, loss and gradient in one call
        {"name": "distill_grad 4096x131072 bf16", "op": "distill_grad", "rows": 4096, "vocab": 131072, "k": 128,
         "dtype": "bf16", "temperature": 1.0, "rest": True, "padded": False},
        # a few rows over a large vocabulary of odd size, some of them without teacher entries
        {"name": "distill_grad 9x131001 f16", "op": "distill_grad", "rows": 9, "vocab": 131001, "k": 32,
         "dtype": "f16", "temperature": 1.5, "rest": True, "padded": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_backward", "norm_product", "product", "product", "epilogue_backward", "distill",
                     "distill_grad"))
    dtype = rng.choice(("bf16", "f16", "f32"))
    if op in ("norm", "norm_backward"):
        cols = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            cols = (cols + 7) // 8 * 8
        rows = _log(rng, 1, min(8192, 8192 * 4096 * 2 // (cols * SIZE[dtype])))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "wdtype": rng.choice((dtype, "f32"))}
    if op in ("norm_product", "product"):
        n, k = _log(rng, 128, 11008), _log(rng, 128, 11008)
        if rng.random() < 0.8:
            k = (k + 15) // 16 * 16
        m = _log(rng, 1, 8192)
        while m * n * k > 8192 * 11008 * 4096 // 4:
            m = (m + 1) // 2
        return {"op": op, "m": m, "n": n, "k": k, "dtype": dtype, "act": rng.choice(ACTS),
                "bias": rng.random() < 0.7, "residual": rng.random() < 0.5}
    if op == "epilogue_backward":
        n = _log(rng, 128, 11008)
        m = _log(rng, 1, min(8192, 8192 * 11008 * 2 // (n * SIZE[dtype])))
        return {"op": op, "m": m, "n": n, "dtype": dtype, "act": rng.choice(ACTS)}
    vocab = _log(rng, 1000, 131072)
    if rng.random() < 0.6:
        vocab = (vocab + 7) // 8 * 8
    rows = _log(rng, 1, min(4096, 4096 * 131072 // 4 // vocab))
    return {"op": op, "rows": rows, "vocab": vocab, "k": _log(rng, 1, 256), "dtype": dtype,
            "temperature": rng.choice((1.0, 1.5, 2.0)), "rest": rng.random() < 0.5, "padded": rng.random() < 0.4}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    if op in ("norm", "norm_backward"):
        rows, cols, wdt = case["rows"], case["cols"], DTYPES[case["wdtype"]]
        x32 = normal(rows, cols) * (0.5 + uniform(rows, 1)) + 0.5 * normal(rows, 1)
        s["x"] = x32.to(dt)
        s["weight"] = (1.0 + 0.2 * normal(cols)).to(wdt)
        if op == "norm":
            s["bias"] = (0.1 * normal(cols)).to(wdt)
        else:   # what the forward pass kept, and what comes back
            x64 = s["x"].double()
            s["mean"] = x64.mean(1).float()
            s["rstd"] = (x64.var(1, correction=0) + EPS).rsqrt().float()
            s["dy"] = normal(rows, cols).to(dt)
        return s
    if op in ("norm_product", "product"):
        m, n, k = case["m"], case["n"], case["k"]
        if op == "norm_product":
            s["x"] = (normal(m, k) * (0.5 + uniform(m, 1)) + 0.5 * normal(m, 1)).to(dt)
            s["weight"] = (1.0 + 0.2 * normal(k)).to(dt)
            s["shift"] = (0.1 * normal(k)).to(dt)
        else:   # codes of roughly normal activations whose largest value is at 127
            s["qx"] = (normal(m, k) * 32).round().clamp(-127, 127).to(torch.int8)
            s["sx"] = (0.5 + uniform(m)) / 32
        s["qw"] = (normal(n, k) * 32).round().clamp(-127, 127).to(torch.int8)
        s["sw"] = (0.5 + uniform(n)) / (32 * math.sqrt(k))
        s["bias"] = (0.5 * normal(n)).to(dt) if case["bias"] else None
        s["residual"] = normal(m, n).to(dt) if case["residual"] else None
        return s
    if op == "epilogue_backward":
        s["dy"] = normal(case["m"], case["n"]).to(dt)
        s["z"] = (1.5 * normal(case["m"], case["n"])).to(dt)
        return s
    rows, vocab = case["rows"], case["vocab"]
    k = min(case["k"], vocab // 2)
    banned = vocab // 100 if case["padded"] else 0   # columns past the tokenizer's own, held at -inf
    live = vocab - banned
    perm = torch.randperm(live, generator=g, device="cuda")
    at = (torch.arange(rows, device="cuda")[:, None] * k + torch.arange(k, device="cuda")[None, :]) % live
    idx = perm[at]
    val = (8.0 + 2.0 * normal(rows, k)).sort(1, descending=True).values
    logits = 2.0 * normal(rows, vocab)
    logits.scatter_add_(1, idx, 0.7 * val + 0.5 * normal(rows, k))   # a student that has begun to follow the teacher
    if banned:
        logits[:, live:] = -math.inf
        left = torch.randint(0, k + 1, (rows, 1), generator=g, device="cuda")   # entries a row has; some have none
        idx = torch.where(torch.arange(k, device="cuda")[None, :] < left, idx, torch.full_like(idx, -1))
    s["logits"] = logits.to(dt)
    s["idx"], s["val"] = idx, val
    inv_t = 1.0 / case["temperature"]
    s["teacher_lse"] = (torch.logsumexp(val.double() * inv_t, 1) + 0.02 + 0.3 * uniform(rows)).float() if case["rest"] else None
    s["dloss"] = (0.5 + uniform(rows)) / rows
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import tensor_quantization_amd as tq
    c = s["case"]
    op = c["op"]
    if op == "norm":
        return tq.tq_layer_norm(s["x"], s["weight"], s["bias"], EPS)
    if op == "norm_backward":
        return tq.tq_layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
    if op == "norm_product":
        qx, sx = tq.tq_layer_norm_quant_per_token(s["x"], s["weight"], s["shift"], EPS)
        return tq.tq_w8a8_linear_epilogue(qx, sx, s["qw"], s["sw"], bias=s["bias"], act=c["act"],
                                          residual=s["residual"], out_dtype=DTYPES[c["dtype"]])
    if op == "product":
        return tq.tq_w8a8_linear_epilogue(s["qx"], s["sx"], s["qw"], s["sw"], bias=s["bias"], act=c["act"],
                                          residual=s["residual"], out_dtype=DTYPES[c["dtype"]])
    if op == "epilogue_backward":
        return tq.tq_linear_epilogue_backward(s["dy"], s["z"], act=c["act"])
    t = c["temperature"]
    if op == "distill":
        loss, stats, rest_sum = tq.tq_topk_distill(s["logits"], s["idx"], s["val"], temperature=t,
                                                   teacher_lse=s["teacher_lse"])
        return loss, tq.tq_topk_distill_backward(s["logits"], s["idx"], s["val"], stats, s["dloss"], temperature=t,
                                                 teacher_lse=s["teacher_lse"], rest_sum=rest_sum)
    return tq.tq_topk_distill_grad(s["logits"], s["idx"], s["val"], dloss=s["dloss"], temperature=t,
                                   teacher_lse=s["teacher_lse"])


def _act32(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope32(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _norm32(x, weight, bias):
    x = x.float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    return d * rstd * weight.float() + bias.float(), mean[:, 0], rstd[:, 0]


def _plain(s):
    c = s["case"]
    op, dt = c["op"], DTYPES[c["dtype"]]
    if op == "norm":
        y, mean, rstd = _norm32(s["x"], s["weight"], s["bias"])
        return y.to(dt), mean, rstd
    if op == "norm_backward":
        x, dy, w, rstd = s["x"].float(), s["dy"].float(), s["weight"].float(), s["rstd"][:, None]
        xhat = (x - s["mean"][:, None]) * rstd
        dxhat = dy * w
        dx = rstd * (dxhat - dxhat.mean(1, keepdim=True) - xhat * (dxhat * xhat).mean(1, keepdim=True))
        return dx.to(dt), (dy * xhat).sum(0).to(s["weight"].dtype), dy.sum(0).to(s["weight"].dtype)
    if op in ("norm_product", "product"):
        if op == "norm_product":   # the normed tokens in their own type, then codes with one scale a token
            h = _norm32(s["x"], s["weight"], s["shift"])[0].to(dt).float()
            sx = h.abs().amax(1) / 127
            sx = torch.where(sx == 0, torch.ones_like(sx), sx)
            qx = torch.round(h / sx[:, None]).clamp(-127, 127)
        else:
            qx, sx = s["qx"].float(), s["sx"]
        z = (qx @ s["qw"].float().t()) * sx[:, None] * s["sw"][None, :]
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act32(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(dt)
    if op == "epilogue_backward":
        dz = s["dy"].float() * _act_slope32(s["z"].float(), c["act"])
        return dz.to(dt), dz.sum(0)
    return _distill32(s, c, dt)


def _distill32(s, c, dt):
    inv_t = 1.0 / c["temperature"]
    idx, here = s["idx"], s["idx"] >= 0
    at = torch.where(here, idx, torch.zeros_like(idx))
    # the teacher: probabilities of its top entries, and what the rest of the vocabulary has
    tv = torch.where(here, s["val"] * inv_t, torch.full_like(s["val"], -math.inf))
    top = tv.amax(1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    if c["rest"]:
        logp = tv - s["teacher_lse"][:, None]
    else:
        logp = tv - (torch.log(torch.exp(tv - top).sum(1, keepdim=True)) + top)
    logp = torch.where(here, logp, torch.zeros_like(logp))
    p = torch.where(here, torch.exp(logp), torch.zeros_like(logp))
    # the student
    z = s["logits"].float() * inv_t
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    lse = torch.log(e.sum(1, keepdim=True)) + m
    loss = (p * (logp - torch.where(here, z.gather(1, at) - lse, torch.zeros_like(p)))).sum(1)
    q = torch.exp(z - lse)
    mass = p.sum(1, keepdim=True)
    some = here.any(1, keepdim=True)
    if c["rest"]:
        p_rest = torch.where(some, (1 - mass).clamp_min(0), torch.zeros_like(mass))
        inside = torch.zeros(z.shape[0], z.shape[1] + 1, dtype=torch.bool, device=z.device)
        inside.scatter_(1, torch.where(here, idx, torch.full_like(idx, z.shape[1])), True)
        inside = inside[:, :-1]
        q_out = torch.where(inside, torch.zeros_like(q), q)
        q_rest = q_out.sum(1, keepdim=True)
        rest = p_rest * (torch.log(p_rest) - torch.log(q_rest))
        loss = loss + torch.where(p_rest > 0, rest, torch.zeros_like(rest))[:, 0]
        grad = q * (mass + p_rest) - q_out * torch.where(p_rest > 0, p_rest / q_rest, torch.zeros_like(p_rest))
    else:
        grad = q * mass
    grad.scatter_add_(1, at, -p)
    return loss, (grad * (inv_t * s["dloss"][:, None])).to(dt)


# ------------------------------------------------------------- work, exact
def work(case):
    op, size = case["op"], SIZE[case["dtype"]]
    if op in ("norm", "norm_backward"):
        n, w = case["rows"] * case["cols"], SIZE[case["wdtype"]] * case["cols"]
        if op == "norm":
            return {"bytes": 2 * n * size + 2 * w + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * size + 3 * w + 8 * case["rows"], "flops": 14 * n}
    if op in ("norm_product", "product"):
        m, n, k = case["m"], case["n"], case["k"]
        b = n * k + 4 * n + m * n * size * (2 if case["residual"] else 1) + (n * size if case["bias"] else 0)
        b += m * k * size + 2 * k * size if op == "norm_product" else m * k + 4 * m
        f = 2 * m * n * k + m * n * (3 + ACT_FLOPS[case["act"]]) + (12 * m * k if op == "norm_product" else 0)
        return {"bytes": b, "flops": f}
    if op == "epilogue_backward":
        n = case["m"] * case["n"]
        return {"bytes": 3 * n * size + 4 * case["n"], "flops": n * (2 + 2 * ACT_FLOPS[case["act"]])}
    n, k = case["rows"] * case["vocab"], min(case["k"], case["vocab"] // 2)
    return {"bytes": 2 * n * size + case["rows"] * (12 * k + 8 + (4 if case["rest"] else 0)), "flops": 10 * n}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS).rsqrt()
        y = torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], s["weight"].double())
        return y, mean, rstd
    if op == "norm_backward":
        # with the statistics that are handed in, dx = rstd (g - <g> - xhat <g xhat>), g = dy w
        xhat = (s["x"].double() - s["mean"].double()[:, None]) * s["rstd"].double()[:, None]
        dy = s["dy"].double()
        g = dy * s["weight"].double()
        both = torch.stack((g.sum(1), (g * xhat).sum(1))) / case["cols"]
        dx = (g - both[0][:, None] - xhat * both[1][:, None]) * s["rstd"].double()[:, None]
        return dx, torch.einsum("ij,ij->j", dy, xhat), dy.sum(0)
    if op in ("norm_product", "product"):
        if op == "norm_product":
            x = s["x"].double()
            var, mean = torch.var_mean(x, 1, correction=0)
            h = (x - mean[:, None]) * (var + EPS).rsqrt()[:, None] * s["weight"].double() + s["shift"].double()
            h = h.to(DTYPES[case["dtype"]]).double()
            sx = h.abs().amax(1) / 127
            sx[sx == 0] = 1
            qx = (h / sx[:, None]).round()
        else:
            qx, sx = s["qx"].double(), s["sx"].double()
        z = torch.mm(qx, s["qw"].double().t()).mul_(sx[:, None]).mul_(s["sw"].double())
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _act64(z, case["act"])
        return y if s["residual"] is None else y + s["residual"].double()
    if op == "epilogue_backward":
        z = s["z"].double().requires_grad_()
        _act64(z, case["act"]).backward(s["dy"].double())
        return z.grad, z.grad.sum(0)
    # distillation: the loss as it is defined, its gradient by differentiating it, a few rows at a time
    losses, grads = [], []
    step = max(1, (1 << 26) // case["vocab"])
    for i in range(0, case["rows"], step):
        loss, grad = _distill64(case, *(None if s[v] is None else s[v][i:i + step]
                                        for v in ("logits", "idx", "val", "teacher_lse", "dloss")))
        losses.append(loss)
        grads.append(grad)
    return torch.cat(losses), torch.cat(grads)


def _act64(z, act):
    f = torch.nn.functional
    return {"none": lambda: z * 1, "relu": lambda: f.relu(z), "silu": lambda: f.silu(z), "gelu": lambda: f.gelu(z),
            "gelu_tanh": lambda: f.gelu(z, approximate="tanh")}[act]()


def _distill64(case, logits, idx, val, teacher_lse, dloss):
    z = logits.double().requires_grad_()
    here = idx >= 0
    logq = torch.log_softmax(z / case["temperature"], 1)
    t = (val.double() / case["temperature"]).masked_fill(~here, -math.inf)
    logp = t - teacher_lse.double()[:, None] if case["rest"] else torch.log_softmax(t, 1)
    logp = logp.masked_fill(~here, 0)
    p = logp.exp().masked_fill(~here, 0)
    loss = (p * (logp - logq.gather(1, idx.clamp_min(0)).masked_fill(~here, 0))).sum(1)
    if case["rest"]:
        p_rest = (1 - p.sum(1)).clamp_min(0) * here.any(1)
        taken = torch.zeros_like(logits, dtype=torch.uint8)
        taken.scatter_add_(1, idx.clamp_min(0), here.to(torch.uint8))
        log_rest = torch.logsumexp(logq.masked_fill(taken > 0, -math.inf), 1)
        loss = loss + torch.where(p_rest > 0, p_rest * (p_rest.log() - log_rest), torch.zeros_like(p_rest))
    loss.backward(dloss.double())
    return loss.detach(), z.grad
