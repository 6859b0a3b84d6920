"""Timed cases of a gated quantized block, of the adapters served beside a
quantized projection and of the policy loss that trains them.

  gated block     both W8A8 projections, the activation and the product in one
                  call, from one token to thousands, with or without the values
                  that training keeps, and the way back through the gate;
  adapters        the W8A8 product beside low-rank adapters, every token with
                  the adapter of its request or none;
  policy loss     a token's log-probability from the logits, the clipped policy
                  loss with its KL term, their gradients.

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
ACTS = ("relu", "silu", "gelu", "gelu_tanh")
ACT_FLOPS = {"none": 0, "relu": 1, "silu": 4, "gelu": 8, "gelu_tanh": 9}
CLIP = 0.2
KL = 0.05


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token in decoding: the two up projections' weights are read, latency counts
        {"name": "gated 1x4096x11008", "op": "gated", "m": 1, "f": 11008, "k": 4096, "dtype": "bf16", "act": "silu",
         "bias": False, "keep": False},
        # a prompt of ragged length
        {"name": "gated 777x4096x4096 f16", "op": "gated", "m": 777, "f": 4096, "k": 4096, "dtype": "f16",
         "act": "gelu_tanh", "bias": True, "keep": False},
        # a training step's forward pass that keeps what the way back needs, at odd sizes in full precision
        {"name": "gated kept 1021x5003x2501 f32", "op": "gated", "m": 1021, "f": 2501, "k": 5003, "dtype": "f32",
         "act": "gelu", "bias": True, "keep": True},
        # a long prompt's or a training step's tokens: the size of the W8A8 benchmark, twice over
        {"name": "gated 8192x4096x11008", "op": "gated", "m": 8192, "f": 11008, "k": 4096, "dtype": "bf16",
         "act": "silu", "bias": False, "keep": False},
        # the way back through the gate of those tokens
        {"name": "gated backward 8192x11008", "op": "gated_backward", "m": 8192, "f": 11008, "dtype": "bf16",
         "act": "silu"},
        # one request's next token with its adapter
        {"name": "adapters 1x4096x11008 r16", "op": "adapters", "m": 1, "n": 11008, "k": 4096, "rank": 16,
         "adapters": 8, "requests": 1, "dtype": "bf16", "act": "none", "bias": False, "residual": False},
        # requests that decode together, each with its own adapter, some with none
        {"name": "adapters 48x11008x4096 r16", "op": "adapters", "m": 48, "n": 4096, "k": 11008, "rank": 16,
         "adapters": 32, "requests": 48, "dtype": "bf16", "act": "none", "bias": True, "residual": True},
        # the prompts of a dozen requests in one batch
        {"name": "adapters 4096x4096x4096 r64 f16", "op": "adapters", "m": 4096, "n": 4096, "k": 4096, "rank": 64,
         "adapters": 9, "requests": 12, "dtype": "f16", "act": "silu", "bias": True, "residual": False},
        # log-probabilities of a batch of next tokens under the reference model
        {"name": "logp 64x131072 bf16", "op": "logp", "rows": 64, "vocab": 131072, "dtype": "bf16",
         "temperature": 1.0, "ref": False, "padded": False},
        # loss, then gradient, as a program with automatic differentiation calls them
        {"name": "policy 512x32000 f32", "op": "policy", "rows": 512, "vocab": 32000, "dtype": "f32",
         "temperature": 1.0, "ref": True, "padded": False},
        # a training step's tokens over a large vocabulary, loss and gradient in one call
        {"name": "policy_grad 4096x131072 bf16", "op": "policy_grad", "rows": 4096, "vocab": 131072, "dtype": "bf16",
         "temperature": 1.0, "ref": True, "padded": False},
        # a few rows over a vocabulary of odd size, some of them a prompt's or padding
        {"name": "policy_grad 9x131001 f16", "op": "policy_grad", "rows": 9, "vocab": 131001, "dtype": "f16",
         "temperature": 1.5, "ref": False, "padded": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gated", "gated", "gated_backward", "adapters", "adapters", "logp", "policy", "policy_grad"))
    dtype = rng.choice(("bf16", "f16", "f32"))
    if op == "gated_backward":
        f = _log(rng, 64, 11008)
        m = _log(rng, 1, min(8192, 8192 * 11008 * 2 // (f * SIZE[dtype])))
        return {"op": op, "m": m, "f": f, "dtype": dtype, "act": rng.choice(ACTS)}
    if op in ("gated", "adapters"):
        n, k = _log(rng, 128, 11008), _log(rng, 128, 11008)
        if rng.random() < 0.8:
            k = (k + 15) // 16 * 16
        m = _log(rng, 1, 8192)
        while m * n * k > 8192 * 11008 * 4096 // 4:
            m = (m + 1) // 2
        if op == "gated":
            return {"op": op, "m": m, "f": n, "k": k, "dtype": dtype, "act": rng.choice(ACTS),
                    "bias": rng.random() < 0.5, "keep": rng.random() < 0.4}
        rank = rng.choice((8, 16, 32, 64, _log(rng, 1, 64)))
        return {"op": op, "m": m, "n": n, "k": k, "rank": rank, "adapters": _log(rng, 1, 48),
                "requests": m if m <= 64 and rng.random() < 0.7 else _log(rng, 1, min(m, 48)), "dtype": dtype,
                "act": rng.choice(("none", "none") + ACTS), "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
    vocab = _log(rng, 1000, 131072)
    if rng.random() < 0.6:
        vocab = (vocab + 7) // 8 * 8
    rows = _log(rng, 1, min(4096, 4096 * 131072 // 4 // vocab))
    return {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "temperature": rng.choice((1.0, 0.7, 1.5)),
            "ref": rng.random() < 0.6, "padded": rng.random() < 0.4}


def _request_adapters(case):
    """The adapter of every request, -1 for none: one request in `adapters` + 1 has none."""
    return [(5 * i + 1) % (case["adapters"] + 1) - 1 for i in range(case["requests"])]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    def codes(rows, cols):   # of roughly normal values whose largest is at 127
        return (normal(rows, cols) * 32).round().clamp(-127, 127).to(torch.int8)

    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    if op == "gated_backward":
        m, f = case["m"], case["f"]
        s["dy"] = normal(m, f).to(dt)
        s["z"] = (1.5 * normal(m, 2 * f)).to(dt)
        return s
    if op == "gated":
        m, f, k = case["m"], case["f"], case["k"]
        s["qx"], s["sx"] = codes(m, k), (0.5 + uniform(m)) / 32
        for name in ("gate", "up"):
            s["q_" + name] = codes(f, k)
            s["s_" + name] = (0.5 + uniform(f)) / (32 * math.sqrt(k))
            s["b_" + name] = (0.3 * normal(f)).to(dt) if case["bias"] else None
        return s
    if op == "adapters":
        m, n, k, r, count = case["m"], case["n"], case["k"], case["rank"], case["adapters"]
        s["x"] = (normal(m, k) * (0.5 + uniform(m, 1))).to(dt)
        x32 = s["x"].float()
        s["sx"] = x32.abs().amax(1) / 127                  # the projection takes the same tokens as codes
        s["qx"] = (x32 / s["sx"][:, None]).round().clamp(-127, 127).to(torch.int8)
        s["qw"] = codes(n, k)
        s["sw"] = (0.5 + uniform(n)) / (32 * math.sqrt(k))
        s["a"] = (normal(count, r, k) / math.sqrt(k)).to(dt)
        s["b"] = (0.3 * normal(count, n, r) / math.sqrt(r)).to(dt)
        s["scale"] = 0.5 + 1.5 * uniform(count)
        # tokens of a request stand together, its length is anything from one
        of = torch.tensor(_request_adapters(case), dtype=torch.int32, device="cuda")
        cuts = torch.randperm(m - 1, generator=g, device="cuda")[:case["requests"] - 1] + 1
        starts = torch.zeros(m, dtype=torch.int64, device="cuda")
        starts[cuts] = 1
        s["adapter"] = of[starts.cumsum(0)]
        s["bias"] = (0.5 * normal(n)).to(dt) if case["bias"] else None
        s["residual"] = normal(m, n).to(dt) if case["residual"] else None
        return s
    rows, vocab, t = case["rows"], case["vocab"], case["temperature"]
    token = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    logits = 2.0 * normal(rows, vocab)
    logits.scatter_add_(1, token[:, None], 5.0 + 2.0 * normal(rows, 1))   # drawn tokens are likely ones
    s["logits"] = logits.to(dt)
    del logits
    # what the policy that drew the tokens and the reference said of them, a few updates ago
    logp = torch.cat([torch.log_softmax(z.float() / t, 1).gather(1, y[:, None])[:, 0]
                      for z, y in zip(s["logits"].split(512), token.split(512))])
    drift = 0.15 * normal(rows)
    ratio = torch.exp(drift)
    edge = torch.minimum((ratio - (1 - CLIP)).abs(), (ratio - (1 + CLIP)).abs()) < 2e-3
    s["old_logp"] = logp - torch.where(edge, 0.5 * drift, drift)   # no ratio where 32 bits cannot tell its side
    s["ref_logp"] = logp + 0.3 * normal(rows) if case["ref"] else None
    s["advantage"] = normal(rows)
    s["dloss"] = (0.5 + uniform(rows)) / rows
    if case["padded"]:
        token = torch.where(uniform(rows) < 0.3, torch.full_like(token, -1), token)
    s["token"] = token
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import tensor_quantization_amd as tq
    c = s["case"]
    op, dt = c["op"], DTYPES[c["dtype"]]
    if op == "gated":
        return tq.tq_w8a8_gated_linear(s["qx"], s["sx"], s["q_gate"], s["s_gate"], s["q_up"], s["s_up"],
                                       bias_gate=s["b_gate"], bias_up=s["b_up"], act=c["act"], out_dtype=dt,
                                       preact=c["keep"])
    if op == "gated_backward":
        return tq.tq_gated_act_backward(s["dy"], s["z"], act=c["act"])
    if op == "adapters":
        return tq.tq_w8a8_linear_adapters(s["x"], s["qx"], s["sx"], s["qw"], s["sw"], s["adapter"], s["a"], s["b"],
                                          scale=s["scale"], bias=s["bias"], act=c["act"], residual=s["residual"],
                                          out_dtype=dt)
    t = c["temperature"]
    if op == "logp":
        return tq.tq_token_logp(s["logits"], s["token"], temperature=t)[0]
    how = {"old_logp": s["old_logp"], "ref_logp": s["ref_logp"], "clip_low": CLIP, "clip_high": CLIP, "kl_coef": KL,
           "temperature": t}
    if op == "policy":
        loss, logp, stats = tq.tq_policy_loss(s["logits"], s["token"], s["advantage"], **how)
        return loss, logp, tq.tq_policy_loss_backward(s["logits"], s["token"], s["advantage"], logp, stats,
                                                      dloss=s["dloss"], **how)
    return tq.tq_policy_loss_grad(s["logits"], s["token"], s["advantage"], dloss=s["dloss"], **how)


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
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _plain(s):
    c = s["case"]
    op, dt = c["op"], DTYPES[c["dtype"]]
    if op == "gated":
        x = s["qx"].float()
        g = (x @ s["q_gate"].float().t()) * s["sx"][:, None] * s["s_gate"][None, :]
        u = (x @ s["q_up"].float().t()) * s["sx"][:, None] * s["s_up"][None, :]
        if c["bias"]:
            g, u = g + s["b_gate"].float(), u + s["b_up"].float()
        y = (_act32(g, c["act"]) * u).to(dt)
        return (y, torch.cat((g, u), 1).to(dt)) if c["keep"] else y
    if op == "gated_backward":
        dy, z, f = s["dy"].float(), s["z"].float(), c["f"]
        g, u = z[:, :f], z[:, f:]
        dz = torch.cat((dy * u * _act_slope32(g, c["act"]), dy * _act32(g, c["act"])), 1)
        return dz.to(dt), dz.sum(0)
    if op == "adapters":
        z = (s["qx"].float() @ s["qw"].float().t()) * s["sx"][:, None] * s["sw"][None, :]
        if s["bias"] is not None:
            z = z + s["bias"].float()
        # every adapter's low-rank values of every token, those of other adapters than its own cleared
        count, r, n = c["adapters"], c["rank"], c["n"]
        h = (s["x"].float() @ s["a"].float().reshape(count * r, -1).t()).view(-1, count, r) * s["scale"][:, None]
        mine = s["adapter"][:, None] == torch.arange(count, device=h.device)
        h = torch.where(mine[:, :, None], h, torch.zeros_like(h)).view(-1, count * r)
        z = z + h @ s["b"].float().transpose(1, 2).reshape(count * r, n)
        y = _act32(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(dt)
    return _policy32(s, c, dt)


def _policy32(s, c, dt):
    inv_t = 1.0 / c["temperature"]
    here = s["token"] >= 0
    at = torch.where(here, s["token"], torch.zeros_like(s["token"]))[:, None]
    z = s["logits"].float() * inv_t
    m = z.amax(1, keepdim=True)
    lse = torch.log(torch.exp(z - m).sum(1, keepdim=True)) + m
    zero = torch.zeros_like(lse[:, 0])
    logp = torch.where(here, (z.gather(1, at) - lse)[:, 0], zero)
    if c["op"] == "logp":
        return logp
    adv = s["advantage"]
    ratio = torch.exp(logp - s["old_logp"])
    free, held = ratio * adv, ratio.clamp(1 - CLIP, 1 + CLIP) * adv
    loss = -torch.minimum(free, held)
    slope = torch.where(free <= held, -free, zero)
    if s["ref_logp"] is not None:
        d = s["ref_logp"] - logp
        loss = loss + KL * (torch.exp(d) - d - 1)
        slope = slope + KL * (1 - torch.exp(d))
    loss = torch.where(here, loss, zero)
    slope = torch.where(here, slope * s["dloss"] * inv_t, zero)[:, None]
    grad = -slope * torch.exp(z - lse)
    grad.scatter_add_(1, at, slope)
    return loss, logp, grad.to(dt)


# ------------------------------------------------------------- work, exact
def work(case):
    op, size = case["op"], SIZE[case["dtype"]]
    if op == "gated_backward":
        n = case["m"] * case["f"]
        return {"bytes": 5 * n * size + 8 * case["f"], "flops": n * (4 + 2 * ACT_FLOPS[case["act"]])}
    if op == "gated":
        m, f, k = case["m"], case["f"], case["k"]
        b = m * k + 4 * m + 2 * f * (k + 4 + (size if case["bias"] else 0)) + m * f * size * (3 if case["keep"] else 1)
        return {"bytes": b, "flops": 4 * m * f * k + m * f * (7 + ACT_FLOPS[case["act"]])}
    if op == "adapters":
        m, n, k, r = case["m"], case["n"], case["k"], case["rank"]
        used = len({a for a in _request_adapters(case) if a >= 0})
        b = m * k * (1 + size) + 8 * m + n * (k + 4) + used * (r * (k + n) * size + 4)
        b += m * n * size * (2 if case["residual"] else 1) + (n * size if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * m * n * k + 2 * m * r * (k + n) + m * n * (4 + ACT_FLOPS[case["act"]])}
    n = case["rows"] * case["vocab"]
    if op == "logp":
        return {"bytes": n * size + 12 * case["rows"], "flops": 4 * n}
    return {"bytes": 2 * n * size + case["rows"] * (32 + (4 if case["ref"] else 0)), "flops": 8 * n}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gated":
        z = []
        for name in ("gate", "up"):
            v = torch.mm(s["qx"].double(), s["q_" + name].double().t())
            v = v.mul_(s["sx"].double()[:, None]).mul_(s["s_" + name].double())
            z.append(v if s["b_" + name] is None else v + s["b_" + name].double())
        y = _act64(z[0], case["act"]).mul_(z[1])
        return (y, torch.cat(z, 1)) if case["keep"] else y
    if op == "gated_backward":
        z = s["z"].double().requires_grad_()
        gate, up = z.chunk(2, 1)
        (_act64(gate, case["act"]) * up).backward(s["dy"].double())
        return z.grad, z.grad.sum(0)
    if op == "adapters":
        z = torch.mm(s["qx"].double(), s["qw"].double().t()).mul_(s["sx"].double()[:, None]).mul_(s["sw"].double())
        if s["bias"] is not None:
            z += s["bias"].double()
        for i in range(case["adapters"]):
            rows = (s["adapter"] == i).nonzero()[:, 0]
            if len(rows):
                low = s["x"][rows].double() @ s["a"][i].double().t()
                z[rows] += s["scale"][i].double() * (low @ s["b"][i].double().t())
        y = _act64(z, case["act"])
        return y if s["residual"] is None else y + s["residual"].double()
    # the policy loss as it is defined, its gradient by differentiating it, a few rows at a time
    parts = []
    step = max(1, (1 << 26) // case["vocab"])
    for i in range(0, case["rows"], step):
        parts.append(_policy64(case, {k: v[i:i + step] for k, v in s.items() if isinstance(v, torch.Tensor)}))
    if op == "logp":
        return torch.cat([p[1] for p in parts])
    return tuple(torch.cat(p) for p in zip(*parts))


def _act64(z, act):
    f = torch.nn.functional
    return {"none": lambda: z * 1, "relu": lambda: f.relu(z), "silu": lambda: f.silu(z), "gelu": lambda: f.gelu(z),
            "gelu_tanh": lambda: f.gelu(z, approximate="tanh")}[act]()


def _policy64(case, s):
    z = s["logits"].double().requires_grad_()
    here = s["token"] >= 0
    logq = torch.log_softmax(z / case["temperature"], 1)
    logp = logq.gather(1, s["token"].clamp_min(0)[:, None])[:, 0].masked_fill(~here, 0)
    if case["op"] == "logp":
        return None, logp.detach(), None
    a = s["advantage"].double()
    ratio = (logp - s["old_logp"].double()).exp()
    loss = torch.maximum(-a * ratio, -a * ratio.clamp(1 - CLIP, 1 + CLIP))
    if "ref_logp" in s:
        apart = s["ref_logp"].double() - logp
        loss = loss + KL * (torch.expm1(apart) - apart)
    loss = loss.masked_fill(~here, 0)
    loss.backward(s["dloss"].double())
    return loss.detach(), logp.detach(), z.grad
