"""The gated block, the adapters and the policy loss together, as a program uses
them: a training step of a quantized policy and its gradients, serving with the
adapters of many requests, replays of a captured graph, two host threads on two
streams, a stream that is not the tensors' own."""
import threading

import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


def deq(tq, q, scale):
    return tq.tq_dequant_per_token(q, q.shape, scale)


def policy_step(tq, p, x, token, adv, old, kl):
    """One forward and backward pass of x -> norm -> gated block -> + x -> norm ->
    head -> policy loss, on s8 codes: (losses, log-probabilities, gradients)."""
    qw = {n: tq.tq_quant_per_token(p[n])[:2] for n in ("gate", "up", "down", "head")}
    q0, s0, m0, r0 = tq.tq_layer_norm_quant_per_token(x, p["g1"], p["c1"], stats=True)
    a, z = tq.tq_w8a8_gated_linear(q0, s0, *qw["gate"], *qw["up"], bias_gate=p["bg"], bias_up=p["bu"], act="silu",
                                   out_dtype=x.dtype, preact=True)
    q1, s1, _ = tq.tq_quant_per_token(a)
    y = tq.tq_w8a8_linear_epilogue(q1, s1, *qw["down"], residual=x, out_dtype=x.dtype)
    q2, s2, m2, r2 = tq.tq_layer_norm_quant_per_token(y, p["g2"], p["c2"], stats=True)
    logits = tq.tq_w8a8_linear_epilogue(q2, s2, *qw["head"], out_dtype=x.dtype)
    mean = torch.full((x.shape[0],), 1.0 / x.shape[0], device=x.device)
    loss, logp, dlogits = tq.tq_policy_loss_grad(logits, token, adv, dloss=mean, old_logp=old, ref_logp=kl, kl_coef=0.1)
    g = {"head": dlogits.float().t() @ deq(tq, q2, s2)}
    dn2 = (dlogits.float() @ deq(tq, *qw["head"])).to(x.dtype)
    dy, g["g2"], g["c2"] = tq.tq_layer_norm_backward(dn2, y, p["g2"], m2, r2)
    g["down"] = dy.float().t() @ deq(tq, q1, s1)
    da = (dy.float() @ deq(tq, *qw["down"])).to(x.dtype)
    dz, db = tq.tq_gated_act_backward(da, z, "silu")
    F = a.shape[1]
    both = dz.float().t() @ deq(tq, q0, s0)
    g["gate"], g["up"], g["bg"], g["bu"] = both[:F], both[F:], db[:F], db[F:]
    weights = torch.cat([deq(tq, *qw["gate"]), deq(tq, *qw["up"])])
    dn1 = (dz.float() @ weights).to(x.dtype)
    _, g["g1"], g["c1"] = tq.tq_layer_norm_backward(dn1, x, p["g1"], m0, r0)
    return loss, logp, logits, g


def policy_params(D, F, V, gen):
    def w(n, k):
        return torch.randn((n, k), generator=gen, device="cuda") / k ** 0.5
    def near(v, n):
        return v + 0.1 * torch.randn(n, generator=gen, device="cuda")
    return {"g1": near(1, D), "c1": near(0, D), "gate": w(F, D), "up": w(F, D), "bg": near(0, F), "bu": near(0, F),
            "down": w(D, F), "g2": near(1, D), "c2": near(0, D), "head": 2 * w(V, D)}


def test_training_step_gradients(tq):
    """The step's gradients against automatic differentiation in 64 bits of the same
    path, its quantizers replaced by the codes that the step used."""
    note("policy step: gradients against 64-bit differentiation")
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, V, D, F = 96, 515, 64, 160
    p = policy_params(D, F, V, gen)
    x = torch.randn((T, D), generator=gen, device="cuda")
    token = torch.randint(0, V, (T,), generator=gen, device="cuda")
    token[::7] = -1
    adv = torch.randn(T, generator=gen, device="cuda")
    _, logp, _, _ = policy_step(tq, p, x, token, adv, None, None)
    drift = 0.3 * torch.randn(T, generator=gen, device="cuda")
    # clear of the clips by more than a code's step moves the ratio
    edge = ((drift.exp() - 0.8).abs() < 0.02) | ((drift.exp() - 1.2).abs() < 0.02)
    old, kl = logp - torch.where(edge, 0 * drift, drift), logp + 0.2
    loss, _, _, grads = policy_step(tq, p, x, token, adv, old, kl)

    def through(v):
        """v's s8 codes' values, its gradient passed straight through."""
        d = v.detach()
        s = d.abs().amax(1, keepdim=True) / 127
        return v + ((d / s).round().clamp(-127, 127) * s - d)

    q = {n: v.double().cpu().requires_grad_() for n, v in p.items()}
    xd = x.double().cpu()

    def norm(v, g, c):
        h = v - v.mean(1, keepdim=True)
        return h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt() * g + c
    h = through(norm(xd, q["g1"], q["c1"]))
    gate, up = h @ through(q["gate"]).t() + q["bg"], h @ through(q["up"]).t() + q["bu"]
    y = through(gate * torch.sigmoid(gate) * up) @ through(q["down"]).t() + xd
    z = through(norm(y, q["g2"], q["c2"])) @ through(q["head"]).t()
    here = token.cpu() >= 0
    l = torch.log_softmax(z, 1).gather(1, token.cpu().clamp_min(0)[:, None])[:, 0]
    a, rho = adv.double().cpu(), (l - old.double().cpu()).exp()
    d = kl.double().cpu() - l
    per = -torch.minimum(rho * a, rho.clamp(0.8, 1.2) * a) + 0.1 * (torch.expm1(d) - d)
    want = per.masked_fill(~here, 0).mean()
    want.backward()
    # a code may fall on the other side of its boundary: agreement is that of the quantized path, not of binary32
    assert abs(loss.mean().item() - want.item()) < 2e-3 * float(per.abs().mean())
    for n, v in q.items():
        g = grads[n].double().cpu()
        assert (g - v.grad).norm() < 1e-2 * v.grad.norm(), n


def _inputs(seed, M=300):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    def codes(*shape):
        return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
    d = {"x": normal(M, 512), "dy": normal(M, 272), "w": [codes(272, 512), codes(272, 512), codes(1040, 272), codes(40, 35)],
         "a": 0.05 * normal(5, 16, 272), "b": normal(5, 1040, 16),
         "ids": torch.randint(-1, 5, (M,), generator=g, device="cuda", dtype=torch.int32),
         "token": torch.randint(-1, 1040, (M,), generator=g, device="cuda"),
         "adv": normal(M).float(), "long": normal(3, 140001)}
    d["sw"] = [torch.full((w.shape[0],), 1 / 4096, device="cuda") for w in d["w"]]
    return d


def _path(tq, d):
    """Every call of this kind once, each kernel variant of a small size."""
    w, sw, M = d["w"], d["sw"], d["x"].shape[0]
    q, s = tq.tq_layer_norm_quant_per_token(d["x"])
    y, z = tq.tq_w8a8_gated_linear(q, s, w[0], sw[0], w[1], sw[1], act="gelu_tanh", preact=True)
    few = tq.tq_w8a8_gated_linear(q[:5], s[:5], w[0], sw[0], w[1], sw[1])
    one = tq.tq_gated_act(z, "relu")
    dz, db = tq.tq_gated_act_backward(d["dy"], z, "gelu_tanh")
    qy, sy, _ = tq.tq_quant_per_token(y)
    qo, so, _ = tq.tq_quant_per_token(y[:, :35].contiguous())
    odd = tq.tq_w8a8_gated_linear(qo, so, w[3], sw[3], w[3], sw[3])
    logits, pre = tq.tq_w8a8_linear_adapters(y, qy, sy, w[2], sw[2], d["ids"], d["a"], d["b"], act="silu", preact=True)
    tokens = tq.tq_w8a8_linear_adapters(y[:7], qy[:7], sy[:7], w[2], sw[2], d["ids"][:7], d["a"], d["b"])
    how = {"old_logp": d["adv"] - 7, "ref_logp": d["adv"] - 7.5, "kl_coef": 0.1}
    loss, logp, stats = tq.tq_policy_loss(logits, d["token"], d["adv"], **how)
    g = tq.tq_policy_loss_backward(logits, d["token"], d["adv"], logp, stats, **how)
    l2, p2, g2 = tq.tq_policy_loss_grad(logits, d["token"], d["adv"], **how)
    l3, p3, g3 = tq.tq_policy_loss_grad(d["long"], d["token"][:3], d["adv"][:3])
    l4, s4 = tq.tq_token_logp(logits[:9], d["token"][:9])
    g4 = tq.tq_token_logp_backward(logits[:9], d["token"][:9], s4)
    return [y, z, few, one, dz, db, odd, logits, pre, tokens, loss, logp, stats, g, l2, p2, g2, l3, p3, g3, l4, s4, g4]


def _bytes(t):
    return t.detach().contiguous().view(torch.uint8)


def test_graph_replays_match_eager(tq):
    note("graph capture: gated block, adapters, policy loss")
    args, other = _inputs(1), _inputs(2)
    want = [_bytes(t).clone() for t in _path(tq, args)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _path(tq, args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _path(tq, args)
    torch.cuda.synchronize()
    for rep in range(4):
        for t in outs:
            t.fill_(77)
        eager = _path(tq, other)                   # eager work on other inputs between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (t, ref) in enumerate(zip(outs, want)):
            assert torch.equal(_bytes(t), ref), "replay %d, output %d differs from the eager result" % (rep, i)
        del eager


def test_two_threads_two_streams(tq):
    note("two host threads, two streams: gated block, adapters, policy loss")
    inputs = [_inputs(3), _inputs(4)]
    want = [[_bytes(t).clone() for t in _path(tq, a)] for a in inputs]
    torch.cuda.synchronize()
    results, errors = [[], []], []

    def worker(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(6):
                    results[k].append(_path(tq, inputs[k]))
            stream.synchronize()
        except Exception as e:  # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=worker, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for k in range(2):
        assert len(results[k]) == 6
        for outs in results[k]:
            for i, (t, ref) in enumerate(zip(outs, want[k])):
                assert torch.equal(_bytes(t), ref), "thread %d, output %d differs" % (k, i)


def test_serving_step_of_many_requests(tq):
    """Prompts of several requests in one batch, then a token of each: a request's
    outputs are those it has alone, up to what a differently shaped launch rounds
    apart, and requests without an adapter have the plain product's bits."""
    note("serving: gated block with adapters on both projections and on the way down")
    gen = torch.Generator(device="cuda").manual_seed(5)
    D, F, R, count, lengths = 256, 352, 8, 3, (37, 1, 90, 5, 200)
    owner = (0, -1, 2, 1, 0)
    x = torch.randn((sum(lengths), D), generator=gen, device="cuda").to(torch.bfloat16)
    ids = torch.repeat_interleave(torch.tensor(owner, dtype=torch.int32), torch.tensor(lengths)).cuda()

    def half(*s):
        return torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16) / s[-1] ** 0.5
    up, down = (tq.tq_quant_per_token(torch.randn(s, generator=gen, device="cuda") / s[1] ** 0.5)[:2]
                for s in ((2 * F, D), (D, F)))
    a1, b1, a2, b2 = half(count, R, D), half(count, 2 * F, R), half(count, R, F), half(count, D, R)

    def block(x, ids):
        n, _, _ = tq.tq_layer_norm(x)
        q, s, _ = tq.tq_quant_per_token(n)
        z = tq.tq_w8a8_linear_adapters(n, q, s, *up, ids, a1, b1)
        h = tq.tq_gated_act(z, "silu")
        q, s, _ = tq.tq_quant_per_token(h)
        return tq.tq_w8a8_linear_adapters(h, q, s, *down, ids, a2, b2, residual=x)
    whole, at = block(x, ids), 0
    plain = block(x, torch.full_like(ids, -1))
    for n, who in zip(lengths, owner):
        part = block(x[at:at + n], ids[at:at + n]).float()
        got = whole[at:at + n].float()
        # intermediate values in bf16, a rounding of which may differ and move a code by one
        assert (got - part).norm() < 1e-2 * part.norm()
        same = torch.equal(whole[at:at + n], plain[at:at + n])
        assert same if who < 0 else not same
        at += n
    # the next token of every request at once
    last = torch.tensor(lengths).cumsum(0) - 1
    nxt = block(x[last.cuda()], torch.tensor(owner, dtype=torch.int32).cuda()).float()
    assert (nxt - whole[last.cuda()].float()).norm() < 1e-2 * nxt.norm()


def test_gated_block_is_the_two_projections_and_the_gate(tq):
    """One kernel against the products and the gate one after the other."""
    d = _inputs(6)
    q, s = tq.tq_layer_norm_quant_per_token(d["x"])
    w, sw = d["w"], d["sw"]
    y, z = tq.tq_w8a8_gated_linear(q, s, w[0], sw[0], w[1], sw[1], out_dtype=torch.float32, preact=True)
    both = torch.cat([tq.tq_w8a8_linear_epilogue(q, s, w[i], sw[i], out_dtype=torch.float32) for i in range(2)], 1)
    assert torch.equal(z, both) and torch.equal(y, tq.tq_gated_act(both))
