"""The router's gate, the few-token expert layer and the adapter projection: cases, inputs and plain forms.

``run`` with ``own`` false computes each operator with elementary torch operations in 32 bits; with ``own`` true it calls
the library. ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the router of one decode batch (128 tokens, 256 experts, top-8)
        dict(name="gate decode", op="gate", T=128, E=256, k=8, logits="fp32", score="softmax", normalize=True, grad=False),
        # one training step's router at 4096 tokens: choice, weights and the logits' gradient, sigmoid scores
        dict(name="gate train 4096", op="gate", T=4096, E=256, k=8, logits="bf16", score="sigmoid", normalize=True, grad=True),
        # many experts and a long batch, weights straight from the softmax (a dense gradient)
        dict(name="gate train 2048 experts", op="gate", T=16384, E=2048, k=8, logits="fp32", score="softmax",
             normalize=False, grad=True),
        # a small layer of the test configuration: launches and latency
        dict(name="layer tiny", op="layer", T=128, H=256, I=256, E=16, k=2, weights="bf16"),
        # one token through one layer: eight experts' weights and nothing else
        dict(name="layer 1 token", op="layer", T=1, H=7168, I=2048, E=64, k=8, weights="bf16"),
        # a small batch with odd sizes
        dict(name="layer 37 tokens odd", op="layer", T=37, H=1160, I=520, E=24, k=3, weights="bf16"),
        # a decode batch over rank-local experts: entries of other ranks are -1
        dict(name="experts local 64", op="experts", T=64, H=7168, I=2048, E=32, k=8, weights="e4m3", masked=0.5),
        # a decode batch over all experts, E4M3 weights: every expert is read
        dict(name="layer decode e4m3", op="layer", T=128, H=7168, I=2048, E=256, k=8, weights="e4m3"),
        # one request's next token through a projection with its adapter
        dict(name="adapter 1 token", op="adapter", T=1, K=7168, N=2048, L=8, r=16, spread="rows"),
        # a decode batch, each row another request's adapter or none
        dict(name="adapter decode 128", op="adapter", T=128, K=7168, N=7168, L=48, r=16, spread="rows"),
        # several prompts at once, uneven lengths, rows of a request next to one another
        dict(name="adapter prompts 4096", op="adapter", T=4096, K=7168, N=4096, L=16, r=64, spread="runs"),
        # odd sizes and an odd rank
        dict(name="adapter odd", op="adapter", T=317, K=1048, N=1336, L=7, r=24, spread="runs"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "layer", "experts", "adapter"])
    if op == "gate":
        E = rng.choice([_log(rng, 8, 2048), 16, 256, 1000])
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=rng.randint(1, min(8, E)), logits=rng.choice(["fp32", "bf16"]),
                    score=rng.choice(["softmax", "sigmoid"]), normalize=rng.random() < 0.5, grad=rng.random() < 0.6)
    if op == "adapter":
        return dict(op=op, T=_log(rng, 1, 3000), K=8 * _log(rng, 16, 896), N=8 * _log(rng, 8, 512), L=_log(rng, 1, 64),
                    r=8 * rng.randint(1, 8), spread=rng.choice(["rows", "runs"]))
    weights = rng.choice(["bf16", "e4m3"])
    step = 8 if weights == "bf16" else 128
    E = _log(rng, 4, 64)
    c = dict(op=op, T=_log(rng, 1, 256), H=step * _log(rng, 256 // step, 7168 // step),
             I=step * _log(rng, 128 // step, 2048 // step), E=E, k=rng.randint(1, min(8, E)), weights=weights)
    if op == "experts":
        c["masked"] = round(rng.uniform(0, 0.9), 2)
    return c


# ------------------------------------------------------------------ inputs

def _normal(gen, *shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, std, generator=gen)


def _weights(gen, kind, E, rows, cols):
    """Expert weights of about unit gain: bf16 [E, rows, cols], or E4M3 codes and their scales [E, rows, cols / 128]."""
    if kind == "bf16":
        return _normal(gen, E, rows, cols, std=cols ** -0.5), None
    codes = torch.empty(E, rows, cols, dtype=torch.uint8, device=DEV)
    for e in range(E):
        v = torch.empty(rows, cols, device=DEV).normal_(0.0, 120.0, generator=gen).clamp_(-448, 448)
        codes[e] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.empty(E, rows, cols // 128, device=DEV).uniform_(0.5, 1.5, generator=gen) / (120.0 * cols ** 0.5)
    return codes, scales


def _choice(gen, T, E, k):
    """k distinct experts a token, and softmax weights."""
    idx = torch.rand(T, E, device=DEV, generator=gen).topk(k, dim=1).indices
    return idx, torch.randn(T, k, device=DEV, generator=gen).softmax(dim=1)


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "gate":
        logits = torch.randn(case["T"], case["E"], device=DEV, generator=gen) * 1.5
        s["logits"] = logits.to(torch.bfloat16) if case["logits"] == "bf16" else logits
        if case["grad"]:
            s["grad_weights"] = torch.randn(case["T"], case["k"], device=DEV, generator=gen)
        return s
    if case["op"] == "adapter":
        T, K, N, L, r = (case[n] for n in ("T", "K", "N", "L", "r"))
        s["x"] = _normal(gen, T, K)
        s["w"] = _normal(gen, N, K, std=K ** -0.5)
        s["a"] = _normal(gen, L, r, K, std=K ** -0.5)
        s["b"] = _normal(gen, L, N, r, std=r ** -0.5)
        s["scales"] = torch.empty(L, device=DEV).uniform_(0.25, 2.0, generator=gen)
        a = torch.randint(-1, L, (T,), device=DEV, generator=gen, dtype=torch.int32)
        if case["spread"] == "runs":   # requests of uneven lengths, one after another
            starts = torch.rand(T, device=DEV, generator=gen) < min(1.0, 2.0 * L / T)
            a = a[torch.cummax(torch.arange(T, device=DEV) * starts, 0).values]
        s["adapter_idx"] = a.contiguous()
        return s
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    s["x"] = _normal(gen, T, H)
    s["w13"], s["w13_scales"] = _weights(gen, case["weights"], E, 2 * I, H)
    s["w2"], s["w2_scales"] = _weights(gen, case["weights"], E, H, I)
    if case["op"] == "layer":
        s["logits"] = torch.randn(T, E, device=DEV, generator=gen) * 1.5
    else:
        idx, s["topk_weights"] = _choice(gen, T, E, k)
        other = torch.rand(T, k, device=DEV, generator=gen) < case["masked"]
        s["topk_idx"] = idx.masked_fill(other, -1)
    return s


# ------------------------------------------------------------------ plain forms

def _plain_gate(logits, k, score, normalize):
    l = logits.float()
    top, idx = torch.sort(l, dim=1, descending=True, stable=True)   # ties go to the lowest index
    top, idx = top[:, :k], idx[:, :k].contiguous()
    if score == "softmax":
        w = torch.exp(top - top[:, :1])
        w = w / (w.sum(1, keepdim=True) if normalize else torch.exp(l - top[:, :1]).sum(1, keepdim=True))
    else:
        w = 1 / (1 + torch.exp(-top))
        w = w / w.sum(1, keepdim=True) if normalize else w
    return idx, w


def _plain_gate_backward(logits, idx, g, score, normalize):
    l = logits.float()
    top = torch.gather(l, 1, idx)
    if score == "softmax" and not normalize:
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        gd = torch.zeros_like(l).scatter(1, idx, g)
        d = p * (gd - (gd * p).sum(1, keepdim=True))
    else:
        if score == "softmax":
            q = torch.exp(top - top.amax(1, keepdim=True))
            q = q / q.sum(1, keepdim=True)
            dt = q * (g - (g * q).sum(1, keepdim=True))
        else:
            sg = 1 / (1 + torch.exp(-top))
            if normalize:
                q = sg / sg.sum(1, keepdim=True)
                dt = q * (1 - sg) * (g - (g * q).sum(1, keepdim=True))
            else:
                dt = g * sg * (1 - sg)
        d = torch.zeros_like(l).scatter(1, idx, dt)
    return d.to(logits.dtype)


def _wide(w, scales):
    """Weights in 32 bits."""
    if scales is None:
        return w.float()
    v = w.view(torch.float8_e4m3fn).float()
    return v.view(*w.shape[:-1], -1, 128).mul_(scales[..., None]).view(w.shape)


def _plain_experts(x, idx, weights, w13, s13, w2, s2):
    T, k = idx.shape
    E, I = w13.shape[0], w2.shape[2]
    weights = torch.where(idx >= 0, weights, 0)
    x = x.float()
    if T * k < E:   # the named experts' weights, entry by entry
        e = idx.clamp_min(0).flatten()
        y = torch.matmul(_wide(w13[e], None if s13 is None else s13[e]), x.repeat_interleave(k, 0)[:, :, None])[:, :, 0]
        h = y[:, :I] / (1 + torch.exp(-y[:, :I])) * y[:, I:]
        y = torch.matmul(_wide(w2[e], None if s2 is None else s2[e]), h[:, :, None])[:, :, 0]
        out = (y.view(T, k, -1) * weights[:, :, None]).sum(1)
    else:           # every expert on every token, weighted
        y = torch.matmul(x, _wide(w13, s13).transpose(1, 2))          # [E, T, 2I]
        h = y[..., :I] / (1 + torch.exp(-y[..., :I])) * y[..., I:]
        wd = torch.zeros(T, E, device=x.device).scatter_add(1, idx.clamp_min(0), weights)
        h = h * wd.t()[:, :, None]
        out = torch.matmul(h, _wide(w2, s2).transpose(1, 2)).sum(0)
    return out.to(torch.bfloat16)


def _plain_adapter(x, w, adapter_idx, a, b, scales):
    L, r, K = a.shape
    x = x.float()
    mine = (adapter_idx[:, None] == torch.arange(L, device=x.device)) * scales        # [T, L]
    v = torch.matmul(x, a.float().view(L * r, K).t()).view(-1, L, r) * mine[:, :, None]
    y = torch.matmul(x, w.float().t())
    y = y + torch.matmul(v.view(-1, L * r), b.float().transpose(1, 2).reshape(L * r, -1))
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    if not own:
        if c["op"] == "gate":
            idx, w = _plain_gate(state["logits"], c["k"], c["score"], c["normalize"])
            out = dict(topk_idx=idx, topk_weights=w)
            if c["grad"]:
                out["grad_logits"] = _plain_gate_backward(state["logits"], idx, state["grad_weights"], c["score"],
                                                          c["normalize"])
            return out
        if c["op"] == "adapter":
            return _plain_adapter(*(state[n] for n in ("x", "w", "adapter_idx", "a", "b", "scales")))
        experts = [state[n] for n in ("w13", "w13_scales", "w2", "w2_scales")]
        if c["op"] == "layer":
            idx, w = _plain_gate(state["logits"], c["k"], "softmax", True)
            return dict(out=_plain_experts(state["x"], idx, w, *experts), topk_idx=idx, topk_weights=w)
        return _plain_experts(state["x"], state["topk_idx"], state["topk_weights"], *experts)

    from combine_moe_get_gb300 import binding as moe
    if "status" not in state:   # what a program keeps from call to call
        state["status"] = moe.new_status(DEV)
        if c["op"] == "adapter":
            n = moe.moe_adapter_linear_workspace_size(c["T"], c["K"], c["N"], c["L"], c["r"])
            state["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        elif c["op"] != "gate":
            n = moe.moe_experts_workspace_size(c["T"], c["H"], c["I"], c["k"], c["E"])
            state["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    if c["op"] == "gate":
        idx, w = moe.moe_topk_gate(state["logits"], c["k"], score=c["score"], normalize=c["normalize"],
                                   status=state["status"])
        out = dict(topk_idx=idx, topk_weights=w)
        if c["grad"]:
            out["grad_logits"] = moe.moe_topk_gate_backward(state["logits"], idx, state["grad_weights"], score=c["score"],
                                                            normalize=c["normalize"], status=state["status"])
        return out
    keep = dict(workspace=state["workspace"], status=state["status"])
    if c["op"] == "adapter":
        return moe.moe_adapter_linear(*(state[n] for n in ("x", "w", "adapter_idx", "a", "b", "scales")), **keep)
    keep |= dict(w13_scales=state["w13_scales"], w2_scales=state["w2_scales"])
    if c["op"] == "layer":
        out, idx, w = moe.moe_layer(state["x"], state["logits"], c["k"], state["w13"], state["w2"], **keep)
        return dict(out=out, topk_idx=idx, topk_weights=w)
    return moe.moe_experts(state["x"], state["topk_idx"], state["topk_weights"], state["w13"], state["w2"], **keep)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        cell = 4 if case["logits"] == "fp32" else 2
        b, f = T * (E * cell + k * 12), T * E * 2
        if case["grad"]:    # the gradient's own reads count once: logits and choice are at hand
            b, f = b + T * (E * cell + k * 4), 2 * f
        return dict(bytes=b, flops=f)
    if case["op"] == "adapter":
        T, K, N, L, r = (case[n] for n in ("T", "K", "N", "L", "r"))
        named = L * (1 - (1 - 1 / (L + 1)) ** T)
        return dict(bytes=int(2 * T * (K + N) + 4 * T + 2 * N * K + named * 2 * r * (K + N)),
                    flops=int(2 * T * N * K + 2 * T * r * (K + N) * L / (L + 1)))
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    valid = 1 - case.get("masked", 0)
    named = E * (1 - (1 - k * valid / E) ** T)
    cell = 2 if case["weights"] == "bf16" else 1 + 4 / 128
    b = named * 3 * H * I * cell + 4 * T * H + T * k * 12 + (4 * T * E if case["op"] == "layer" else 0)
    return dict(bytes=int(b), flops=int(6 * H * I * T * k * valid))


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_scores(top, everything, score, normalize):
    """Weights of the chosen logits `top` among `everything`."""
    if score == "sigmoid":
        w = torch.sigmoid(top)
        return w / w.sum(-1, keepdim=True) if normalize else w
    base = top if normalize else everything
    return torch.exp(top - torch.logsumexp(base, -1, keepdim=True))


def _exact_choice(logits, k):
    l = logits.double()
    # the k largest, and the lowest index among equals: a second key that decreases with the index
    order = torch.argsort(torch.arange(l.shape[1], device=l.device).expand_as(l) +
                          l.shape[1] * torch.unique(-l, return_inverse=True)[1], dim=1)
    return l, order[:, :k].contiguous()


def _row64(w, scales, e):
    v = w[e].double() if scales is None else w[e].view(torch.float8_e4m3fn).double()
    return v if scales is None else v * scales[e].double().repeat_interleave(128, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gate":
        l, idx = _exact_choice(s["logits"], case["k"])
        l = l.requires_grad_(case["grad"])
        w = _exact_scores(l.gather(1, idx), l, case["score"], case["normalize"])
        out = dict(topk_idx=idx, topk_weights=w.detach())
        if case["grad"]:
            out["grad_logits"] = torch.autograd.grad(w, l, s["grad_weights"].double())[0]
        return out
    if case["op"] == "adapter":
        x = s["x"].double()
        y = x @ s["w"].double().t()
        for i in range(case["L"]):
            t = (s["adapter_idx"] == i).nonzero()[:, 0]
            y[t] += s["scales"][i].double() * (x[t] @ s["a"][i].double().t()) @ s["b"][i].double().t()
        return y
    if case["op"] == "layer":
        l, idx = _exact_choice(s["logits"], case["k"])
        w = _exact_scores(l.gather(1, idx), l, "softmax", True)
    else:
        idx, w = s["topk_idx"], s["topk_weights"].double()
    x, I = s["x"].double(), case["I"]
    y = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t):
            u = x[t] @ _row64(s["w13"], s["w13_scales"], e).t()
            h = torch.nn.functional.silu(u[:, :I]) * u[:, I:]
            y.index_add_(0, t, (h @ _row64(s["w2"], s["w2_scales"], e).t()) * w[t, j, None])
    return dict(out=y, topk_idx=idx, topk_weights=w) if case["op"] == "layer" else y
