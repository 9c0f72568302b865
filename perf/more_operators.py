"""What stands between a dispatch's rows and the combine, and in front of the router: matrix products grouped by expert
with their gradients, the gated activation of their rows, and the root-mean-square norm behind the residual's addition.
Cases, inputs and plain forms.

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
        # one token's eight rows through its experts' first product: latency and the stream of eight experts' weights
        dict(name="grouped 1 token", op="grouped", rows=8, capacity=8, E=64, K=7168, N=4096, weights="bf16", routing="uniform"),
        # a decode batch of 128 tokens over all experts in 8 bits: every expert's weights for a few rows each
        dict(name="grouped decode e4m3", op="grouped", rows=1024, capacity=1024, E=256, K=7168, N=4096, weights="e4m3",
             routing="uniform"),
        # prompts of 4096 tokens, the experts' second product
        dict(name="grouped prompts bf16", op="grouped", rows=32768, capacity=32768, E=256, K=2048, N=7168, weights="bf16",
             routing="uniform"),
        # the same prompts as an 8-bit dispatch delivers them, the experts' first product
        dict(name="grouped prompts e4m3", op="grouped", rows=32768, capacity=32768, E=256, K=7168, N=4096, weights="e4m3",
             routing="uniform"),
        # odd sizes, a skewed choice with experts that get nothing, and a receive buffer with room to spare
        dict(name="grouped odd", op="grouped", rows=1531, capacity=2048, E=24, K=1160, N=1048, weights="bf16", routing="zipf"),
        # one training step of a rank's 32 experts: gradients of the rows and of the weights (32 bits, as an optimizer adds them up)
        dict(name="grouped gradients 16384", op="grouped_grad", rows=16384, capacity=16384, E=32, K=7168, N=4096, grad_w="fp32",
             routing="uniform"),
        # the gradients of a small layer, skewed, with room to spare
        dict(name="grouped gradients small", op="grouped_grad", rows=251, capacity=256, E=16, K=256, N=520, grad_w="bf16",
             routing="zipf"),
        # the activation between two 8-bit products, 4096 tokens of eight rows
        dict(name="swiglu prompts e4m3", op="swiglu", rows=32768, capacity=32768, I=2048, out="e4m3", weighted=False, grad=False),
        # the activation of one training step and its gradient, the router's weights folded in, odd sizes
        dict(name="swiglu train odd", op="swiglu", rows=12345, capacity=16384, I=1416, out="bf16", weighted=True, grad=True),
        # the norm of a decode batch: rows for the router in bf16, rows for the dispatch in 8 bits, the new residual
        dict(name="norm decode e4m3", op="norm", T=128, H=7168, residual=True, out="both", grad=False),
        # the norm of long prompts, straight into 8 bits
        dict(name="norm prompts e4m3", op="norm", T=16384, H=7168, residual=True, out="e4m3", grad=False),
        # the norm of a training step with its gradients
        dict(name="norm train 4096", op="norm", T=4096, H=7168, residual=True, out="bf16", grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grouped_grad", "swiglu", "norm"])
    if op in ("grouped", "grouped_grad"):
        rows, E = _log(rng, 1, 16384), _log(rng, 1, 64)
        capacity = rows + (rng.randint(0, rows) if rng.random() < 0.3 else 0)
        c = dict(op=op, rows=rows, capacity=capacity, E=E, routing=rng.choice(["uniform", "zipf"]))
        step = 8
        if op == "grouped":
            c["weights"] = rng.choice(["bf16", "e4m3"])
            step = 128 if c["weights"] == "e4m3" else 8
        else:
            c["grad_w"] = rng.choice(["fp32", "bf16"])
        c.update(K=step * _log(rng, max(1, 64 // step), 7168 // step), N=8 * _log(rng, 8, 512))
        return c
    if op == "swiglu":
        rows, out = _log(rng, 1, 32768), rng.choice(["bf16", "e4m3"])
        step = 128 if out == "e4m3" else 8
        return dict(op=op, rows=rows, capacity=rows + (rng.randint(0, rows) if rng.random() < 0.3 else 0),
                    I=step * _log(rng, 128 // step, 2048 // step), out=out, weighted=rng.random() < 0.5,
                    grad=out == "bf16" and rng.random() < 0.7)
    out = rng.choice(["bf16", "e4m3", "both"])
    step = 8 if out == "bf16" else 128
    return dict(op=op, T=_log(rng, 1, 16384), H=step * _log(rng, 128 // step, 7168 // step), residual=rng.random() < 0.7, out=out,
                grad=out == "bf16" and rng.random() < 0.7)


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


def _shares(case):
    """The part of the rows that each expert gets on average."""
    p = torch.ones(case["E"], dtype=torch.float64)
    if case["routing"] == "zipf":
        p = 1 / torch.arange(1, case["E"] + 1, dtype=torch.float64)
    return p / p.sum()


def _groups(case, seed):
    """Rows of each expert, on the host; zipf shares go to experts in a random order."""
    host = torch.Generator().manual_seed(seed)
    p = _shares(case)[torch.randperm(case["E"], generator=host)]
    return torch.bincount(torch.multinomial(p, case["rows"], replacement=True, generator=host), minlength=case["E"])


def _quantised(v):
    """E4M3 codes (uint8) and scales of rows in 32 bits, 128 channels to a scale."""
    blocks = v.unflatten(-1, (-1, 128))
    scales = blocks.abs().amax(-1) / 448.0
    codes = torch.where(scales[..., None] > 0, blocks / scales[..., None], 0.0).to(torch.float8_e4m3fn)
    return codes.flatten(-2).view(torch.uint8), scales


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    s = dict(case=case)
    if case["op"] in ("grouped", "grouped_grad"):
        rows, M, E, K, N = (case[n] for n in ("rows", "capacity", "E", "K", "N"))
        counts = _groups(case, seed)
        prefix = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
        s["expert_prefix"] = prefix.to(torch.int32).to(DEV)
        # for the plain form: each row's expert and place among its expert's rows
        s["expert"] = torch.repeat_interleave(torch.arange(E), counts).to(DEV)
        s["place"] = (torch.arange(rows) - torch.repeat_interleave(prefix[:-1], counts)).to(DEV)
        s["most"] = int(counts.max())
        s["x"], s["x_scales"] = _normal(gen, M, K), None
        s["w"], s["w_scales"] = _weights(gen, case.get("weights", "bf16"), E, N, K)
        if case.get("weights") == "e4m3":
            s["x"], s["x_scales"] = _quantised(s["x"].float())
        if case["op"] == "grouped_grad":
            s["grad"] = _normal(gen, M, N)
        return s
    if case["op"] == "swiglu":
        M, I = case["capacity"], case["I"]
        s["gate_up"] = _normal(gen, M, 2 * I)
        s["num_rows"] = torch.tensor([case["rows"]], dtype=torch.int32, device=DEV)
        s["row_weights"] = torch.rand(M, device=DEV, generator=gen) if case["weighted"] else None
        if case["grad"]:
            s["grad"] = _normal(gen, M, I)
        return s
    T, H = case["T"], case["H"]
    loud = 1 + 15 * (torch.rand(H, device=DEV, generator=gen) < 0.003)   # a few channels stand out, as in trained models
    s["x"] = _normal(gen, T, H)
    s["residual"] = (_normal(gen, T, H, std=2.0) * loud.to(torch.bfloat16)) if case["residual"] else None
    s["weight"] = (1 + 0.2 * torch.randn(H, device=DEV, generator=gen)).to(torch.bfloat16)
    if case["grad"]:
        s["grad"] = _normal(gen, T, H)
        s["grad_residual"] = _normal(gen, T, H) if case["residual"] else None
    return s


EPS = 1e-6


# ------------------------------------------------------------------ plain forms

def _wide(w, scales):
    """Weights or rows in 32 bits."""
    if scales is None:
        return w.float()
    v = w.view(torch.float8_e4m3fn).float()
    return v.view(*w.shape[:-1], -1, 128).mul_(scales[..., None]).view(w.shape)


def _by_expert(s, rows):
    """Rows in 32 bits, each expert's with zeros behind them: [E, most, columns]."""
    out = torch.zeros(s["case"]["E"], s["most"], rows.shape[1], device=rows.device)
    out[s["expert"], s["place"]] = rows[: s["case"]["rows"]]
    return out


def _in_order(s, y):
    """The rows of [E, most, columns], rounded, and zeros behind the last one."""
    out = torch.zeros(s["case"]["capacity"], y.shape[2], dtype=torch.bfloat16, device=y.device)
    out[: s["case"]["rows"]] = y[s["expert"], s["place"]].to(torch.bfloat16)
    return out


def _plain_grouped(s):
    x = _by_expert(s, _wide(s["x"], s["x_scales"]))
    return _in_order(s, torch.matmul(x, _wide(s["w"], s["w_scales"]).transpose(1, 2)))


def _plain_grouped_grad(s):
    g = _by_expert(s, s["grad"].float())
    gx = _in_order(s, torch.matmul(g, s["w"].float()))
    gw = torch.matmul(g.transpose(1, 2), _by_expert(s, s["x"].float()))
    return dict(grad_x=gx, grad_w=gw if s["case"]["grad_w"] == "fp32" else gw.to(torch.bfloat16))


def _plain_swiglu(s):
    c, n, I = s["case"], s["case"]["rows"], s["case"]["I"]
    gu = s["gate_up"][:n].float()
    g, u = gu[:, :I], gu[:, I:]
    sig = 1 / (1 + torch.exp(-g))
    silu = g * sig
    h = silu * u
    w = s["row_weights"][:n, None] if c["weighted"] else None
    y = h if w is None else h * w
    if c["out"] == "e4m3":
        codes, scales = _quantised(y)
        out = dict(codes=torch.zeros(c["capacity"], I, dtype=torch.uint8, device=y.device),
                   scales=torch.zeros(c["capacity"], I // 128, device=y.device))
        out["codes"][:n], out["scales"][:n] = codes, scales
        out["codes"] = out["codes"].view(torch.float8_e4m3fn)
        return out
    out = dict(out=torch.zeros(c["capacity"], I, dtype=torch.bfloat16, device=y.device))
    out["out"][:n] = y.to(torch.bfloat16)
    if c["grad"]:
        d = s["grad"][:n].float()
        dh = d if w is None else d * w
        out["grad_gate_up"] = torch.zeros(c["capacity"], 2 * I, dtype=torch.bfloat16, device=y.device)
        out["grad_gate_up"][:n, :I] = (dh * u * sig * (1 + g * (1 - sig))).to(torch.bfloat16)
        out["grad_gate_up"][:n, I:] = (dh * silu).to(torch.bfloat16)
        if w is not None:
            out["grad_row_weights"] = torch.zeros(c["capacity"], device=y.device)
            out["grad_row_weights"][:n] = (d * h).sum(1)
    return out


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
    w = s["weight"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * w
    out = {}
    if c["out"] != "e4m3":
        out["out"] = y.to(torch.bfloat16)
    if c["out"] != "bf16":
        codes, out["scales"] = _quantised(y)
        out["codes"] = codes.view(torch.float8_e4m3fn)
    if s["residual"] is not None:
        out["residual"] = h.to(torch.bfloat16)
    if c["grad"]:   # at the residual that the forward pass kept
        h = h.to(torch.bfloat16).float()
        r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        n, g = h * r, s["grad"].float()
        d = g * w
        dx = r * (d - n * (d * n).mean(1, keepdim=True))
        out["grad_x"] = (dx if s["grad_residual"] is None else dx + s["grad_residual"].float()).to(torch.bfloat16)
        out["grad_weight"] = (g * n).sum(0)
    return out


# ------------------------------------------------------------------ one pass

def _kept(s, name, *shape, dtype):
    """A buffer that a program keeps from call to call, zero where no call writes."""
    if name not in s:
        s[name] = torch.zeros(*shape, dtype=dtype, device=DEV)
    return s[name]


def run(state):
    s, c = state, state["case"]
    if not own:
        return dict(grouped=_plain_grouped, grouped_grad=_plain_grouped_grad, swiglu=_plain_swiglu, norm=_plain_norm)[c["op"]](s)

    from combine_moe_get_gb300 import binding as moe
    status = s["status"] if "status" in s else s.setdefault("status", moe.new_status(DEV))
    bf16 = torch.bfloat16
    if c["op"] == "grouped":
        out = _kept(s, "out", c["capacity"], c["N"], dtype=bf16)
        return moe.moe_grouped_linear(s["x"], s["w"], s["expert_prefix"], x_scales=s["x_scales"], w_scales=s["w_scales"],
                                      out=out, status=status)
    if c["op"] == "grouped_grad":
        gx = _kept(s, "grad_x", c["capacity"], c["K"], dtype=bf16)
        gw = _kept(s, "grad_w", c["E"], c["N"], c["K"], dtype=torch.float32 if c["grad_w"] == "fp32" else bf16)
        moe.moe_grouped_linear_grad_x(s["grad"], s["w"], s["expert_prefix"], out=gx, status=status)
        moe.moe_grouped_linear_grad_w(s["grad"], s["x"], s["expert_prefix"], out=gw, status=status)
        return dict(grad_x=gx, grad_w=gw)
    if c["op"] == "swiglu":
        M, I = c["capacity"], c["I"]
        keep = dict(row_weights=s["row_weights"], num_rows=s["num_rows"], status=status)
        if c["out"] == "e4m3":
            codes, scales = moe.moe_swiglu(s["gate_up"], quantize_fp8=True, out=_kept(s, "out", M, I, dtype=torch.uint8),
                                           out_scales=_kept(s, "scales", M, I // 128, dtype=torch.float32), **keep)
            return dict(codes=codes.view(torch.float8_e4m3fn), scales=scales)
        out = dict(out=moe.moe_swiglu(s["gate_up"], out=_kept(s, "out", M, I, dtype=bf16), **keep)[0])
        if c["grad"]:
            weights = _kept(s, "grad_weights", M, dtype=torch.float32) if c["weighted"] else None
            out["grad_gate_up"], weights = moe.moe_swiglu_backward(
                s["gate_up"], s["grad"], out=_kept(s, "grad_gate_up", M, 2 * I, dtype=bf16), grad_row_weights=weights, **keep)
            if weights is not None:
                out["grad_row_weights"] = weights
        return out
    r = moe.moe_add_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, bf16_out=c["out"] != "e4m3",
                             quantize_fp8=c["out"] != "bf16", status=status)
    out = {}
    if r.out is not None:
        out["out"] = r.out
    if r.codes is not None:
        out["codes"], out["scales"] = r.codes.view(torch.float8_e4m3fn), r.scales
    if r.residual is not None:
        out["residual"] = r.residual
    if c["grad"]:
        h = s["x"] if r.residual is None else r.residual
        if "workspace" not in s:
            n = moe.moe_add_rms_norm_backward_workspace_size(c["T"], c["H"])
            s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        out["grad_x"], out["grad_weight"] = moe.moe_add_rms_norm_backward(
            h, s["weight"], s["grad"], grad_residual=s["grad_residual"], eps=EPS, workspace=s["workspace"], status=status)
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] in ("grouped", "grouped_grad"):
        rows, K, N = case["rows"], case["K"], case["N"]
        named = float((1 - (1 - _shares(case)) ** rows).sum())   # experts with a row
        if case["op"] == "grouped":
            cell = 2 if case["weights"] == "bf16" else 1 + 4 / 128
            return dict(bytes=int(named * N * K * cell + rows * K * cell + rows * N * 2), flops=2 * rows * N * K)
        gw = case["E"] * N * K * (4 if case["grad_w"] == "fp32" else 2)
        return dict(bytes=int(named * N * K * 2 + rows * (2 * N + 4 * K) + gw), flops=4 * rows * N * K)
    if case["op"] == "swiglu":
        rows, I = case["rows"], case["I"]
        b = rows * I * (4 + (2 if case["out"] == "bf16" else 1 + 4 / 128)) + (4 * rows if case["weighted"] else 0)
        f = 8 * rows * I
        if case["grad"]:
            b, f = b + rows * I * (2 + 4) + (4 * rows if case["weighted"] else 0), f + 16 * rows * I
        return dict(bytes=int(b), flops=f)
    T, H = case["T"], case["H"]
    cells = 2 + (4 if case["residual"] else 0) + (2 if case["out"] != "e4m3" else 0) + (1 + 4 / 128 if case["out"] != "bf16" else 0)
    f = 6 * T * H
    if case["grad"]:   # the kept residual's own reads count once: the rows are at hand
        cells, f = cells + 4 + (2 if case["residual"] else 0), f + 10 * T * H
    return dict(bytes=int(T * H * cells + 2 * H + (4 * H if case["grad"] else 0)), flops=f)


# ------------------------------------------------------------------ the definition in 64 bits

def _values64(w, scales):
    v = w.double() if scales is None else w.view(torch.float8_e4m3fn).double()
    return v if scales is None else v * scales.double().repeat_interleave(128, -1)


def _exact_blocks(y):
    """What E4M3 codes of rows stand for before they are rounded, and the scales."""
    scales = torch.stack([b.abs().max(1).values for b in y.split(128, 1)], 1) / 448
    wide = scales.repeat_interleave(128, 1)
    return torch.where(wide > 0, y / wide.clamp_min(1e-300), 0.0), scales


def _behind(y, capacity):
    """Zeros behind the last row."""
    return torch.cat([y, y.new_zeros(capacity - y.shape[0], *y.shape[1:])])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("grouped", "grouped_grad"):
        M, E, K, N = (case[n] for n in ("capacity", "E", "K", "N"))
        p = s["expert_prefix"].tolist()
        if case["op"] == "grouped":
            y = torch.zeros(M, N, dtype=torch.float64, device=DEV)
            for e in range(E):
                r = slice(p[e], p[e + 1])
                if p[e] < p[e + 1]:
                    x = _values64(s["x"][r], None if s["x_scales"] is None else s["x_scales"][r])
                    y[r] = x @ _values64(s["w"][e], None if s["w_scales"] is None else s["w_scales"][e]).t()
            return y
        gx = torch.zeros(M, K, dtype=torch.float64, device=DEV)
        gw = torch.zeros(E, N, K, dtype=torch.float64, device=DEV)
        for e in range(E):
            r = slice(p[e], p[e + 1])
            gx[r] = s["grad"][r].double() @ s["w"][e].double()
            gw[e] = s["grad"][r].double().t() @ s["x"][r].double()
        return dict(grad_x=gx, grad_w=gw)
    if case["op"] == "swiglu":
        n, M = case["rows"], case["capacity"]
        gu = s["gate_up"][:n].double().requires_grad_(case["grad"])
        w = (s["row_weights"][:n] if case["weighted"] else torch.ones(n, device=DEV)).double().requires_grad_(case["grad"])
        g, u = gu.chunk(2, 1)
        y = torch.nn.functional.silu(g) * u * w[:, None]
        if case["out"] == "e4m3":
            codes, scales = _exact_blocks(y)
            return dict(codes=_behind(codes, M), scales=_behind(scales, M))
        out = dict(out=_behind(y.detach(), M))
        if case["grad"]:
            dgu, dw = torch.autograd.grad(y, (gu, w), s["grad"][:n].double())
            out["grad_gate_up"] = _behind(dgu, M)
            if case["weighted"]:
                out["grad_row_weights"] = _behind(dw, M)
        return out
    h = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
    w = s["weight"].double()

    def norm(h, w):
        return h / (h.pow(2).sum(1, keepdim=True) / case["H"] + EPS).sqrt() * w

    y, out = norm(h, w), {}
    if case["out"] != "e4m3":
        out["out"] = y
    if case["out"] != "bf16":
        out["codes"], out["scales"] = _exact_blocks(y)
    if s["residual"] is not None:
        out["residual"] = h
    if case["grad"]:
        # the sum of two bf16 rounds the same from 64 bits as from 32, where it is exact or so near that it cannot tell
        kept = h.float().to(torch.bfloat16).double().requires_grad_()
        w = w.requires_grad_()
        dx, out["grad_weight"] = torch.autograd.grad(norm(kept, w), (kept, w), s["grad"].double())
        out["grad_x"] = dx if s["grad_residual"] is None else dx + s["grad_residual"].double()
    return out
