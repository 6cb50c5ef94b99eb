"""Cases for the operators around the dispatch and the combine: the experts'
products over the receive rows (BF16 in its three directions, and with 4-bit
weights), and the RMS norm that stands before the dispatch, with its backward.

`run` computes them with elementary torch operations in binary32, or, with
`own` set, through combine_ep_layout_10_amd.ops.

Sizes follow the workloads of ep_workloads.py: hidden 7168 with top-8 routing
(a rank's share of 8,192 tokens: 32 experts with about 2,048 rows each),
hidden 4096 with 64 experts and top-6, 128-token decode steps, and small odd
ones.
"""
import math

import torch

own = False

GEMMS = ("forward", "grad_input", "grad_weight")


def listed():
    return [
        # one rank's experts over a training batch of 8,192 tokens: up and gate
        # projections at once, rows packed without padding
        dict(name="forward rank", op="forward", tokens=8192, experts=32, topk=8, n=4096, k=7168, align=1, skew=0.0),
        # a small serving batch: about six rows an expert, bound by the weights
        dict(name="forward decode", op="forward", tokens=64, experts=64, topk=6, n=4096, k=4096, align=1, skew=0.0),
        # the same products' input gradient in a training step, rows padded to 128
        dict(name="grad_input train", op="grad_input", tokens=4096, experts=64, topk=6, n=4096, k=4096, align=128,
             skew=0.0),
        # a small model's step with a hot expert and sizes that no tile divides
        dict(name="grad_input odd", op="grad_input", tokens=515, experts=24, topk=3, n=1000, k=1416, align=16, skew=0.6),
        # weight gradients of a training step, kept in BF16
        dict(name="grad_weight train", op="grad_weight", tokens=4096, experts=64, topk=6, n=4096, k=4096, align=128,
             skew=0.0, f32=False),
        # weight gradients kept in binary32, odd sizes
        dict(name="grad_weight odd", op="grad_weight", tokens=900, experts=16, topk=2, n=1416, k=1000, align=1, skew=0.6,
             f32=True),
        # serving one token: eight experts' weights, each read for a single row
        dict(name="mxfp4 token", op="mxfp4", tokens=1, experts=32, topk=8, n=4096, k=7168, align=1, skew=0.0),
        # a 128-token decode step on one rank's experts: 16 rows an expert
        dict(name="mxfp4 decode", op="mxfp4", tokens=128, experts=64, topk=8, n=4096, k=7168, align=1, skew=0.0),
        # the norm before the FP8 dispatch of a training or prefill batch
        dict(name="norm prefill", op="norm", tokens=8192, hidden=7168, fp8=True, residual=True),
        # the norm of a decode step, BF16 output: latency counts
        dict(name="norm decode", op="norm", tokens=16, hidden=7168, fp8=False, residual=True),
        # backward of the norm in the training batch
        dict(name="norm backward", op="norm_backward", tokens=8192, hidden=7168, residual=True),
        # backward of the norm in a small model's step, no residual branch
        dict(name="norm backward small", op="norm_backward", tokens=300, hidden=1024, residual=False),
    ]


def _log(rng, low, high, step=1):
    """A multiple of step, spread evenly over the logarithm of [low, high]."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return min(high // step * step, max(-(-low // step) * step, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(GEMMS + ("mxfp4", "norm", "norm_backward"))
    if op in ("norm", "norm_backward"):
        fp8 = op == "norm" and rng.random() < 0.6
        hidden = _log(rng, 256, 8192, 128 if fp8 else 8)
        c = dict(op=op, tokens=_log(rng, 1, 8192), hidden=hidden, residual=rng.random() < 0.7)
        if op == "norm":
            c["fp8"] = fp8
        return c
    experts = rng.choice((8, 16, 32, 64))
    c = dict(op=op, tokens=_log(rng, 1, 4096) if op != "mxfp4" else _log(rng, 1, 256), experts=experts,
             topk=rng.choice((1, 2, 4, 6, 8)), n=_log(rng, 256, 4096, 8),
             k=_log(rng, 256, 4096, 32 if op == "mxfp4" else 8), align=rng.choice((1, 1, 16, 128)),
             skew=rng.choice((0.0, 0.0, 0.6)))
    if op == "grad_weight":
        c["f32"] = rng.random() < 0.5
    return c


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0):
    """BF16 normal values, drawn a slab of the first axis at a time."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    per = max(1, (1 << 28) // max(1, math.prod(shape[1:])))
    for i in range(0, shape[0], per):
        part = torch.randn((min(per, shape[0] - i),) + shape[1:], generator=g, device="cuda")
        out[i:i + per] = part.mul_(scale)
    return out


def _routing(case, g):
    """Distinct experts for every token: the largest of log p + Gumbel noise."""
    p = -case["skew"] * torch.arange(1, case["experts"] + 1, device="cuda").double().log()
    noise = torch.rand((case["tokens"], case["experts"]), generator=g, device="cuda", dtype=torch.float64)
    return (p - (-noise.log()).log()).topk(case["topk"], dim=1).indices


def _counts(idx, case):
    """Rows of each expert, the first row of each, and the rows that hold them
    all when every expert's rows are padded to the alignment."""
    count = torch.bincount(idx.flatten(), minlength=case["experts"])
    padded = (count + case["align"] - 1) // case["align"] * case["align"]
    bound = case["tokens"] * case["topk"] + case["experts"] * (case["align"] - 1)
    return count, padded.cumsum(0) - padded, bound


def _live(idx, case):
    """Receive rows that hold a token, expert by expert."""
    count, first, _ = _counts(idx, case)
    expert = torch.repeat_interleave(torch.arange(case["experts"], device="cuda"), count)
    within = torch.arange(expert.numel(), device="cuda") - (count.cumsum(0) - count)[expert]
    return expert, within, first[expert] + within


def _rows(g, bound, live, width, scale=1.0):
    """Receive rows: normal values where a token is, zeros on padding."""
    out = torch.zeros((bound, width), dtype=torch.bfloat16, device="cuda")
    out[live] = _normal(g, live.numel(), width, scale=scale)
    return out


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("norm", "norm_backward"):
        T, H = case["tokens"], case["hidden"]
        s["x"] = _normal(g, T, H)
        s["weight"] = (1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
        s["residual"] = _normal(g, T, H, scale=3.0) if case["residual"] else None
        if op == "norm_backward":  # x is then the normalised rows' input, residual the gradient that skips the norm
            s["rstd"] = (s["x"].double().square().mean(1) + 1e-6).rsqrt().float()
            s["grad_y"] = _normal(g, T, H)
            if own:
                from combine_ep_layout_10_amd import ops
                s["workspace"] = ops.rms_norm_workspace(T, H)
        return s

    E, n, k = case["experts"], case["n"], case["k"]
    idx = _routing(case, g)
    _, _, bound = _counts(idx, case)
    expert, within, live = _live(idx, case)
    if own:
        from combine_ep_layout_10_amd import ops
        cfg = ops.Config(max_tokens=case["tokens"], hidden=8, num_experts=E, num_topk=case["topk"],
                         expert_alignment=case["align"])
        s["handle"] = ops.layout(cfg, idx)
    # where each live row stands in a batch of the experts that have rows
    used, place = expert.unique(return_inverse=True)
    most = int(within.max()) + 1
    s["live"], s["used"], s["place"], s["batch"] = live, used, place * most + within, (used.numel(), most)
    if op == "mxfp4":
        s["a"] = _rows(g, bound, live, k)
        s["b"] = torch.randint(0, 256, (E, n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
        # block scales 2^-9 .. 2^-6: weights of the size that initialisation gives
        s["b_scales"] = torch.randint(118, 122, (E, n, k // 32), dtype=torch.uint8, device="cuda", generator=g)
    else:
        if op != "grad_input":
            s["a"] = _rows(g, bound, live, k)
        if op != "forward":
            s["grad_out"] = _rows(g, bound, live, n)
        if op != "grad_weight":
            s["b"] = _normal(g, E, n, k, scale=1.0 / math.sqrt(k))
    if op == "grad_weight":
        s["out"] = torch.zeros((E, n, k), dtype=torch.float32 if case["f32"] else torch.bfloat16, device="cuda")
    else:
        s["out"] = torch.zeros((bound, k if op == "grad_input" else n), dtype=torch.bfloat16, device="cuda")
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    if op == "norm":
        return _norm(state)
    if op == "norm_backward":
        return _norm_backward(state)
    if op == "grad_weight":
        g, a = _batched(state, "grad_out"), _batched(state, "a")
        state["out"][state["used"]] = torch.bmm(g.transpose(1, 2).contiguous(), a).to(state["out"].dtype)
        return state["out"]
    if op == "grad_input":
        prod = torch.bmm(_batched(state, "grad_out"), _used(state, state["b"]).float())
    elif op == "forward":
        prod = torch.bmm(_batched(state, "a"), _used(state, state["b"]).float().transpose(1, 2).contiguous())
    else:
        prod = torch.bmm(_batched(state, "a"), _mxfp4(state).transpose(1, 2).contiguous())
    state["out"][state["live"]] = prod.flatten(0, 1)[state["place"]].to(torch.bfloat16)
    return state["out"]


def _run_own(state, op):
    from combine_ep_layout_10_amd import ops
    if op == "norm":
        fp8 = state["case"]["fp8"]
        y, scales, total, rstd = ops.rms_norm(state["x"], state["weight"], 1e-6, residual=state["residual"],
                                              dtype=ops.FP8_QUANTIZE if fp8 else ops.BF16)
        return dict(y=y.view(torch.float8_e4m3fn), scales=scales, total=total, rstd=rstd) if fp8 else \
            dict(y=y, total=total, rstd=rstd)
    if op == "norm_backward":
        grad_x, grad_weight = ops.rms_norm_backward(state["x"], state["weight"], state["rstd"], state["grad_y"],
                                                    grad_total=state["residual"], workspace=state["workspace"])
        return dict(grad_x=grad_x, grad_weight=grad_weight)
    h, out = state["handle"], state["out"]
    if op == "forward":
        return ops.grouped_gemm_bf16(h, state["a"], state["b"], out=out)
    if op == "grad_input":
        return ops.grouped_gemm_bf16_grad_input(h, state["grad_out"], state["b"], grad_a=out)
    if op == "grad_weight":
        return ops.grouped_gemm_bf16_grad_weight(h, state["grad_out"], state["a"], grad_b=out)
    return ops.grouped_gemm_mxfp4(h, state["a"], state["b"], state["b_scales"], out=out)


def _batched(state, name):
    """The live rows as a batch [experts with rows, most rows, width], zeros behind."""
    x = state[name]
    experts, most = state["batch"]
    out = torch.zeros((experts * most, x.shape[1]), dtype=torch.float32, device=x.device)
    out[state["place"]] = x[state["live"]].float()
    return out.view(experts, most, x.shape[1])


def _used(state, w):
    """The weights of the experts that have rows."""
    return w if state["used"].numel() == w.shape[0] else w[state["used"]]


def _mxfp4(state):
    """The 4-bit weights of the experts that have rows, as binary32: sign,
    two exponent bits, one mantissa bit, times their group's power of two."""
    b, scales = _used(state, state["b"]), _used(state, state["b_scales"])
    value = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    value = torch.cat([value, -value])
    w = torch.stack([value[(b & 15).int()], value[(b >> 4).int()]], dim=-1)
    w = w.view(scales.shape + (32,)) * torch.exp2(scales.float() - 127.0).unsqueeze(-1)
    return w.flatten(2)


def _norm(state):
    x = state["x"]
    total = x if state["residual"] is None else (x.float() + state["residual"].float()).to(torch.bfloat16)
    s = total.float()
    rstd = torch.rsqrt(s.square().mean(1) + 1e-6)
    u = s * state["weight"].float()
    if not state["case"]["fp8"]:
        return dict(y=(u * rstd[:, None]).to(torch.bfloat16), total=total, rstd=rstd)
    u = u.view(u.shape[0], -1, 128)
    q = u.abs().amax(2, keepdim=True) / 448.0
    code = torch.where(q > 0, u / q, torch.zeros_like(u)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return dict(y=code.view(x.shape), scales=q.squeeze(2) * rstd[:, None], total=total, rstd=rstd)


def _norm_backward(state):
    s, g, rstd = state["x"].float(), state["grad_y"].float(), state["rstd"][:, None]
    gw = g * state["weight"].float()
    xhat = s * rstd
    grad_x = rstd * (gw - xhat * (gw * xhat).mean(1, keepdim=True))
    if state["residual"] is not None:
        grad_x = grad_x + state["residual"].float()
    return dict(grad_x=grad_x.to(torch.bfloat16), grad_weight=(g * xhat).sum(0))


def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        T, H = case["tokens"], case["hidden"]
        extra = 2 if case["residual"] else 0
        if op == "norm":
            out = 1 + 4 / 128 if case["fp8"] else 2
            return dict(bytes=T * H * (2 + 2 * extra + out) + 4 * T + 2 * H, flops=6 * T * H)
        return dict(bytes=T * H * (2 + 2 + extra + 2) + 4 * T + 6 * H, flops=10 * T * H)
    E, n, k = case["experts"], case["n"], case["k"]
    rows = case["tokens"] * case["topk"]
    # experts that have rows, when routing is even
    used = min(E, rows) if rows > 4 * E else E * (1 - (1 - min(1.0, case["topk"] / E)) ** case["tokens"])
    weight = dict(forward=2.0, grad_input=2.0, mxfp4=0.5 + 1 / 32, grad_weight=4.0 if case.get("f32") else 2.0)[op]
    return dict(bytes=rows * 2 * (n + k) + (E if op == "grad_weight" else used) * n * k * weight, flops=2 * rows * n * k)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        total = s["x"].double() if s["residual"] is None else \
            (s["x"].double() + s["residual"].double()).to(torch.bfloat16).double()
        rstd = 1.0 / (total.pow(2).sum(1) / case["hidden"] + 1e-6).sqrt()
        y = total * s["weight"].double() * rstd[:, None]
        if not case["fp8"]:
            return dict(y=y, total=total, rstd=rstd)
        blocks = y.unflatten(1, (-1, 128))
        scales = blocks.abs().max(2).values / 448.0
        unit = blocks / scales.clamp(min=1e-300).unsqueeze(2)
        return dict(y=unit.flatten(1), scales=scales, total=total, rstd=rstd)
    if op == "norm_backward":
        x, g, w, r = s["x"].double(), s["grad_y"].double(), s["weight"].double(), s["rstd"].double()
        inner = (g * w * x).sum(1) / case["hidden"]
        grad = g * w * r[:, None] - x * (inner * r.pow(3))[:, None]
        if s["residual"] is not None:
            grad += s["residual"].double()
        return dict(grad_x=grad, grad_weight=(g * x * r[:, None]).sum(0))
    idx = _routing(case, _generator(seed))
    count, first, _ = _counts(idx, case)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    levels = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
    for e, (c, f) in enumerate(zip(count.tolist(), first.tolist())):
        rows = slice(f, f + c)
        if c == 0:
            continue
        if op == "grad_weight":
            out[e] = s["grad_out"][rows].double().t() @ s["a"][rows].double()
        elif op == "grad_input":
            out[rows] = s["grad_out"][rows].double() @ s["b"][e].double()
        elif op == "forward":
            out[rows] = s["a"][rows].double() @ s["b"][e].double().t()
        else:
            w = torch.empty((case["n"], case["k"]), dtype=torch.float64, device="cuda")
            for half in (0, 1):
                code = (s["b"][e] >> (4 * half)) & 15
                w[:, half::2] = levels[(code & 7).long()] * (1 - 2 * (code >> 3).double())
            w *= torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), s["b_scales"][e].int() - 127) \
                .repeat_interleave(32, dim=1)
            out[rows] = s["a"][rows].double() @ w.t()
    return out
