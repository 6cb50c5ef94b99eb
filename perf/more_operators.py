"""Cases for the router (choice and weights of a token's experts, the balance
loss with the counts, and the gradient of both with respect to the logits) and
for 4-bit rows (MXFP4 quantisation, and the experts' products with both operands
in MXFP4).

`run` computes them with elementary torch operations in binary32 (the keys that
decide a choice, and sums over a batch, in binary64), or, with `own` set, through
combine_ep_layout_10_amd.ops.

Sizes follow the workloads of ep_workloads.py: 8,192 tokens with 256 experts and
top-8, 4,096 tokens with 64 experts and top-6, 128-token and one-token decode
steps at hidden 7168, and small odd ones.
"""
import math

import torch

own = False

ROUTER = ("route", "balance", "backward")


def listed():
    return [
        # the router of a training or prefill batch: sigmoid scores, a choice that a bias
        # steers, four of eight groups, weights normalised and scaled; some padding tokens
        dict(name="route batch", op="route", tokens=8192, experts=256, topk=8, score="sigmoid", f32=True, bias=True,
             groups=8, keep=4, best=2, renormalize=True, masked=0.02),
        # a decode step: plain softmax scores, latency counts
        dict(name="route decode", op="route", tokens=128, experts=256, topk=8, score="softmax", f32=False, bias=False,
             groups=1, keep=1, best=1, renormalize=True, masked=0.0),
        # the balance loss over a whole training batch
        dict(name="balance batch", op="balance", tokens=8192, experts=256, topk=8, score="sigmoid", f32=True, sequences=1,
             masked=0.02),
        # the same for every sequence of a packed batch, of uneven lengths
        dict(name="balance sequences", op="balance", tokens=4096, experts=64, topk=6, score="softmax", f32=False,
             sequences=19, masked=0.0),
        # the router's gradient in a training step: of the weights and of the loss
        dict(name="backward batch", op="backward", tokens=8192, experts=256, topk=8, score="sigmoid", f32=True,
             renormalize=True, sequences=1, loss=True, masked=0.02),
        # a small model's step, odd sizes, no loss
        dict(name="backward odd", op="backward", tokens=515, experts=60, topk=3, score="softmax", f32=False,
             renormalize=False, sequences=1, loss=False, masked=0.0),
        # the receive rows of a rank's prompt, quantised ahead of the experts' products
        dict(name="quantize rows", op="quantize", tokens=8192, experts=32, topk=8, k=7168, align=128, skew=0.0),
        # master weights of eight experts in binary32, with the values that the codes stand for (training with 4-bit weights)
        dict(name="quantize weights", op="quantize", experts=8, n=4096, k=4096, f32=True, values=True),
        # one rank's experts over a prompt of 8,192 tokens
        dict(name="product prompt", op="product", tokens=8192, experts=32, topk=8, n=4096, k=7168, align=1, skew=0.0),
        # a 128-token decode step on one rank's experts: 16 rows an expert
        dict(name="product decode", op="product", tokens=128, experts=64, topk=8, n=4096, k=7168, align=1, skew=0.0),
        # serving one token: eight experts' weights, each read for a single row
        dict(name="product token", op="product", tokens=1, experts=32, topk=8, n=4096, k=7168, align=1, skew=0.0),
        # a small model's step with a hot expert and sizes that no tile divides
        dict(name="product odd", op="product", tokens=515, experts=24, topk=3, n=1000, k=1440, align=16, skew=0.6),
    ]


def _log(rng, low, high, step=1):
    """A multiple of step, spread evenly over the logarithm of [low, high]."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return min(high // step * step, max(-(-low // step) * step, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(ROUTER + ("quantize", "product", "product"))
    if op in ROUTER:
        experts = rng.choice((8, 16, 60, 64, 160, 256, rng.randint(9, 256)))
        c = dict(op=op, tokens=_log(rng, 1, 8192), experts=experts, topk=rng.choice((1, 2, 4, 6, 8)),
                 score=rng.choice(("softmax", "sigmoid")), f32=rng.random() < 0.5, masked=rng.choice((0.0, 0.0, 0.1)))
        if op == "route":
            c["bias"] = rng.random() < 0.5
            groups = rng.choice([g for g in (1, 4, 8) if experts % g == 0 and experts // g >= 8] or [1])
            c["groups"], c["keep"] = groups, max(1, groups // 2)
            c["best"] = 2 if groups > 1 and c["bias"] else 1
        if op != "balance":
            c["renormalize"] = rng.random() < 0.5
        if op != "route":
            c["sequences"] = rng.choice((1, 1, _log(rng, 2, 64)))
        if op == "backward":
            c["loss"] = rng.random() < 0.7
        return c
    if op == "quantize" and rng.random() < 0.5:
        return dict(op=op, experts=rng.choice((1, 3, 8)), n=_log(rng, 1, 4096), k=_log(rng, 256, 4096, 32),
                    f32=rng.random() < 0.5, values=rng.random() < 0.5)
    c = dict(op=op, tokens=_log(rng, 1, 4096), experts=rng.choice((8, 16, 32, 64)), topk=rng.choice((1, 2, 4, 6, 8)),
             k=_log(rng, 256, 4096, 32), align=rng.choice((1, 1, 16, 128)), skew=rng.choice((0.0, 0.0, 0.6)))
    if op == "product":
        c["n"] = _log(rng, 256, 4096, 8)
    return c


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    """Normal values, drawn a slab of the first axis at a time."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    per = max(1, (1 << 28) // max(1, math.prod(shape[1:])))
    for i in range(0, shape[0], per):
        part = torch.randn((min(per, shape[0] - i),) + shape[1:], generator=g, device="cuda")
        out[i:i + per] = part.mul_(scale)
    return out


# ---------------------------------------------------------------- what a program has before the call

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


def _prepare_router(case, g):
    T, E, k = case["tokens"], case["experts"], case["topk"]
    s = dict(case=case)
    popular = 0.5 * torch.randn(E, generator=g, device="cuda")
    logits = 1.5 * torch.randn((T, E), generator=g, device="cuda") + popular
    s["logits"] = logits if case["f32"] else logits.to(torch.bfloat16)
    routed = torch.rand(T, generator=g, device="cuda") >= case["masked"]
    if case["op"] == "route":
        s["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        s["mask"] = routed if case["masked"] else None
    else:
        s["idx"] = s["logits"].float().topk(k, dim=1).indices.masked_fill(~routed[:, None], -1)
        cuts = torch.randint(0, T + 1, (case["sequences"] - 1,), generator=g, device="cuda").sort().values
        ends = torch.tensor([0, T], device="cuda")
        s["seq_off"] = torch.cat([ends[:1], cuts, ends[1:]]).int() if case["sequences"] > 1 else None
    if case["op"] == "backward":
        s["grad_w"] = torch.randn((T, k), generator=g, device="cuda")
        if case["loss"]:
            # the forward's counts, and a factor for each sequence of the size it gives them
            counts, tokens = _count(s["idx"], _sequence_of(s), case)
            s["counts"] = counts.int()
            s["coef"] = (E / (k * tokens.clamp(min=1).double().square() * max(1, case["sequences"]))).float()
            s["grad_loss"] = 0.5 + torch.rand((), generator=g, device="cuda")
    if own:
        from combine_ep_layout_10_amd import ops
        s["router"] = ops.Router(num_experts=E, num_topk=k,
                                 score=ops.SCORE_SIGMOID if case["score"] == "sigmoid" else ops.SCORE_SOFTMAX,
                                 num_groups=case.get("groups", 1), topk_groups=case.get("keep", 1),
                                 group_best=case.get("best", 1), renormalize=case.get("renormalize", False),
                                 scale=_SCALE)
        if case["op"] == "balance":
            s["workspace"] = ops.balance_loss_workspace(s["router"], T, case["sequences"])
    return s


_SCALE = 2.5  # factor of the weights


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op in ROUTER:
        return _prepare_router(case, g)
    E, k = case["experts"], case["k"]
    s = dict(case=case)
    if op == "quantize" and "n" in case:
        s["x"] = _normal(g, E, case["n"], k, scale=1.0 / math.sqrt(k),
                         dtype=torch.float32 if case["f32"] else torch.bfloat16)
        return s
    idx = _routing(case, g)
    _, _, bound = _counts(idx, case)
    expert, within, live = _live(idx, case)
    s["live"] = live
    if own:
        from combine_ep_layout_10_amd import ops
        cfg = ops.Config(max_tokens=case["tokens"], hidden=8, num_experts=E, num_topk=case["topk"],
                         expert_alignment=case["align"])
        s["handle"] = ops.layout(cfg, idx)
    if op == "quantize":
        s["x"] = torch.zeros((bound, k), dtype=torch.bfloat16, device="cuda")
        s["x"][live] = _normal(g, live.numel(), k)
        s["codes"] = torch.zeros((bound, k // 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros((bound, k // 32), dtype=torch.uint8, device="cuda")
        return s
    n = case["n"]
    # where each live row stands in a batch of the experts that have rows
    used, place = expert.unique(return_inverse=True)
    most = int(within.max()) + 1
    s["used"], s["place"], s["batch"] = used, place * most + within, (used.numel(), most)
    s["a"] = torch.zeros((bound, k // 2), dtype=torch.uint8, device="cuda")
    s["a_scales"] = torch.zeros((bound, k // 32), dtype=torch.uint8, device="cuda")
    s["a"][live], s["a_scales"][live] = _quantize(_normal(g, live.numel(), k))
    s["b"] = torch.empty((E, n, k // 2), dtype=torch.uint8, device="cuda")
    s["b_scales"] = torch.empty((E, n, k // 32), dtype=torch.uint8, device="cuda")
    for e in range(E):
        s["b"][e], s["b_scales"][e] = _quantize(_normal(g, n, k, scale=1.0 / math.sqrt(k)))
    s["out"] = torch.zeros((bound, n), dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    if op == "route":
        return _route(state)
    if op == "balance":
        return _balance(state)
    if op == "backward":
        return _backward(state)
    if op == "quantize":
        if "live" not in state:
            codes, scales = _quantize(state["x"])
            out = dict(codes=codes, scales=scales)
            if state["case"]["values"]:
                out["values"] = _values(codes, scales).to(torch.bfloat16)
            return out
        state["codes"][state["live"]], state["scales"][state["live"]] = _quantize(state["x"][state["live"]])
        return dict(codes=state["codes"], scales=state["scales"])
    experts, most = state["batch"]
    a = torch.zeros((experts * most, state["case"]["k"]), dtype=torch.float32, device="cuda")
    a[state["place"]] = _values(state["a"][state["live"]], state["a_scales"][state["live"]])
    whole = state["used"].numel() == state["b"].shape[0]
    b, b_scales = (state["b"], state["b_scales"]) if whole else (state["b"][state["used"]], state["b_scales"][state["used"]])
    prod = torch.bmm(a.view(experts, most, -1), _values(b, b_scales).transpose(1, 2).contiguous())
    state["out"][state["live"]] = prod.flatten(0, 1)[state["place"]].to(torch.bfloat16)
    return state["out"]


def _run_own(state, op):
    from combine_ep_layout_10_amd import ops
    case = state["case"]
    if op == "route":
        idx, w = ops.route(state["router"], state["logits"], bias=state["bias"], token_mask=state["mask"])
        return dict(idx=idx, weights=w)
    if op == "balance":
        loss, counts, coef = ops.balance_loss(state["router"], state["logits"], state["idx"], seq_off=state["seq_off"],
                                              workspace=state["workspace"])
        return dict(loss=loss, counts=counts, coef=coef)
    if op == "backward":
        return ops.route_backward(state["router"], state["logits"], state["idx"], grad_topk_w=state["grad_w"],
                                  counts=state.get("counts"), coef=state.get("coef"), grad_loss=state.get("grad_loss"),
                                  seq_off=state["seq_off"] if case["loss"] else None)  # read with the counts alone
    if op == "quantize":
        if "live" not in state:
            values = torch.empty(state["x"].shape, dtype=torch.bfloat16, device="cuda") if case["values"] else None
            codes, scales = ops.quantize_mxfp4(state["x"], values=values)
            return dict(codes=codes, scales=scales) if values is None else dict(codes=codes, scales=scales, values=values)
        codes, scales = ops.quantize_mxfp4(state["x"], state["handle"], codes=state["codes"], scales=state["scales"])
        return dict(codes=codes, scales=scales)
    return ops.grouped_gemm_mxfp4_rows(state["handle"], state["a"], state["a_scales"], state["b"], state["b_scales"],
                                       out=state["out"])


def _probabilities(logits, score, dtype):
    """Scores that sum to one over a token's experts, and the scores themselves."""
    l = logits.to(dtype)
    if score == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
        return s / s.sum(1, keepdim=True), s
    e = torch.exp(l - l.amax(1, keepdim=True))
    p = e / e.sum(1, keepdim=True)
    return p, p


def _route(state):
    case, logits = state["case"], state["logits"]
    T, E, k = case["tokens"], case["experts"], case["topk"]
    # what decides a choice, in 64 bits: scores next to each other must not change places
    key = logits.double()
    if case["bias"] or case["best"] > 1:
        key = _probabilities(logits, case["score"], torch.float64)[1]
        if case["bias"]:
            key = key + state["bias"].double()
    if case["groups"] > 1:
        grouped = key.view(T, case["groups"], -1)
        best = grouped.sort(dim=2, descending=True).values[:, :, :case["best"]].sum(2)
        rank = best.sort(dim=1, descending=True, stable=True).indices[:, :case["keep"]]
        kept = torch.zeros((T, case["groups"]), dtype=torch.bool, device="cuda").scatter_(1, rank, True)
        key = grouped.masked_fill(~kept[:, :, None], -math.inf).view(T, E)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = _probabilities(logits, case["score"], torch.float32)[1].gather(1, idx)
    if case["renormalize"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    w = w * _SCALE
    if state["mask"] is not None:
        idx = idx.masked_fill(~state["mask"][:, None], -1)
        w = w.masked_fill(~state["mask"][:, None], 0.0)
    return dict(idx=idx, weights=w)


def _sequence_of(state):
    """The sequence of each token."""
    if state["seq_off"] is None:
        return torch.zeros(state["case"]["tokens"], dtype=torch.int64, device="cuda")
    t = torch.arange(state["case"]["tokens"], device="cuda")
    return (t[:, None] >= state["seq_off"][None, 1:]).sum(1)


def _count(idx, seq, case):
    """Pairs of each sequence and expert, and routed tokens of each sequence."""
    member = (seq[None, :] == torch.arange(case["sequences"], device="cuda")[:, None]).float()
    chosen = torch.zeros((case["tokens"], case["experts"]), device="cuda")
    chosen.scatter_add_(1, idx.clamp(min=0), (idx >= 0).float())
    return (member @ chosen).long(), (member @ (idx >= 0).any(1).float()).long()


def _balance(state):
    case, idx = state["case"], state["idx"]
    S, E, k = case["sequences"], case["experts"], case["topk"]
    seq = _sequence_of(state)
    counts, tokens = _count(idx, seq, case)
    p = _probabilities(state["logits"], case["score"], torch.float32)[0] * (idx >= 0).any(1, keepdim=True)
    member = seq[None, :] == torch.arange(S, device="cuda")[:, None]
    sums = member.double() @ p.double()
    used = (tokens > 0).sum().clamp(min=1)
    coef = torch.where(tokens > 0, E / (k * tokens.clamp(min=1).double().square() * used), 0.0)
    loss = (coef * (counts * sums).sum(1)).sum()
    return dict(loss=loss.float(), counts=counts.int(), coef=coef.float())


def _backward(state):
    case, logits, idx = state["case"], state["logits"], state["idx"]
    routed = (idx >= 0).any(1, keepdim=True)
    at = idx.clamp(min=0)
    p, s = _probabilities(logits, case["score"], torch.float32)
    chosen = s.gather(1, at)
    grad_s = state["grad_w"] * _SCALE
    if case["renormalize"]:
        total = chosen.sum(1, keepdim=True) + 1e-20
        grad_s = (grad_s - (grad_s * chosen).sum(1, keepdim=True) / total) / total
    grad_s = torch.zeros_like(s).scatter_add_(1, at, grad_s.masked_fill(idx < 0, 0.0))
    if case["loss"]:
        # in 64 bits: counts of a balanced batch are nearly equal, and their mean goes out again
        b = state["counts"].double() * (state["coef"].double() * state["grad_loss"].double())[:, None]
        b = b[_sequence_of(state)]
        b = (b - (p * b).sum(1, keepdim=True)).float()
        grad_s = grad_s + (b / s.sum(1, keepdim=True) if case["score"] == "sigmoid" else b)
    if case["score"] == "sigmoid":
        grad = grad_s * s * (1.0 - s)
    else:
        grad = p * (grad_s - (p * grad_s).sum(1, keepdim=True))
    return grad.masked_fill(~routed, 0.0).to(logits.dtype)


def _quantize(x):
    """Codes (sign, two exponent bits, one mantissa bit; two a byte, the first in
    the low half) and a power of two for each 32 values: the largest magnitude's
    power lies two below, so that it is a 4 or more; nearest even, at most 6."""
    v = x.float().unflatten(-1, (-1, 32))
    most = v.abs().amax(-1, keepdim=True)
    power = torch.where(most > 0, torch.frexp(most).exponent - 3, -127).clamp(min=-127)
    y = torch.ldexp(v.abs(), -power)
    code = torch.where(y < 2.0, (2.0 * y).round(), torch.where(y < 4.0, y.round() + 2.0, (0.5 * y).round() + 4.0))
    code = code.clamp(max=7.0).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    finite = torch.isfinite(most)
    code = code.masked_fill(~finite, 0).flatten(-2)
    scales = (power + 127).masked_fill(~finite, 255).to(torch.uint8).squeeze(-1)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def _values(codes, scales):
    """What MXFP4 codes and scales stand for, in binary32."""
    value = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    value = torch.cat([value, -value])
    v = torch.stack([value[(codes & 15).int()], value[(codes >> 4).int()]], dim=-1)
    return (v.view(scales.shape + (32,)) * torch.exp2(scales.float() - 127.0).unsqueeze(-1)).flatten(-2)


# ---------------------------------------------------------------- work and exact results

def work(case):
    op = case["op"]
    if op in ROUTER:
        T, E, k = case["tokens"], case["experts"], case["topk"]
        logits = T * E * (4 if case["f32"] else 2)
        if op == "route":
            return dict(bytes=logits + T * k * 12 + (4 * E if case["bias"] else 0) + (T if case["masked"] else 0),
                        flops=8 * T * E)
        S = case["sequences"]
        extra = 4 * (S + 1) if S > 1 else 0
        if op == "balance":
            return dict(bytes=logits + 8 * T * k + 4 * S * E + 4 * S + extra, flops=8 * T * E)
        loss = 4 * S * E + 4 * S + extra if case["loss"] else 0
        return dict(bytes=2 * logits + 12 * T * k + loss, flops=12 * T * E)
    E, k = case["experts"], case["k"]
    if op == "quantize":
        values = case["tokens"] * case["topk"] * k if "tokens" in case else E * case["n"] * k
        size = (4 if case.get("f32") else 2) + 17 / 32 + (2 if case.get("values") else 0)
        return dict(bytes=values * size, flops=4 * values)
    n, rows = case["n"], case["tokens"] * case["topk"]
    # experts that have rows, when routing is even
    used = min(E, rows) if rows > 4 * E else E * (1 - (1 - min(1.0, case["topk"] / E)) ** case["tokens"])
    return dict(bytes=rows * (k * 17 / 32 + 2 * n) + used * n * k * 17 / 32, flops=2 * rows * n * k)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ROUTER:
        return _exact_router(case, s)
    levels = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
    if op == "quantize":
        if not case.get("values"):
            return None  # bytes alone
        values = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            x = s["x"][e].double().view(case["n"], -1, 32)
            top = x.abs().max(2, keepdim=True).values
            # the power of two at or below the largest magnitude, a quarter of it
            unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -125)))) / 4
            unit = torch.where(unit * 4 > top, unit / 2, unit).clamp(min=2.0 ** -127)
            y = x.abs() / unit
            below = (torch.searchsorted(levels, y.contiguous(), right=True) - 1).clamp(max=6)
            down, up = y - levels[below], levels[below + 1] - y
            step = (up < down) | ((up == down) & (below % 2 == 1))
            values[e] = (torch.where(step, levels[below + 1], levels[below]) * torch.sign(x) * unit).view(case["n"], -1)
        return dict(codes=None, scales=None, values=values)

    def operand(codes, scales):
        w = torch.empty((codes.shape[0], case["k"]), dtype=torch.float64, device="cuda")
        for half in (0, 1):
            code = (codes >> (4 * half)) & 15
            w[:, half::2] = levels[(code & 7).long()] * (1 - 2 * (code >> 3).double())
        return w * torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"),
                               scales.int() - 127).repeat_interleave(32, dim=1)

    count, first, _ = _counts(_routing(case, _generator(seed)), case)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for e, (c, f) in enumerate(zip(count.tolist(), first.tolist())):
        if c:
            rows = slice(f, f + c)
            out[rows] = operand(s["a"][rows], s["a_scales"][rows]) @ operand(s["b"][e], s["b_scales"][e]).t()
    return out


def _exact_router(case, s):
    T, E, k = case["tokens"], case["experts"], case["topk"]
    l = s["logits"].double()
    if case["score"] == "sigmoid":
        score = torch.sigmoid(l)
        share = score / score.sum(1)[:, None]
    else:
        score = share = torch.softmax(l, 1)
    if case["op"] == "route":
        key = l.clone()
        if case["bias"] or case["best"] == 2:
            key = score + (s["bias"].double() if case["bias"] else 0.0)
        size = E // case["groups"]
        if case["groups"] > 1:
            best = torch.stack([key[:, g * size:(g + 1) * size].topk(case["best"], 1).values.sum(1)
                                for g in range(case["groups"])], 1)
            place = torch.argsort(torch.argsort(best, dim=1, descending=True, stable=True), dim=1)
            key = torch.where((place < case["keep"]).repeat_interleave(size, 1), key, -math.inf)
        w = score.gather(1, torch.argsort(key, dim=1, descending=True, stable=True)[:, :k])
        if case["renormalize"]:
            w = w / w.sum(1)[:, None]
        w = _SCALE * w
        if s["mask"] is not None:
            w = torch.where(s["mask"][:, None], w, 0.0)
        return dict(idx=None, weights=w)
    S, idx = case["sequences"], s["idx"]
    cuts = [0, T] if s["seq_off"] is None else s["seq_off"].tolist()
    parts = [slice(a, b) for a, b in zip(cuts, cuts[1:])]
    routed = idx[:, 0] >= 0
    if case["op"] == "balance":
        terms, sizes = [], []
        for p in parts:
            live = routed[p]
            sizes.append(int(live.sum()))
            f = torch.bincount(idx[p][live].flatten(), minlength=E).double()
            terms.append((f * share[p][live].sum(0)).sum())
        used = max(1, sum(n > 0 for n in sizes))
        coef = torch.tensor([E / (k * n * n * used) if n else 0.0 for n in sizes], dtype=torch.float64, device="cuda")
        return dict(loss=(coef * torch.stack(terms)).sum(), counts=None, coef=coef)
    # the gradient, from automatic differentiation in 64 bits
    l.requires_grad_(True)
    score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    share = score / score.sum(1, keepdim=True)
    w = score.gather(1, idx.clamp(min=0))
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    loss = (_SCALE * w * s["grad_w"].double())[routed].sum()
    if case["loss"]:
        for i, p in enumerate(parts):
            f = s["counts"][i].double() * s["coef"][i].double() * s["grad_loss"].double()
            loss = loss + (share[p][routed[p]] * f).sum()
    return torch.autograd.grad(loss, l)[0]
