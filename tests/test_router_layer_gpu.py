"""The router and the 4-bit products where a model has them. Training: norm, router with its
balance loss, dispatch, BF16 experts, combine, and the whole backward through both uses of the
router's weights; the same with experts on 4-bit operands. Serving: a captured decode step
from the router on, every operand of the experts in MXFP4. Stages are held to their own
formulas in 64 bits on the inputs they really had, the BF16 layer also as a whole."""
import numpy as np
import pytest
import torch

import mxfp4_reference as mx
from test_expert_layer_gpu import bf, gate
from test_expert_products_gpu import decode_mxfp4, ranges
from test_router_gpu import check_backward, check_balance, check_route

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_ep_layout_10_amd import ops


def seeded(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def layer64(x, w, wr, w1, w2, idx, r, off):
    """(output, balance loss) in 64 bits, for experts chosen already: norm, router, experts,
    weighted sum. Padding (indices of -1) enters neither."""
    y = x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt() * w
    l = y @ wr.t()
    s = torch.sigmoid(l) if r.score == ops.SCORE_SIGMOID else torch.softmax(l, 1)
    part = s.gather(1, idx.clamp(min=0))
    tw = r.scale * part / part.sum(1, keepdim=True) * (idx >= 0)
    p, loss, parts = s / s.sum(1, keepdim=True), 0.0, list(zip(off, off[1:]))
    for a, b in parts:
        live = idx[a:b, 0] >= 0
        counts = torch.bincount(idx[a:b][live].flatten(), minlength=r.num_experts)
        n = int(live.sum())
        loss = loss + r.num_experts / (r.num_topk * n * n * len(parts)) * (counts * p[a:b][live].sum(0)).sum()
    out = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        for j in range(idx.shape[1]):
            t = (idx[:, j] == e).nonzero()[:, 0]
            if t.numel():
                a, b = (y[t] @ w1[e].t()).chunk(2, 1)
                out = out.index_add(0, t, tw[t, j:j + 1] * ((torch.nn.functional.silu(a) * b) @ w2[e].t()))
    return x + out, loss


def check_router_stages(r, logits, idx, tw, bias, mask, off, loss, counts, coef, g_tw, g_loss, g_logits):
    """Choice, weights, loss and gradient, on the logits that the layer had: the calls once more,
    held to their formulas and bounds, and the layer's to theirs bit for bit."""
    for got, again in zip((idx, tw, loss, counts, coef, g_logits),
                          (*check_route(r, logits, bias, mask), *check_balance(r, logits, idx, off),
                           check_backward(r, logits, idx, g_tw, counts, coef, g_loss, off))):
        assert torch.equal(got, again)


@pytest.mark.parametrize("score,T", [("softmax", 70), ("sigmoid", 300)])
def test_training_step(score, T):
    """Seven bf16 roundings (2^-8 each, at most) stand between x and the output and as many
    again to a gradient, each of a random sign over hundreds of terms: relative errors in the
    2-norm stay below their plain sum, 14 * 2^-8; one more for the gradient of y, which is the
    rounded sum of two. The router's weight sees the gradient of the weights less its mean
    over a token's experts (they add up to one): what that takes from the value it may leave
    in the error, for two experts with gradients of a random sign half of the square, so 2^0.5
    times the bound; 2 times is allowed."""
    H, I, E, k, alpha = 256, 192, 8, 2, 0.5
    gen = seeded(T)
    x, w = bf(gen, T, H), (1 + 0.1 * torch.randn(H, device="cuda", generator=gen)).to(torch.bfloat16)
    wr = torch.randn((E, H), device="cuda", generator=gen) * H ** -0.5
    bias = 0.1 * torch.randn(E, device="cuda", generator=gen)
    w1, w2 = bf(gen, E, 2 * I, H, scale=H ** -0.5), bf(gen, E, H, I, scale=I ** -0.5)
    mask = torch.rand(T, device="cuda", generator=gen) < 0.9
    off = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    grad, g_loss = bf(gen, T, H), torch.tensor(alpha, device="cuda")
    r = ops.Router(E, k, ops.SCORE_SIGMOID if score == "sigmoid" else ops.SCORE_SOFTMAX, num_groups=4, topk_groups=3,
                   renormalize=True, scale=2.0)
    cfg = ops.Config(max_tokens=T, hidden=H, num_experts=E, num_topk=k, expert_alignment=16)

    y, _, total, rstd = ops.rms_norm(x, w)
    logits = (y.float() @ wr.t()).contiguous()
    idx, tw = ops.route(r, logits, bias, mask)
    loss, counts, coef = ops.balance_loss(r, logits, idx, off)
    h, recv = ops.dispatch_forward(cfg, idx, y, topk_w=tw)
    up = ops.grouped_gemm_bf16(h, recv, w1).requires_grad_()
    act = gate(up)
    down = ops.grouped_gemm_bf16(h, act.detach(), w2)
    out = total + ops.combine(h, down, tw)

    g_down = ops.combine_backward(h, grad, topk_w=tw)
    g_tw = ops.combine_weight_grad(h, grad, down)
    g_act = ops.grouped_gemm_bf16_grad_input(h, g_down, w2)
    g_w2 = ops.grouped_gemm_bf16_grad_weight(h, g_down, act.detach())
    rows = int(h.read_counts()[2])
    act.backward(torch.cat([g_act[:rows], torch.zeros_like(g_act[rows:])]))
    g_up = up.grad.contiguous()
    g_recv = ops.grouped_gemm_bf16_grad_input(h, g_up, w1)
    g_w1 = ops.grouped_gemm_bf16_grad_weight(h, g_up, recv)
    g_logits = ops.route_backward(r, logits, idx, g_tw, counts, coef, g_loss, off)
    g_y = (ops.dispatch_backward(h, g_recv).float() + g_logits @ wr).to(torch.bfloat16)
    g_wr = g_logits.t() @ y.float()
    g_x, g_w = ops.rms_norm_backward(total, w, rstd, g_y, grad_total=grad)

    assert bool((idx[~mask] == -1).all()) and not bool(tw[~mask].any()) and not bool(g_logits[~mask].any())
    check_router_stages(r, logits, idx, tw, bias, mask, off, loss, counts, coef, g_tw, g_loss, g_logits)

    leaves = [t.double().requires_grad_() for t in (x, w, wr, w1, w2)]
    X, W, WR, W1, W2 = leaves
    want, want_loss = layer64(X, W, WR, W1, W2, idx, r, off.tolist())
    ((want * grad.double()).sum() + alpha * want_loss).backward()
    far = lambda got, ref: float((got.double() - ref).norm() / ref.norm())
    step = 2.0 ** -8
    assert far(out, want.detach()) < 14 * step
    assert abs(float(loss) - want_loss.item()) < 14 * step * want_loss.item()
    for name, got, leaf, steps in (("x", g_x, X, 15), ("weight", g_w, W, 15), ("router", g_wr, WR, 28), ("w1", g_w1, W1, 14),
                                   ("w2", g_w2, W2, 14)):
        assert far(got, leaf.grad) < steps * step, name


def product_close(h, got, a, s, b, t):
    """Rows of a product with both operands in MXFP4 (test_mxfp4_gpu.py has the bound)."""
    n = 0
    for e, (first, live, _) in enumerate(ranges(h)):
        rows = slice(first, first + live)
        if live:
            x, w = decode_mxfp4(a[rows], s[rows]), decode_mxfp4(b[e], t[e])
            want, acc = x @ w.t(), (129 * -(-x.shape[1] // 128) + 8) * 2.0 ** -23 * (x.abs() @ w.abs().t())
            assert bool(((got[rows].double() - want).abs() <= acc + 2.0 ** -8 * (want.abs() + acc)).all()), e
            n += live
    return n


def quantised_close(h, x, codes, scales):
    for first, live, _ in ranges(h):
        rows = slice(first, first + live)
        if live == 0:
            continue
        want = mx.quantize(x[rows].double().cpu().numpy())
        assert np.array_equal(codes[rows].cpu().numpy(), want[0]) and np.array_equal(scales[rows].cpu().numpy(), want[1])


@pytest.mark.parametrize("T", [1, 200])
def test_training_step_on_4_bit_operands(T):
    """Rows and weights quantised in the step; the products' backward takes the values that
    the codes stand for, as bf16, in the BF16 products. A gradient sums n (or rows) products in
    binary32, half a step and a last cut for each, and is rounded to bf16 once."""
    H, I, E, k = 256, 192, 6, 2
    gen = seeded(T)
    y, w1, w2 = bf(gen, T, H), bf(gen, E, 2 * I, H, scale=H ** -0.5), bf(gen, E, H, I, scale=I ** -0.5)
    r = ops.Router(E, k, renormalize=True)
    idx, tw = ops.route(r, torch.randn((T, E), device="cuda", generator=gen))
    cfg = ops.Config(max_tokens=T, hidden=H, num_experts=E, num_topk=k)
    h, recv = ops.dispatch_forward(cfg, idx, y, topk_w=tw)

    def quantised(x, hh=None):
        v = torch.zeros(x.shape, dtype=torch.bfloat16, device="cuda")
        c, s = ops.quantize_mxfp4(x, hh, values=v)
        if hh is not None:
            quantised_close(hh, x, c, s)
        return c, s, v

    (b1, t1, v1), (b2, t2, v2) = quantised(w1), quantised(w2)
    for v, b, t in ((v1, b1, t1), (v2, b2, t2)):
        assert torch.equal(v.double(), decode_mxfp4(b, t))
    a1, s1, x1 = quantised(recv, h)
    up = ops.grouped_gemm_mxfp4_rows(h, a1, s1, b1, t1)
    assert product_close(h, up, a1, s1, b1, t1) == T * k
    a2, s2, x2 = quantised(gate(up), h)
    down = ops.grouped_gemm_mxfp4_rows(h, a2, s2, b2, t2)
    assert product_close(h, down, a2, s2, b2, t2) == T * k
    assert bool(torch.isfinite(ops.combine(h, down, tw)).all())

    grad = bf(gen, T, H)
    g_down = ops.combine_backward(h, grad, topk_w=tw)
    g_act = ops.grouped_gemm_bf16_grad_input(h, g_down, v2)
    g_w2 = ops.grouped_gemm_bf16_grad_weight(h, g_down, x2)
    for e, (first, live, _) in enumerate(ranges(h)):
        rows = slice(first, first + live)
        g, x, w = g_down[rows].double(), x2[rows].double(), v2[e].double()
        for got, want, size, terms in ((g_act[rows], g @ w, g.abs() @ w.abs(), H), (g_w2[e], g.t() @ x, g.abs().t() @ x.abs(), live)):
            acc = (terms + 8) * 2.0 ** -23 * size
            assert bool(((got.double() - want).abs() <= acc + 2.0 ** -8 * (want.abs() + acc)).all()), e


def test_serving_step_captured():
    """A decode step from the router on, FIXED layout, padded batch, in one graph: replayed on
    new logits, tokens and masks with eager work between, and equal to the eager calls bit for
    bit; each stage of the eager calls against its formula."""
    T, H, I, E, k, C = 6, 256, 128, 16, 2, 8
    gen = seeded(3)
    r = ops.Router(E, k, ops.SCORE_SIGMOID, num_groups=4, topk_groups=2, group_best=2, renormalize=True, scale=2.5)
    cfg = ops.Config(max_tokens=T, hidden=H, num_experts=E, num_topk=k, capacity=C, mode=ops.MODE_FIXED)
    (b1, t1), (b2, t2) = (ops.quantize_mxfp4(bf(gen, *s, scale=s[2] ** -0.5)) for s in ((E, 2 * I, H), (E, H, I)))
    x, logits = bf(gen, T, H), torch.randn((T, E), device="cuda", generator=gen)
    bias, mask = 0.1 * torch.randn(E, device="cuda", generator=gen), torch.ones(T, dtype=torch.bool, device="cuda")
    ws, R = ops.new_workspace(cfg), E * C
    recv = torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    up = torch.zeros((R, 2 * I), dtype=torch.bfloat16, device="cuda")
    down = torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    a1, s1, a2, s2 = (torch.zeros((R, n), dtype=torch.uint8, device="cuda") for n in (H // 2, H // 32, I // 2, I // 32))

    def step(stages=False):
        idx, tw = ops.route(r, logits, bias, mask)
        h, _ = ops.dispatch_forward(cfg, idx, x, workspace=ws, recv=recv)
        ops.quantize_mxfp4(recv, h, a1, s1)
        ops.grouped_gemm_mxfp4_rows(h, a1, s1, b1, t1, out=up)
        act = gate(up)
        ops.quantize_mxfp4(act, h, a2, s2)
        ops.grouped_gemm_mxfp4_rows(h, a2, s2, b2, t2, out=down)
        out = ops.combine(h, down, tw)
        if stages:
            for got, again in zip((idx, tw), check_route(r, logits, bias, mask)):
                assert torch.equal(got, again)
            quantised_close(h, recv, a1, s1)
            quantised_close(h, act, a2, s2)
            pairs = int(mask.sum()) * k
            assert product_close(h, up, a1, s1, b1, t1) == pairs and product_close(h, down, a2, s2, b2, t2) == pairs
        return out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(4):
        x.copy_(bf(gen, T, H))
        logits.copy_(torch.randn((T, E), device="cuda", generator=gen))
        mask.copy_(torch.arange(T, device="cuda") < (T, 3, 1, 5)[rep])
        graph.replay()
        torch.cuda.synchronize()
        kept = out.clone()
        assert torch.equal(step(stages=True), kept), rep
        assert bool(torch.isfinite(kept).all()) and float(kept[mask].float().abs().max()) > 0
        assert not bool(kept[~mask].any())
