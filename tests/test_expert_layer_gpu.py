"""The operators together, as a model's expert layer uses them: norm, dispatch,
two products with a gate between them, combine; then the whole backward; and
the serving form on 4-bit weights. Each stage is held to its own formula in 64
bits on the inputs it really had, and the whole to the layer's formula in 64 bits."""
import numpy as np
import pytest
import torch

from ep_workloads import random_routing_table
from gpu_common import to_dev

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_ep_layout_10_amd import ops


def bf(gen, *shape, scale=1.0):
    return (scale * torch.randn(shape, device="cuda", generator=gen)).to(torch.bfloat16)


def gate(x):
    """silu(first half) * second half, the elementwise part a model brings."""
    a, b = x.float().chunk(2, 1)
    return (torch.nn.functional.silu(a) * b).to(torch.bfloat16)


def layer64(x, r, w, idx, tw, w1, w2, eps=1e-6):
    """The layer in 64 bits: norm(x + r), top-k experts, weighted sum, plus the stream."""
    s = x + r
    y = s / (s.square().mean(1, keepdim=True) + eps).sqrt() * w
    out = torch.zeros_like(s)
    for e in range(w1.shape[0]):
        for j in range(idx.shape[1]):
            t = (idx[:, j] == e).nonzero()[:, 0]
            if t.numel():
                a, b = (y[t] @ w1[e].t()).chunk(2, 1)
                out = out.index_add(0, t, tw[t, j:j + 1] * ((torch.nn.functional.silu(a) * b) @ w2[e].t()))
    return s + out


@pytest.mark.parametrize("A,T", [(1, 70), (16, 1), (128, 300)])
def test_training_step(A, T):
    """Forward and backward of the layer. bf16 keeps 2^-8 a rounding; seven
    roundings stand between x and the layer's output and as many again to a
    gradient, each of a random sign over hundreds of terms: the relative error
    in the 2-norm stays below their plain sum, 14 * 2^-8 = 5.5 %."""
    H, I, E, k = 256, 192, 6, 2
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    x, r, w = bf(gen, T, H), bf(gen, T, H), (1 + 0.1 * torch.randn(H, device="cuda", generator=gen)).to(torch.bfloat16)
    w1, w2 = bf(gen, E, 2 * I, H, scale=H ** -0.5), bf(gen, E, H, I, scale=I ** -0.5)
    idx = to_dev(random_routing_table(np.random.default_rng(T), T, E, k))
    tw = torch.softmax(torch.randn((T, k), device="cuda", generator=gen), 1)
    grad = bf(gen, T, H)

    cfg = ops.Config(max_tokens=T, hidden=H, num_experts=E, num_topk=k, expert_alignment=A)
    y, _, total, rstd = ops.rms_norm(x, w, residual=r)
    h, recv = ops.dispatch_forward(cfg, idx, y, topk_w=tw)
    up = ops.grouped_gemm_bf16(h, recv, w1)
    up_req = up.detach().requires_grad_()
    act = gate(up_req)
    down = ops.grouped_gemm_bf16(h, act.detach(), w2)
    out = total + ops.combine(h, down, tw)

    g_down = ops.combine_backward(h, grad, topk_w=tw)
    g_tw = ops.combine_weight_grad(h, grad, down)
    g_act = ops.grouped_gemm_bf16_grad_input(h, g_down, w2)
    g_w2 = ops.grouped_gemm_bf16_grad_weight(h, g_down, act.detach())
    rows = int(h.read_counts()[2])
    act.backward(torch.cat([g_act[:rows], torch.zeros_like(g_act[rows:])]))
    g_up = up_req.grad.contiguous()
    g_recv = ops.grouped_gemm_bf16_grad_input(h, g_up, w1)
    g_w1 = ops.grouped_gemm_bf16_grad_weight(h, g_up, recv)
    g_y = ops.dispatch_backward(h, g_recv)
    g_x, g_w = ops.rms_norm_backward(total, w, rstd, g_y, grad_total=grad)

    leaves = [t.double().requires_grad_() for t in (x, r, w, tw, w1, w2)]
    X, R, W, TW, W1, W2 = leaves
    want = layer64(X, R, W, idx, TW, W1, W2)
    want.backward(grad.double())
    far = lambda got, ref: float((got.double() - ref).norm() / ref.norm())
    assert far(out, want.detach()) < 14 * 2.0 ** -8
    for name, got, leaf in (("x", g_x, X), ("residual", g_x, R), ("weight", g_w, W), ("topk_w", g_tw, TW),
                            ("w1", g_w1, W1), ("w2", g_w2, W2)):
        assert far(got, leaf.grad) < 14 * 2.0 ** -8, name


def test_serving_step_captured():
    """A decode step on 4-bit weights: FIXED layout, one graph, replayed on new
    tokens with eager work between; equal to the eager calls bit for bit."""
    T, H, I, E, k, C = 5, 256, 128, 8, 2, 8
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    cfg = ops.Config(max_tokens=T, hidden=H, num_experts=E, num_topk=k, capacity=C, mode=ops.MODE_FIXED)
    codes = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=gen)
    b1, b2 = codes(E, 2 * I, H // 2), codes(E, H, I // 2)
    s1, s2 = (torch.randint(118, 122, s, dtype=torch.uint8, device="cuda", generator=gen)
              for s in ((E, 2 * I, H // 32), (E, H, I // 32)))
    x, w = bf(gen, T, H), torch.ones(H, dtype=torch.bfloat16, device="cuda")
    idx = to_dev(random_routing_table(np.random.default_rng(0), T, E, k))
    tw = torch.full((T, k), 0.5, device="cuda")
    ws = ops.new_workspace(cfg)
    recv = torch.zeros((E * C, H), dtype=torch.bfloat16, device="cuda")
    up = torch.zeros((E * C, 2 * I), dtype=torch.bfloat16, device="cuda")
    down = torch.zeros((E * C, H), dtype=torch.bfloat16, device="cuda")

    def step():
        y = ops.rms_norm(x, w)[0]
        h, _ = ops.dispatch_forward(cfg, idx, y, workspace=ws, recv=recv)
        ops.grouped_gemm_mxfp4(h, recv, b1, s1, out=up)
        ops.grouped_gemm_mxfp4(h, gate(up), b2, s2, out=down)
        return ops.combine(h, down, tw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(3):
        x.copy_(bf(gen, T, H))
        idx.copy_(to_dev(random_routing_table(np.random.default_rng(rep + 1), T, E, k)))
        graph.replay()
        torch.cuda.synchronize()
        kept = out.clone()
        assert torch.equal(step(), kept), rep
        assert bool(torch.isfinite(kept).all()) and float(kept.float().abs().max()) > 0
