"""RMS norm with the residual's addition (BF16 and FP8 outputs) and its
backward against the formulas in 64 bits.

Tolerances, u = 2^-24 the binary32 half step: a sum of H squares in any order
is within H u relative of the exact one (all terms positive), so rstd (root,
division, addition: 4 more roundings) is within r = (H / 2 + 8) u; a bf16
output adds 2^-8 of its value. The FP8 code is E4M3(u / q) with u exact, q one
rounding and u / q one more: 2^-4 of the quotient, or half the smallest
subnormal step 2^-10, plus 3 u; scales are q rstd, within r + 2 u."""
import numpy as np
import pytest
import torch

from ep_workloads import random_routing_table
from gpu_common import log, to_dev

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_ep_layout_10_amd import ops

U = 2.0 ** -24
SIZES = [(1, 8), (3, 64), (1, 128), (5, 136), (130, 256), (2, 504), (7, 512), (33, 1024), (4, 1416), (600, 768),
         (1030, 128), (9, 7168), (3, 8192), (2, 8200), (2, 16384), (2, 20480), (1, 32768)]


def data(T, H, residual, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + T + H)
    n = lambda *s: torch.randn(s, device="cuda", generator=gen)
    x, w = n(T, H).to(torch.bfloat16), (1 + 0.2 * n(H)).to(torch.bfloat16)
    r = (3 * n(T, H)).to(torch.bfloat16) if residual else None
    return x, w, r


def total_of(x, r):
    return x if r is None else (x.double() + r.double()).to(torch.bfloat16)


def quantise(u):
    """The definition of the FP8 form on the host, whose binary32 divisions are
    correctly rounded (a GPU division by a number multiplies by its reciprocal):
    codes and q of u [T, blocks, 128]."""
    uf = u.float().cpu().numpy()
    q = np.abs(uf).max(2, keepdims=True) / np.float32(448)
    with np.errstate(divide="ignore", invalid="ignore"):
        v = np.where(q > 0, uf / q, np.float32(0)).clip(-448, 448)
    code = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8)
    return code.flatten(1).cuda(), torch.from_numpy(q[:, :, 0]).cuda()


def rtol(H):
    return (H / 2 + 8) * U


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_bf16(T, H, residual):
    log("norm bf16 T=%d H=%d residual=%d" % (T, H, residual))
    x, w, r = data(T, H, residual)
    y, scales, total, rstd = ops.rms_norm(x, w, 1e-5, residual=r)
    assert scales is None
    # bf16 + bf16 rounds once to bf16 through binary32 when the sum fits 24 bits; otherwise the binary32 sum is
    # itself rounded first, which moves a bf16 result only where the exact sum is within 2^-24 of a tie
    want_total = total_of(x, r)
    if residual:
        exact = x.double() + r.double()
        assert bool(((total.double() - exact).abs() <= exact.abs() * (2.0 ** -8 + U)).all())
        assert float((total != want_total).float().mean()) < 1e-3
    else:
        assert total is x
    s = total.double()
    want = 1.0 / (s.square().mean(1) + float(np.float32(1e-5))).sqrt()
    assert bool(((rstd.double() - want).abs() <= rtol(H) * want).all())
    want_y = s * want[:, None] * w.double()
    assert bool(((y.double() - want_y).abs() <= (2.0 ** -8 + rtol(H) + 2 * U) * (1 + 2.0 ** -8) * want_y.abs()).all())


@pytest.mark.parametrize("T,H", [s for s in SIZES if s[1] % 128 == 0])
@pytest.mark.parametrize("residual", [False, True])
def test_fp8(T, H, residual):
    log("norm fp8 T=%d H=%d residual=%d" % (T, H, residual))
    x, w, r = data(T, H, residual)
    x[0, :128] = 0
    if r is not None:
        r[0, :128] = 0                              # a block of zeros: scale 0, codes 0
    y, scales, total, rstd = ops.rms_norm(x, w, 1e-5, residual=r, dtype=ops.FP8_QUANTIZE)
    s = total.double()
    want = 1.0 / (s.square().mean(1) + float(np.float32(1e-5))).sqrt()
    assert bool(((rstd.double() - want).abs() <= rtol(H) * want).all())
    u = (s * w.double()).view(T, H // 128, 128)
    q = u.abs().amax(2) / 448.0
    assert bool(((scales.double() - q * want[:, None]).abs() <= (rtol(H) + 2 * U) * q * want[:, None]).all())
    assert bool((scales[0, 0] == 0)) and bool((y[0, :128] == 0).all())
    code = y.view(torch.float8_e4m3fn).double().view(u.shape)
    ratio = torch.where(q[:, :, None] > 0, u / q.clamp(min=1e-300)[:, :, None], torch.zeros_like(u))
    lim = torch.maximum(ratio.abs() * 2.0 ** -4, torch.full_like(ratio, 2.0 ** -10)) + 4 * U * ratio.abs()
    assert bool(((code - ratio).abs() <= lim).all())
    # the definition, with binary32 quotients: the same codes and scales bit for bit
    ref, qf = quantise(u)
    assert torch.equal(ref, y)
    assert torch.equal(scales, qf * rstd[:, None])


def test_fp8_extreme_blocks():
    """Outliers, the largest finite values, subnormal values, negative zeros."""
    x, w, _ = data(4, 512, False)
    x[0, 7] = 3.0e38
    x[1] = 1e-39
    x[1, 0] = 1e-40
    x[2, ::2] = -0.0
    x[3, 128:256] = 2.0 ** -126
    y, scales, _, rstd = ops.rms_norm(x, w, 1e-6, dtype=ops.FP8_QUANTIZE)
    ref, q = quantise((x.double() * w.double()).view(4, 4, 128))
    assert torch.equal(ref, y)
    assert torch.equal(scales, q * rstd[:, None])
    assert float(rstd[0]) == 0.0                    # its square overflows binary32, as the formula in binary32 does


@pytest.mark.parametrize("fp8", [False, True])
def test_total_in_place(fp8):
    """total may be residual's or x's own buffer."""
    x, w, r = data(40, 1024, True)
    dt = ops.FP8_QUANTIZE if fp8 else ops.BF16
    want = ops.rms_norm(x, w, residual=r, dtype=dt)
    for which in (0, 1):
        x2, r2 = x.clone(), r.clone()
        into = (x2, r2)[which]
        got = ops.rms_norm(x2, w, residual=r2, dtype=dt, total=into)
        assert got[2] is into
        for p, q in zip(got, want):
            assert (p is None and q is None) or torch.equal(p, q)


def formula(s, w, g, gt, eps):
    """Gradients of sum(y g) + sum(s gt) in 64 bits, y = s rstd w."""
    rstd = 1.0 / (s.square().mean(1, keepdim=True) + eps).sqrt()
    gw = g * w
    gx = rstd * (gw - s * rstd.square() * (gw * s).mean(1, keepdim=True))
    return gx if gt is None else gx + gt, (g * s * rstd).sum(0)


@pytest.mark.parametrize("T,H", SIZES + [(2000, 264)])
@pytest.mark.parametrize("branch", [False, True])
def test_backward(T, H, branch):
    """grad_x: the mean of H products is within (H + 4) u of the terms' sum of
    magnitudes, s rstd and the two outer products add 6 u of theirs, the output
    2^-8. grad_weight: T terms in any order, (T + 4) u of their magnitudes.
    (rstd is an input of the backward: taken as given.)"""
    log("norm backward T=%d H=%d branch=%d" % (T, H, branch))
    s, w, gt = data(T, H, branch)
    g = data(T, H, False, seed=99)[0]
    rstd = (1.0 / (s.double().square().mean(1) + 1e-5).sqrt()).float()
    gx, gw = ops.rms_norm_backward(s, w, rstd, g, grad_total=gt)
    S, W, G, R = s.double(), w.double(), g.double(), rstd.double()[:, None]
    inner = (G * W * S * R).mean(1, keepdim=True)
    first, second = R * G * W, R * R * S * inner
    want = first - second + (0 if gt is None else gt.double())
    mag = (G * W * S * R).abs().mean(1, keepdim=True)
    err = (H + 4) * U * (R * R * S).abs() * mag + 6 * U * (first.abs() + second.abs()) + 2 * U * want.abs()
    lim = err + 2.0 ** -8 * (want.abs() + err)
    assert bool(((gx.double() - want).abs() <= lim).all())
    terms = G * S * R
    assert bool(((gw.double() - terms.sum(0)).abs() <= (T + 4) * U * terms.abs().sum(0)).all())


def test_formula_is_the_gradient():
    """The formula the kernel is held to, against central differences in 64 bits."""
    gen = torch.Generator().manual_seed(4)
    s, g, gt = (torch.randn(3, 40, dtype=torch.float64, generator=gen) for _ in range(3))
    w = 1 + 0.2 * torch.randn(40, dtype=torch.float64, generator=gen)
    eps, h = 1e-5, 1e-6
    loss = lambda s, w: float(((s / (s.square().mean(1, keepdim=True) + eps).sqrt() * w) * g).sum() + (s * gt).sum())
    gx, gw = formula(s, w, g, gt, eps)
    for i in range(40):
        d = torch.zeros(40, dtype=torch.float64)
        d[i] = h
        assert abs((loss(s, w + d) - loss(s, w - d)) / (2 * h) - float(gw[i])) < 1e-6
        dx = torch.zeros(3, 40, dtype=torch.float64)
        dx[i % 3, i] = h
        assert abs((loss(s + dx, w) - loss(s - dx, w)) / (2 * h) - float(gx[i % 3, i])) < 1e-6


def test_backward_in_place_and_workspace():
    s, w, gt = data(700, 512, True)
    g = data(700, 512, False, seed=5)[0]
    rstd = (1.0 / (s.double().square().mean(1) + 1e-5).sqrt()).float()
    want = ops.rms_norm_backward(s, w, rstd, g, grad_total=gt)
    ws = ops.rms_norm_workspace(700, 512)
    ws.fill_(0xFF)                                  # NaN partial sums left by another use
    into = gt.clone()
    gx, gw = ops.rms_norm_backward(s, w, rstd, g, grad_total=into, grad_x=into, workspace=ws)
    assert gx is into and torch.equal(gx, want[0]) and torch.equal(gw, want[1])


def test_empty_batch():
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    y, scales, total, rstd = ops.rms_norm(x, w, dtype=ops.FP8_QUANTIZE)
    assert y.shape == (0, 256) and scales.shape == (0, 2) and rstd.shape == (0,)
    gx, gw = ops.rms_norm_backward(x, w, rstd, x, grad_weight=torch.full((256,), 7.0, device="cuda"))
    assert gx.shape == (0, 256) and bool((gw == 0).all())


def test_bits_do_not_depend_on_the_batch():
    """A row's results are the same alone and inside a batch, and under another launch size."""
    import os
    x, w, r = data(300, 1024, True)
    full = ops.rms_norm(x, w, residual=r, dtype=ops.FP8_QUANTIZE)
    one = ops.rms_norm(x[37:38].contiguous(), w, residual=r[37:38].contiguous(), dtype=ops.FP8_QUANTIZE)
    for f, o in zip(full, one):
        assert torch.equal(f[37:38], o)
    g = data(300, 1024, False, seed=6)[0]
    a = ops.rms_norm_backward(full[2], w, full[3], g)
    try:
        os.environ["EP_LAUNCH_CUS"] = "3"
        b = ops.rms_norm_backward(full[2], w, full[3], g)
        again = ops.rms_norm(x, w, residual=r, dtype=ops.FP8_QUANTIZE)
    finally:
        os.environ.pop("EP_LAUNCH_CUS", None)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for f, o in zip(full, again):
        assert torch.equal(f, o)


def test_graph_replay_forward_and_backward():
    x, w, r = data(200, 1024, True)
    g = data(200, 1024, False, seed=7)[0]
    ws = ops.rms_norm_workspace(200, 1024)

    def step():
        y, sc, total, rstd = ops.rms_norm(x, w, residual=r, dtype=ops.FP8_QUANTIZE)
        return (y, sc, total, rstd) + ops.rms_norm_backward(total, w, rstd, g, grad_total=r, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for rep in range(3):
        x2, w2, r2 = data(200, 1024, True, seed=20 + rep)
        x.copy_(x2), w.copy_(w2), r.copy_(r2)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        ws.fill_(0xFF)
        for p, q in zip(kept, step()):
            assert torch.equal(p, q), rep


def test_fp8_rows_are_the_dispatch_input():
    """The norm's codes and scales through a pre-quantised dispatch: copied bitwise to the receive rows."""
    T, H, E = 96, 512, 8
    x, w, r = data(T, H, True)
    idx = random_routing_table(np.random.default_rng(21), T, E, 2)
    y, scales, _, _ = ops.rms_norm(x, w, residual=r, dtype=ops.FP8_QUANTIZE)
    cfg = ops.Config(max_tokens=T, hidden=H, num_experts=E, num_topk=2, expert_alignment=16)
    h, recv, rs = ops.dispatch_forward(cfg, to_dev(idx), y, ops.FP8_PREQUANT, x_scales=scales)
    slot = h.slot.view(T, 2).long()
    for j in range(2):
        assert torch.equal(recv[slot[:, j]], y)
        assert torch.equal(rs[slot[:, j]], scales)


def test_refusals():
    x, w, r = data(8, 256, True)
    y = torch.full((8, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    for bad in (x.float(), x[:, :248], x.cpu(), x.view(-1)):
        with pytest.raises(ValueError):
            ops.rms_norm(bad, w, y=y)
    with pytest.raises(ValueError):
        ops.rms_norm(x, w[:128], y=y)
    with pytest.raises(ValueError):
        ops.rms_norm(x, w, y=y, total=torch.empty_like(x))        # total without a residual
    with pytest.raises(ValueError):
        ops.rms_norm(x, w, residual=r[:4], y=y)
    with pytest.raises(ValueError):
        ops.rms_norm(x, w, y=y.float())
    with pytest.raises(ops.F.EPError, match="eps"):
        ops.rms_norm(x, w, 0.0, y=y)
    with pytest.raises(ops.F.EPError, match="eps"):
        ops.rms_norm(x, w, float("nan"), y=y)
    with pytest.raises(ops.F.EPError, match="dtype"):
        ops.rms_norm(x, w, y=y, dtype=ops.FP8_PREQUANT)
    x2 = torch.zeros((2, 200), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ops.F.EPError, match="128"):
        ops.rms_norm(x2, torch.zeros(200, dtype=torch.bfloat16, device="cuda"), dtype=ops.FP8_QUANTIZE)
    x3 = torch.zeros((1, 32776), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ops.F.EPError, match="exceeds"):
        ops.rms_norm(x3, x3[0])
    rstd = torch.ones(8, device="cuda")
    with pytest.raises(ops.F.EPError, match="workspace"):
        ops.rms_norm_backward(x, w, rstd, x, grad_x=y, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ops.rms_norm_backward(x, w, rstd[:4], x, grad_x=y)
    with pytest.raises(ValueError):
        ops.rms_norm_backward(x, w, rstd, x.float(), grad_x=y)
    torch.cuda.synchronize()
    assert bool((y == 7).all())
