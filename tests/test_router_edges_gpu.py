"""The router on the GPU where its formulas are hardest to keep: the lowest finite
logits beside NaN, sigmoids that underflow, scores that are equal where their logits are not,
logits past 2^31, the largest sizes. References and bounds are test_router_gpu.py's."""
import numpy as np
import pytest
import torch

import router_reference as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_ep_layout_10_amd import ops
    from test_router_gpu import U, check_route, gen, make_logits, routing


@pytest.mark.parametrize("E,k,G,keep", [(24, 3, 1, 1), (100, 4, 4, 2), (128, 8, 1, 1), (160, 6, 1, 1), (256, 8, 8, 3),
                                        (256, 2, 8, 8), (700, 32, 1, 1), (1024, 8, 16, 2)])
def test_nan_ties_with_the_lowest_logit(E, k, G, keep):
    """A NaN key counts as the lowest finite number, which the logits hold, too: the lower index goes first,
    however many experts there are."""
    lowest, nan = torch.finfo(torch.float32).min, float("nan")
    logits = torch.full((8, E), -torch.inf, device="cuda")
    logits[0, 0], logits[0, 1] = nan, lowest
    logits[1, 0], logits[1, 1] = lowest, nan
    logits[2, ::2], logits[2, 1::2] = nan, lowest
    logits[3, ::2], logits[3, 1::2] = lowest, nan
    logits[4] = nan
    logits[4, -1] = lowest
    logits[5] = lowest
    logits[5, -1] = nan
    logits[6, ::3], logits[6, 1::3], logits[6, E // 2] = lowest, nan, -3.0e38
    logits[7, 1::5], logits[7, 2::5], logits[7, -1] = nan, lowest, 0.5
    for sigmoid in (0, 1):
        for renorm in (False, True):
            check_route(ops.Router(E, k, sigmoid, G, keep, 1, renorm), logits)


# ---------------------------------------------------------------- sigmoids that underflow

def shares(l):
    """Shares of sigmoid scores, with the scores and one minus them, of any finite or infinite logits: from logarithms."""
    up, down = -np.logaddexp(0, -l), -np.logaddexp(0, l)
    top = up.max(1, keepdims=True)
    x = np.exp(up - np.where(np.isfinite(top), top, 0.0))
    total = x.sum(1, keepdims=True)
    return x / np.where(total == 0, 1.0, total), np.exp(up), np.exp(down)


def faint_logits(g, E, f32):
    """Rows whose highest logit lies at many levels below 0, from where 1 + e^l is 1 in binary32 to where e^l is 0,
    some with an ordinary logit or closed experts among them."""
    levels = [-12.0, -16.0, -17.5, -18.5, -21.0, -40.0, -80.0, -87.0, -88.5, -95.0, -104.0, -110.0, -300.0, -2000.0, -3e4]
    l = torch.tensor(levels, device="cuda").repeat_interleave(3)[:, None] + 1.5 * torch.randn((45, E), generator=g, device="cuda")
    l[1::3, E // 2] = -torch.inf
    l[2::9, E // 3] = 0.25
    flat = torch.full((3, E), -1e30, device="cuda")
    flat[1], flat[2, 0] = torch.finfo(torch.float32).min / 2, -torch.inf
    l = torch.cat([l, flat])
    return l if f32 else l.to(torch.bfloat16)


def reach(l):
    """What the exponentials' arguments can be off by, in units of 2^-24: a row's spread, as far as a term counts,
    and the 30 that an ordinary sigmoid's argument has before e^l drops out of 1 + e^l."""
    l = np.where(np.isfinite(l), l, np.nan)
    return min(111.0, np.nanmax(np.nanmax(l, 1) - np.nanmin(l, 1))) + 30.0


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("E,k", [(5, 2), (64, 4), (250, 8), (256, 8), (700, 8), (1024, 3)])
def test_shares_of_sigmoids_that_underflow(E, k, f32):
    """Balance loss and gradient where all of a token's sigmoids are tiny or 0 in binary32: the shares are ratios
    and stay. The weights' part of the gradient has the scores themselves, which are 0 below 2^-126: its bound
    adds what that times its other factor makes."""
    g = gen(E)
    logits = faint_logits(g, E, f32)
    T = logits.shape[0]
    idx = routing(g, T, E, k, dropped=0.1)
    l, ids = logits.double().cpu().numpy(), idx.cpu().numpy()
    p, s, rest = shares(l)
    R, out = reach(l), U if f32 else 2.0 ** -8
    live = (ids >= 0) & (ids < E)
    grad_w = torch.randn((T, k), generator=g, device="cuda")
    gw, grad_loss = grad_w.double().cpu().numpy(), torch.tensor(0.7, device="cuda")
    n, ge, ga = (np.zeros((T, E)) for _ in range(3))
    for t, j in zip(*np.nonzero(live)):
        n[t, ids[t, j]] += 1
        ge[t, ids[t, j]] += gw[t, j]
        ga[t, ids[t, j]] += abs(gw[t, j])
    for cuts in (None, list(range(T + 1)), [0, T // 3, T // 3, T - 1]):
        off = None if cuts is None else torch.tensor(cuts, dtype=torch.int32, device="cuda")
        r = ops.Router(E, k, ops.SCORE_SIGMOID)
        loss, counts, coef = ops.balance_loss(r, logits, idx, off)
        c, f = counts.double().cpu().numpy(), coef.double().cpu().numpy()
        at = np.zeros(T, int) if cuts is None else np.searchsorted(cuts, np.arange(T), side="right") - 1
        inside, at = at < len(f), np.minimum(at, len(f) - 1)
        routed = live.any(1)
        want = float((f[at] * (p * c[at]).sum(1))[inside & routed].sum())
        ref.close(loss.item(), want, (2 * R + 60) * U * want, "loss")
        scale = 0.7 * (f[at] * inside)[:, None]
        c = c[at]
        c = c - c[:, :1]  # a constant of all counts changes nothing, and would hide shares far below 2^-53 here
        b, ba = scale * (c - (p * c).sum(1, keepdims=True)), scale * (abs(c) + (p * abs(c)).sum(1, keepdims=True))
        for weights, renorm in ((None, False), (grad_w, False), (grad_w, True)):
            u, ua = np.zeros((T, E)), np.zeros((T, E))
            if weights is not None:
                u, ua = ge, ga
                if renorm:
                    D = (n * s).sum(1, keepdims=True) + 1e-20
                    u, ua = (ge - n * (ge * s).sum(1, keepdims=True) / D) / D, (ga + n * (ga * s).sum(1, keepdims=True) / D) / D
            r = ops.Router(E, k, ops.SCORE_SIGMOID, renormalize=renorm)
            got = ops.route_backward(r, logits, idx, weights, counts, coef, grad_loss, off)
            want = np.where(routed[:, None], s * rest * u + p * rest * b, 0.0)
            size = s * rest * ua + p * rest * ba
            ref.close(got.double().cpu().numpy(), want,
                      (8 * R + 240) * U * size + out * abs(want) + 1e-37 + 2.0 ** -126 * ua, "gradient %s %s" % (cuts is None, renorm))


def test_equal_faint_sigmoids_have_equal_shares():
    """The same logit for all experts, however low: shares of 1 / E, and a loss of 1 for an even choice."""
    E, T = 64, 32
    idx = torch.arange(2 * T, device="cuda").view(T, 2) % E
    for level in (0.0, -20.0, -87.5, -90.0, -103.0, -104.0, -500.0, -1e30):
        loss, counts, coef = ops.balance_loss(ops.Router(E, 2, 1), torch.full((T, E), level, device="cuda"), idx)
        assert abs(loss.item() - 1.0) <= 60 * U, level


# ---------------------------------------------------------------- scores as keys

@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("E,k,G,keep", [(24, 4, 1, 1), (64, 6, 8, 8), (128, 8, 4, 4), (256, 8, 1, 1), (256, 8, 8, 8), (256, 8, 8, 4),
                                        (700, 9, 1, 1), (1024, 32, 16, 16)])
def test_scores_are_the_keys_where_two_of_a_group_count(E, k, G, keep, f32):
    """With group_best 2 a key is the score in binary64, whether groups are dropped or not: sigmoids of logits from
    40 on are 1 there, and terms 800 below a row's largest logit 0, so those experts tie and the lowest
    index goes first."""
    g = gen(E)
    high = 40.0 + 20.0 * torch.rand((6, E), generator=g, device="cuda")
    some = torch.where(torch.rand((6, E), generator=g, device="cuda") < 0.9, -800.0 - high, -high)
    some[:, 1] = 0.0
    logits = torch.cat([high, some])
    logits = logits if f32 else logits.to(torch.bfloat16)
    check_route(ops.Router(E, k, ops.SCORE_SIGMOID, G, keep, 2), logits[:6])
    check_route(ops.Router(E, k, ops.SCORE_SOFTMAX, G, keep, 2), logits[6:])


@pytest.mark.parametrize("sigmoid", [0, 1])
@pytest.mark.parametrize("E,k,G,keep", [(60, 6, 4, 2), (128, 8, 8, 3), (160, 6, 8, 3), (256, 8, 8, 4), (256, 8, 8, 8), (512, 10, 64, 9),
                                        (384, 8, 8, 3), (1024, 32, 64, 2), (1024, 8, 1, 1)])
def test_two_of_a_group_of_bf16_logits(E, k, G, keep, sigmoid):
    """bf16 logits without a bias, which tie. Two groups' sums of different scores may be equal but for their last
    bit (s(x) + s(-x) is 1), and then either may go first: tokens whose sums at the border lie within 1e-12 without being
    sums of the same logits are left out, all others compared exactly."""
    g, T = gen(E + k), 200
    logits = make_logits(g, T, E, False)
    clear = torch.ones(T, dtype=torch.bool)
    if keep < G:
        top = logits.double().cpu().view(T, G, -1).topk(2, 2).values.numpy()
        for t in range(T):
            s = np.exp(top[t] - logits[t].double().max().item()) if not sigmoid else 1.0 / (1.0 + np.exp(-top[t]))
            total = 1.0 if sigmoid else np.exp(logits[t].double().cpu().numpy() - logits[t].double().max().item()).sum()
            sums = s.sum(1) / total
            order = np.argsort(-sums, kind="stable")
            border = sums[order[keep - 1]]
            for a in order:
                for b in order:
                    if abs(sums[a] - border) < 1e-12 and abs(sums[b] - border) < 1e-12 and not np.array_equal(top[t][a], top[t][b]):
                        clear[t] = False
    assert clear.sum() >= T // 2
    for renorm in (False, True):
        check_route(ops.Router(E, k, sigmoid, G, keep, 2, renorm), logits[clear.cuda()].contiguous())


# ---------------------------------------------------------------- far rows

@pytest.mark.parametrize("E,f32", [(1024, True), (1000, False), (999, True)])
def test_rows_past_2_31_logits(E, f32):
    """Tokens whose logits start past 2^31 elements (8 GB in binary32): all calls give them what they give a batch of those
    tokens alone."""
    k, last = 8, 70
    T = (1 << 31) // E + last + 1
    g = gen(E)
    logits = torch.zeros((T, E), device="cuda", dtype=torch.float32 if f32 else torch.bfloat16)
    logits[-last:] = make_logits(g, last, E, f32)
    some = logits[-last:].clone()
    bias = 0.2 * torch.randn(E, generator=g, device="cuda")
    r = ops.Router(E, k, ops.SCORE_SIGMOID, renormalize=True)
    idx, w = ops.route(r, logits, bias)
    few_idx, few_w = check_route(r, some, bias)
    assert torch.equal(idx[-last:], few_idx) and torch.equal(w[-last:], few_w)
    # the last tokens as two sequences, those before them none
    off = torch.tensor([T - last, T - 30, T], dtype=torch.int32, device="cuda")
    loss, counts, coef = ops.balance_loss(r, logits, idx, off)
    want, want_counts, want_coef, _ = ref.balance(some, few_idx, [0, last - 30, last], r)
    assert np.array_equal(counts.cpu().numpy(), want_counts)
    ref.close(coef.cpu().numpy(), want_coef, 2 * U * want_coef, "coef")
    ref.close(loss.item(), want, (2 * ref.spread(some) + 60) * U * want, "loss")
    # written over the logits
    few = ops.route_backward(r, some, few_idx, few_w, counts, coef, loss, off - (T - last))
    grad = ops.route_backward(r, logits, idx, w, counts, coef, loss, off, grad_logits=logits)
    assert torch.equal(grad[-last:], few) and few.any()


# ---------------------------------------------------------------- the largest sizes

def test_the_most_tokens():
    """2^25 tokens: slices of them as in a call of their own, the loss against torch in 64 bits."""
    T, E, k = 1 << 25, 8, 2
    logits = make_logits(gen(25), T, E, False)
    r = ops.Router(E, k, ops.SCORE_SIGMOID, renormalize=True)
    idx, w = ops.route(r, logits)
    loss, counts, coef = ops.balance_loss(r, logits, idx)
    assert torch.equal(counts[0].long(), torch.bincount(idx.flatten(), minlength=E))
    assert abs(coef.item() - E / (k * float(T) ** 2)) <= 2 * U * coef.item()
    total = torch.zeros(E, dtype=torch.float64, device="cuda")
    for part in logits.split(1 << 22):
        s = torch.sigmoid(part.double())
        total += (s / s.sum(1, keepdim=True)).sum(0)
    want = (E / (k * float(T) ** 2) * (counts[0].double() * total).sum()).item()
    spread = 2.0 * float(logits.abs().max())  # at least the distances within a token
    assert abs(loss.item() - want) <= (2 * (spread + float(logits.abs().max())) + 60) * U * want
    grad = ops.route_backward(r, logits, idx, w, counts, coef, loss)
    for first in (0, T // 2 - 7, T - 300):
        some = logits[first:first + 300].clone()
        few_idx, few_w = check_route(r, some)
        assert torch.equal(idx[first:first + 300], few_idx) and torch.equal(w[first:first + 300], few_w)
        assert torch.equal(grad[first:first + 300], ops.route_backward(r, some, few_idx, few_w, counts, coef, loss))
    with pytest.raises(RuntimeError, match="num_tokens"):
        ops.route(r, torch.empty((T + 1, E), dtype=torch.bfloat16, device="cuda"))


def test_the_most_sequences_and_experts():
    """2^17 sequences, most of them empty, of 1024 experts."""
    T, E, k, S = 5000, 1024, 2, 1 << 17
    g = gen(17)
    logits, idx = make_logits(g, T, E, True), torch.randint(0, E, (T, k), generator=g, device="cuda")
    off = torch.sort(torch.randint(0, T + 1, (S + 1,), generator=g, device="cuda").int())[0]
    r = ops.Router(E, k)
    loss, counts, coef = ops.balance_loss(r, logits, idx, off)
    q = torch.searchsorted(off[1:].long(), torch.arange(T, device="cuda"), right=True)
    inside = (q < S) & (torch.arange(T, device="cuda") >= off[0])
    q = q.clamp(max=S - 1)
    want_counts = torch.zeros((S, E), dtype=torch.int32, device="cuda")
    want_counts.index_put_((q[inside].repeat_interleave(k), idx[inside].flatten()), torch.ones((), dtype=torch.int32, device="cuda"),
                           accumulate=True)
    assert torch.equal(counts, want_counts)
    n = torch.bincount(q[inside], minlength=S).double()
    want_coef = torch.where(n > 0, E / (k * n.clamp(min=1).square() * (n > 0).sum()), 0.0)
    assert ((coef.double() - want_coef).abs() <= 2 * U * want_coef).all()
    p = torch.softmax(logits.double(), 1)
    want = (want_coef[q] * (p * want_counts[q].double()).sum(1))[inside].sum().item()
    assert abs(loss.item() - want) <= (2 * ref.spread(logits) + 60) * U * want
    grad = ops.route_backward(r, logits, idx, None, counts, coef, torch.ones((), device="cuda"), off)
    c = want_counts[q].double() * (want_coef[q] * inside)[:, None]
    want = p * (c - (p * c).sum(1, keepdim=True))
    size = p * (c + (p * c).sum(1, keepdim=True))
    assert ((grad.double() - want).abs() <= (8 * ref.spread(logits) + 240) * U * size + U * want.abs() + 1e-37).all()


# ---------------------------------------------------------------- one expert alone

@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("sigmoid", [0, 1])
@pytest.mark.parametrize("E", [1, 16, 60, 256, 700])
def test_a_renormalised_weight_alone_has_no_gradient(E, sigmoid, f32):
    """Where all of a token's ids name one expert, its renormalised weights are shares of 1 that nothing changes, as long
    as their sum takes up 1e-20 in binary32: gradients are 0 exactly, not what rounding leaves of them."""
    g, T = gen(E), 200
    logits = make_logits(g, T, E, f32)
    one = torch.randint(0, E, (T, 1), generator=g, device="cuda")
    for k in (1, 2, 4):
        if k > E:
            continue
        idx = one.repeat(1, k)
        if k > 1:
            idx[::3, 1:] = -1          # one pair of several
            idx[1::3, :k // 2] = E + 3
        r = ops.Router(E, k, sigmoid, renormalize=True, scale=-1.5)
        grad = ops.route_backward(r, logits, idx, torch.randn((T, k), generator=g, device="cuda"))
        assert not grad.any()


@pytest.mark.parametrize("level", [-38.0, -44.0, -46.0, -48.0, -60.0, -80.0])
def test_a_renormalised_faint_weight_alone(level):
    """The same where 1e-20 counts: s / (s + 1e-20) has the slope 1e-20 / (s + 1e-20)^2 times the sigmoid's."""
    T, E = 100, 40
    g = gen(int(-level))
    logits = level + make_logits(g, T, E, True)
    idx = torch.randint(0, E, (T, 1), generator=g, device="cuda")
    grad_w = torch.randn((T, 1), generator=g, device="cuda")
    got = ops.route_backward(ops.Router(E, 1, 1, renormalize=True, scale=2.5), logits, idx, grad_w).double()
    s = torch.sigmoid(logits.double()).gather(1, idx)
    want = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    want.scatter_(1, idx, 2.5 * grad_w.double() * s * (1 - s) * 1e-20 / (s + 1e-20).square())
    assert ((got - want).abs() <= (8 * 30 + 240) * U * want.abs()).all()
