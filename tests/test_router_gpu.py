"""The router on the GPU against its formulas in 64 bits: the choice exactly, the
weights, the balance loss and the gradient within what their binary32 steps can be off.

Bounds, u = 2^-24. An exponential is off by 2 u and by what its argument's rounding
gives, at most R u with R the logits' spread plus magnitude; a sum of positive terms
adds one u for each addition a term passes through (at most 16 in a lane, 4 within
the rows of 16 lanes, 2 across them); a product or quotient adds u each. A share
has two exponentials and one sum behind it: (2 R + 32) u. A weight that is
renormalised has two shares and another sum: (4 R + 80) u. A gradient multiplies a
score by differences of such weights: (8 R + 240) u of the sum of its terms'
magnitudes. An output in bf16 adds 2^-8 of its value, in binary32 u."""
import numpy as np
import pytest
import torch

import router_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24

if torch.cuda.is_available():
    from combine_ep_layout_10_amd import ops


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make_logits(g, T, E, f32, scale=1.5):
    l = scale * torch.randn((T, E), generator=g, device="cuda")
    return l if f32 else l.to(torch.bfloat16)


def check_route(r, logits, bias=None, mask=None, **kw):
    idx, w = ops.route(r, logits, bias=bias, token_mask=mask, **kw)
    want_idx, want_w = ref.route(logits, bias, mask, r)
    assert idx.dtype == (torch.int64 if r.idx_bits == 64 else torch.int32)
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    tol = (4 * ref.spread(logits) + 80) * U * abs(want_w) + 1e-37
    ref.close(w.cpu().numpy(), want_w, np.nan_to_num(tol), "weights")
    return idx, w


# tokens, experts, topk, groups, kept groups, best
SIZES = [(1, 1, 1, 1, 1, 1), (5, 2, 2, 1, 1, 1), (7, 3, 1, 3, 2, 1), (130, 24, 3, 1, 1, 1), (9, 60, 6, 4, 2, 2),
         (65, 64, 8, 8, 4, 2), (3, 65, 8, 5, 3, 2), (17, 100, 4, 4, 1, 1), (33, 128, 32, 1, 1, 1), (12, 160, 6, 8, 3, 1),
         (200, 256, 8, 8, 4, 2), (31, 256, 8, 1, 1, 1), (4, 257, 32, 1, 1, 1), (6, 384, 8, 3, 2, 2), (6, 512, 10, 64, 9, 2),
         (5, 513, 8, 9, 4, 1), (3, 1000, 20, 8, 7, 2), (9, 1024, 32, 64, 2, 2), (6, 1024, 8, 1, 1, 1), (3, 1023, 31, 1, 1, 2)]


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("sigmoid", [0, 1])
@pytest.mark.parametrize("T,E,k,G,keep,best", SIZES)
def test_route(T, E, k, G, keep, best, sigmoid, f32):
    if best > E // G:
        pytest.skip("a group has fewer experts")
    g = gen(T * 1000 + E)
    logits = make_logits(g, T, E, f32)
    for bias, renorm, bits in ((None, False, 64), (0.3 * torch.randn(E, generator=g, device="cuda"), True, 32)):
        if bias is None and best == 2 and not f32:
            continue  # sums of scores of coarse logits tie up to the last bit of binary64
        r = ops.Router(E, k, sigmoid, G, keep, best, renorm, 1.0 if bias is None else 2.5, bits)
        check_route(r, logits, bias)
        check_route(r, logits, bias, torch.rand(T, generator=g, device="cuda") < 0.7)


@pytest.mark.parametrize("E,G", [(8, 1), (64, 4), (100, 4), (256, 8), (1024, 8)])
@pytest.mark.parametrize("biased", [False, True])
def test_ties_go_to_the_lowest_index(E, G, biased):
    """Few distinct logits, both zeros among them, equal biases: groups and experts tie."""
    g = gen(E)
    logits = torch.randint(-2, 3, (60, E), generator=g, device="cuda").float()
    logits = torch.where((logits == 0) & (torch.rand((60, E), generator=g, device="cuda") < 0.5), -0.0, logits)
    bias = torch.full((E,), 0.25, device="cuda") if biased else None
    for score in (0, 1):
        check_route(ops.Router(E, 6, score, G, max(1, G // 2), 1), logits, bias)
    check_route(ops.Router(E, 6, 1, 1, 1, 1), logits[:1] * 0, bias)


@pytest.mark.parametrize("sigmoid", [1, 0])
@pytest.mark.parametrize("E,k,G,keep,best", [(24, 4, 1, 1, 1), (64, 6, 8, 3, 2), (100, 5, 1, 1, 1), (256, 8, 8, 4, 2), (256, 8, 8, 4, 1),
                                             (384, 8, 1, 1, 1), (160, 6, 8, 3, 2), (1024, 32, 16, 4, 2)])
def test_scores_closer_than_binary32(E, k, G, keep, best, sigmoid):
    """Scores a fraction of a binary32 unit apart, at the border of the choice, within it, or for all
    experts, under biases that are equal or exact; the choice is that of scores in 64 bits. Logits of
    8 differ by steps of 2^-20, which is more than 10^-10 in a sigmoid and 2^-20 of itself in a
    softmax's share: far more than 64 bits' rounding."""
    g, T = gen(E + k), 60
    r = ops.Router(E, k, sigmoid, G, keep, best, renormalize=True)
    logits = torch.randn((T, E), device="cuda", generator=g) * 1.5
    near = 8.0 + 2.0 ** -20 * torch.randint(0, 1 << 17, (T, E), device="cuda", generator=g).float()
    share = torch.linspace(0, 1.2, T, device="cuda")[:, None]    # from no expert to all of them
    logits = torch.where(torch.rand((T, E), device="cuda", generator=g) < share, near, logits)
    for bias in (torch.zeros(E, device="cuda"), torch.randint(0, 3, (E,), device="cuda", generator=g).float() * 0.25):
        check_route(r, logits, bias=bias)
    check_route(r, logits)


@pytest.mark.parametrize("E", [40, 64, 250, 256, 700])
@pytest.mark.parametrize("biased", [False, True])
def test_closed_experts(E, biased):
    """-infinity closes experts: some, all but few, all of a row, all of a group; by the bias as well."""
    g = gen(E)
    logits = make_logits(g, 40, E, True)
    logits[torch.rand((40, E), generator=g, device="cuda") < 0.5] = -torch.inf
    logits[3] = -torch.inf
    logits[4, 5:] = -torch.inf
    logits[5, :E - 1] = -torch.inf
    logits[6, : E // 2] = -torch.inf
    logits[7] = torch.finfo(torch.float32).min
    logits[8, 2:] = torch.finfo(torch.float32).min
    bias = None
    if biased:
        bias = 0.2 * torch.randn(E, generator=g, device="cuda")
        bias[::3] = -torch.inf
    for score in (0, 1):
        for renorm in (False, True):
            idx, w = check_route(ops.Router(E, 8, score, 1, 1, 1, renorm), logits, bias)
            assert (idx[3] == -1).all() and (w[3] == 0).all()
            check_route(ops.Router(E, 8, score, 2, 1, 1, renorm), logits, bias)
            if biased:
                check_route(ops.Router(E, 8, score, 2, 1, 2, renorm), logits, bias)


def test_nan_and_infinity_reach_the_weights():
    E, nan, inf = 70, float("nan"), float("inf")
    logits = make_logits(gen(1), 8, E, True)
    logits[0, 7] = nan
    logits[1] = nan
    logits[2, 9] = inf
    logits[3, [4, 60]] = inf
    logits[4, 3:] = nan
    logits[5, 3:] = -inf
    logits[5, 1] = nan
    for score in (0, 1):
        for bias in (None, torch.zeros(E, device="cuda")):
            check_route(ops.Router(E, 4, score), logits, bias)
            check_route(ops.Router(E, 4, score, 7, 3), logits, bias)
    bias = torch.zeros(E, device="cuda")
    bias[11], bias[12] = inf, nan
    idx, _ = check_route(ops.Router(E, 4, 1), logits[6:], bias)
    assert (idx[:, 0] == 11).all() and not (idx == 12).any()


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("E,k,G,keep", [(160, 6, 1, 1), (256, 8, 8, 3), (257, 4, 1, 1), (700, 32, 1, 1), (1024, 8, 16, 2)])
def test_nan_and_infinity_among_many_experts(E, k, G, keep, f32):
    """NaN, infinities and the largest finite numbers of either sign among logits and biases,
    from a few of a token's experts to all of them."""
    g, T = gen(E), 80
    top = 3.3e38                                     # a finite number in either type
    special = torch.tensor([float("nan"), float("inf"), -float("inf"), top, -top, 0.0, -0.0], device="cuda")
    pick = lambda *shape: special[torch.randint(0, 7, shape, device="cuda", generator=g)]
    share = torch.linspace(0, 1, T, device="cuda")[:, None]
    logits = torch.where(torch.rand((T, E), device="cuda", generator=g) < share, pick(T, E), torch.randn((T, E), device="cuda", generator=g))
    logits = logits if f32 else logits.to(torch.bfloat16)
    noise = torch.randn(E, device="cuda", generator=g)
    odd = torch.where(torch.rand(E, device="cuda", generator=g) < 0.1, pick(E), noise)
    for bias in (None, torch.zeros(E, device="cuda"), noise, odd, 1e30 * noise):
        for sigmoid in (0, 1):
            check_route(ops.Router(E, k, sigmoid, G, keep, 1), logits, bias)


def test_masked_tokens_are_not_read():
    """NaN in the padding of a batch goes nowhere."""
    logits = make_logits(gen(2), 6, 48, True)
    mask = torch.tensor([True, False, True, False, False, True], device="cuda")
    logits[~mask] = float("nan")
    r = ops.Router(48, 4, 0, renormalize=True)
    idx, w = check_route(r, logits, None, mask)
    assert (idx[~mask] == -1).all() and (w[~mask] == 0).all()
    loss, counts, coef = ops.balance_loss(r, logits, idx)
    assert torch.isfinite(loss) and int(counts.sum()) == 12
    grad = ops.route_backward(r, logits, idx, torch.ones_like(w), counts, coef, torch.ones((), device="cuda"))
    assert torch.isfinite(grad).all() and (grad[~mask] == 0).all()


def test_route_into_buffers_and_unaligned_rows():
    """Rows that start anywhere (a slice of tokens of an odd number of experts), buffers of the caller's."""
    for f32 in (True, False):
        for E in (63, 201, 256):
            base = make_logits(gen(E), 20, E, f32)
            logits = base[1:]
            idx = torch.full((19, 5), -7, dtype=torch.int64, device="cuda")
            w = torch.full((19, 5), -7.0, device="cuda")
            got = check_route(ops.Router(E, 5), logits, topk_idx=idx, topk_w=w)
            assert got[0].data_ptr() == idx.data_ptr() and got[1].data_ptr() == w.data_ptr()


def test_no_tokens():
    r = ops.Router(16, 2)
    logits = torch.empty((0, 16), device="cuda")
    idx, w = ops.route(r, logits)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    loss, counts, coef = ops.balance_loss(r, logits, idx)
    assert float(loss) == 0 and not counts.any() and float(coef) == 0
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    loss, counts, coef = ops.balance_loss(r, logits, idx, off)
    assert float(loss) == 0 and counts.shape == (3, 16) and not counts.any() and not coef.any()
    assert ops.route_backward(r, logits, idx, w).shape == (0, 16)


# ---------------------------------------------------------------- balance loss

def routing(g, T, E, k, dropped=0.2, bits=64):
    """Ids as a user may have them: duplicates, masked and bad ones, tokens without any."""
    idx = torch.randint(-1, E, (T, k), generator=g, device="cuda")
    bad = torch.rand((T, k), generator=g, device="cuda")
    idx = torch.where(bad < 0.03, E + 5, idx)
    if bits == 64:
        idx = torch.where(bad > 0.97, (1 << 32) + 1, idx)
    idx = torch.where(torch.rand((T, 1), generator=g, device="cuda") < dropped, -1, idx)
    return idx if bits == 64 else idx.int()


def check_balance(r, logits, idx, off, **kw):
    loss, counts, coef = ops.balance_loss(r, logits, idx, off, **kw)
    want, want_counts, want_coef, _ = ref.balance(logits, idx, off, r)
    assert loss.shape == () and counts.dtype == torch.int32
    assert np.array_equal(counts.cpu().numpy(), want_counts)
    ref.close(coef.cpu().numpy(), want_coef, 2 * U * want_coef, "coef")
    # each term is a share, summed over at most 4 tokens of a wave and 16 waves in binary32
    ref.close(loss.item(), want, (2 * ref.spread(logits) + 60) * U * want, "loss")
    return loss, counts, coef


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("sigmoid", [0, 1])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 5, 2), (63, 24, 3), (64, 64, 6), (65, 60, 8), (300, 256, 8), (129, 257, 2),
                                   (200, 1024, 32), (1000, 8, 2)])
def test_balance(T, E, k, sigmoid, f32):
    g = gen(T + E)
    logits, idx = make_logits(g, T, E, f32), routing(g, T, E, k)
    check_balance(ops.Router(E, k, sigmoid), logits, idx, None)
    idx = routing(g, T, E, k, bits=32)
    r = ops.Router(E, k, sigmoid, idx_bits=32)
    for cuts in ([0, T], [0, 0, T // 2, T // 2, T // 2, T], [T // 3, T // 3 + 1, max(T - 2, T // 3 + 1)],
                 list(range(T + 1)), [-5, 1, T + 9], [0] * 40 + [T] * 40):
        check_balance(r, logits, idx, torch.tensor(cuts, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("T,S", [(33, 30), (1, 40), (7, 3), (512, 512), (700, 2000), (2048, 100), (20000, 600),
                                 (40, 1 << 17)])
def test_balance_of_short_sequences(T, S):
    """Fewer tokens a sequence than a block takes at once, empty sequences among them, tokens
    before the first and past the last."""
    g = gen(T + S)
    off = torch.sort(torch.randint(T // 20, T + 1, (S + 1,), device="cuda", generator=g).int())[0]
    for E, k in ((138, 4), (16, 2)):
        r, logits, idx = ops.Router(E, k, 1), make_logits(g, T, E, True), routing(g, T, E, k)
        loss, counts, coef = check_balance(r, logits, idx, off)
        check_backward(r, logits, idx, None, counts, coef, torch.tensor(1.5, device="cuda"), off)


def test_balance_of_long_and_of_even_batches():
    g = gen(3)
    T, E = 40000, 8
    logits = make_logits(g, T, E, True)
    idx = logits.topk(2, 1).indices
    r = ops.Router(E, 2)
    # against the formula with torch in 64 bits, the reference takes too long
    loss, counts, coef = ops.balance_loss(r, logits, idx)
    f = torch.bincount(idx.flatten(), minlength=E)
    assert torch.equal(counts[0].long(), f)
    want = (f * logits.double().softmax(1).sum(0)).sum() * E / (2.0 * T * T)
    assert abs(loss.item() - want.item()) <= (2 * ref.spread(logits) + 60) * U * want.item()
    # even scores and counts: 1
    even = torch.arange(64, device="cuda").view(32, 2) % E
    for score in (0, 1):
        loss, _, _ = ops.balance_loss(ops.Router(E, 2, score), torch.zeros((32, E), device="cuda"), even)
        assert abs(loss.item() - 1.0) <= 60 * U


def test_rows_without_a_finite_logit():
    """A routed token whose logits are all -infinity has no shares and no gradient."""
    logits = torch.full((3, 20), -torch.inf, device="cuda")
    logits[1] = make_logits(gen(4), 1, 20, True)[0]
    idx = torch.tensor([[1, 2], [3, 4], [5, -1]], device="cuda")
    for score in (0, 1):
        r = ops.Router(20, 2, score)
        loss, counts, coef = check_balance(r, logits, idx, None)
        grad = ops.route_backward(r, logits, idx, torch.ones((3, 2), device="cuda"), counts, coef, loss)
        assert torch.isfinite(grad).all() and not grad[0].any() and not grad[2].any()


# ---------------------------------------------------------------- gradient

def check_backward(r, logits, idx, grad_w, counts, coef, grad_loss, off, **kw):
    got = ops.route_backward(r, logits, idx, grad_w, counts, coef, grad_loss, off, **kw)
    want, size = ref.backward(logits, idx, grad_w, counts, coef, grad_loss, off, r)
    assert got.dtype == logits.dtype and got.shape == logits.shape
    out = U if logits.dtype == torch.float32 else 2.0 ** -8
    least = 1e-37 if logits.dtype == torch.float32 else 1e-37
    ref.close(got.double().cpu().numpy(), want, (8 * ref.spread(logits) + 240) * U * size + out * abs(want) + least, "grad")
    return got


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("sigmoid", [0, 1])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 2), (63, 24, 3), (30, 64, 6), (65, 60, 8), (50, 256, 8), (9, 257, 2),
                                   (20, 1000, 32), (7, 1024, 8)])
def test_backward(T, E, k, sigmoid, f32):
    g = gen(T * 7 + E)
    logits = make_logits(g, T, E, f32)
    idx = routing(g, T, E, k)
    grad_w = torch.randn((T, k), generator=g, device="cuda")
    grad_loss = torch.tensor(0.7, device="cuda")
    off = torch.tensor([0, T // 3, T // 3, max(T // 3, T - 1)], dtype=torch.int32, device="cuda")
    for renorm in (False, True):
        r = ops.Router(E, k, sigmoid, renormalize=renorm, scale=-1.5)
        check_backward(r, logits, idx, grad_w, None, None, None, None)
        for cuts in (None, off):
            _, counts, coef = ops.balance_loss(r, logits, idx, cuts)
            check_backward(r, logits, idx, grad_w, counts, coef, grad_loss, cuts)
            check_backward(r, logits, idx, None, counts, coef, grad_loss, cuts)


@pytest.mark.parametrize("sigmoid", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward_against_differences(sigmoid, renorm):
    """The gradient against central differences of the reference's own forward in 64
    bits, the choice held: their error is the third derivative's, below 1e-3 step^2,
    and the rounding of the forward, 1e-15 / step."""
    T, E, k = 4, 12, 3
    g = gen(9)
    logits = make_logits(g, T, E, True)
    r = ops.Router(E, k, sigmoid, renormalize=renorm, scale=1.5)
    idx, _ = ops.route(r, logits)
    grad_w = torch.randn((T, k), generator=g, device="cuda")
    _, counts, coef = ops.balance_loss(r, logits, idx)
    got = ops.route_backward(r, logits, idx, grad_w, counts, coef, torch.tensor(2.0, device="cuda")).double().cpu().numpy()
    l, ids, gw = logits.double().cpu().numpy(), idx.cpu().numpy(), grad_w.double().cpu().numpy()
    c, f = counts.double().cpu().numpy(), float(coef[0])

    def total(x):
        v = 0.0
        for t in range(T):
            s, p = ref.scores(x[t], sigmoid)
            w = s[ids[t]]
            if renorm:
                w = w / w.sum()
            v += (1.5 * w * gw[t]).sum() + 2.0 * f * (c[0] * p).sum()
        return v

    step = 1e-4
    for t in range(T):
        for e in range(E):
            up, down = l.copy(), l.copy()
            up[t, e] += step
            down[t, e] -= step
            want = (total(up) - total(down)) / (2 * step)
            assert abs(got[t, e] - want) <= 1e-6, (t, e)


def test_backward_of_a_balanced_batch_keeps_its_digits():
    """Counts of a million each, a few apart: their common part must cancel exactly."""
    E, k = 64, 2
    g = gen(10)
    logits = make_logits(g, 16, E, True)
    idx = logits.topk(k, 1).indices
    counts = (1_000_000 + torch.randint(-3, 4, (1, E), generator=g, device="cuda")).int()
    coef = torch.tensor([1e-6], device="cuda")
    for score in (0, 1):
        check_backward(ops.Router(E, k, score), logits, idx, None, counts, coef, torch.ones((), device="cuda"), None)


def test_backward_may_write_over_the_logits():
    for E in (60, 256):
        logits = make_logits(gen(E), 33, E, True)
        r = ops.Router(E, 4, 1, renormalize=True)
        idx, w = ops.route(r, logits)
        want = ops.route_backward(r, logits, idx, torch.ones_like(w))
        got = ops.route_backward(r, logits, idx, torch.ones_like(w), grad_logits=logits)
        assert got.data_ptr() == logits.data_ptr() and torch.equal(got, want)


# ---------------------------------------------------------------- how calls go together

def test_the_same_call_gives_the_same_bits():
    g = gen(11)
    T, E, k = 3000, 256, 8
    logits = make_logits(g, T, E, True)
    r = ops.Router(E, k, 1, 8, 4, 2, True, 2.5)
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    off = torch.tensor([0, 1000, 1001, 3000], dtype=torch.int32, device="cuda")
    first = None
    for _ in range(3):
        idx, w = ops.route(r, logits, bias)
        loss, counts, coef = ops.balance_loss(r, logits, idx, off)
        grad = ops.route_backward(r, logits, idx, w, counts, coef, loss, off)
        now = [idx, w, loss, counts, coef, grad]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


@pytest.mark.parametrize("T,E,S", [(8192, 256, 1), (4096, 64, 19), (3000, 1024, 130)])
def test_balance_again_and_again_in_one_workspace(T, E, S):
    """Two batches in turn through the same workspace and outputs: what an earlier call left there
    never shows."""
    r, g = ops.Router(E, 4), gen(T)
    off = torch.linspace(0, T, S + 1, device="cuda").int()
    batches = [(make_logits(g, T, E, True), routing(g, T, E, 4)) for _ in range(2)]
    want = [tuple(t.clone() for t in ops.balance_loss(r, l, i, off)) for l, i in batches]
    ws = ops.balance_loss_workspace(r, T, S)
    out = tuple(torch.empty_like(t) for t in want[0])
    for rep in range(300):
        ops.balance_loss(r, *batches[rep % 2], off, *out, workspace=ws)
        kept = tuple(t.clone() for t in out)
        assert all(torch.equal(a, b) for a, b in zip(kept, want[rep % 2])), rep


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, against the same calls one after the other."""
    E, k = 160, 6
    r = ops.Router(E, k, 1, renormalize=True)
    logits = [make_logits(gen(20 + i), 4000, E, True) for i in range(2)]

    def step(l, ws):
        idx, w = ops.route(r, l)
        loss, counts, coef = ops.balance_loss(r, l, idx, workspace=ws)
        return idx, w, loss, counts, coef, ops.route_backward(r, l, idx, w, counts, coef, loss)

    want = [step(l, None) for l in logits]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [ops.balance_loss_workspace(r, 4000) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, l, ws in zip(streams, logits, spaces):
            with torch.cuda.stream(s):
                got.append(step(l, ws))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured():
    """A captured training step of the router, replayed on new logits, with eager work between."""
    T, E, k = 500, 256, 8
    r = ops.Router(E, k, 1, 8, 4, 2, True, 2.5)
    bias = 0.1 * torch.randn(E, generator=gen(30), device="cuda")
    off = torch.tensor([0, 100, 350, 500], dtype=torch.int32, device="cuda")
    logits = make_logits(gen(31), T, E, True)
    ws = ops.balance_loss_workspace(r, T, 3)

    def step(l, w_space):
        idx, w = ops.route(r, l, bias)
        loss, counts, coef = ops.balance_loss(r, l, idx, off, workspace=w_space)
        return idx, w, loss, counts, coef, ops.route_backward(r, l, idx, w, counts, coef, loss, off)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(logits, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(logits, ws)
    for i in range(4):
        logits.copy_(make_logits(gen(40 + i), T, E, True))
        graph.replay()
        want = step(logits, None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i


def test_refused_tensors():
    r = ops.Router(16, 2)
    l = torch.zeros((4, 16), device="cuda")
    idx, w = ops.route(r, l)
    for bad in (l[:, :8], l.half(), l.t().contiguous().t(), l.cpu(), torch.zeros((4, 17), device="cuda"), l[0]):
        with pytest.raises(ValueError):
            ops.route(r, bad)
    with pytest.raises(ValueError, match="bias"):
        ops.route(r, l, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError, match="token_mask"):
        ops.route(r, l, token_mask=torch.zeros(4, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="topk_idx"):
        ops.route(r, l, topk_idx=idx.int())
    with pytest.raises(ValueError, match="topk_idx"):
        ops.balance_loss(r, l, idx[:, :1].contiguous())
    with pytest.raises(ValueError, match="seq_off"):
        ops.balance_loss(r, l, idx, torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="seq_off"):
        ops.balance_loss(r, l, idx, torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(RuntimeError, match="workspace"):
        ops.balance_loss(r, l, idx, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    loss, counts, coef = ops.balance_loss(r, l, idx)
    with pytest.raises(RuntimeError, match="together"):
        ops.route_backward(r, l, idx, w, counts, coef)
    with pytest.raises(RuntimeError, match="given"):
        ops.route_backward(r, l, idx)
    with pytest.raises(ValueError, match="grad_logits"):
        ops.route_backward(r, l, idx, w, grad_logits=l.bfloat16())
