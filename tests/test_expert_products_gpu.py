"""The experts' products over the receive rows (BF16 in three directions,
MXFP4 weights) against plain products in 64 bits.

Tolerance: bf16 (and MXFP4) operands have exact products in binary32; the MFMA
adds at most K of them, each addition off by at most one binary32 ulp of the
running sum (2^-23 relative, whatever the rounding mode and order), so the sum
is within acc = K * 2^-23 * (1 + 2^-9) * sum|a b| of the exact one (K <= 2^13
here, so second-order terms stay below the factor); a bf16 output adds half a
step, 2^-8 of the rounded value at most. Inputs are far from bf16's subnormals."""
import math

import numpy as np
import pytest
import torch

from ep_workloads import random_routing_table
from gpu_common import log, to_dev

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_ep_layout_10_amd import ops

DIRS = ("forward", "grad_input", "grad_weight", "mxfp4")
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def routing(counts, k=1):
    """A [T, 1] table giving expert e exactly counts[e] tokens, interleaved."""
    ids = np.concatenate([np.full(c, e, np.int64) for e, c in enumerate(counts)] + [np.zeros(0, np.int64)])
    return np.random.default_rng(3).permutation(ids).reshape(-1, k)


def make_handle(idx, E, A=1, mode=0, C=0, flags=0, max_tokens=None):
    cfg = ops.Config(max_tokens=max_tokens or idx.shape[0], hidden=8, num_experts=E, num_topk=idx.shape[1],
                     expert_alignment=A, capacity=C, mode=mode, flags=flags)
    return ops.layout(cfg, to_dev(idx))


def ranges(h):
    """(first row, live rows, owned rows) of every expert, on the host."""
    cnt, pad, _ = h.read_counts()
    if h.cfg.mode == ops.MODE_FIXED:
        return [(e * h.cfg.capacity, int(p), int(p)) for e, p in enumerate(pad)]
    off = h.expert_off.cpu().numpy()
    return [(int(off[e]), int(cnt[e]), int(off[e + 1] - off[e])) for e in range(h.cfg.num_experts)]


def bf16(gen, *shape):
    return torch.randn(shape, device="cuda", generator=gen).to(torch.bfloat16)


def poison(x, rr):
    """NaN in every row that holds no pair."""
    keep = torch.zeros(x.shape[0], dtype=torch.bool, device=x.device)
    for first, live, _ in rr:
        keep[first:first + live] = True
    x[~keep] = float("nan")
    return x


def decode_mxfp4(b, s):
    lv = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device=b.device)
    codes = torch.stack([b & 15, b >> 4], -1).flatten(-2).long()
    return lv[codes] * torch.exp2(s.double() - 127.0).repeat_interleave(32, -1)


def operands(direction, h, n, k, seed=0):
    """Operands with NaN wherever the contract says nothing is read, and the
    weights in 64 bits."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    R, E = h.cfg.recv_rows_bound(), h.cfg.num_experts
    rr = ranges(h)
    o = dict(rr=rr)
    if direction != "grad_input":
        o["a"] = poison(bf16(gen, R, k), rr)
    if direction in ("grad_input", "grad_weight"):
        o["g"] = poison(bf16(gen, R, n), rr)
    if direction in ("forward", "grad_input"):
        o["b"] = bf16(gen, E, n, k)
        for e, (_, live, _) in enumerate(rr):
            if live == 0:
                o["b"][e] = float("nan")
        o["w64"] = lambda e: o["b"][e].double()
    if direction == "mxfp4":
        o["b"] = torch.randint(0, 256, (E, n, k // 2), dtype=torch.uint8, device="cuda", generator=gen)
        o["s"] = torch.randint(120, 135, (E, n, k // 32), dtype=torch.uint8, device="cuda", generator=gen)
        for e, (_, live, _) in enumerate(rr):
            if live == 0:
                o["s"][e] = 255
        o["w64"] = lambda e: decode_mxfp4(o["b"][e], o["s"][e])
    return o


def call(direction, h, o, out=None):
    if direction == "forward":
        return ops.grouped_gemm_bf16(h, o["a"], o["b"], out=out)
    if direction == "grad_input":
        return ops.grouped_gemm_bf16_grad_input(h, o["g"], o["b"], grad_a=out)
    if direction == "grad_weight":
        return ops.grouped_gemm_bf16_grad_weight(h, o["g"], o["a"], grad_b=out)
    return ops.grouped_gemm_mxfp4(h, o["a"], o["b"], o["s"], out=out)


def check(got, x, y, K, what):
    """got against x @ y (64 bits): the tolerance of the module's docstring."""
    want, size = x @ y, x.abs() @ y.abs()
    acc = K * 2.0 ** -23 * (1 + 2.0 ** -9) * size
    lim = acc if got.dtype == torch.float32 else acc + 2.0 ** -8 * (want.abs() + acc)
    err = (got.double() - want).abs()
    assert bool((err <= lim).all()), (what, float((err / lim.clamp(min=1e-300)).max()))


def verify(direction, h, o, got, n, k):
    """Every expert's values, zeros on padding, everything else untouched
    (got was filled with 7 before the call)."""
    touched = torch.zeros(got.shape[0], dtype=torch.bool, device="cuda")
    zero_pad = not (h.cfg.flags & ops.FLAG_NO_ZERO_PAD)
    for e, (first, live, owned) in enumerate(o["rr"]):
        rows = slice(first, first + live)
        if direction == "grad_weight":
            if live == 0:
                assert bool((got[e] == 0).all()), e
            else:
                check(got[e], o["g"][rows].double().t(), o["a"][rows].double(), live, e)
            continue
        if live:
            x = o["g" if direction == "grad_input" else "a"][rows].double()
            w = o["w64"](e)
            check(got[rows], x, w if direction == "grad_input" else w.t(), n if direction == "grad_input" else k, e)
        assert not zero_pad or bool((got[first + live:first + owned] == 0).all()), e
        touched[first:first + (owned if zero_pad else live)] = True
    if direction != "grad_weight":
        assert bool((got[~touched] == 7).all())


def run_case(direction, h, n, k, seed=0, f32=True):
    log("%s: T=%d E=%d k=%d A=%d mode=%d n=%d k=%d" % (direction, h.num_tokens, h.cfg.num_experts, h.cfg.num_topk,
                                                      h.cfg.expert_alignment, h.cfg.mode, n, k))
    o = operands(direction, h, n, k, seed)
    R, E = h.cfg.recv_rows_bound(), h.cfg.num_experts
    if direction == "grad_weight":
        out = torch.full((E, n, k), 7.0, device="cuda", dtype=torch.float32 if f32 else torch.bfloat16)
    else:
        out = torch.full((R, k if direction == "grad_input" else n), 7.0, device="cuda", dtype=torch.bfloat16)
    got = call(direction, h, o, out)
    assert got is out
    torch.cuda.synchronize()
    verify(direction, h, o, got, n, k)
    return o, got


# rows an expert: none, one, around the 16-, 64-, 128- and 256-row steps, and more than one tile
COUNTS = [0, 1, 15, 16, 17, 0, 31, 33, 64, 65, 127, 128, 129, 255, 256, 257, 300, 0, 511, 513, 2, 0]


@pytest.mark.parametrize("direction", DIRS)
@pytest.mark.parametrize("A", [1, 16, 300])
def test_every_count(direction, A):
    run_case(direction, make_handle(routing(COUNTS), len(COUNTS), A), 264, 288)


@pytest.mark.parametrize("direction", DIRS)
@pytest.mark.parametrize("n,k", [(8, 32), (16, 64), (24, 96), (8, 1056), (1000, 32), (248, 160), (256, 256), (264, 224),
                                 (520, 544), (512, 64), (128, 512), (1032, 2080)])
def test_sizes(direction, n, k):
    rng = np.random.default_rng(5)
    h = make_handle(random_routing_table(rng, 150, 7, 3, masked_frac=0.2), 7, 8)
    run_case(direction, h, n, k, seed=n + k)


@pytest.mark.parametrize("direction", DIRS[:3])
@pytest.mark.parametrize("n,k", [(8, 8), (40, 72), (200, 8), (8, 200), (1416, 1000), (312, 328)])
def test_sizes_off_any_tile(direction, n, k):
    """Widths that are multiples of 8 alone."""
    rng = np.random.default_rng(6)
    h = make_handle(random_routing_table(rng, 333, 5, 2), 5, 1)
    run_case(direction, h, n, k, seed=n + k, f32=False)


@pytest.mark.parametrize("direction", DIRS)
def test_one_token(direction):
    h = make_handle(np.array([[3, 0, 6]], np.int64), 8)
    run_case(direction, h, 136, 352)
    h = make_handle(np.array([[0]], np.int64), 1)
    run_case(direction, h, 264, 288)


@pytest.mark.parametrize("direction", DIRS)
def test_no_rows(direction):
    """Every pair masked, and an empty batch: nothing but grad_weight's zeros is written."""
    run_case(direction, make_handle(np.full((9, 2), -1, np.int64), 4, 16), 72, 96)
    cfg = ops.Config(max_tokens=4, hidden=8, num_experts=4, num_topk=2)
    h = ops.layout(cfg, torch.empty((0, 2), dtype=torch.int64, device="cuda"))
    run_case(direction, h, 72, 96)


@pytest.mark.parametrize("direction", DIRS)
def test_many_experts(direction):
    """More experts than a wave has lanes, most of them with few rows, bad ids among the pairs."""
    rng = np.random.default_rng(7)
    h = make_handle(random_routing_table(rng, 400, 1024, 4, masked_frac=0.1, bad_frac=0.05), 1024, 4)
    run_case(direction, h, 40, 64)


@pytest.mark.parametrize("direction", DIRS)
def test_duplicate_experts_and_hot_expert(direction):
    """The same expert several times in a token's row, and one expert with everything."""
    rng = np.random.default_rng(8)
    run_case(direction, make_handle(random_routing_table(rng, 120, 3, 5, distinct=False), 3, 1), 136, 160)
    run_case(direction, make_handle(np.full((700, 1), 2, np.int64), 5, 128), 136, 160)


@pytest.mark.parametrize("direction", DIRS)
@pytest.mark.parametrize("C", [3, 40, 160])
def test_fixed_capacity(direction, C):
    """FIXED: experts that overflow, rows past each count left as they were."""
    rng = np.random.default_rng(9)
    h = make_handle(random_routing_table(rng, 200, 6, 2), 6, 1, mode=ops.MODE_FIXED, C=C)
    run_case(direction, h, 264, 96)


@pytest.mark.parametrize("direction", ("forward", "grad_input", "mxfp4"))
def test_no_zero_pad(direction):
    rng = np.random.default_rng(10)
    h = make_handle(random_routing_table(rng, 90, 6, 2), 6, 32, flags=ops.FLAG_NO_ZERO_PAD)
    run_case(direction, h, 136, 96)


@pytest.mark.parametrize("direction", DIRS)
def test_fewer_tokens_than_configured(direction):
    rng = np.random.default_rng(11)
    h = make_handle(random_routing_table(rng, 50, 6, 2), 6, 8, max_tokens=300)
    run_case(direction, h, 72, 96)


@pytest.mark.parametrize("direction", DIRS)
def test_large_batch(direction):
    """Many tiles of every kind: a mid-size training batch."""
    rng = np.random.default_rng(12)
    h = make_handle(random_routing_table(rng, 3000, 8, 2), 8, 128)
    run_case(direction, h, 1032, 1056, f32=False)


@pytest.mark.parametrize("direction", DIRS)
def test_same_bits_again(direction):
    """The sums have a fixed order: two calls, and a call sized for other
    hardware, give the same bits."""
    import os
    rng = np.random.default_rng(13)
    h = make_handle(random_routing_table(rng, 500, 6, 2), 6, 1)
    o = operands(direction, h, 520, 544)
    first = call(direction, h, o)
    rows = torch.cat([torch.arange(f, f + l) for f, l, _ in o["rr"]]).cuda() if direction != "grad_weight" else slice(None)
    try:
        for cus in (None, "3", "1024"):
            if cus:
                os.environ["EP_LAUNCH_CUS"] = cus
            assert torch.equal(call(direction, h, o)[rows], first[rows]), cus
    finally:
        os.environ.pop("EP_LAUNCH_CUS", None)


@pytest.mark.parametrize("direction", DIRS)
def test_infinite_and_nan_values(direction):
    """Infinities and NaN in live rows reach exactly the outputs that the
    formula says; neighbouring experts' rows stay finite."""
    h = make_handle(routing([20, 30, 10]), 3, 1)
    o = operands(direction, h, 72, 96)
    for first, live, _ in o["rr"]:
        for x in [o[i] for i in ("a", "g") if i in o]:
            x[first + 3, 5] = float("inf") if first == 0 else 2.0
    name = "g" if direction == "grad_input" else "a"
    o[name][o["rr"][2][0]] = float("nan")          # one whole row of the last expert
    got = call(direction, h, o)
    for e, (first, live, _) in enumerate(o["rr"]):
        rows = slice(first, first + live)
        if direction == "grad_weight":
            g, want = got[e], o["g"][rows].double().t() @ o["a"][rows].double()
        else:
            w = o["w64"](e)
            g, want = got[rows], o[name][rows].double() @ (w if direction == "grad_input" else w.t())
        assert torch.equal(torch.isnan(g), torch.isnan(want)), e
        assert torch.equal(torch.isinf(g), torch.isinf(want)), e
        assert torch.equal(g[torch.isinf(want)].double(), want[torch.isinf(want)]), e


def test_mxfp4_every_code_and_scale():
    """Each of the 16 codes under each of the 256 scales, alone in its group:
    one nonzero activation selects it."""
    E, n, k = 1, 256, 32 * 16
    b = torch.zeros((E, n, k // 2), dtype=torch.uint8, device="cuda")
    for c in range(16):                            # group c holds code c at its position 5 (byte 2, high nibble)
        b[:, :, 16 * c + 2] = c << 4
    s = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, n, 1).expand(E, n, 16).contiguous()
    h = make_handle(np.zeros((16, 1), np.int64), E)
    a = torch.zeros((16, k), dtype=torch.bfloat16, device="cuda")
    for c in range(16):
        a[c, 32 * c + 5] = 1.0
    got = ops.grouped_gemm_mxfp4(h, a, b, s).double()
    lv = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device="cuda")
    for c in range(16):
        want = lv[c] * torch.exp2(torch.arange(256, device="cuda").double() - 127.0)
        want = want.to(torch.bfloat16).double()
        sound = slice(0, 253)                      # above, another group's 6 is infinite, and 0 * inf is NaN
        assert torch.equal(got[c, sound], want[sound]), c
        assert bool(torch.isnan(got[c, 255])), c   # a NaN scale makes its whole group NaN


def test_mxfp4_top_scale():
    """2^127: codes of 2 and more are infinite in bf16, the others exact."""
    b = torch.zeros((1, 16, 16), dtype=torch.uint8, device="cuda")
    b[0, :, 2] = torch.arange(16, dtype=torch.uint8, device="cuda") << 4
    s = torch.full((1, 16, 1), 254, dtype=torch.uint8, device="cuda")
    a = torch.zeros((1, 32), dtype=torch.bfloat16, device="cuda")
    a[0, 5] = 1.0
    got = ops.grouped_gemm_mxfp4(make_handle(np.zeros((1, 1), np.int64), 1), a, b, s)[0].double()
    lv = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device="cuda") * 2.0 ** 127
    assert torch.equal(got, lv.to(torch.bfloat16).double())


@pytest.mark.parametrize("rows", [1, 9, 40])
@pytest.mark.parametrize("n,k", [(72, 4128), (520, 2080), (1000, 1056), (2056, 1024), (264, 8192)])
def test_mxfp4_long_reductions(rows, n, k):
    """One to many rows an expert, reductions that are split over more and
    fewer parts and end inside a slice, scales at an odd address."""
    h = make_handle(routing([rows, 0, rows + 2, 1, 3 * rows]), 5, 1)
    o = operands("mxfp4", h, n, k, seed=rows + k)
    odd = torch.empty(o["s"].numel() + 1, dtype=torch.uint8, device="cuda")[1:].view(o["s"].shape)
    o["s"] = odd.copy_(o["s"])
    out = torch.full((h.cfg.recv_rows_bound(), n), 7.0, dtype=torch.bfloat16, device="cuda")
    verify("mxfp4", h, o, call("mxfp4", h, o, out), n, k)


def test_gradients_are_differences():
    """Integer operands small enough that every product and sum is exact in
    bf16: the change of <out, g> along a direction equals the gradient's inner
    product with it, exactly."""
    rng = np.random.default_rng(14)
    h = make_handle(random_routing_table(rng, 60, 4, 2), 4, 4)
    R, E, n, k = h.cfg.recv_rows_bound(), 4, 48, 56
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    ints = lambda m, *shape: torch.randint(-m, m + 1, shape, device="cuda", generator=gen).to(torch.bfloat16)
    rr = ranges(h)
    live = torch.cat([torch.arange(f, f + l) for f, l, _ in rr]).cuda()
    a, b, g = ints(1, R, k), ints(1, E, n, k), ints(1, R, n)
    da, db = ints(1, R, k), ints(1, E, n, k)
    inner = lambda x, y: float((x.double() * y.double()).sum())
    f = lambda x, w: ops.grouped_gemm_bf16(h, x, w)[live]
    ga = ops.grouped_gemm_bf16_grad_input(h, g, b)[live]
    gb = ops.grouped_gemm_bf16_grad_weight(h, g, a)
    assert inner(f(a + da, b) - f(a, b), g[live]) == inner(ga, da[live])
    assert inner(f(a, b + db) - f(a, b), g[live]) == inner(gb, db)


@pytest.mark.parametrize("direction", DIRS)
def test_graph_replay(direction):
    """Captured once and replayed on new routing and operands, with eager calls
    between the replays."""
    rng = np.random.default_rng(15)
    T, E, n, k = 300, 6, 264, 288
    h = make_handle(random_routing_table(rng, T, E, 2), E, 16)
    idx = h.topk_idx
    o = operands(direction, h, n, k)
    out = torch.full_like(call(direction, h, o), 7.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(direction, h, o, out)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h2 = ops.layout(h.cfg, idx, workspace=h.workspace)
        call(direction, h2, o, out)
    for rep in range(3):
        idx.copy_(to_dev(random_routing_table(rng, T, E, 2)))
        he = ops.layout(h.cfg, idx)
        new = operands(direction, he, n, k, seed=rep)
        for name in ("a", "g", "b", "s"):
            if name in o:
                o[name].copy_(new[name])
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        eager = torch.full_like(out, 7.0)
        call(direction, he, new, eager)
        assert torch.equal(out, eager), rep
        verify(direction, he, new, out, n, k)


@pytest.mark.parametrize("direction", DIRS)
def test_two_streams_at_once(direction):
    """Two calls on two streams share nothing."""
    rng = np.random.default_rng(16)
    hs = [make_handle(random_routing_table(rng, 700, 6, 2), 6, 1) for _ in range(2)]
    os_ = [operands(direction, h, 520, 544, seed=i) for i, h in enumerate(hs)]
    want = [call(direction, h, o) for h, o in zip(hs, os_)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for s, h, o in zip(streams, hs, os_):
        with torch.cuda.stream(s):
            got.append([call(direction, h, o) for _ in range(4)])
    torch.cuda.synchronize()
    for w, g, o in zip(want, got, os_):
        rows = torch.cat([torch.arange(f, f + l) for f, l, _ in o["rr"]]).cuda() if direction != "grad_weight" else slice(None)
        for x in g:
            assert torch.equal(x[rows], w[rows])


@pytest.mark.parametrize("direction", DIRS)
def test_widest(direction):
    """The widest rows of either side that are accepted. (The tolerance's K 2^-23
    is 1/8 here: gamma = K u / (1 - K u) in its place.)"""
    W = 1 << 20
    gamma = W * 2.0 ** -23 / (1 - W * 2.0 ** -23)
    h = make_handle(routing([1, 0, 2]), 3, 1)
    for n, k in ((8, W), (W, 32)):
        o = operands(direction, h, n, k)
        got = call(direction, h, o)
        for e, (first, live, _) in enumerate(o["rr"]):
            rows = slice(first, first + live)
            if direction == "grad_weight":
                check(got[e], o["g"][rows].double().t(), o["a"][rows].double(), live, e)
            elif live:
                x = o["g" if direction == "grad_input" else "a"][rows].double()
                w = o["w64"](e) if direction == "grad_input" else o["w64"](e).t()
                want, size = x @ w, gamma * (x.abs() @ w.abs())
                err = (got[rows].double() - want).abs()
                assert bool((err <= size + 2.0 ** -8 * (want.abs() + size)).all()), e


def test_far_offsets():
    """Operands and outputs past 2^32 bytes: the last experts of a wide stack."""
    E, n, k = 40, 4096, 16384                      # 5.4 GB of weights
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    h = make_handle(np.array([[0], [E - 2], [E - 1], [E - 1]], np.int64), E)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    b = torch.zeros((E, n, k), dtype=torch.bfloat16, device="cuda")
    for e in (0, E - 2, E - 1):
        b[e] = bf16(gen, n, k)
    a, g = bf16(gen, 4, k), bf16(gen, 4, n)
    out, ga = ops.grouped_gemm_bf16(h, a, b), ops.grouped_gemm_bf16_grad_input(h, g, b)
    gb = ops.grouped_gemm_bf16_grad_weight(h, g, a, grad_b=torch.full_like(b, 7.0))
    for e, rows in ((0, slice(0, 1)), (E - 2, slice(1, 2)), (E - 1, slice(2, 4))):
        w = b[e].double()
        check(out[rows], a[rows].double(), w.t(), k, e)
        check(ga[rows], g[rows].double(), w, n, e)
        check(gb[e], g[rows].double().t(), a[rows].double(), 2, e)
    assert bool((gb[1:E - 2] == 0).all())


def test_refusals():
    rng = np.random.default_rng(17)
    h = make_handle(random_routing_table(rng, 20, 4, 2), 4, 1)
    R = h.cfg.recv_rows_bound()
    z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")
    a, g, b = z(R, 64), z(R, 40), z(4, 40, 64)
    codes, scales = z(4, 40, 32, dtype=torch.uint8), z(4, 40, 2, dtype=torch.uint8)
    out = torch.full((R, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    for bad in (z(R - 1, 64), z(R, 72), a.float(), a.cpu(), z(R, 128)[:, ::2]):
        with pytest.raises(ValueError):
            ops.grouped_gemm_bf16(h, bad, b, out=out)
        with pytest.raises(ValueError):
            ops.grouped_gemm_mxfp4(h, bad, codes, scales, out=out)
    for bad in (z(3, 40, 64), z(4, 40 * 64), b.float(), z(4, 64, 40).transpose(1, 2)):
        with pytest.raises(ValueError):
            ops.grouped_gemm_bf16(h, a, bad, out=out)
    with pytest.raises(ValueError):
        ops.grouped_gemm_bf16(h, a, b, out=z(R, 48))
    with pytest.raises(ValueError):
        ops.grouped_gemm_bf16_grad_input(h, z(R, 48), b)
    with pytest.raises(ValueError):
        ops.grouped_gemm_bf16_grad_weight(h, g, a[:R - 1])
    with pytest.raises(ValueError):
        ops.grouped_gemm_bf16_grad_weight(h, g, a, grad_b=z(4, 40, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        ops.grouped_gemm_mxfp4(h, a, codes, scales[:, :, :1].contiguous(), out=out)
    with pytest.raises(ops.F.EPError, match="multiple of 8"):
        ops.grouped_gemm_bf16(h, a, z(4, 36, 64))
    with pytest.raises(ops.F.EPError, match="multiple of 32"):
        ops.grouped_gemm_mxfp4(h, z(R, 48), z(4, 40, 24, dtype=torch.uint8), z(4, 40, 1, dtype=torch.uint8))
    with pytest.raises(ops.F.EPError, match="16-byte"):
        ops.grouped_gemm_bf16(h, z(R * 64 + 1)[1:].view(R, 64), b, out=out)
    torch.cuda.synchronize()
    assert bool((out == 7).all())
