"""The experts' products on each of their kernels: whole tiles (8 waves, 256 x
256), half tiles and the kernel that streams the weights, which the launchers
choose by sizes alone. Every test names the kernel that it is about and fails
when another one ran, so that a change of the rules cannot move it elsewhere.

Values are held to the tolerance of test_expert_products_gpu.py's docstring; the
widest reductions to equality, on integers whose sums are exact in any order."""
import re

import numpy as np
import pytest
import torch

from ep_workloads import random_routing_table
from gpu_common import log, to_dev
from test_expert_products_gpu import call, check, decode_mxfp4, make_handle, operands, ranges, routing, verify

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_ep_layout_10_amd import ops


@pytest.fixture
def launched(monkeypatch, capfd):
    """A function that returns the launches of the products since the last call
    of it, as (kernel, the launcher's remarks)."""
    monkeypatch.setenv("EP_BUFFER_DEBUG", "1")

    def read():
        return re.findall(r"\[ep\] (k_grouped_gemm\w*) grid \d+ block \d+ (.*)", capfd.readouterr().err)

    yield read


def output(direction, h, n, k, f32=True):
    R, E = h.cfg.recv_rows_bound(), h.cfg.num_experts
    if direction == "grad_weight":
        return torch.full((E, n, k), 7.0, device="cuda", dtype=torch.float32 if f32 else torch.bfloat16)
    return torch.full((R, k if direction == "grad_input" else n), 7.0, device="cuda", dtype=torch.bfloat16)


def run_case(direction, h, n, k, launched, kernel, seed=0, remark=""):
    o = operands(direction, h, n, k, seed)
    out = output(direction, h, n, k)
    launched()
    call(direction, h, o, out)
    torch.cuda.synchronize()
    ran = launched()
    assert [r[0] for r in ran] == [kernel] and remark in ran[0][1], ran
    verify(direction, h, o, out, n, k)


def wide(direction, width, reduction):
    """n and k for an output of `width` columns."""
    return (width, reduction) if direction == "forward" else (reduction, width)


# every number of 32-row steps that a whole tile is compiled for (1 to 8), experts of one tile, two, three, and
# more than a group of the block order, empty ones first, in the middle and last
WHOLE_COUNTS = [0, 1, 15, 32, 33, 64, 65, 96, 97, 0, 128, 129, 160, 161, 192, 193, 224, 225, 255, 256, 257, 300, 513,
                1100, 2, 2306, 0]


@pytest.mark.parametrize("direction", ("forward", "grad_input"))
@pytest.mark.parametrize("A", [1, 300])
@pytest.mark.parametrize("reduction", [8, 64, 72, 136, 328, 1056])
def test_whole_tiles(direction, A, reduction, launched):
    """Whole tiles of every height and ring, reductions below, at and past the
    64 of a step, a last column tile of 8."""
    h = make_handle(routing(WHOLE_COUNTS), len(WHOLE_COUNTS), A)
    n, k = wide(direction, 2056, reduction)
    run_case(direction, h, n, k, launched, "k_grouped_gemm_bf16", seed=reduction)


@pytest.mark.parametrize("direction", ("forward", "grad_input"))
def test_whole_tiles_fixed_capacity(direction, launched):
    """FIXED: experts that overflow, rows past each count left as they were."""
    h = make_handle(random_routing_table(np.random.default_rng(9), 1500, 6, 2), 6, 1, mode=ops.MODE_FIXED, C=499)
    n, k = wide(direction, 5640, 200)
    run_case(direction, h, n, k, launched, "k_grouped_gemm_bf16")


@pytest.mark.parametrize("direction", ("forward", "grad_input"))
def test_whole_tiles_no_zero_pad_masked_and_bad_ids(direction, launched):
    idx = random_routing_table(np.random.default_rng(10), 1500, 6, 2, masked_frac=0.2, bad_frac=0.05)
    h = make_handle(idx, 6, 32, flags=ops.FLAG_NO_ZERO_PAD)
    n, k = wide(direction, 5640, 200)
    run_case(direction, h, n, k, launched, "k_grouped_gemm_bf16")


@pytest.mark.parametrize("direction", ("forward", "grad_input"))
def test_whole_tiles_infinite_and_nan_values(direction, launched):
    """Infinities and NaN reach exactly the outputs that the formula says."""
    h = make_handle(routing([300, 40, 700]), 3, 1)
    n, k = wide(direction, 11272, 136)
    o = operands(direction, h, n, k)
    x = o["g" if direction == "grad_input" else "a"]
    x[3, 5] = float("inf")
    x[301, 7] = float("-inf")
    x[340 + 511] = float("nan")
    launched()
    got = call(direction, h, o)
    torch.cuda.synchronize()
    assert [r[0] for r in launched()] == ["k_grouped_gemm_bf16"]
    for e, (first, live, _) in enumerate(o["rr"]):
        rows = slice(first, first + live)
        w = o["w64"](e)
        g, want = got[rows], x[rows].double() @ (w if direction == "grad_input" else w.t().contiguous())
        assert torch.equal(torch.isnan(g), torch.isnan(want)), e
        assert torch.equal(torch.isinf(g), torch.isinf(want)), e
        assert torch.equal(g[torch.isinf(want)].double(), want[torch.isinf(want)]), e


@pytest.mark.parametrize("direction", ("forward", "grad_input"))
def test_whole_tiles_far_rows(direction, launched):
    """Rows whose output stands past 2^32 bytes, behind a long padding that is
    cleared: experts 2^18 rows apart, 8200 columns."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    A, counts = 1 << 18, [260, 1, 40, 129, 300]
    h = make_handle(routing(counts), len(counts), A)
    n, k = wide(direction, 8200, 24)
    o = operands(direction, h, n, k)
    x = o["g" if direction == "grad_input" else "a"]
    launched()
    got = call(direction, h, o)
    torch.cuda.synchronize()
    assert [r[0] for r in launched()] == ["k_grouped_gemm_bf16"]
    for e, (first, live, owned) in enumerate(ranges(h)):
        assert first == e * A and owned == A
        w = o["w64"](e)
        check(got[first:first + live], x[first:first + live].double(), w if direction == "grad_input" else w.t(), 24, e)
        for r in range(first + live, first + owned, 1 << 15):
            end = min(r + (1 << 15), first + owned)
            assert int(torch.count_nonzero(got[r:end].view(torch.int16))) == 0, (e, r)


# ---------------------------------------------------------------- BF16 weights streamed

# rows of five experts: one each, the most that 16-row tiles take on the mean, the least and the most of 32-row
# tiles, and one expert with nearly everything (several row tiles of it)
FEW = {"one": ([1, 0, 1, 1, 2], 16), "six": ([6, 3, 9, 0, 12], 16), "seven": ([0, 7, 16, 1, 11], 32),
       "sixteen": ([16, 31, 1, 0, 32], 32), "hot16": ([0, 28, 0, 1, 0], 16), "hot32": ([0, 0, 79, 0, 1], 32)}
# n, k and the parts the reduction is split in; k ends inside a slice (512 or 1024) and off every chunk of 128
SPLITS = [(72, 4104, 8), (1416, 4104, 4), (264, 2088, 4), (2600, 1032, 2), (40, 1032, 2), (5200, 1032, 1), (264, 8, 1),
          (1000, 520, 1)]


@pytest.mark.parametrize("rows", sorted(FEW))
@pytest.mark.parametrize("n,k,split", SPLITS)
def test_streamed_weights(rows, n, k, split, launched):
    counts, tile = FEW[rows]
    h = make_handle(routing(counts), 5, 4)
    run_case("forward", h, n, k, launched, "k_grouped_gemm_stream", seed=n + k,
             remark="rows %d split %d n %d k %d" % (tile, split, n, k))


def test_streamed_weights_fixed_capacity(launched):
    """FIXED: experts that overflow; rows past each count left as they were."""
    h = make_handle(random_routing_table(np.random.default_rng(9), 40, 6, 2), 6, 1, mode=ops.MODE_FIXED, C=11)
    run_case("forward", h, 520, 1096, launched, "k_grouped_gemm_stream", remark="rows 32 split 2")


def test_streamed_weights_infinite_and_nan_values(launched):
    h = make_handle(routing([6, 14, 2]), 3, 1)
    o = operands("forward", h, 72, 2088)
    o["a"][2, 2087] = float("inf")
    o["a"][7] = float("nan")
    o["b"][2, 5, 1000] = float("nan")
    launched()
    got = call("forward", h, o)
    torch.cuda.synchronize()
    assert [r[0] for r in launched()] == ["k_grouped_gemm_stream"]
    for e, (first, live, _) in enumerate(o["rr"]):
        rows = slice(first, first + live)
        want = o["a"][rows].double() @ o["w64"](e).t().contiguous()
        assert torch.equal(torch.isnan(got[rows]), torch.isnan(want)), e
        assert torch.equal(torch.isinf(got[rows]), torch.isinf(want)), e
        assert torch.equal(got[rows][torch.isinf(want)].double(), want[torch.isinf(want)]), e


# ---------------------------------------------------------------- the widest reductions, exactly

@pytest.mark.parametrize("direction", ("forward", "grad_input", "mxfp4"))
@pytest.mark.parametrize("counts", [[1, 0, 2], [9, 40, 2]])
def test_widest_exact(direction, counts, launched):
    """Reductions of 2^20, the widest that are accepted. Operands are -1, 0 and 1
    (4-bit weights: every code, in halves up to 6), so every partial sum is a
    multiple of 1/2 of at most 6 * 2^20 < 2^23: exact in binary32 in any order.
    The outputs are the exact sums rounded to bf16, bit for bit."""
    W = 1 << 20
    h = make_handle(routing(counts), 3, 1)
    n, k = (W, 32) if direction == "grad_input" else (8, W)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(sum(counts))
    R, rr = h.cfg.recv_rows_bound(), ranges(h)
    ints = lambda *shape: torch.randint(-1, 2, shape, device="cuda", generator=gen).to(torch.bfloat16)
    o = dict(rr=rr)
    x = o["g" if direction == "grad_input" else "a"] = ints(R, W)
    if direction == "mxfp4":
        o["b"] = torch.randint(0, 256, (3, n, k // 2), dtype=torch.uint8, device="cuda", generator=gen)
        o["s"] = torch.full((3, n, k // 32), 127, dtype=torch.uint8, device="cuda")
        w64 = lambda e: decode_mxfp4(o["b"][e], o["s"][e])
    else:
        o["b"] = ints(3, n, k)
        w64 = lambda e: o["b"][e].double()
    launched()
    out = output(direction, h, n, k)
    got = call(direction, h, o, out)
    torch.cuda.synchronize()
    log("%s %s: %s" % (direction, counts, launched()))
    for e, (first, live, _) in enumerate(rr):
        if live == 0:
            continue
        rows, w = slice(first, first + live), w64(e)
        want = x[rows].double() @ (w if direction == "grad_input" else w.t().contiguous())
        assert float(want.abs().max()) > 256.0     # sums that the output's rounding has to round
        assert torch.equal(got[rows], want.to(torch.bfloat16)), e


# ---------------------------------------------------------------- the same bits: again, captured, on two streams

# direction, tokens, experts, top-k, n, k, kernel, the launcher's remark
KERNELS = {
    "whole forward": ("forward", 600, 6, 2, 5640, 200, "k_grouped_gemm_bf16", ""),
    "whole grad_input": ("grad_input", 600, 6, 2, 200, 5640, "k_grouped_gemm_bf16", ""),
    "half forward": ("forward", 600, 6, 2, 520, 544, "k_grouped_gemm_bf16_half", ""),
    "bf16 16 rows split 8": ("forward", 12, 8, 2, 264, 4104, "k_grouped_gemm_stream", "rows 16 split 8"),
    "bf16 16 rows split 4": ("forward", 12, 8, 2, 1032, 2088, "k_grouped_gemm_stream", "rows 16 split 4"),
    "bf16 16 rows split 2": ("forward", 12, 8, 2, 2056, 1032, "k_grouped_gemm_stream", "rows 16 split 2"),
    "bf16 32 rows split 8": ("forward", 40, 8, 2, 264, 4104, "k_grouped_gemm_stream", "rows 32 split 8"),
    "bf16 32 rows split 4": ("forward", 40, 8, 2, 1032, 2088, "k_grouped_gemm_stream", "rows 32 split 4"),
    "bf16 32 rows split 2": ("forward", 40, 8, 2, 2056, 1032, "k_grouped_gemm_stream", "rows 32 split 2"),
    "bf16 32 rows split 1": ("forward", 40, 8, 2, 4104, 136, "k_grouped_gemm_stream", "rows 32 split 1"),
    "mxfp4 16 rows split 8": ("mxfp4", 12, 8, 2, 264, 4128, "k_grouped_gemm_stream", "rows 16 split 8"),
    "mxfp4 16 rows split 4": ("mxfp4", 12, 8, 2, 1032, 2080, "k_grouped_gemm_stream", "rows 16 split 4"),
    "mxfp4 32 rows split 2": ("mxfp4", 40, 8, 2, 2056, 1056, "k_grouped_gemm_stream", "rows 32 split 2"),
    "mxfp4 32 rows split 1": ("mxfp4", 40, 8, 2, 4104, 160, "k_grouped_gemm_stream", "rows 32 split 1"),
    "mxfp4 64 rows": ("mxfp4", 300, 8, 2, 520, 544, "k_grouped_gemm_stream", "rows 64 split 1"),
}


def live_rows(o):
    return torch.cat([torch.arange(f, f + l) for f, l, _ in o["rr"]]).cuda()


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_same_bits_again(name, launched):
    """A second call, with other work on the card between, gives the same bits."""
    direction, T, E, top, n, k, kernel, remark = KERNELS[name]
    h = make_handle(random_routing_table(np.random.default_rng(13), T, E, top), E)
    o = operands(direction, h, n, k)
    launched()
    first = call(direction, h, o, output(direction, h, n, k))
    for _ in range(2):
        torch.randn((1 << 24,), device="cuda").sort()
        assert torch.equal(call(direction, h, o, output(direction, h, n, k)), first)
    torch.cuda.synchronize()
    ran = launched()
    assert len(ran) == 3 and all(r[0] == kernel and remark in r[1] for r in ran), ran
    verify(direction, h, o, first, n, k)


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_graph_replay(name, launched):
    """Captured once with its layout and replayed on new routing and operands,
    with eager calls between the replays."""
    direction, T, E, top, n, k, kernel, remark = KERNELS[name]
    rng = np.random.default_rng(15)
    h = make_handle(random_routing_table(rng, T, E, top), E, 16)
    idx = h.topk_idx
    o = operands(direction, h, n, k)
    out = output(direction, h, n, k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(direction, h, o, out)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    launched()
    with torch.cuda.graph(graph):
        h2 = ops.layout(h.cfg, idx, workspace=h.workspace)
        call(direction, h2, o, out)
    ran = launched()
    assert [r[0] for r in ran] == [kernel] and remark in ran[0][1], ran
    for rep in range(3):
        idx.copy_(to_dev(random_routing_table(rng, T, E, top)))
        he = ops.layout(h.cfg, idx)
        new = operands(direction, he, n, k, seed=rep)
        for key in ("a", "g", "b", "s"):
            if key in o:
                o[key].copy_(new[key])
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        eager = output(direction, he, n, k)
        call(direction, he, new, eager)
        assert torch.equal(out, eager), rep
        verify(direction, he, new, out, n, k)


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_two_streams_at_once(name):
    """Two calls on two streams share nothing."""
    direction, T, E, top, n, k, _, _ = KERNELS[name]
    rng = np.random.default_rng(16)
    hs = [make_handle(random_routing_table(rng, T, E, top), E) for _ in range(2)]
    os_ = [operands(direction, h, n, k, seed=i) for i, h in enumerate(hs)]
    want = [call(direction, h, o) for h, o in zip(hs, os_)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for s, h, o in zip(streams, hs, os_):
        with torch.cuda.stream(s):
            got.append([call(direction, h, o) for _ in range(4)])
    torch.cuda.synchronize()
    for w, g, o in zip(want, got, os_):
        rows = live_rows(o)
        for x in g:
            assert torch.equal(x[rows], w[rows])
