"""MXFP4 quantisation and the experts' products with both operands in MXFP4.

Quantisation is exact by definition (powers of two divide exactly, one rounding to
a code), so codes, scales and values are compared bit by bit.

Products, most tests: codes under scales of 2^-2 .. 2^2, so products are multiples
of 2^-6 and sum |a b| stays below 2^18 (asserted): every term and partial sum, in any
order, is below 2^18 and so has a leading bit of 2^17 at most, 23 places above 2^-6, and is
a binary32 number; the matrix unit cuts off only what lies further below the largest
term, so nothing, and the result is the exact sum rounded to bf16, bit for bit.

With scales far apart: one matrix instruction cuts each of its 128 products and its
running sum off at 2^-23 of the largest of them, none of which exceeds
S = sum |a b|, so ceil(K / 128) instructions (and the sum of up to 8 parts) are off by at most
(129 ceil(K / 128) + 8) 2^-23 S; the bf16 output adds 2^-8 of its value."""
import os

import numpy as np
import pytest
import torch

import mxfp4_reference as ref
from ep_workloads import random_routing_table
from gpu_common import to_dev
from test_expert_products_gpu import decode_mxfp4, make_handle, ranges, routing

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_ep_layout_10_amd import ops


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------- quantisation

def check_quantize(x, values=True):
    out = torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") if values else None
    codes, scales = ops.quantize_mxfp4(x, values=out)
    want_codes, want_scales, want_values = ref.quantize(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_scales)
    assert np.array_equal(codes.cpu().numpy(), want_codes)
    if values:
        got = out.double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want_values))
        fine = ~np.isnan(want_values)
        assert np.array_equal(got[fine], want_values[fine]) and np.array_equal(np.signbit(got[fine]), np.signbit(want_values[fine]))
    return codes, scales


def test_every_bf16_value():
    """Each of the 65,536 bf16 bit patterns as the largest of its 32, and beside 1.0, 3.5 and 448."""
    bits = torch.arange(65536, device="cuda").int() << 16
    v = bits.view(torch.float32).to(torch.bfloat16)
    g = gen(0)
    share = (torch.rand((65536, 31), generator=g, device="cuda") * 2 - 1)
    check_quantize(torch.cat([v[:, None], (v[:, None].float() * share).to(torch.bfloat16)], 1))
    for other in (1.0, 3.5, 448.0):
        x = v.view(-1, 16).repeat(1, 2)
        x[:, 16:] = other
        check_quantize(x)


@pytest.mark.parametrize("f32", [True, False])
def test_ties_and_borders(f32):
    """Values at, just below and just above every place where a code, or the scale, changes, at
    many magnitudes: subnormal ones, zeros of either sign, the largest."""
    places = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0, 7.99], device="cuda").double()
    rows = []
    for e in list(range(-149 if f32 else -133, -120)) + [-60, -3, 0, 1, 40, 100, 124, 125]:
        for top in (4.0, 5.0, 6.0, 7.0):
            p = places * 2.0 ** e
            near = torch.cat([p, -p])[:31]
            for tilt in (0.0, 2.0 ** -23, -2.0 ** -23, 2.0 ** -8, -2.0 ** -8):
                rows.append(torch.cat([torch.tensor([top * 2.0 ** e], device="cuda").double(), near * (1 + tilt)]))
    x = torch.stack(rows)
    x = x.float() if f32 else x.float().to(torch.bfloat16)
    check_quantize(x)
    check_quantize(-x)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("shape", [(1, 32), (3, 32), (1, 64), (7, 96), (5, 1440), (33, 2048), (2, 5, 7168), (1000, 32), (32,), (1, 1 << 20)])
def test_shapes(shape, f32):
    x = torch.randn(shape, generator=gen(sum(shape)), device="cuda") * 3
    x = x if f32 else x.to(torch.bfloat16)
    codes, scales = check_quantize(x)
    assert codes.shape == shape[:-1] + (shape[-1] // 2,) and scales.shape == shape[:-1] + (shape[-1] // 32,)
    check_quantize(x, values=False)


def test_nan_and_infinity():
    x = torch.randn((6, 96), generator=gen(1), device="cuda")
    x[0, 3], x[1, 40], x[2, 95], x[3, 0] = float("nan"), float("inf"), -float("inf"), -float("nan")
    x[4, 32:64] = float("nan")
    for t in (x, x.to(torch.bfloat16)):
        _, scales = check_quantize(t)
        assert (scales == 255).sum() == 5


def test_no_rows():
    codes, scales = ops.quantize_mxfp4(torch.empty((0, 64), device="cuda"))
    assert codes.shape == (0, 32) and scales.shape == (0, 2)
    h = make_handle(np.zeros((0, 1), np.int64), 4, max_tokens=8)
    codes, scales = ops.quantize_mxfp4(torch.full((8, 64), float("nan"), device="cuda"), h, codes=torch.full((8, 32), 9, dtype=torch.uint8, device="cuda"))
    assert (codes == 9).all()


def test_values_over_the_input():
    x = torch.randn((300, 1024), generator=gen(2), device="cuda").to(torch.bfloat16)
    _, _, want = ref.quantize(x.double().cpu().numpy())
    ops.quantize_mxfp4(x, values=x)
    assert np.array_equal(x.double().cpu().numpy(), want)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("mode,A,C", [("compact", 1, 0), ("compact", 128, 0), ("fixed", 1, 40), ("fixed", 1, 3), ("unpadded", 64, 0)])
def test_live_rows_only(mode, A, C, f32):
    """With a handle: rows of pairs, and no other byte."""
    h = make_handle(routing([0, 5, 130, 1, 39, 40, 0]), 7, A, ops.MODE_FIXED if mode == "fixed" else ops.MODE_COMPACT, C,
                    flags=ops.FLAG_NO_ZERO_PAD if mode == "unpadded" else 0)
    R = h.cfg.recv_rows_bound()
    for k in (32, 96, 7168):
        x = torch.randn((R, k), generator=gen(k), device="cuda")
        x = x if f32 else x.to(torch.bfloat16)
        live = torch.zeros(R, dtype=torch.bool, device="cuda")
        for first, n, _ in ranges(h):
            live[first:first + n] = True
        x[~live] = float("nan")
        codes = torch.full((R, k // 2), 9, dtype=torch.uint8, device="cuda")
        scales = torch.full((R, k // 32), 9, dtype=torch.uint8, device="cuda")
        values = torch.full((R, k), 9.0, dtype=torch.bfloat16, device="cuda")
        ops.quantize_mxfp4(x, h, codes, scales, values)
        wc, ws, wv = ref.quantize(x[live].double().cpu().numpy())
        assert np.array_equal(codes[live].cpu().numpy(), wc) and np.array_equal(scales[live].cpu().numpy(), ws)
        assert np.array_equal(values[live].double().cpu().numpy(), wv)
        assert (codes[~live] == 9).all() and (scales[~live] == 9).all() and (values[~live] == 9).all()


def test_far_offsets_of_rows():
    """More than 2^32 bytes of input and of values."""
    rows, k = 300_000, 8192
    x = torch.zeros((rows, k), dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.randn(k, generator=gen(3), device="cuda").to(torch.bfloat16)
    values = torch.empty_like(x)
    codes, scales = ops.quantize_mxfp4(x, values=values)
    wc, ws, wv = ref.quantize(x[-1:].double().cpu().numpy())
    assert np.array_equal(codes[-1:].cpu().numpy(), wc) and np.array_equal(scales[-1:].cpu().numpy(), ws)
    assert np.array_equal(values[-1:].double().cpu().numpy(), wv)
    assert not codes[:-1].any() and not scales[:-1].any()


# ---------------------------------------------------------------- products

def operands(h, n, k, seed=0, low=125, high=129):
    """Codes and scales; NaN scales wherever the contract says nothing is read."""
    g = gen(seed)
    R, E = h.cfg.recv_rows_bound(), h.cfg.num_experts
    rr = ranges(h)
    byte = lambda lo, hi, *shape: torch.randint(lo, hi, shape, dtype=torch.uint8, device="cuda", generator=g)
    o = dict(rr=rr, a=byte(0, 256, R, k // 2), s=byte(low, high + 1, R, k // 32), b=byte(0, 256, E, n, k // 2),
             t=byte(low, high + 1, E, n, k // 32))
    live = torch.zeros(R, dtype=torch.bool, device="cuda")
    for e, (first, rows, _) in enumerate(rr):
        live[first:first + rows] = True
        if rows == 0:
            o["t"][e] = 255
    o["s"][~live] = 255
    return o


def call(h, o, out=None):
    return ops.grouped_gemm_mxfp4_rows(h, o["a"], o["s"], o["b"], o["t"], out=out)


def verify(h, o, got, exact=True, fill=7.0):
    """Every expert's values, zeros on padding, everything else untouched (got was filled before the call)."""
    touched = torch.zeros(got.shape[0], dtype=torch.bool, device="cuda")
    K = 2 * o["a"].shape[1]
    for e, (first, live, owned) in enumerate(o["rr"]):
        rows = slice(first, first + live)
        if live:
            x, w = decode_mxfp4(o["a"][rows], o["s"][rows]), decode_mxfp4(o["b"][e], o["t"][e])
            want, size = x @ w.t(), x.abs() @ w.abs().t()
            if exact:
                assert float(size.max()) < 2.0 ** 18
                bad = got[rows] != want.to(torch.bfloat16)
                assert not bool(bad.any()), (e, bad.nonzero()[:4].tolist(), int(bad.sum()))
            else:
                acc = (129 * -(-K // 128) + 8) * 2.0 ** -23 * size
                err = (got[rows].double() - want).abs()
                assert bool((err <= acc + 2.0 ** -8 * (want.abs() + acc)).all()), e
        touched[rows] = True
        if h.cfg.mode == ops.MODE_COMPACT and not h.cfg.flags & ops.FLAG_NO_ZERO_PAD:
            assert not got[first + live:first + owned].any(), e
            touched[first + live:first + owned] = True
    assert bool((got[~touched] == fill).all())


def run_case(h, n, k, seed=0, **kw):
    o = operands(h, n, k, seed, **kw)
    out = torch.full((h.cfg.recv_rows_bound(), n), 7.0, dtype=torch.bfloat16, device="cuda")
    assert call(h, o, out).data_ptr() == out.data_ptr()
    verify(h, o, out, exact=not kw)
    return o, out


EVERY = [0, 1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 96, 127, 128, 129, 191, 192, 193, 255, 256, 257, 320, 511,
         513]


@pytest.mark.parametrize("A", [1, 16, 300])
def test_every_count(A):
    for k in (544, 640):
        run_case(make_handle(routing(EVERY), len(EVERY), A), 264, k)


def kernels(capfd, h, o, out):
    """The kernels that a call launches, as the library says."""
    os.environ["EP_BUFFER_DEBUG"] = "1"
    try:
        capfd.readouterr()
        call(h, o, out)
        return [l.split()[1] for l in capfd.readouterr().err.splitlines() if l.startswith("[ep]")]
    finally:
        os.environ.pop("EP_BUFFER_DEBUG", None)


def run_whole(capfd, h, n, k, seed=0, **kw):
    """A case that whole tiles take."""
    o, out = run_case(h, n, k, seed, **kw)
    assert kernels(capfd, h, o, out) == ["k_grouped_gemm_fp4"]
    return o, out


@pytest.mark.parametrize("A", [1, 16, 300])
@pytest.mark.parametrize("k", [128, 640, 1024])
def test_whole_tiles_every_count(capfd, A, k):
    run_whole(capfd, make_handle(routing(EVERY), len(EVERY), A), 1032, k)


@pytest.mark.parametrize("n,k", [(1032, 256), (1040, 384), (1024, 512), (1272, 896), (1280, 1152), (1032, 1408), (1536, 1664),
                                 (1032, 2048), (1032, 3200), (2056, 7168)])
def test_whole_tiles_sizes(capfd, n, k):
    """Reductions that end anywhere in a step and in a slab of scales; widths off the tile."""
    counts = [0, 5, 100, 64, 300, 1, 700, 2] * 3
    run_whole(capfd, make_handle(routing(counts), len(counts), 1), n, k, seed=n + k)


def test_whole_tiles_fixed_capacity_and_no_zero_pad(capfd):
    counts = [0, 5, 130, 1, 39, 40, 700, 256] * 4
    for C in (3, 40, 160, 600):
        run_whole(capfd, make_handle(routing(counts), len(counts), 1, ops.MODE_FIXED, C), 1032, 640)
    run_whole(capfd, make_handle(routing(counts), len(counts), 64, flags=ops.FLAG_NO_ZERO_PAD), 1032, 640)


@pytest.mark.parametrize("k", [128, 384, 1152, 2048, 160, 416, 1184, 2080, 448])
def test_whole_tiles_nan_scales(capfd, k):
    """A row's NaN scales stay out of the rows before and behind it, though its last slab's loads run on into the next row."""
    counts = [70, 3, 260, 64] * 8
    h = make_handle(routing(counts), len(counts), 1)
    o = operands(h, 1032, k, seed=k)
    for first, live, _ in o["rr"]:
        o["s"][first + 1, 0] = 255
        o["s"][first + 2, k // 32 - 1] = 255
    o["t"][:, 1, 0] = 255
    o["t"][:, 1029, k // 32 - 1] = 255
    o["t"][:, 1031, k // 64] = 255
    out = torch.full((h.cfg.recv_rows_bound(), 1032), 7.0, dtype=torch.bfloat16, device="cuda")
    assert kernels(capfd, h, o, out) == ["k_grouped_gemm_fp4"]
    for e, (f, n, _) in enumerate(o["rr"]):
        x, w = decode_mxfp4(o["a"][f:f + n], o["s"][f:f + n]), decode_mxfp4(o["b"][e], o["t"][e])
        rows, cols = (o["s"][f:f + n] == 255).any(1), (o["t"][e] == 255).any(1)
        nan = rows[:, None] | cols[None, :]
        assert torch.equal(torch.isnan(out[f:f + n]), nan), e
        x[rows], w[cols] = 0, 0
        assert torch.equal(out[f:f + n][~nan], (x @ w.t()).to(torch.bfloat16)[~nan]), e


def run_odd_whole(capfd, h, n, k, seed=0):
    """A case that whole tiles take whose rows of scales are no whole words."""
    o, out = run_whole(capfd, h, n, k, seed)
    os.environ["EP_BUFFER_DEBUG"] = "1"
    try:
        capfd.readouterr()
        call(h, o, out)
        assert "words 0" in capfd.readouterr().err
    finally:
        os.environ.pop("EP_BUFFER_DEBUG", None)


@pytest.mark.parametrize("A", [1, 16, 300])
@pytest.mark.parametrize("k", [160, 416, 992, 1440])
def test_whole_tiles_of_odd_scales_every_count(capfd, A, k):
    run_odd_whole(capfd, make_handle(routing(EVERY), len(EVERY), A), 1032, k)


@pytest.mark.parametrize("n,k", [(1032, 160), (1040, 192), (1024, 224), (1272, 288), (1280, 480), (1032, 544), (1536, 736),
                                 (1032, 1056), (1160, 1504), (1032, 1696), (1296, 2016), (1032, 3232), (2056, 7200)])
def test_whole_tiles_of_odd_scales_sizes(capfd, n, k):
    """Rows of scales that start at any byte of a word, by any number of groups past a step's
    eight and a slab's 24; tiles whose last rows and columns end at any byte."""
    counts = [0, 5, 100, 64, 300, 1, 701, 2] * 3
    run_odd_whole(capfd, make_handle(routing(counts), len(counts), 1), n, k, seed=n + k)


def test_whole_tiles_of_odd_scales_fixed_capacity(capfd):
    counts = [0, 5, 130, 1, 39, 40, 700, 256] * 4
    for C in (3, 41, 162, 600):
        run_odd_whole(capfd, make_handle(routing(counts), len(counts), 1, ops.MODE_FIXED, C), 1032, 672)
    run_odd_whole(capfd, make_handle(routing(counts), len(counts), 64, flags=ops.FLAG_NO_ZERO_PAD), 1032, 672)


def test_whole_tiles_far_offsets(capfd):
    """Codes past 2^32 bytes, under whole tiles."""
    E, n, k = 160, 8192, 8192
    rows = {0: 300, E - 2: 320, E - 1: 380}
    h = make_handle(np.concatenate([np.full((c, 1), e, np.int64) for e, c in rows.items()]), E)
    g = gen(2)
    b = torch.zeros((E, n, k // 2), dtype=torch.uint8, device="cuda")
    t = torch.zeros((E, n, k // 32), dtype=torch.uint8, device="cuda")
    for e in rows:
        b[e], t[e] = ops.quantize_mxfp4(torch.randn((n, k), generator=g, device="cuda"))
    a, s = ops.quantize_mxfp4(torch.randn((1000, k), generator=g, device="cuda"))
    o = dict(a=a, s=s, b=b, t=t)
    out = torch.empty((1000, n), dtype=torch.bfloat16, device="cuda")
    assert kernels(capfd, h, o, out) == ["k_grouped_gemm_fp4"]
    for e, (first, live, _) in enumerate(ranges(h)):
        if live:
            x, w = decode_mxfp4(a[first:first + live], s[first:first + live]), decode_mxfp4(b[e], t[e])
            want, acc = x @ w.t(), (129 * (k // 128) + 8) * 2.0 ** -23 * (x.abs() @ w.abs().t())
            assert bool(((out[first:first + live].double() - want).abs() <= acc + 2.0 ** -8 * (want.abs() + acc)).all()), e


@pytest.mark.parametrize("counts,n,k,want", [([1], 72, 4096, "rows 16 split 8"), ([2, 3], 4104, 4096, "rows 16 split 4"),
                                             ([3] * 8, 1536, 2080, "rows 16 split 2"), ([5] * 16, 1600, 1024, "rows 16 split 1"),
                                             ([40, 7], 520, 2080, "rows 64 split 2"), ([100, 9] * 4, 1600, 1440, "rows 64 split 1")])
def test_streamed_splits(capfd, counts, n, k, want):
    """Each tile height and split of the kernel that streams the weights."""
    h = make_handle(routing(counts), len(counts), 1)
    o, out = run_case(h, n, k)
    os.environ["EP_BUFFER_DEBUG"] = "1"
    try:
        capfd.readouterr()
        call(h, o, out)
        assert want in capfd.readouterr().err
    finally:
        os.environ.pop("EP_BUFFER_DEBUG", None)


@pytest.mark.parametrize("n,k", [(8, 32), (16, 64), (24, 96), (8, 1056), (1000, 32), (248, 160), (256, 256), (264, 224),
                                 (1000, 1440), (504, 2048), (520, 4128), (72, 7168), (136, 128), (264, 384), (264, 1152), (264, 1664)])
def test_sizes(n, k):
    for counts in ([3, 0, 1], [30, 5, 17], [100, 0, 64, 1], [300, 700, 2]):
        run_case(make_handle(routing(counts), len(counts), 1), n, k, seed=n + k)


@pytest.mark.parametrize("rows", [1, 5, 20, 40])
@pytest.mark.parametrize("n,k", [(72, 4128), (520, 2080), (1000, 1056), (2056, 1024), (264, 8192), (4096, 7168)])
def test_long_reductions(rows, n, k):
    """Split reductions, slices that end anywhere, scales at an odd address."""
    h = make_handle(routing([rows, 0, rows + 2, 1, 3 * rows]), 5, 1)
    o = operands(h, n, k, seed=rows + k)
    for name in ("s", "t"):
        odd = torch.empty(o[name].numel() + 1, dtype=torch.uint8, device="cuda")[1:].view(o[name].shape)
        o[name] = odd.copy_(o[name])
    out = torch.full((h.cfg.recv_rows_bound(), n), 7.0, dtype=torch.bfloat16, device="cuda")
    verify(h, o, call(h, o, out))


@pytest.mark.parametrize("counts", [[1, 0, 3], [20, 9, 30], [70, 1, 300], [600, 900, 10]])
@pytest.mark.parametrize("k", [96, 1024, 1440, 7168])
def test_scales_far_apart(counts, k):
    run_case(make_handle(routing(counts), 3, 1), 264, k, low=90, high=160)


def test_one_token_and_no_rows():
    run_case(make_handle(np.array([[5, 2, 7]], np.int64), 8, 1), 520, 1024)
    run_case(make_handle(np.full((3, 2), -1, np.int64), 4, 16), 64, 64)
    run_case(make_handle(np.zeros((0, 1), np.int64), 4, max_tokens=9), 64, 64)


def test_many_experts():
    rng = np.random.default_rng(5)
    run_case(make_handle(random_routing_table(rng, 700, 1024, 2), 1024, 4), 72, 96)


@pytest.mark.parametrize("T", [40, 400, 3000])
def test_duplicate_experts_and_hot_expert(T):
    idx = np.zeros((T, 2), np.int64)
    idx[::7, 1] = 3
    run_case(make_handle(idx, 5, 16), 264, 544)
    run_case(make_handle(idx, 5, 16), 520, 1024)


@pytest.mark.parametrize("C", [3, 40, 160, 600])
def test_fixed_capacity(C):
    h = make_handle(routing([0, 5, 130, 1, 39, 40, 700]), 7, 1, ops.MODE_FIXED, C)
    run_case(h, 264, 544)
    run_case(h, 264, 1024)


def test_no_zero_pad():
    for counts in ([5, 30, 2], [500, 30, 300]):
        run_case(make_handle(routing(counts), 3, 64, flags=ops.FLAG_NO_ZERO_PAD), 264, 1024)


@pytest.mark.parametrize("counts", [[2, 3], [10, 20], [60, 30], [300, 600]])
@pytest.mark.parametrize("k", [160, 640, 1440, 2048])
def test_nan_scales(counts, k):
    """A NaN scale of a row, or of a weight column, reaches its own row or column only, whichever of its groups it is."""
    h = make_handle(routing(counts), 2, 1)
    for group in (0, k // 64, k // 32 - 1):
        o = operands(h, 264, k, seed=group)
        first, live, _ = o["rr"][1]
        o["s"][first + 1, group] = 255
        o["t"][0, 261, group] = 255
        out = call(h, o)
        for e, (f, n, _) in enumerate(o["rr"]):
            x, w = decode_mxfp4(o["a"][f:f + n], o["s"][f:f + n]), decode_mxfp4(o["b"][e], o["t"][e])
            nan = (o["s"][f:f + n] == 255).any(1)[:, None] | (o["t"][e] == 255).any(1)[None, :]
            assert torch.equal(torch.isnan(out[f:f + n]), nan), (e, group)
            x[(o["s"][f:f + n] == 255).any(1)] = 0
            w[(o["t"][e] == 255).any(1)] = 0
            assert torch.equal(out[f:f + n][~nan], (x @ w.t()).to(torch.bfloat16)[~nan]), (e, group)


def test_extreme_scales():
    """Scales of 2^-127 and 2^127 meet: their product, exactly."""
    h = make_handle(np.zeros((2, 1), np.int64), 1)
    for k in (32, 1024):
        o = operands(h, 64, k)
        o["a"][:], o["b"][:] = 0x22, 0x42              # all 1; 2 and 1 in turn
        o["s"][0], o["s"][1] = 0, 254
        o["t"][0] = torch.arange(64, device="cuda").to(torch.uint8)[:, None] + 100
        want = k * 1.5 * torch.exp2(o["s"][:, :1].double() - 127 + o["t"][0, :, 0].double()[None] - 127)
        got = call(h, o)[:2].double()
        fine = (want >= 2.0 ** -126) & (want < 2.0 ** 127)
        assert torch.equal(got[fine], want[fine])
        assert bool(torch.isinf(got[want >= 2.0 ** 128]).all()) and bool((got[want < 2.0 ** -134] == 0).all())


def test_same_bits_again_and_two_streams():
    rng = np.random.default_rng(16)
    for T, k in ((30, 4096), (700, 544), (3000, 1024)):
        hs = [make_handle(random_routing_table(rng, T, 6, 2), 6, 1) for _ in range(2)]
        os_ = [operands(h, 520, k, seed=i, low=100, high=150) for i, h in enumerate(hs)]
        live = [torch.cat([torch.arange(f, f + l) for f, l, _ in o["rr"]]).cuda() for o in os_]
        want = [call(h, o)[l] for h, o, l in zip(hs, os_, live)]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        got = []
        for s, h, o in zip(streams, hs, os_):
            with torch.cuda.stream(s):
                got.append([call(h, o) for _ in range(4)])
        torch.cuda.synchronize()
        for w, g, l in zip(want, got, live):
            assert all(torch.equal(x[l], w) for x in g)


@pytest.mark.parametrize("T", [20, 300, 2500])
def test_graph_replay(T):
    """Quantisation and product captured once, replayed on new rows and routing, with eager calls between."""
    rng = np.random.default_rng(15)
    E, n, k = 6, 264, 1024
    idx = to_dev(random_routing_table(rng, T, E, 2))
    cfg = ops.Config(max_tokens=T, hidden=8, num_experts=E, num_topk=2, expert_alignment=16)
    R = cfg.recv_rows_bound()
    g = gen(4)
    x = torch.randn((R, k), generator=g, device="cuda").to(torch.bfloat16)
    b, t = ops.quantize_mxfp4(torch.randn((E, n, k), generator=g, device="cuda"))

    def step():
        h = ops.layout(cfg, idx)
        a, s = ops.quantize_mxfp4(x, h)
        return h, ops.grouped_gemm_mxfp4_rows(h, a, s, b, t)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, held = step()
    for i in range(3):
        idx.copy_(to_dev(random_routing_table(rng, T, E, 2)))
        x.copy_(torch.randn((R, k), generator=g, device="cuda").to(torch.bfloat16))
        graph.replay()
        h, want = step()
        torch.cuda.synchronize()
        live = torch.cat([torch.arange(f, f + l) for f, l, _ in ranges(h)]).cuda()
        assert torch.equal(held[live], want[live]), i


def test_widest():
    """The widest rows of either side that are accepted."""
    W = 1 << 20
    for counts in ([1, 0, 2], [30, 0, 40]):
        h = make_handle(routing(counts), 3, 1)
        for n, k in ((8, W), (W, 32)):
            o = operands(h, n, k, low=126, high=127)
            out = torch.full((h.cfg.recv_rows_bound(), n), 7.0, dtype=torch.bfloat16, device="cuda")
            call(h, o, out)
            for e, (f, l, _) in enumerate(o["rr"]):
                if l:
                    x, w = decode_mxfp4(o["a"][f:f + l], o["s"][f:f + l]), decode_mxfp4(o["b"][e], o["t"][e])
                    want = x @ w.t()
                    if k == W:  # partial sums may pass what is exact: terms cut at 2^-23 of a partial sum of at most S
                        S = x.abs() @ w.abs().t()
                        err = (out[f:f + l].double() - want).abs()
                        assert bool((err <= 129 * (W // 128) * 2.0 ** -23 * S + 2.0 ** -8 * want.abs()).all())
                    else:
                        assert torch.equal(out[f:f + l], want.to(torch.bfloat16))


def test_far_offsets():
    """Weights and outputs past 2^32 bytes: the last experts of a wide stack."""
    E, n, k = 160, 8192, 8192                      # 5.7 GB of codes
    h = make_handle(np.array([[0], [E - 2], [E - 1], [E - 1]], np.int64), E)
    g = gen(2)
    b = torch.zeros((E, n, k // 2), dtype=torch.uint8, device="cuda")
    t = torch.zeros((E, n, k // 32), dtype=torch.uint8, device="cuda")
    for e in (0, E - 2, E - 1):
        b[e], t[e] = ops.quantize_mxfp4(torch.randn((n, k), generator=g, device="cuda"))
    a, s = ops.quantize_mxfp4(torch.randn((4, k), generator=g, device="cuda"))
    out = ops.grouped_gemm_mxfp4_rows(h, a, s, b, t)
    for e, rows in ((0, slice(0, 1)), (E - 2, slice(1, 2)), (E - 1, slice(2, 4))):
        x, w = decode_mxfp4(a[rows], s[rows]), decode_mxfp4(b[e], t[e])
        want, acc = x @ w.t(), (129 * (k // 128) + 8) * 2.0 ** -23 * (x.abs() @ w.abs().t())
        assert bool(((out[rows].double() - want).abs() <= acc + 2.0 ** -8 * (want.abs() + acc)).all()), e


def test_against_the_product_with_bf16_rows():
    """Where rows are MXFP4 values already, grouped_gemm_mxfp4 on those values is the same product."""
    h = make_handle(routing([40, 3, 90]), 3, 1)
    o = operands(h, 264, 544)
    for first, live, _ in o["rr"]:
        o["s"][first:first + live] = 127
    values = decode_mxfp4(o["a"], o["s"].clamp(max=127)).to(torch.bfloat16)
    got, want = call(h, o), ops.grouped_gemm_mxfp4(h, values, o["b"], o["t"])
    for first, live, _ in o["rr"]:
        assert torch.equal(got[first:first + live], want[first:first + live])


def test_refused_tensors():
    h = make_handle(routing([3, 4]), 2, 1)
    o = operands(h, 64, 96)
    with pytest.raises(ValueError, match="a_scales"):
        ops.grouped_gemm_mxfp4_rows(h, o["a"], o["t"], o["b"], o["t"])
    with pytest.raises(ValueError, match="a has shape"):
        ops.grouped_gemm_mxfp4_rows(h, o["a"][:, :32].contiguous(), o["s"], o["b"], o["t"])
    with pytest.raises(ValueError, match="b_scales"):
        ops.grouped_gemm_mxfp4_rows(h, o["a"], o["s"], o["b"], o["t"].float())
    with pytest.raises(ValueError, match="out"):
        ops.grouped_gemm_mxfp4_rows(h, o["a"], o["s"], o["b"], o["t"], out=torch.empty((7, 64), device="cuda"))
    for bad in (torch.zeros((4, 48), device="cuda"), torch.zeros((4, 64), device="cuda").half(), torch.zeros((4, 64)),
                torch.zeros((4, 128), device="cuda")[:, ::2], torch.zeros((), device="cuda")):
        with pytest.raises(ValueError):
            ops.quantize_mxfp4(bad)
    x = torch.zeros((4, 64), device="cuda")
    with pytest.raises(ValueError, match="x has shape"):
        ops.quantize_mxfp4(x, h)
    with pytest.raises(ValueError, match="codes"):
        ops.quantize_mxfp4(x, codes=torch.zeros((4, 64), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="values"):
        ops.quantize_mxfp4(x, values=torch.zeros((4, 64), device="cuda"))
    with pytest.raises(RuntimeError, match="16-byte"):
        ops.quantize_mxfp4(torch.zeros(257, device="cuda")[1:].view(4, 64))
