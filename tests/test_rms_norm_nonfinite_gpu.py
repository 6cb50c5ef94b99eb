"""NaN and infinities through the RMS norm, its FP8 form and its backward: each
reaches what the formulas say, and nothing else."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_ep_layout_10_amd import ops

NAN, INF = float("nan"), float("inf")


def data(T, H, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n = lambda *s: torch.randn(s, device="cuda", generator=gen)
    return n(T, H).to(torch.bfloat16), (1 + 0.2 * n(H)).to(torch.bfloat16), n(T, H).to(torch.bfloat16)


def same(a, b):
    """Equal, NaN where NaN."""
    a, b = a.double(), b.double()
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(0.0, INF, -INF),
                                                                      b.nan_to_num(0.0, INF, -INF))


def definition(s, w, rstd):
    """Codes (as values) and scales of the FP8 form on the host, in binary32:
    q = max|u| / 448, a NaN among the |u| being the largest; u / q unless q is 0."""
    u = (s.float() * w.float()).cpu().numpy().reshape(s.shape[0], -1, 128)
    with np.errstate(all="ignore"):
        q = np.abs(u).max(2, keepdims=True) / np.float32(448)
        v = np.where(q == 0, np.float32(0), (u / q).clip(-448, 448))
    code = torch.from_numpy(v.reshape(s.shape)).to(torch.float8_e4m3fn).double().cuda()
    return code, torch.from_numpy(q[:, :, 0]).cuda() * rstd[:, None]


# place in the row (which block of 128 and whether its other values are ordinary, zero or tiny), and the value
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("rest", ["ordinary", "zero", "tiny"])
@pytest.mark.parametrize("H,at", [(128, 0), (512, 255), (1024, 511), (7168, 6000), (16384, 16383)])
def test_weight(value, rest, H, at):
    """A NaN or an infinity in the weight: the channel's own block has a NaN or
    an infinite scale, and NaN codes where u / q is; other blocks are as ever."""
    x, w, _ = data(3, H)
    block = slice(at // 128 * 128, at // 128 * 128 + 128)
    if rest != "ordinary":
        x[:, block] = 0.0 if rest == "zero" else 1e-38
    x[:, at] = 1.0
    clean = ops.rms_norm(x, w, 1e-5, dtype=ops.FP8_QUANTIZE)
    bad = w.clone()
    bad[at] = value
    if rest == "zero":
        x[1, at] = 0.0                              # 0 * inf and 0 * NaN are NaN
        clean = ops.rms_norm(x, w, 1e-5, dtype=ops.FP8_QUANTIZE)
    y, scales, _, rstd = ops.rms_norm(x, bad, 1e-5, dtype=ops.FP8_QUANTIZE)
    code, want = definition(x, bad, rstd)
    got = y.view(torch.float8_e4m3fn).double()
    assert same(got, code)
    assert same(scales, want)
    assert not bool(torch.isfinite(scales[:, at // 128]).any())
    assert bool(torch.isnan((got.view(3, -1, 128) * scales.double()[:, :, None]).flatten(1)[:, at]).all())
    other = [b for b in range(H // 128) if b != at // 128]
    assert torch.equal(y.view(3, -1, 128)[:, other], clean[0].view(3, -1, 128)[:, other])
    assert torch.equal(scales[:, other], clean[1][:, other])
    plain = ops.rms_norm(x, bad, 1e-5)
    assert same(plain[0][:, at], (x[:, at].float() * bad[at].float() * plain[3]).to(torch.bfloat16))
    rest_of_row = torch.arange(H, device="cuda") != at
    assert bool(torch.isfinite(plain[0][:, rest_of_row]).all())


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("residual", [False, True])
def test_row(value, residual):
    """A NaN or an infinity in a row of x: that row's results follow the
    formulas, the other rows' are those of the same call without it."""
    x, w, r = data(5, 1024, 1)
    r = r if residual else None
    for dtype in (ops.BF16, ops.FP8_QUANTIZE):
        clean = ops.rms_norm(x, w, 1e-5, residual=r, dtype=dtype)
        bad = x.clone()
        bad[2, 300] = value
        y, scales, total, rstd = ops.rms_norm(bad, w, 1e-5, residual=r, dtype=dtype)
        assert bool(torch.isnan(rstd[2])) if value != value else float(rstd[2]) == 0.0
        others = [0, 1, 3, 4]
        for a, b in zip((y, total, rstd), (clean[0], total if r is None else clean[2], clean[3])):
            assert torch.equal(a[others], b[others])
        if dtype == ops.BF16:
            assert same(y[2], (total[2].float() * w.float() * rstd[2]).to(torch.bfloat16))
        else:
            code, want = definition(total, w, rstd)
            assert same(y.view(torch.float8_e4m3fn).double(), code) and same(scales, want)
            assert torch.equal(scales[others], clean[1][others])


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("T,H", [(5, 1024), (2000, 264), (4, 16384)])
def test_backward(value, T, H):
    """In one row's gradient of y: that row of grad_x, and that channel of
    grad_weight; the rest as without it."""
    s, w, g = data(T, H, 2)
    rstd = (1.0 / (s.double().square().mean(1) + 1e-5).sqrt()).float()
    gx, gw = ops.rms_norm_backward(s, w, rstd, g)
    bad = g.clone()
    bad[T // 2, 100] = value
    bx, bw = ops.rms_norm_backward(s, w, rstd, bad)
    rows, channels = torch.arange(T, device="cuda") != T // 2, torch.arange(H, device="cuda") != 100
    assert not bool(torch.isfinite(bx[T // 2]).any())
    assert torch.equal(bx[rows], gx[rows])
    assert not bool(torch.isfinite(bw[100])) and torch.equal(bw[channels], gw[channels])
