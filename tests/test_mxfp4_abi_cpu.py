"""Argument checks of the MXFP4 quantisation and of the product with MXFP4 rows on
the CPU: every call below fails a check before anything reaches the GPU, so no
pointer is dereferenced."""
import ctypes

import numpy as np
import pytest

import mxfp4_reference as ref
from combine_ep_layout_10_amd import _ffi as F
from test_abi_cpu import fake_handle

FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)
BAD, UNSUP = F.EP_ERR_INVALID_ARG, F.EP_ERR_UNSUPPORTED


def test_quantize():
    q = F.lib().ep_quantize_mxfp4
    for k in (0, -32, 16, 33, 48):
        assert q(None, 4, k, 0, FAKE, FAKE, FAKE, None, None) == BAD, k
    assert q(None, 4, (1 << 20) + 32, 0, FAKE, FAKE, FAKE, None, None) == UNSUP
    assert q(None, -1, 32, 0, FAKE, FAKE, FAKE, None, None) == BAD
    assert q(None, (1 << 37) + 1, 32, 0, FAKE, FAKE, FAKE, None, None) == UNSUP
    for f32 in (-1, 2):
        assert q(None, 4, 32, f32, FAKE, FAKE, FAKE, None, None) == BAD
    for bad in (None, ODD):
        assert q(None, 4, 32, 0, bad, FAKE, FAKE, None, None) == BAD
        assert q(None, 4, 32, 0, FAKE, bad, FAKE, None, None) == BAD
        assert "16-byte" in F.last_error_message()
    assert q(None, 4, 32, 0, FAKE, FAKE, None, None, None) == BAD
    assert q(None, 4, 32, 0, FAKE, FAKE, FAKE, ODD, None) == BAD
    assert q(None, 0, 32, 0, None, None, None, None, None) == F.EP_OK
    h = fake_handle()
    bound = F.ep_recv_rows_bound(h.cfg)
    assert q(ctypes.byref(h), bound - 1, 32, 0, FAKE, FAKE, FAKE, None, None) == BAD
    assert "bound" in F.last_error_message()
    assert q(ctypes.byref(h), bound, 32, 0, None, FAKE, FAKE, None, None) == BAD
    h.row_src = None
    assert q(ctypes.byref(h), bound, 32, 0, FAKE, FAKE, FAKE, None, None) == BAD
    h = fake_handle()
    h.num_tokens = 0
    assert q(ctypes.byref(h), bound, 32, 0, None, None, None, None, None) == F.EP_OK


def test_product():
    f = F.lib().ep_grouped_gemm_mxfp4_rows
    h = ctypes.byref(fake_handle())
    assert f(None, FAKE, FAKE, FAKE, FAKE, 64, 64, FAKE, None) == BAD
    for n in (0, -8, 4, 12):
        assert f(h, FAKE, FAKE, FAKE, FAKE, n, 64, FAKE, None) == BAD, n
    for k in (0, -32, 8, 16, 48):
        assert f(h, FAKE, FAKE, FAKE, FAKE, 64, k, FAKE, None) == BAD, k
    assert f(h, FAKE, FAKE, FAKE, FAKE, (1 << 20) + 8, 64, FAKE, None) == UNSUP
    assert f(h, FAKE, FAKE, FAKE, FAKE, 64, (1 << 20) + 32, FAKE, None) == UNSUP
    for i in (1, 2, 3, 4, 7):
        a = [h, FAKE, FAKE, FAKE, FAKE, 64, 64, FAKE, None]
        a[i] = None
        assert f(*a) == BAD, i
        if i in (1, 3, 7):
            a[i] = ODD
            assert f(*a) == BAD and "16-byte" in F.last_error_message()
    empty = fake_handle()
    empty.num_tokens = 0
    assert f(ctypes.byref(empty), None, None, None, None, 64, 64, None, None) == F.EP_OK


@pytest.mark.parametrize("tokens", [(1 << 31) - (1 << 24) + 1, (1 << 31) - 1])
def test_pairs(tokens):
    h = fake_handle(max_tokens=tokens, num_experts=1, num_topk=1)
    h.num_tokens = tokens
    f = F.lib().ep_grouped_gemm_mxfp4_rows
    assert f(ctypes.byref(h), FAKE, FAKE, FAKE, FAKE, 8, 32, FAKE, None) == UNSUP
    assert "pairs" in F.last_error_message()


# tokens, top-k (1,024 experts), n, k, and the tiles of the header's rule: rows and columns of one
@pytest.mark.parametrize("tokens,topk,n,k,rows,cols", [
    (6 * 1024, 1, 5957 * 128 + 8, 64, 16, 128), (8 * 1024, 1, 7281 * 128 + 8, 32, 64, 128), (1 << 26, 16, 264, 128, 256, 256),
    (1 << 26, 16, 264, 160, 192, 256)])
def test_tiles_of_a_launch(tokens, topk, n, k, rows, cols):
    """The smallest width past the header's limit of 2^23 - 1 tiles."""
    tiles = lambda w: (tokens * topk // rows + 1024) * -(-w // cols)
    assert tiles(n) > (1 << 23) - 1 >= tiles(n - 8)
    h = fake_handle(max_tokens=tokens, num_experts=1024, num_topk=topk)
    h.num_tokens = tokens
    f = F.lib().ep_grouped_gemm_mxfp4_rows
    assert f(ctypes.byref(h), FAKE, FAKE, FAKE, FAKE, n, k, FAKE, None) == UNSUP
    assert "tiles" in F.last_error_message()


def test_reference_on_known_values():
    """The tests' own quantiser on values worked out by hand."""
    x = np.zeros((1, 32))
    x[0, :9] = [6.0, -5.0, 0.25, -0.75, 3.5, 2.5, 0.2, -0.0, 1.0]     # largest 6: X = 0
    codes, scales, values = ref.quantize(x)
    assert scales[0, 0] == 127
    assert values[0, :9].tolist() == [6.0, -4.0, 0.0, -1.0, 4.0, 2.0, 0.0, -0.0, 1.0]
    assert codes[0, :5].tolist() == [0x7 | 0xE << 4, 0x0 | 0xA << 4, 0x6 | 0x4 << 4, 0x0 | 0x8 << 4, 0x2]
    assert ref.quantize(np.full((1, 32), 7.99))[2][0, 0] == 6.0       # saturated
    assert ref.quantize(np.full((1, 32), 8.0))[1][0, 0] == 128
    assert ref.quantize(np.zeros((1, 32)))[1][0, 0] == 0
    assert np.array_equal(ref.decode(codes, scales), values)


def test_dma_loads_bring_their_wait_states(tmp_path):
    """The LDS DMA loads are inline assembly, into which the compiler's hazard pass
    does not look: they bring the five wait states behind a scalar's write themselves."""
    import os
    import re
    import subprocess

    from combine_ep_layout_10_amd import build as B
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc not installed")
    out = tmp_path / "fp4.s"
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([B.HIPCC] + flags + ["--cuda-device-only", "-S", "-o", str(out),
                                        os.path.join(B.CSRC, "ep_gemm_fp4.hip")], check=True, capture_output=True)
    lines = [l.split(";")[0].strip() for l in out.read_text().splitlines()]
    lines = [l for l in lines if l and not l.startswith(".")]
    loads = [i for i, l in enumerate(lines) if l.startswith("buffer_load_dwordx4") and l.endswith(" lds")]
    assert len(loads) > 50
    for i in loads:
        m = re.fullmatch(r"s_nop (\d+)", lines[i - 1])
        assert m and int(m.group(1)) >= 4, lines[i - 3:i + 1]
