"""Sizes that the experts' products refuse on the host, one past what the header
states: nothing is launched, and no pointer is dereferenced."""
import ctypes

import pytest

from combine_ep_layout_10_amd import _ffi as F
from test_abi_cpu import fake_handle

FAKE = ctypes.c_void_p(1 << 20)


def handle(tokens, experts=1, topk=1):
    h = fake_handle(max_tokens=tokens, num_experts=experts, num_topk=topk)
    h.num_tokens = tokens
    return h


@pytest.mark.parametrize("tokens", [(1 << 31) - (1 << 24) + 1, (1 << 31) - 31, (1 << 31) - 1])
def test_pairs(tokens):
    """An expert's rows and the tiles they make are added in 32 bits: more pairs
    than leave room for that are refused in every direction."""
    l, h = F.lib(), ctypes.byref(handle(tokens))
    assert l.ep_grouped_gemm_bf16(h, FAKE, FAKE, 8, 8, FAKE, None) == F.EP_ERR_UNSUPPORTED
    assert "pairs" in F.last_error_message()
    assert l.ep_grouped_gemm_bf16_grad_input(h, FAKE, FAKE, 8, 8, FAKE, None) == F.EP_ERR_UNSUPPORTED
    assert "pairs" in F.last_error_message()
    for f32 in (0, 1):
        assert l.ep_grouped_gemm_bf16_grad_weight(h, FAKE, FAKE, 8, 8, f32, FAKE, None) == F.EP_ERR_UNSUPPORTED
        assert "pairs" in F.last_error_message()
    assert l.ep_grouped_gemm_mxfp4(h, FAKE, FAKE, FAKE, 8, 32, FAKE, None) == F.EP_ERR_UNSUPPORTED


def row_tiles(pairs, experts, rows):
    return pairs // rows + min(pairs, experts)


# call, tokens, top-k (1,024 experts), n, k, and the tiles of the header's rule: rows and columns of one
@pytest.mark.parametrize("call,tokens,topk,n,k,rows,cols", [
    ("forward", 6 * 1024, 1, 5957 * 128 + 8, 64, 16, 128), ("forward", 8 * 1024, 1, 6553 * 128 + 8, 64, 32, 128),
    ("forward", 16 * 1024, 1, 5461 * 128 + 8, 64, 32, 128), ("forward", 1 << 26, 16, 264, 64, 256, 256),
    ("grad_input", 1 << 26, 16, 64, 264, 256, 256), ("mxfp4", 6 * 1024, 1, 5957 * 128 + 8, 64, 16, 128),
    ("mxfp4", 1 << 21, 1, 248 * 256 + 8, 64, 64, 256)])
def test_tiles_of_rows(call, tokens, topk, n, k, rows, cols):
    """The smallest width past the header's limit of 2^23 - 1 tiles."""
    width, E = k if call == "grad_input" else n, 1024
    tiles = row_tiles(tokens * topk, E, rows)
    assert tiles * -(-width // cols) > (1 << 23) - 1 >= tiles * -(-(width - 8) // cols)
    l, h = F.lib(), ctypes.byref(handle(tokens, E, topk))
    if call == "forward":
        st = l.ep_grouped_gemm_bf16(h, FAKE, FAKE, n, k, FAKE, None)
    elif call == "grad_input":
        st = l.ep_grouped_gemm_bf16_grad_input(h, FAKE, FAKE, n, k, FAKE, None)
    else:
        st = l.ep_grouped_gemm_mxfp4(h, FAKE, FAKE, FAKE, n, k, FAKE, None)
    assert st == F.EP_ERR_UNSUPPORTED and "tiles" in F.last_error_message()


@pytest.mark.parametrize("f32", [0, 1])
def test_tiles_of_the_weight_gradient(f32):
    n, k, E = 1 << 20, 3 * 128 + 8, 1024
    assert E * (n // 256) * -(-k // 128) > (1 << 24) - 1 >= E * (n // 256) * -(-(k - 8) // 128)
    h = ctypes.byref(handle(64, E))
    st = F.lib().ep_grouped_gemm_bf16_grad_weight(h, FAKE, FAKE, n, k, f32, FAKE, None)
    assert st == F.EP_ERR_UNSUPPORTED and "tiles" in F.last_error_message()
