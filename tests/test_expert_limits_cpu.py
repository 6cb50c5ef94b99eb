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
