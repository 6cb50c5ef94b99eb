"""Padding rows of the experts' products under alignments so large that rows
times the vectors of a row pass 2^31: zeroed to the last, nothing beside them
touched. (16 vectors of 8 columns a row for half tiles and for streamed weights,
32 for whole tiles.)"""
import numpy as np
import pytest
import torch

from test_expert_products_gpu import check, decode_mxfp4, make_handle

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_ep_layout_10_amd import ops

GUARD = 4096  # values in front of and behind the output


# direction, tokens (all of one expert), padding rows
@pytest.mark.parametrize("direction,T,padding", [
    ("forward", 1, 2 ** 27 - 1), ("forward", 1, 2 ** 27), ("mxfp4", 1, 2 ** 27), ("grad_input", 20, 2 ** 27 - 1),
    ("grad_input", 20, 2 ** 27), ("forward", 33024, 2 ** 26 - 1), ("grad_input", 33024, 2 ** 26 + 5)])
def test_padding_past_int32(direction, T, padding):
    if torch.cuda.mem_get_info()[0] < 32 << 30:
        pytest.skip("needs 32 GB of device memory")
    rows = T + padding
    h = make_handle(np.zeros((T, 1), np.int64), 1, rows)
    assert h.cfg.recv_rows_bound() >= rows
    bound, red = h.cfg.recv_rows_bound(), 32 if direction == "mxfp4" else 8
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    buffer = torch.full((bound * 8 + 2 * GUARD,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buffer[GUARD:GUARD + bound * 8].view(bound, 8)
    x = torch.full((bound, red), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[:T] = torch.randn((T, red), device="cuda", generator=gen).to(torch.bfloat16)
    if direction == "mxfp4":
        b = torch.randint(0, 256, (1, 8, 16), dtype=torch.uint8, device="cuda", generator=gen)
        s = torch.full((1, 8, 1), 127, dtype=torch.uint8, device="cuda")
        ops.grouped_gemm_mxfp4(h, x, b, s, out=out)
        w = decode_mxfp4(b[0], s[0]).t()
    else:
        b = torch.randn((1, 8, 8), device="cuda", generator=gen).to(torch.bfloat16)
        if direction == "forward":
            ops.grouped_gemm_bf16(h, x, b, out=out)
        else:
            ops.grouped_gemm_bf16_grad_input(h, x, b, grad_a=out)
        w = b[0].double().t() if direction == "forward" else b[0].double()
    torch.cuda.synchronize()
    check(out[:T], x[:T].double(), w, red, direction)
    bits = buffer.view(torch.int16)
    for r in range(T, rows, 1 << 25):
        end = min(r + (1 << 25), rows)
        assert int(torch.count_nonzero(bits[GUARD + 8 * r:GUARD + 8 * end])) == 0, r
    assert bool((buffer[:GUARD] == 7).all()) and bool((buffer[GUARD + 8 * rows:] == 7).all())
