"""The router on the GPU where its formulas are hardest to keep: the lowest finite
logits beside NaN. References and bounds are test_router_gpu.py's."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_ep_layout_10_amd import ops
    from test_router_gpu import check_route


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
