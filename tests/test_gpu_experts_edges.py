"""The operators of a layer of experts where a comparison, a mask or a tensor that the
call makes could go wrong unseen."""
import itertools

import pytest
import torch

from test_gpu_experts import _check_route, _gen

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- routing

def _pairs_of_near_sums(g, T, groups, score, spread):
    """Logits of `groups` groups of two experts whose scores add up to nearly the same in
    every group (times a common factor for softmax)."""
    a = 0.3 + 0.4 * torch.rand((T, groups), generator=g, device="cuda", dtype=torch.float64)
    d = spread * torch.randn((T, groups), generator=g, device="cuda", dtype=torch.float64)
    s = torch.stack([a, 1.0 + d - a], 2).view(T, 2 * groups)
    return (torch.logit(s) if score == "sigmoid" else torch.log(s)).float()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [32.0, 100.0, 3000.0])
@pytest.mark.parametrize("groups,kept", [(2, 1), (8, 3)])
def test_route_groups_whose_biases_cancel(score, size, groups, kept):
    """Biases of opposite sign leave a group's sum small, and its error as large as theirs."""
    g = _gen(int(size) + groups)
    sign = torch.tensor([size, -size], device="cuda").repeat(groups)
    unlike = sign * torch.repeat_interleave(1 + torch.arange(groups, device="cuda") % 3, 2)
    for spread, bias in itertools.product((1e-5, 1e-6 * size), (sign, unlike)):
        logits = _pairs_of_near_sums(g, 1500, groups, score, spread)
        _check_route(logits, min(3, 2 * kept), score=score, bias=bias, groups=groups,
                     groups_kept=kept, group_top=2)
