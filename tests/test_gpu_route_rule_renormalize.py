"""`renormalize` is read as Python reads a truth value, whichever way the call takes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from quantized_routed_expert_router_amd import qmoe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [True, 1, 2, "yes", np.True_, False, 0, None, "", np.False_])
@pytest.mark.parametrize("given", [False, True])
def test_truth_values(value, given):
    logits = torch.randn((9, 16), generator=torch.Generator().manual_seed(6)).cuda()
    ref = qmoe.route_scored(logits, 3, qmoe.RouteRule(renormalize=bool(value)))
    out = qmoe.Routing.empty(9, 16, 3) if given else None
    got = qmoe.route_scored(logits, 3, qmoe.RouteRule(renormalize=value), out=out)
    assert torch.equal(got.topk_ids, ref.topk_ids) and torch.equal(got.topk_w, ref.topk_w)
