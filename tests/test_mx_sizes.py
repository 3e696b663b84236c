"""Sizes that do not fit the C ABI's integers do not reach it as other sizes: tensors without
memory (device "meta") stand for the large ones."""
from __future__ import annotations

import pytest
import torch

from quantized_routed_expert_router_amd import mx, qmoe

WRAPS = 2 ** 32  # 2 ** 32 + 64 columns would arrive as 64


def _meta(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("rows", [1, 3])
def test_quantize_columns(rows):
    with pytest.raises(ValueError, match=f"{WRAPS + 64} columns"):
        mx.quantize(_meta(rows, WRAPS + 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match=f"{WRAPS + 64} columns"):
        mx.quantize(_meta(2, rows, WRAPS + 64, dtype=torch.float32))


@pytest.mark.parametrize("n,E,k", [(WRAPS + 4, 8, 2), (4, WRAPS + 8, 2), (4, 8, WRAPS + 2), (4, 8, 2 - WRAPS)])
def test_route_sizes(n, E, k):
    with pytest.raises(ValueError, match="rows of"):
        qmoe.route_scored(_meta(n, E, dtype=torch.bfloat16), k, qmoe.RouteRule())


def test_rule_sizes():
    for rule in (qmoe.RouteRule(groups=WRAPS + 1, top_groups=1), qmoe.RouteRule(groups=1, top_groups=WRAPS + 1),
                 qmoe.RouteRule(groups=1 - WRAPS, top_groups=1)):
        st = rule._struct()
        assert (st.groups, st.top_groups) != (1, 1) and {st.groups, st.top_groups} <= {-1, 1, 0x7fffffff}


def _layer(E=4, f=32, d=64, top_k=2):
    m = lambda rows, cols: mx.MxMatrix(_meta(E, rows, cols // 2), _meta(E, rows, cols // 32))  # noqa: E731
    return mx.MxLayer(m(f, d), m(f, d), m(d, f), top_k)


def test_ffn_workspace_sizes():
    good = mx.ffn_workspace_bytes(_layer(), 4)
    assert good > 0
    for n in (WRAPS + 4, 4 - WRAPS, 2 ** 70):
        assert mx.ffn_workspace_bytes(_layer(), n) == 0
    for over in (dict(E=WRAPS + 4), dict(f=WRAPS + 32), dict(d=WRAPS + 64), dict(top_k=WRAPS + 2),
                 dict(top_k=2 - WRAPS)):
        assert mx.ffn_workspace_bytes(_layer(**over), 4) == 0


def test_layer_sizes():
    for over, field in ((dict(E=WRAPS + 4), "n_experts"), (dict(f=WRAPS + 32), "d_ff"), (dict(d=WRAPS + 64), "d_model"),
                        (dict(top_k=WRAPS + 2), "top_k")):
        st = _layer(**over).check(qmoe._Args())
        assert getattr(st, field) == 0x7fffffff
