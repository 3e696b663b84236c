"""Norm, rotation and append reject a call whose outputs lie on anything that it reads: rows,
positions, slots, norm weights, frequencies and scales. Fake device addresses, never
dereferenced: a call that is not rejected fails at its launch (there is no GPU here), which is
another status."""
from __future__ import annotations

import ctypes

import pytest

from quantized_routed_expert_router_amd import attention as att
from quantized_routed_expert_router_amd.qmoe import lib

INVALID, HIP = 1, 4
BASE = 0x7f0000000000
N, D, HQ, HKV = 8, 64, 4, 2

PLACES = {"positions": 0x7200000, "slots": 0x7300000, "q_norm": 0x6000000, "k_norm": 0x6001000,
          "inv_freq": 0x6002000, "k_scale": 0x6003000, "v_scale": 0x6004000}
SIZES = {"positions": 4 * N, "slots": 4 * N, "q_norm": 4 * D, "k_norm": 4 * D, "inv_freq": 2 * D,
         "k_scale": 4 * HKV, "v_scale": 4 * HKV}
ROPE = ("positions", "q_norm", "k_norm", "inv_freq")


def _heads(at, heads):
    return att._Heads(BASE + at, heads * D, D, heads)


class Call:
    """A good call; every place may be moved."""

    def __init__(self, **moved):
        at = {name: BASE + moved.get(name, PLACES[name]) for name in PLACES}
        self.q, self.k, self.v = _heads(0x1000000, HQ), _heads(0x2000000, HKV), _heads(0x3000000, HKV)
        self.q_out = _heads(moved.get("q_out", 0x4000000), HQ)
        self.k_out = _heads(moved.get("k_out", 0x5000000), HKV)
        self.p = att._NormRope(at["q_norm"], at["k_norm"], at["inv_freq"], 1e-6, 0.0, D, 0)
        self.cache = att._KVCache(BASE + 0x10000000, BASE + 0x20000000, at["k_scale"], at["v_scale"],
                                  2, 64, 16, HKV, D)
        self.at = at

    def rope(self):
        r = ctypes.byref
        return lib.moe_qk_norm_rope(r(self.q), r(self.k), self.at["positions"], N, 0, D, r(self.p),
                                    r(self.q_out), r(self.k_out), None)

    def append(self, with_q=True):
        r = ctypes.byref
        q, q_out = (r(self.q), r(self.q_out)) if with_q else (None, None)
        return lib.moe_kv_append(r(self.cache), r(self.k), r(self.v), self.at["slots"],
                                 self.at["positions"], N, 0, r(self.p), q, q_out, None)


@pytest.fixture(autouse=True)
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("calls that are not rejected would launch on the GPU")


def test_the_good_call_reaches_its_launch():
    assert Call().rope() == HIP and Call().append() == HIP and Call().append(False) == HIP


@pytest.mark.parametrize("what", ROPE)
@pytest.mark.parametrize("out,heads", [("q_out", HQ), ("k_out", HKV)])
def test_norm_rope_outputs_on_parameters(what, out, heads):
    bytes_out = 2 * N * heads * D
    for at in (PLACES[what], PLACES[what] + SIZES[what] - 16, PLACES[what] - bytes_out + 16):
        assert Call(**{out: at}).rope() == INVALID, hex(at)
    # side by side is fine
    for at in (PLACES[what] + SIZES[what], PLACES[what] - bytes_out):
        alone = {"positions": 0x7200000, "q_norm": 0x8000000, "k_norm": 0x9000000,
                 "inv_freq": 0xa000000}
        alone[what] = PLACES[what]
        assert Call(**{out: at}, **alone).rope() == HIP, hex(at)


@pytest.mark.parametrize("what", sorted(PLACES))
def test_append_outputs_on_parameters(what):
    bytes_out = 2 * N * HQ * D
    size = max(SIZES[what], 16)
    for at in (PLACES[what], PLACES[what] + size - 16, PLACES[what] - bytes_out + 16):
        assert Call(q_out=at).append() == INVALID, hex(at)
    cache_bytes = 64 * 16 * HKV * D
    for cache in (0x10000000, 0x20000000):
        for at in (cache, cache + cache_bytes - 4, cache - SIZES[what] + 4):
            assert Call(**{what: at}).append() == INVALID, hex(at)
            assert Call(**{what: at}).append(False) == INVALID, hex(at)
        for at in (cache + cache_bytes, cache - SIZES[what]):
            assert Call(**{what: at}).append() == HIP, hex(at)


def test_unused_frequencies_may_lie_anywhere():
    # rot_dim == 0: no frequency is read
    c = Call(inv_freq=0x4000000)
    c.p.rot_dim = 0
    assert c.rope() == HIP
