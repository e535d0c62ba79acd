"""Attention over a 4-bit cache whose steps differ by many powers of two, between
the groups of a row and between tokens: every head's every group is as exact as
if the other groups and the tokens without weight were not there (the bound:
q4_cases.attend_reference, own_units)."""
import numpy as np
import pytest
import torch

import q4_cases as C
from oracle import q4 as Q
from paged_kv_cache_162_gb300 import _lib as L
from paged_kv_cache_162_gb300 import engine as E

pytestmark = pytest.mark.gpu


def check(c, most=0):
    d = C.on_gpu(c)
    out = torch.full(d["q"].shape, 7.0, dtype=d["q"].dtype, device="cuda")
    E.paged_attention_decode_q4(out, d["q"], d["k"], d["v"], d["tables"], d["lens"], c["scale"], max_context_len=most)
    ref, bound = C.attend_reference(c, own_units=True)
    got = Q.widen(C.bits_of(out), c["dtype"])
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= bound).all(), float((np.abs(got - ref) / bound).max())
    assert L.pkv_get_device_errors() == 0


def scaled(c, up):
    """V's steps and centres times 2^up [NB, bs, Hkv, groups] (broadcast)."""
    step, centre, code = Q.parts(c["v"], c["D"])
    step, centre = (Q.narrow(Q.widen(x, c["dtype"]) * np.exp2(up), c["dtype"]) for x in (step, centre))
    return dict(c, v=Q.pack(step, centre, code))


@pytest.mark.parametrize("dtype,ups", [("f16", (11, -15)), ("f16", (-15, 11)), ("bf16", (0, -30)), ("bf16", (-100, 60))])
@pytest.mark.parametrize("S,Hkv,G,lens,MB", [
    (3, 2, 2, [200, 40, 1000], None),      # (head, group) columns
    (3, 2, 7, [200, 40, 1000], None),      # one block of heads
    (2, 1, 16, [130, 900], None),          # two
    (2, 2, 4, [9000, 5000], 4096),         # split
    (2, 2, 12, [3000, 700], 4096),
])
def test_groups_of_far_other_sizes(dtype, ups, S, Hkv, G, lens, MB):
    c = C.attend_case(31, S, Hkv * G, Hkv, 128, 16, dtype, lens, MB=MB, spread=0.0)
    check(scaled(c, np.array(ups, float)))


@pytest.mark.parametrize("dtype,up", [("f16", 13), ("bf16", 30), ("bf16", 90)])
@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 1), (128, 2, 4), (64, 1, 7), (128, 1, 16)])
@pytest.mark.parametrize("first", [False, True])
def test_a_large_token_without_weight(dtype, up, D, Hkv, G, first):
    """One token's V is far above the others', its weight farther below theirs."""
    n = 300
    c = C.attend_case(32, 1, Hkv * G, Hkv, D, 16, dtype, [n], spread=0.0)
    j, low = 0 if first else 70, -15.0 if dtype == "f16" else 0.0
    rows = c["tables"][0, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16
    # its K: against all of the group's heads
    q = Q.widen(c["q"], dtype)[0].reshape(Hkv, G, D)
    parts = [x.reshape(-1, Hkv, x.shape[-1]).copy() for x in Q.parts(c["k"], D)]
    for x, new in zip(parts, Q.quantise(-24 * q.sum(1), dtype)):
        x[rows[j]] = new
    c["k"] = Q.pack(*(x.reshape(-1, 16, Hkv, x.shape[-1]) for x in parts))
    z = c["scale"] * np.einsum("gqd,ngd->gqn", q, Q.values(c["k"], D, dtype).reshape(-1, Hkv, D)[rows])
    assert ((z.max(-1) - z[:, :, j]) / np.log(2) > up - low + 20).all()
    ups = np.full((c["k"].shape[0] * 16, Hkv, 1), low)
    ups[rows[j]] = up
    check(scaled(c, ups.reshape(-1, 16, Hkv, 1)))


@pytest.mark.parametrize("G,split", [(1, False), (3, True), (6, False), (6, True), (12, True)])
@pytest.mark.parametrize("climbs", [1, -1])
def test_weights_that_climb_while_steps_fall(G, split, climbs):
    """Logits that rise by 7 powers of two from tile to tile, and V that falls as fast: every token
    counts alike.  And the other way round."""
    n, D, bs = 700, 64, 16
    c = C.attend_case(33, 1, G, 1, D, bs, "bf16", [n], MB=8192 if split else None, spread=0.0)
    rows = c["tables"][0, np.arange(n) // bs].astype(np.int64) * bs + np.arange(n) % bs
    at = np.arange(n) if climbs > 0 else np.arange(n)[::-1]
    powers = np.floor(at * 7 / 64)                    # of two
    c["q"] = Q.narrow(np.ones((1, G, D)), "bf16")
    c["scale"] = np.log(2.0) / D                      # a K of x everywhere: a weight of 2^x
    step, centre, code = (x.reshape(-1, 1, x.shape[-1]).copy() for x in Q.parts(c["k"], D))
    step[rows], code[rows] = 0, 8
    centre[rows, 0] = Q.narrow(powers, "bf16")[:, None]
    c["k"] = Q.pack(*(x.reshape(-1, bs, 1, x.shape[-1]) for x in (step, centre, code)))
    ups = np.zeros((c["k"].shape[0] * bs, 1, 1))
    ups[rows, 0, 0] = -powers
    check(scaled(c, ups.reshape(-1, bs, 1, 1)))


@pytest.mark.parametrize("G", [2, 5, 11])
def test_the_largest_queries(G):
    """Up to 2^113 (not itself): the elements' units, and the logits'."""
    c = C.attend_case(35, 2, G, 1, 64, 16, "bf16", [90, 700], spread=0.0)
    q = Q.widen(c["q"], "bf16").reshape(2, G, 64)
    q *= 1.99 * 2.0 ** 112 / np.abs(q).max(-1, keepdims=True)
    step, centre, code = Q.parts(c["k"], 64)
    step, centre = (Q.narrow(Q.widen(x, "bf16") * 2.0 ** -112, "bf16") for x in (step, centre))
    check(dict(c, q=Q.narrow(q, "bf16"), k=Q.pack(step, centre, code)))
