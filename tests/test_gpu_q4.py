"""Attention over a 4-bit cache against its definition in 64 bits (the bound and
where it comes from: q4_cases.attend_reference), and the calls around it."""
import numpy as np
import pytest
import torch

import q4_cases as C
from oracle import q4 as Q
from paged_kv_cache_162_gb300 import _lib as L
from paged_kv_cache_162_gb300 import engine as E

pytestmark = pytest.mark.gpu


def run(c, d=None, **kw):
    d = d or C.on_gpu(c)
    out = torch.full(d["q"].shape, 7.0, dtype=d["q"].dtype, device="cuda")
    E.paged_attention_decode_q4(out, d["q"], d["k"], d["v"], d["tables"], d["lens"], c["scale"], **kw)
    return out


def check(c, out):
    ref, bound = C.attend_reference(c)
    got = Q.widen(C.bits_of(out), c["dtype"])
    assert np.isfinite(got).all()
    over = np.abs(got - ref) - bound
    assert over.max() <= 0, (float(over.max()), float((np.abs(got - ref) / bound).max()))
    assert L.pkv_get_device_errors() == 0


def spread(rng, S, hi):
    """Lengths with the edges of units, tiles and blocks among them."""
    edge = [0, 1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, hi]
    lens = rng.integers(1, hi + 1, S)
    lens[:min(S, len(edge))] = np.minimum(edge, hi)[:S]
    return lens


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,bs", [(64, 8), (64, 64), (128, 8), (128, 16), (128, 32)])
@pytest.mark.parametrize("Hkv,G", [(4, 1), (2, 4), (1, 7), (3, 8), (1, 9), (2, 16), (8, 2)])
def test_few_short_contexts(dtype, D, bs, Hkv, G):
    rng = np.random.default_rng(D + bs + Hkv)
    c = C.attend_case(11, 17, Hkv * G, Hkv, D, bs, dtype, spread(rng, 17, 300))
    check(c, run(c))


@pytest.mark.parametrize("S,Hkv,G,D,bs,dtype,hi", [
    (1, 8, 4, 128, 16, "bf16", 5000),    # clusters share a sequence
    (1, 1, 1, 64, 8, "f16", 16384),
    (2, 2, 16, 128, 32, "f16", 9001),
    (1, 1, 1, 128, 16, "bf16", 40000),   # split, four warps on a head
    (3, 3, 2, 64, 16, "f16", 20000),
    (5, 2, 9, 128, 64, "bf16", 18000),
    (2, 4, 1, 128, 16, "f16", 33000),
    (2, 2, 7, 128, 16, "f16", 3000),     # 5 to 8 query heads per KV head
    (3, 1, 5, 64, 8, "bf16", 6000),
    (1, 1, 1, 128, 16, "f16", 70000),    # too long for the clusters: split
    (1, 2, 6, 64, 64, "bf16", 95000),
])
def test_long_contexts(S, Hkv, G, D, bs, dtype, hi):
    rng = np.random.default_rng(hi)
    lens = rng.integers(hi // 2, hi + 1, S)
    lens[0] = hi
    c = C.attend_case(12, S, Hkv * G, Hkv, D, bs, dtype, lens)
    check(c, run(c))


@pytest.mark.parametrize("S,Hkv,G,D,bs,dtype,hi", [
    (300, 8, 1, 64, 16, "f16", 130),
    (620, 4, 2, 128, 8, "bf16", 100),
    (1300, 2, 1, 64, 8, "f16", 70),
    (2500, 1, 3, 64, 16, "bf16", 60),
    (900, 3, 10, 64, 32, "f16", 64),
    (160, 16, 1, 128, 16, "bf16", 400),
    (80, 4, 6, 128, 16, "bf16", 1300),
    (80, 4, 2, 64, 8, "f16", 1300),
    (200, 2, 1, 64, 16, "f16", 1100),
    (45, 8, 10, 64, 32, "f16", 1100),
])
def test_many_sequences(S, Hkv, G, D, bs, dtype, hi):
    """Enough units that tiles are cut into ranges; empty sequences in between."""
    rng = np.random.default_rng(hi)
    lens = spread(rng, S, hi)
    lens[rng.integers(0, S, S // 5)] = 0
    c = C.attend_case(13, S, Hkv * G, Hkv, D, bs, dtype, lens)
    check(c, run(c))


def test_all_empty_and_one_token():
    for lens in ([0, 0, 0], [1, 1, 1]):
        c = C.attend_case(14, 3, 8, 2, 128, 16, "f16", lens, MB=2)
        out = run(c)
        check(c, out)
        if not any(lens):
            assert (out == 0).all()


@pytest.mark.parametrize("scale", [0.0, -0.125, 3.0])
def test_scales(scale):
    """3: a weight of nearly 1 and the others next to nothing."""
    c = C.attend_case(15, 4, 8, 2, 128, 16, "f16", [100, 33, 500, 64])
    c["scale"] = scale
    check(c, run(c))


@pytest.mark.parametrize("dtype,k_exp,q_exp", [("f16", 8, -8), ("f16", -10, 9), ("bf16", 40, -40), ("bf16", -50, 50),
                                               ("bf16", 60, -90), ("bf16", 110, -110), ("bf16", -100, 100)])
def test_far_from_one(dtype, k_exp, q_exp):
    """Steps, centres and queries of far other sizes; steps that differ by orders from token to token."""
    c = C.attend_case(16, 3, 12, 3, 64, 16, dtype, [200, 40, 1000], spread=3.0 if dtype == "bf16" else 1.0)
    for name, up in (("k", k_exp), ("v", k_exp // 2)):
        step, centre, code = Q.parts(c[name], 64)
        step, centre = (Q.narrow(Q.widen(x, dtype) * 2.0 ** up, dtype) for x in (step, centre))
        c[name] = Q.pack(step, centre, code)
    c["q"] = Q.narrow(Q.widen(c["q"], dtype) * 2.0 ** q_exp, dtype)
    check(c, run(c))


def test_equal_bits_and_any_workspace_contents():
    c = C.attend_case(17, 40, 32, 8, 128, 16, "bf16", np.random.default_rng(1).integers(1, 3000, 40))
    d = C.on_gpu(c)
    ws = E.new_q4_workspace(40, 32, 8, 128)
    ws.random_(0, 256)
    first = run(c, d, workspace=ws)
    for _ in range(3):
        assert torch.equal(run(c, d, workspace=ws), first)
    assert torch.equal(run(c, d), first)
    check(c, first)


def test_bad_blocks_and_lengths():
    """A block out of range: its tokens are passed over and its bit is set; lengths are clamped."""
    c = C.attend_case(18, 3, 4, 2, 64, 16, "f16", [40, 100, 10])
    d = C.on_gpu(c)
    d["tables"][1, 2] = 10 ** 6
    out = run(c, d)
    torch.cuda.synchronize()
    assert L.pkv_get_device_errors() == L.PKV_DEVERR_BLOCK_ID
    # the same without those 16 tokens
    c2 = dict(c, tables=c["tables"].copy(), lens=np.array([40, 84, 10], np.int32))
    c2["tables"][1, 2:6] = c["tables"][1, 3:7]
    ref, bound = C.attend_reference(c2)
    assert (np.abs(Q.widen(C.bits_of(out), "f16") - ref) <= bound).all()
    d = C.on_gpu(c)
    d["lens"] = torch.tensor([-5, 200, 10], dtype=torch.int32, device="cuda")
    out = run(c, d, max_context_len=100)
    torch.cuda.synchronize()
    assert L.pkv_get_device_errors() == L.PKV_DEVERR_CONTEXT
    ref, bound = C.attend_reference(dict(c, lens=np.array([0, 100, 10], np.int32)))
    assert (np.abs(Q.widen(C.bits_of(out), "f16") - ref) <= bound).all()


def test_a_group_that_is_not_finite():
    """A NaN group of V shows in its 64 dims, one of K in the whole row; other heads do not see it."""
    c = C.attend_case(19, 2, 4, 2, 128, 16, "f16", [50, 50])
    for name, dims in (("v", slice(64, 128)), ("k", slice(0, 128))):
        step, centre, code = Q.parts(c[name], 128)
        slot = c["tables"][1, 1] * 16 + 3
        step.reshape(-1, 2, 2)[slot, 1, 1] = C.NAN_BITS["f16"]
        out = run({**c, name: Q.pack(step, centre, code)}).isnan().cpu()
        want = torch.zeros(2, 4, 128, dtype=torch.bool)
        want[1, 2:, dims] = True
        assert torch.equal(out, want)


def test_stream_and_graph():
    c = C.attend_case(20, 6, 16, 4, 128, 16, "bf16", [3000, 1, 0, 700, 64, 2222])
    d = C.on_gpu(c)
    ws = E.new_q4_workspace(6, 16, 4, 128)
    first = run(c, d, workspace=ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.empty_like(first)
    E.paged_attention_decode_q4(out, d["q"], d["k"], d["v"], d["tables"], d["lens"], c["scale"], stream=side)
    side.synchronize()
    assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(g):
        E.paged_attention_decode_q4(out, d["q"], d["k"], d["v"], d["tables"], d["lens"], c["scale"], workspace=ws)
    d["lens"][3] = 650
    g.replay()
    torch.cuda.synchronize()
    check(dict(c, lens=np.array([3000, 1, 0, 650, 64, 2222], np.int32)), out)


def test_calls_without_a_workspace_on_two_streams():
    """Each takes scratch of its own stream's memory."""
    c = C.attend_case(21, 40, 8, 8, 64, 16, "f16", np.random.default_rng(3).integers(900, 3000, 40))
    d = C.on_gpu(c)
    want = run(c, d)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(want) for _ in range(8)]
    for i, o in enumerate(outs):
        E.paged_attention_decode_q4(o, d["q"], d["k"], d["v"], d["tables"], d["lens"], c["scale"], stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("D", [64, 128])
def test_copy_and_swap_blocks(D):
    NB, Hkv, bs = 12, 3, 16
    RB = Q.row_bytes(D)
    k, v = (torch.randint(0, 256, (NB, Hkv, bs, RB), dtype=torch.uint8, device="cuda") for _ in range(2))
    want_k, want_v = k.clone(), v.clone()
    pairs = torch.tensor([[3, 0], [3, 11], [5, 2]], device="cuda")
    E.copy_blocks(k, v, pairs)
    for a, b in pairs.tolist():
        want_k[b], want_v[b] = want_k[a], want_v[a]
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    host = [torch.zeros((5, Hkv, bs, RB), dtype=torch.uint8).pin_memory() for _ in range(2)]
    E.swap_blocks(k, v, *host, torch.tensor([[4, 0], [9, 4]], device="cuda"), L.PKV_SWAP_OUT)
    torch.cuda.synchronize()
    assert torch.equal(host[0][0], k[4].cpu()) and torch.equal(host[1][4], v[9].cpu()) and not host[0][1:4].any()
    E.swap_blocks(k, v, *host, torch.tensor([[4, 1]], device="cuda"), L.PKV_SWAP_IN)
    want_k[1], want_v[1] = want_k[9], want_v[9]
    torch.cuda.synchronize()
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    assert L.pkv_get_device_errors() == 0


def test_values_near_the_end_of_bf16():
    """V of 2^113: a weight's units and a code's together must not leave fp32."""
    c = C.attend_case(22, 2, 4, 2, 128, 16, "bf16", [70, 20], spread=0.0)
    step, centre, code = Q.parts(c["v"], 128)
    step, centre = (Q.narrow(Q.widen(x, "bf16") * 2.0 ** 113, "bf16") for x in (step, centre))
    c["v"] = Q.pack(step, centre, code)
    check(c, run(c))
