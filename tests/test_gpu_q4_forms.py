"""Attention over a 4-bit cache in the forms that only large calls take: tiles
handed out in large and small ranges as CTAs come free, and CTAs that fill half
of an SM.  Bounds: q4_cases.attend_reference, here for sequences that share
their blocks, in torch."""
import numpy as np
import pytest
import torch

import q4_cases as C
from oracle import q4 as Q
from paged_kv_cache_162_gb300 import _lib as L
from paged_kv_cache_162_gb300 import engine as E

pytestmark = pytest.mark.gpu


def shared_case(seed, S, Hkv, G, D, bs, dtype, lens):
    """attend_case's inputs where every sequence's context begins the longest one's: one pool's blocks for all."""
    n = int(max(lens))
    c = C.attend_case(seed, 1, Hkv * G, Hkv, D, bs, dtype, [n])
    rng = np.random.default_rng(seed + 1)
    return dict(c, S=S, lens=np.asarray(lens, np.int32), tables=np.repeat(c["tables"], S, 0),
                q=Q.narrow(rng.standard_normal((S, Hkv * G, D)), dtype))


def reference(c):
    """attend_reference's (out, bound) of shared_case, as CUDA tensors."""
    S, H, Hkv, D, dtype = (c[x] for x in ("S", "H", "Hkv", "D", "dtype"))
    G, u, n, e = H // Hkv, C.U[dtype], int(c["lens"].max()), C.E32
    pos = np.arange(n)
    rows = c["tables"][0, pos // c["bs"]].astype(np.int64) * c["bs"] + pos % c["bs"]
    sides = []
    for pool in (c["k"], c["v"]):
        step, centre, code = Q.parts(pool, D)
        step, centre = (np.repeat(Q.widen(x, dtype), 64, -1).reshape(-1, Hkv, D)[rows] for x in (step, centre))
        sides.append([torch.from_numpy(np.ascontiguousarray(x.transpose(1, 0, 2))).cuda().double()
                      for x in (step, centre, code.reshape(-1, Hkv, D)[rows] - 8)])
    (ks, ka, kc), (vs, va, vc) = sides
    k, v = ka + ks * kc, va + vs * vc
    kmag, vmag = ka.abs() + ks * (kc.abs() + 16), va.abs() + vs * vc.abs()
    out, bound = (torch.zeros(S, Hkv, G, D, dtype=torch.float64, device="cuda") for _ in range(2))
    q = torch.from_numpy(Q.widen(c["q"], dtype)).cuda().view(S, Hkv, G, D)
    r16, s = 2.0 ** -22 if dtype == "f16" else 2.0 ** -11, abs(c["scale"])
    for i, m in enumerate(c["lens"].tolist()):
        if m == 0:
            bound[i] = 2.0 ** -25
            continue
        p = torch.softmax(c["scale"] * (q[i] @ k[:, :m].transpose(1, 2)), -1)
        Z = s * (q[i].abs() @ kmag[:, :m].transpose(1, 2)).amax(-1)
        Zq = s * (q[i].abs().amax(-1) * kmag[:, :m].sum(-1).amax(-1)[:, None])
        w = (4 * (144 * e * Z + e * Zq) + 2.0 ** -21 + (m / 8 + 100) * 4 * e)[..., None]
        A, r = p @ vmag[:, :m], p @ v[:, :m]
        A16 = A + 16 * (p @ vs[:, :m])
        out[i] = r
        bound[i] = u * r.abs() + (1 + u) * (A * r16 + A16 * w + m * 2.0 ** -30 * vs[:, :m].max()) + 2.0 ** -25
    return out.view(S, H, D), bound.view(S, H, D)


def run(c, d, workspace=None):
    out = torch.full(d["q"].shape, 7.0, dtype=d["q"].dtype, device="cuda")
    E.paged_attention_decode_q4(out, d["q"], d["k"], d["v"], d["tables"], d["lens"], c["scale"], workspace=workspace)
    return out


def check(c, out):
    ref, bound = reference(c)
    off = (out.double() - ref).abs()
    assert (off <= bound).all(), float((off / bound).max())
    assert L.pkv_get_device_errors() == 0


def test_the_reference_is_the_other_one():
    c = shared_case(40, 5, 2, 3, 128, 16, "bf16", [300, 0, 17, 64, 129])
    for got, want in zip(reference(c), C.attend_reference(c)):
        assert np.allclose(got.cpu().numpy(), want, rtol=1e-10, atol=1e-14)


SMALL_RANGES = 64 * 608  # tiles from which a call on any number of CTAs per SM (up to 4) has them


@pytest.mark.parametrize("Hkv,G,D,dtype", [
    (4, 1, 128, "f16"), (4, 4, 64, "bf16"),      # (head, group) columns
    (4, 5, 128, "bf16"), (4, 8, 64, "f16"),      # one block of heads
    (4, 9, 128, "f16"), (4, 16, 64, "bf16"),     # two
    (8, 2, 128, "bf16"),                         # two units per sequence
])
def test_large_and_small_ranges(Hkv, G, D, dtype):
    """Rings that run over units and ranges, pieces of units in both kinds; equal bits whoever takes which."""
    rng = np.random.default_rng(Hkv + G + D)
    S = 64 if Hkv == 4 else 32
    most = 47000
    lens = np.concatenate([rng.integers(most - 9000, most + 1, S), [most, 0, 1, 64, 63, 0, 500, 0, 65, 2000, 129, 0]])
    lens = rng.permutation(lens)
    units = Hkv // 4                                     # per sequence
    assert units * np.maximum(1, -(-lens // 64)).sum() >= SMALL_RANGES
    c = shared_case(41, len(lens), Hkv, G, D, 32, dtype, lens)
    d = C.on_gpu(c)
    ws = E.new_q4_workspace(len(lens), Hkv * G, Hkv, D)
    ws.random_(0, 256)
    first = run(c, d, ws)
    check(c, first)
    for _ in range(4):
        ws.random_(0, 256)
        assert torch.equal(run(c, d, ws), first)


def test_many_ranges_for_few_tokens():
    """A table that allows contexts long enough for small ranges, which these few are not cut into."""
    c = C.attend_case(42, 70, 8, 4, 64, 16, "f16", np.random.default_rng(5).integers(0, 900, 70), MB=2400)
    assert 70 * 2400 * 16 // 64 >= SMALL_RANGES
    d = C.on_gpu(c)
    out = run(c, d)
    ref, bound = C.attend_reference(c)
    assert (np.abs(Q.widen(C.bits_of(out), "f16") - ref) <= bound).all()
    assert L.pkv_get_device_errors() == 0


@pytest.mark.parametrize("S,Hkv,G,D,dtype,hi", [
    (20, 8, 8, 128, "bf16", 1024), (38, 8, 5, 64, "f16", 2048), (100, 3, 7, 128, "f16", 1500), (25, 8, 6, 64, "bf16", 5600),
    (160, 1, 8, 128, "bf16", 4000), (19, 9, 4, 128, "bf16", 1100), (33, 9, 12, 64, "f16", 1200), (20, 8, 10, 128, "bf16", 2000),
])
def test_two_units_per_sm(S, Hkv, G, D, dtype, hi):
    """Between one and two units for every SM: a CTA each that fills half of one."""
    rng = np.random.default_rng(hi)
    lens = rng.integers(1, hi + 1, S)
    lens[:3] = [hi, 0, 1]
    assert 152 < S * Hkv <= 304
    c = C.attend_case(43, S, Hkv * G, Hkv, D, 16, dtype, lens)
    out = run(c, C.on_gpu(c))
    ref, bound = C.attend_reference(c)
    assert (np.abs(Q.widen(C.bits_of(out), dtype) - ref) <= bound).all()
    assert L.pkv_get_device_errors() == 0


def test_large_and_small_ranges_captured():
    """Launch control in a replayed graph, after the lengths have changed."""
    rng = np.random.default_rng(7)
    lens = rng.integers(38000, 47001, 64)
    lens[5] = 47000
    c = shared_case(44, 64, 4, 2, 64, 32, "bf16", lens)
    d = C.on_gpu(c)
    ws = E.new_q4_workspace(64, 8, 4, 64)
    out = run(c, d, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        E.paged_attention_decode_q4(out, d["q"], d["k"], d["v"], d["tables"], d["lens"], c["scale"], workspace=ws)
    for low in (38000, 1):
        now = rng.integers(low, 47001, 64)
        now[9] = 47000
        d["lens"].copy_(torch.from_numpy(now))
        out.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        check(dict(c, lens=now.astype(np.int32)), out)
