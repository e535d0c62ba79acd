"""Window attention, weight-accumulating attention and eviction against their
definitions in 64 bits.

Tolerances, from the arithmetic.  u = half a step of the output type (2^-11
fp16, 2^-8 bf16), e = 2^-24 (fp32).  A logit is D products and sums in fp32,
scaled: |dz| <= (D + 4) e Z with Z = scale max_j sum_d |q_d K_jd|; a weight
2^(z - M) then errs by 2 |dz| + 4 e relative (the maximum errs as a logit
does), the normaliser by as much, and n sums in tiles of 16 add (n / 16 + 24) e:
    w = 4 (D + 4) e Z + (n / 16 + 40) e
In P.V the weight is the sum of two 16-bit numbers: relative error u^2; in
fp16 the second one may fall below the smallest subnormal, 2^-25 absolute
against a largest weight of 1 per piece.  With A = sum_j p_j |V_j|:
    |out - ref| <= u |ref| + (1 + u) (A (w + u^2) + n 2^-25 max|V| [fp16])
               + 2^-25 [fp16: subnormal outputs]
    |score - ref| <= e |ref| + (w + G e) sum_h p_hj + 2^-126
Indices, copies and eviction are exact.
"""
import math

import numpy as np
import pytest
import torch

from oracle import bounded as B
from paged_kv_cache_162_gb300 import _lib as L
from paged_kv_cache_162_gb300 import engine as E

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def make(seed, S, H, Hkv, D, bs, dtype, lens, extra_blocks=3, MB=None):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    lens = np.asarray(lens, np.int32)
    need = [-(-int(n) // bs) for n in lens]
    MB = MB or max(1, max(need, default=1))
    NB = sum(need) + extra_blocks
    ids = torch.randperm(NB, generator=g).tolist()
    tables = np.full((S, MB), -1, np.int32)
    for s in range(S):
        for j in range(need[s]):
            tables[s, j] = ids.pop()
    c = dict(q=torch.randn(S, H, D, generator=g).to(dt), k=torch.randn(NB, bs, Hkv, D, generator=g).to(dt),
             v=torch.randn(NB, bs, Hkv, D, generator=g).to(dt), tables=tables, lens=lens,
             scale=1.0 / math.sqrt(D), S=S, H=H, Hkv=Hkv, D=D, bs=bs, NB=NB, MB=MB, dtype=dtype)
    # rows without a token hold NaN: one that reaches a result shows
    live = torch.zeros(NB * bs, dtype=torch.bool)
    for s in range(S):
        if lens[s]:
            live[torch.from_numpy(B.rows_of(tables[s], range(int(lens[s])), bs))] = True
    for x in (c["k"], c["v"]):
        x.view(-1, Hkv, D)[~live] = float("nan")
    return c


def dev(c):
    d = {k: (c[k].cuda() if isinstance(c[k], torch.Tensor) else torch.from_numpy(c[k]).cuda())
         for k in ("q", "k", "v", "tables", "lens")}
    d["out"] = torch.full(c["q"].shape, float("nan"), dtype=c["q"].dtype, device="cuda")
    return d


def f64(x):
    return x.double().numpy()


def weight_error(c, window=None, sinks=0):
    e = 2.0 ** -24
    k = np.nan_to_num(np.abs(f64(c["k"])).reshape(-1, c["Hkv"], c["D"]))
    Z = abs(c["scale"]) * float(np.einsum("shd,d->sh", np.abs(f64(c["q"])), k.max(axis=(0, 1))).max(initial=0.0))
    return 4 * (c["D"] + 4) * e * Z + (int(c["lens"].max(initial=0)) / 16 + 40) * e


def check_out(c, got, ref, mag, w):
    u = torch.finfo(DT[c["dtype"]]).eps / 2
    tiny = 2.0 ** -25 if c["dtype"] == "f16" else 0.0
    vmax = np.nan_to_num(np.abs(f64(c["v"]))).max(initial=0.0)
    n = int(c["lens"].max(initial=0))
    tol = u * np.abs(ref) + (1 + u) * (mag * (w + u * u) + n * tiny * vmax) + tiny
    err = np.abs(f64(got.cpu()) - ref)
    assert np.all(np.isfinite(f64(got.cpu())))
    assert np.all(err <= tol), f"worst excess {np.max(err - tol):.3g}, error {err.max():.3g}"


def check_window(c, window, sinks, **kw):
    d = dev(c)
    E.paged_attention_decode_window(d["out"], d["q"], d["k"], d["v"], d["tables"], d["lens"], window, sinks,
                                    c["scale"], **kw)
    torch.cuda.synchronize()
    ref, _, mag = B.attend(f64(c["q"]), f64(c["k"]), f64(c["v"]), c["tables"], c["lens"], c["scale"], window, sinks)
    check_out(c, d["out"], ref, mag, weight_error(c))
    return d


def check_accumulate(c, cap=None, seed=0, **kw):
    d = dev(c)
    cap = cap or c["MB"] * c["bs"]
    before = torch.rand(c["S"], c["Hkv"], cap, generator=torch.Generator().manual_seed(seed))
    scores = before.cuda()
    E.paged_attention_decode_accumulate(d["out"], scores, d["q"], d["k"], d["v"], d["tables"], d["lens"], c["scale"],
                                        **kw)
    torch.cuda.synchronize()
    ref, weights, mag = B.attend(f64(c["q"]), f64(c["k"]), f64(c["v"]), c["tables"], c["lens"], c["scale"])
    w = weight_error(c)
    check_out(c, d["out"], ref, mag, w)
    want = B.accumulate(before.numpy(), weights, c["Hkv"])
    e = 2.0 ** -24
    added = want - before.double().numpy()
    tol = e * np.abs(want) + (w + (c["H"] // c["Hkv"]) * e) * added + 2.0 ** -126
    got = scores.cpu()
    assert np.all(np.abs(f64(got) - want) <= tol), f"worst {np.abs(f64(got) - want).max():.3g}"
    for s in range(c["S"]):  # entries past the context as they were
        assert torch.equal(got[s, :, int(c["lens"][s]):], before[s, :, int(c["lens"][s]):])
    return d, scores


# lengths around tiles, blocks, the window and the sinks; empty and one-token
# contexts; first the one-CTA form (short visible lengths), then the split form
SHORT = [0, 1, 2, 15, 16, 17, 31, 33, 64, 100]
LONG = [0, 1, 700, 513, 64, 1300, 2049]


@pytest.mark.parametrize("dtype,D,bs,H,Hkv", [
    ("f16", 64, 8, 4, 4), ("bf16", 128, 16, 8, 2), ("f16", 128, 32, 5, 5), ("bf16", 64, 64, 14, 2),
    ("f16", 128, 16, 16, 1), ("bf16", 128, 8, 9, 1), ("bf16", 64, 16, 6, 6)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (17, 4), (5, 33), (64, 16), (1000, 0), (1, 1)])
def test_window_short(dtype, D, bs, H, Hkv, window, sinks):
    c = make(7 + D + H, len(SHORT), H, Hkv, D, bs, dtype, SHORT)
    check_window(c, window, sinks, max_context_len=100)


@pytest.mark.parametrize("dtype,D,bs,H,Hkv", [
    ("f16", 128, 16, 4, 4), ("bf16", 128, 32, 16, 4), ("f16", 64, 8, 6, 2), ("bf16", 64, 64, 12, 1),
    ("f16", 128, 64, 3, 3), ("bf16", 128, 16, 32, 2)])
@pytest.mark.parametrize("window,sinks", [(600, 4), (1021, 33), (5000, 0), (1, 512)])
def test_window_long(dtype, D, bs, H, Hkv, window, sinks):
    c = make(11 + D + H, len(LONG), H, Hkv, D, bs, dtype, LONG)
    check_window(c, window, sinks)


@pytest.mark.parametrize("dtype,D,bs,H,Hkv", [
    ("f16", 64, 8, 4, 4), ("bf16", 128, 16, 8, 2), ("f16", 128, 64, 16, 1), ("bf16", 64, 32, 27, 3)])
def test_accumulate_short(dtype, D, bs, H, Hkv):
    c = make(5 + D + H, len(SHORT), H, Hkv, D, bs, dtype, SHORT)
    check_accumulate(c)


@pytest.mark.parametrize("dtype,D,bs,H,Hkv", [
    ("f16", 128, 16, 4, 4), ("bf16", 128, 32, 16, 4), ("f16", 64, 8, 6, 2), ("bf16", 64, 64, 12, 1),
    ("f16", 128, 64, 3, 3), ("bf16", 128, 16, 32, 2)])
def test_accumulate_long(dtype, D, bs, H, Hkv):
    c = make(13 + D + H, len(LONG), H, Hkv, D, bs, dtype, LONG)
    check_accumulate(c, cap=c["MB"] * bs + 5)


def evict_case(seed, S, Hkv, D, bs, dtype, lens, budget, again=True, cap=None):
    """Scores with ties, infinities and NaN; half of the sequences evicted
    before (shuffled stored positions)."""
    rng = np.random.default_rng(seed)
    c = make(seed, S, Hkv, Hkv, D, bs, dtype, lens)
    cap = cap or c["MB"] * bs
    score = np.exp(rng.standard_normal((S, Hkv, cap))).astype(np.float32)
    score[rng.random(score.shape) < 0.3] = 0.5
    score[rng.random(score.shape) < 0.1] = 0.0
    score[rng.random(score.shape) < 0.05] = -0.0
    for v in (np.nan, np.inf, -np.inf, -1.0):
        score[rng.random(score.shape) < 0.02] = v
    pos = np.full((S, Hkv, cap), -1, np.int32)
    seen = c["lens"].copy()
    for s in range(S):
        old = min(int(c["lens"][s]), budget)
        if again and s % 2 and old:
            seen[s] += 2 * old
            for g in range(Hkv):
                pos[s, g, :old] = rng.permutation(3 * old)[:old]
    c.update(score=score, pos=pos, seen=seen, cap=cap)
    return c


def check_evict(c, budget, recent, sinks, in_place=False):
    d = dev(c)
    score, pos = torch.from_numpy(c["score"].copy()).cuda(), torch.from_numpy(c["pos"].copy()).cuda()
    if in_place:
        so, po = score, pos
    else:
        so, po = torch.full_like(score, 7.0), torch.full_like(pos, -7)
    so0, po0 = so.cpu().numpy().copy(), po.cpu().numpy().copy()
    new = torch.full_like(d["lens"], -1)
    E.evict_tokens(d["k"], d["v"], score, pos, d["tables"], d["lens"], torch.from_numpy(c["seen"]).cuda(), new, budget,
                   recent, sinks, scores_out=None if in_place else so, positions_out=None if in_place else po)
    torch.cuda.synchronize()
    k, v = c["k"].view(torch.int16).numpy().copy(), c["v"].view(torch.int16).numpy().copy()
    ws, wp = c["score"].copy(), c["pos"].copy()
    lens = B.evict(k, v, ws, wp, c["tables"], c["lens"], c["seen"], budget, recent, sinks)
    for s in range(c["S"]):  # entries past the context are not touched
        n = int(c["lens"][s])
        ws[s, :, n:], wp[s, :, n:] = so0[s, :, n:], po0[s, :, n:]
    assert np.array_equal(new.cpu().numpy(), lens)
    assert np.array_equal(po.cpu().numpy(), wp), "positions"
    assert np.array_equal(so.cpu().numpy(), ws, equal_nan=True), "scores"
    assert np.array_equal(d["k"].view(torch.int16).cpu().numpy(), k), "K"
    assert np.array_equal(d["v"].view(torch.int16).cpu().numpy(), v), "V"


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype,D,bs,Hkv,budget,recent,sinks", [
    ("f16", 64, 8, 3, 32, 8, 4), ("bf16", 128, 16, 2, 33, 0, 0), ("f16", 128, 64, 1, 1, 1, 0),
    ("bf16", 64, 16, 5, 1, 0, 0), ("bf16", 128, 32, 4, 60, 56, 4), ("f16", 64, 8, 2, 500, 100, 7)])
def test_evict(dtype, D, bs, Hkv, budget, recent, sinks, in_place):
    lens = SHORT + [257, 1000, 1025]
    c = evict_case(3 * D + budget, len(lens), Hkv, D, bs, dtype, lens, budget)
    check_evict(c, budget, recent, sinks, in_place)


@pytest.mark.parametrize("n,budget,S,Hkv", [(9000, 4100, 1, 1), (20001, 300, 2, 1), (33000, 32999, 1, 2)])
def test_evict_long_rows_over_several_ctas(n, budget, S, Hkv):
    c = evict_case(n, S, Hkv, 64, 64, "f16", [n] * S, budget)
    check_evict(c, budget, 100, 4)
