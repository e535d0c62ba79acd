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


# --------------------------------------------------- shapes of the work split
@pytest.mark.parametrize("S,H,Hkv,n,window", [
    (1, 1, 1, 40000, 39000), (1, 16, 1, 20000, 19999), (3, 8, 4, 9000, 8500), (1, 6, 3, 2000, 1800),
    (2, 4, 4, 12000, 5000), (9, 12, 6, 1500, 1400)])
def test_window_few_rows_many_pieces(S, H, Hkv, n, window):
    """One sequence over many CTAs: clusters, and units cut into many pieces."""
    c = make(n + H, S, H, Hkv, 64, 16, "bf16", [n - 37 * s for s in range(S)])
    check_window(c, window, 5)


@pytest.mark.parametrize("S,H,Hkv,n", [(1, 4, 1, 30000), (2, 8, 8, 5000), (16, 4, 4, 3000), (5, 32, 2, 2500)])
def test_accumulate_few_rows_many_pieces(S, H, Hkv, n):
    c = make(n + H, S, H, Hkv, 64, 32, "f16", [n - 41 * s for s in range(S)])
    check_accumulate(c)


@pytest.mark.parametrize("S", [700, 3001])
def test_many_short_sequences(S):
    """More sequences than threads that plan, lengths 0 to 40, some long."""
    rng = np.random.default_rng(S)
    lens = rng.integers(0, 41, S)
    lens[rng.integers(0, S, 3)] = 700
    c = make(S, S, 2, 2, 64, 8, "f16", lens)
    check_window(c, 600, 2)
    check_accumulate(c)
    check_window(c, 20, 3)


def test_contexts_much_shorter_than_the_bound():
    """max_context_len says little about the lengths: the split form, with
    ranges and stretches that hold nothing."""
    c = make(3, 4, 8, 2, 128, 16, "bf16", [5, 0, 130, 33], MB=4096)
    check_window(c, 60000, 4)
    check_accumulate(c, max_context_len=4096)


def test_rows_behind_the_last_sequence_stay():
    c = make(4, 3, 8, 4, 64, 16, "f16", [700, 20, 1])
    d = dev(c)
    out = torch.full((5, 8, 64), 7.0, dtype=torch.float16, device="cuda")
    cap = c["MB"] * 16
    scores = torch.full((5, 4, cap), 3.0, device="cuda")
    ws = E.new_accumulate_workspace(3, 8, 4, 64, cap)
    E.paged_attention_decode_window(out[:3], d["q"], d["k"], d["v"], d["tables"], d["lens"], 600, 2)
    E.paged_attention_decode_accumulate(out[:3], scores[:3], d["q"], d["k"], d["v"], d["tables"], d["lens"],
                                        workspace=ws)
    torch.cuda.synchronize()
    assert (out[3:] == 7).all() and (scores[3:] == 3).all()


@pytest.mark.parametrize("offset,cap_extra", [(1, 0), (0, 1), (3, 2)])
def test_unaligned_rows(offset, cap_extra):
    """Score and position rows that do not start on 16 bytes."""
    c = make(6, 4, 4, 4, 64, 16, "f16", [900, 100, 513, 64])
    d = dev(c)
    cap = c["MB"] * 16 + cap_extra
    before = torch.rand(4 * 4 * cap + offset)
    flat = before.cuda()
    scores = flat[offset:].view(4, 4, cap)
    E.paged_attention_decode_accumulate(d["out"], scores, d["q"], d["k"], d["v"], d["tables"], d["lens"], c["scale"])
    ref, weights, _ = B.attend(f64(c["q"]), f64(c["k"]), f64(c["v"]), c["tables"], c["lens"], c["scale"])
    want = B.accumulate(before[offset:].view(4, 4, cap).numpy(), weights, 4)
    e, w = 2.0 ** -24, weight_error(c)
    assert np.all(np.abs(f64(scores.cpu()) - want) <= e * np.abs(want) + (w + e) * 1.0)
    ev = evict_case(7, 4, 4, 64, 16, "f16", [900, 100, 513, 64], 90, cap=cap)
    d = dev(ev)
    flat_s = torch.zeros(4 * 4 * cap + offset, device="cuda")
    flat_p = torch.zeros(4 * 4 * cap + offset, dtype=torch.int32, device="cuda")
    s2, p2 = flat_s[offset:].view(4, 4, cap), flat_p[offset:].view(4, 4, cap)
    s2.copy_(torch.from_numpy(ev["score"]))
    p2.copy_(torch.from_numpy(ev["pos"]))
    new = torch.empty_like(d["lens"])
    E.evict_tokens(d["k"], d["v"], s2, p2, d["tables"], d["lens"], torch.from_numpy(ev["seen"]).cuda(), new, 90, 20, 4)
    k, v = ev["k"].view(torch.int16).numpy().copy(), ev["v"].view(torch.int16).numpy().copy()
    B.evict(k, v, ev["score"], ev["pos"], ev["tables"], ev["lens"], ev["seen"], 90, 20, 4)
    assert np.array_equal(s2.cpu().numpy(), ev["score"], equal_nan=True)
    assert np.array_equal(p2.cpu().numpy(), ev["pos"])
    assert np.array_equal(d["k"].view(torch.int16).cpu().numpy(), k)


def test_offsets_past_32_bits():
    """Blocks whose element offsets pass 2^31: the last ones of 5 GB caches."""
    Hkv, D, bs = 32, 128, 64
    NB = 10000                       # 2.6e9 elements each
    k = torch.zeros(NB, bs, Hkv, D, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    c = make(8, 2, Hkv, Hkv, D, bs, "f16", [900, 130], extra_blocks=0)
    used = c["NB"]
    k[NB - used:] = c["k"].cuda().nan_to_num_()
    v[NB - used:] = c["v"].cuda().nan_to_num_()
    tables = np.where(c["tables"] >= 0, c["tables"] + NB - used, -1).astype(np.int32)
    out = torch.empty(2, Hkv, D, dtype=torch.float16, device="cuda")
    q, lens = c["q"].cuda(), torch.from_numpy(c["lens"]).cuda()
    cap = c["MB"] * bs
    scores = torch.zeros(2, Hkv, cap, device="cuda")
    ref, weights, mag = B.attend(f64(c["q"]), np.nan_to_num(f64(c["k"])), np.nan_to_num(f64(c["v"])), c["tables"],
                                 c["lens"], c["scale"])
    t = torch.from_numpy(tables).cuda()
    E.paged_attention_decode_accumulate(out, scores, q, k, v, t, lens, c["scale"])
    check_out(c, out, ref, mag, weight_error(c))
    E.paged_attention_decode_window(out, q, k, v, t, lens, 100, 4, c["scale"])
    ref, _, mag = B.attend(f64(c["q"]), np.nan_to_num(f64(c["k"])), np.nan_to_num(f64(c["v"])), c["tables"], c["lens"],
                           c["scale"], 100, 4)
    check_out(c, out, ref, mag, weight_error(c))
    pos = torch.full((2, Hkv, cap), -1, dtype=torch.int32, device="cuda")
    sc, new = scores.cpu().numpy().copy(), torch.empty_like(lens)
    E.evict_tokens(k, v, scores, pos, t, lens, lens.clone(), new, 128, 32, 4)
    kk = c["k"].nan_to_num().view(torch.int16).numpy().copy()
    vv = c["v"].nan_to_num().view(torch.int16).numpy().copy()
    B.evict(kk, vv, sc, np.full(sc.shape, -1, np.int32), c["tables"], c["lens"], c["lens"], 128, 32, 4)
    assert np.array_equal(k[NB - used:].view(torch.int16).cpu().numpy(), kk)
    assert np.array_equal(v[NB - used:].view(torch.int16).cpu().numpy(), vv)
    assert (k[:NB - used] == 0).all()


# ------------------------------------------------------------- bad pages
def test_released_blocks_outside_the_window_are_not_looked_up():
    """Entries the window has passed may be anything."""
    L.pkv_get_device_errors()
    for lens, window in (([100, 64, 33], 20), ([1500, 1900], 600)):
        c = make(12, len(lens), 4, 2, 64, 16, "bf16", lens)
        ref, _, mag = B.attend(f64(c["q"]), f64(c["k"]), f64(c["v"]), c["tables"], c["lens"], c["scale"], window, 5)
        for s, n in enumerate(lens):
            seen = {j // 16 for j in B.visible(n, window, 5)}
            for lb in range(c["MB"]):
                if lb not in seen:
                    c["tables"][s, lb] = [-1, 1 << 30, -(1 << 31)][lb % 3]
        d = dev(c)
        E.paged_attention_decode_window(d["out"], d["q"], d["k"], d["v"], d["tables"], d["lens"], window, 5, c["scale"])
        check_out(c, d["out"], ref, mag, weight_error(c))
        assert L.pkv_get_device_errors() == 0


@pytest.mark.parametrize("lens", [[40, 90], [900, 1300]])
def test_bad_blocks_and_lengths_are_flagged_and_skipped(lens):
    """A visible block out of range holds no tokens; lengths are clamped."""
    L.pkv_get_device_errors()
    c = make(13, 2, 4, 2, 64, 16, "f16", lens)
    good = c["tables"].copy()
    c["tables"][0, 1] = c["NB"]
    c["tables"][1, 0] = -7
    d = dev(c)
    cap = c["MB"] * 16
    scores = torch.zeros(2, 2, cap, device="cuda")
    E.paged_attention_decode_accumulate(d["out"], scores, d["q"], d["k"], d["v"], d["tables"], d["lens"], c["scale"])
    assert L.pkv_get_device_errors() == L.PKV_DEVERR_BLOCK_ID
    assert torch.isfinite(d["out"].float()).all()
    # the tokens of the bad blocks weigh nothing, the others 1 per query head
    assert (scores[0, :, 16:32] == 0).all() and (scores[1, :, :16] == 0).all()
    assert torch.allclose(scores.sum(-1), torch.full((2, 2), 2.0, device="cuda"), atol=1e-4)
    E.paged_attention_decode_window(d["out"], d["q"], d["k"], d["v"], d["tables"], d["lens"], 30, 20, c["scale"])
    assert L.pkv_get_device_errors() == L.PKV_DEVERR_BLOCK_ID
    d["tables"] = torch.from_numpy(good).cuda()
    for bad in (-5, cap + 1, 2 ** 31 - 1, -2 ** 31):
        n = torch.tensor([bad, lens[1]], dtype=torch.int32, device="cuda")
        E.paged_attention_decode_window(d["out"], d["q"], d["k"], d["v"], d["tables"], n, 30, 4, c["scale"],
                                        max_context_len=lens[0])
        flags = L.pkv_get_device_errors()
        assert flags == L.PKV_DEVERR_CONTEXT
        if bad < 0:
            assert (d["out"][0] == 0).all()
    new = torch.empty_like(d["lens"])
    pos = torch.full((2, 2, cap), -1, dtype=torch.int32, device="cuda")
    E.evict_tokens(d["k"], d["v"], scores, pos, d["tables"], d["lens"], d["lens"] - 1, new, 20, 4)  # seen < cached
    assert L.pkv_get_device_errors() == L.PKV_DEVERR_CONTEXT and new.tolist() == [20, 20]
    d = dev(c)                                     # the bad tables again
    k0 = d["k"].clone()
    scores = torch.rand(2, 2, cap, device="cuda")
    pos.fill_(-1)
    E.evict_tokens(d["k"], d["v"], scores, pos, d["tables"], d["lens"], d["lens"], new, 20, 4)
    flags = L.pkv_get_device_errors()
    assert flags in (0, L.PKV_DEVERR_BLOCK_ID)
    untouched = torch.ones(c["NB"], dtype=torch.bool)
    untouched[c["tables"][(c["tables"] >= 0) & (c["tables"] < c["NB"])]] = False
    assert torch.equal(d["k"].view(torch.int16)[untouched.cuda()], k0.view(torch.int16)[untouched.cuda()])


def test_infinities_in_keys_and_large_logits():
    """K = -inf and +-60000 logits: weights 0 or 1, nothing overflows."""
    c = make(14, 2, 2, 2, 64, 16, "f16", [40, 700])
    c["q"].abs_()
    r = B.rows_of(c["tables"][1], [3, 4, 699], 16)
    rows = c["k"].view(-1, 2, 64)
    rows[r[0]] = -float("inf")
    rows[r[1]] = -60000.0
    rows[r[2]] = 3000.0
    d = dev(c)
    scores = torch.zeros(2, 2, c["MB"] * 16, device="cuda")
    E.paged_attention_decode_accumulate(d["out"], scores, d["q"], d["k"], d["v"], d["tables"], d["lens"], c["scale"])
    assert torch.equal(scores[1, :, 699], torch.ones(2, device="cuda"))
    assert (scores[1, :, :699] == 0).all()
    assert torch.equal(d["out"][1], d["v"].view(-1, 2, 64)[int(r[2])])


# ---------------------------------------- calls that follow and overlap others
def all_three(c, d, ws, scores, pos, new, outs):
    E.paged_attention_decode_window(outs[0], d["q"], d["k"], d["v"], d["tables"], d["lens"], 500, 4, c["scale"],
                                    workspace=ws[0])
    E.paged_attention_decode_accumulate(outs[1], scores, d["q"], d["k"], d["v"], d["tables"], d["lens"], c["scale"],
                                        workspace=ws[1])
    E.evict_tokens(d["k"], d["v"], scores, pos, d["tables"], d["lens"], d["lens"], new, 300, 50, 4, workspace=ws[2])


def state_of(c, d):
    cap = c["MB"] * c["bs"]
    ws = (E.new_window_workspace(c["S"], c["H"], c["Hkv"], c["D"]),
          E.new_accumulate_workspace(c["S"], c["H"], c["Hkv"], c["D"], cap),
          E.new_evict_workspace(c["S"], c["Hkv"], 300))
    for w in ws:
        w.fill_(0xff)               # no initial contents are needed
    scores = torch.rand(c["S"], c["Hkv"], cap, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    pos = torch.full((c["S"], c["Hkv"], cap), -1, dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(d["q"]) for _ in range(2)]
    return ws, scores, pos, torch.zeros_like(d["lens"]), outs


def results(d, st):
    ws, scores, pos, new, outs = st
    torch.cuda.synchronize()
    return [x.clone() for x in (d["k"], d["v"], scores, pos, new, *outs)]


def same(a, b):
    return all(torch.equal(x.view(torch.int16) if x.element_size() == 2 else x.view(torch.int32),
                           y.view(torch.int16) if y.element_size() == 2 else y.view(torch.int32))
               for x, y in zip(a, b))


@pytest.mark.parametrize("H,Hkv,D,dtype", [(8, 8, 128, "f16"), (12, 3, 64, "bf16"), (32, 4, 128, "bf16")])
def test_same_bits_every_time_in_graphs_and_on_streams(H, Hkv, D, dtype):
    c = make(21, 6, H, Hkv, D, 16, dtype, [2000, 1, 700, 0, 513, 1300])
    d = dev(c)
    st = state_of(c, d)
    all_three(c, d, *st)
    want = results(d, st)
    for _ in range(5):
        d2 = dev(c)
        st2 = state_of(c, d2)
        all_three(c, d2, *st2)
        assert same(results(d2, st2), want)
    # captured twice over the same workspaces, replayed in turn
    d3 = dev(c)
    st3 = state_of(c, d3)
    k0, v0, s0 = d3["k"].clone(), d3["v"].clone(), st3[1].clone()
    graphs = []
    side = torch.cuda.Stream()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            d3["k"].copy_(k0)
            d3["v"].copy_(v0)
            st3[1].copy_(s0)
            st3[2].fill_(-1)
            all_three(c, d3, *st3)
        graphs.append(g)
    for g in graphs + graphs[::-1]:
        for o in st3[4]:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        assert same(results(d3, st3), want)
    # two streams at once, each with its own state; torch's current stream, and one given by handle
    streams = [torch.cuda.Stream() for _ in range(2)]
    ds = [dev(c) for _ in range(2)]
    sts = [state_of(c, x) for x in ds]
    torch.cuda.synchronize()
    for x, y, stream in zip(ds, sts, streams):
        with torch.cuda.stream(stream):
            all_three(c, x, *y)
    for x, y in zip(ds, sts):
        assert same(results(x, y), want)
    d4 = dev(c)
    ws, scores, pos, new, outs = state_of(c, d4)
    torch.cuda.synchronize()
    sd = streams[0]
    E.paged_attention_decode_window(outs[0], d4["q"], d4["k"], d4["v"], d4["tables"], d4["lens"], 500, 4, c["scale"],
                                    stream=sd)
    E.paged_attention_decode_accumulate(outs[1], scores, d4["q"], d4["k"], d4["v"], d4["tables"], d4["lens"],
                                        c["scale"], stream=sd.cuda_stream)
    E.evict_tokens(d4["k"], d4["v"], scores, pos, d4["tables"], d4["lens"], d4["lens"], new, 300, 50, 4, stream=sd)
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]  # freed memory is not theirs yet
    assert same(results(d4, (ws, scores, pos, new, outs)), want)
    del junk


def test_queries_and_output_in_pinned_host_memory():
    c = make(22, 4, 8, 4, 64, 16, "f16", [900, 3, 0, 64])
    d = dev(c)
    for window in (30, 800):
        q, out = c["q"].pin_memory(), torch.zeros_like(c["q"]).pin_memory()
        E.paged_attention_decode_window(out, q, d["k"], d["v"], d["tables"], d["lens"], window, 4, c["scale"])
        E.paged_attention_decode_window(d["out"], d["q"], d["k"], d["v"], d["tables"], d["lens"], window, 4, c["scale"])
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), d["out"].cpu().view(torch.int16))


def test_refusals_of_tensor_calls():
    c = make(23, 2, 4, 2, 64, 16, "f16", [40, 20])
    d = dev(c)
    a = dict(out=d["out"], q=d["q"], k_cache=d["k"], v_cache=d["v"], block_tables=d["tables"], context_lens=d["lens"],
             window=8)
    for kw in (dict(q=d["q"].float()), dict(q=d["q"].transpose(0, 1)), dict(out=d["out"][:1]), dict(v_cache=d["v"][:1]),
               dict(block_tables=d["tables"].long()), dict(context_lens=d["lens"].cpu()), dict(out=d["out"].cpu()),
               dict(context_lens=d["lens"][:1]), dict(v_cache=d["v"].bfloat16()), dict(window=0), dict(sink_tokens=-1),
               dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
               dict(workspace=torch.empty(1 << 20, dtype=torch.uint8)), dict(max_context_len=49),
               dict(k_cache=d["k"].float(), v_cache=d["v"].float(), q=d["q"].float(), out=d["out"].float())):
        with pytest.raises(L.PkvError):
            E.paged_attention_decode_window(**{**a, **kw})
    q = torch.zeros(2, 34, 64, dtype=torch.float16, device="cuda")   # 17 query heads per KV head
    with pytest.raises(L.PkvError):
        E.paged_attention_decode_window(torch.empty_like(q), q, d["k"], d["v"], d["tables"], d["lens"], 8)
    with pytest.raises(L.PkvError):                                  # not a multiple
        E.paged_attention_decode_window(torch.empty_like(q[:, :3].contiguous()), q[:, :3].contiguous(), d["k"], d["v"],
                                        d["tables"], d["lens"], 8)
    sc = torch.zeros(2, 2, 48, device="cuda")
    del a["window"]
    for bad in (sc.double(), sc[:, :1], sc[..., :47].contiguous(), sc.transpose(1, 2), sc.cpu(), sc[0]):
        with pytest.raises(L.PkvError):
            E.paged_attention_decode_accumulate(scores=bad, **a)
    pos, new = torch.full((2, 2, 48), -1, dtype=torch.int32, device="cuda"), torch.zeros_like(d["lens"])
    e = dict(k_cache=d["k"], v_cache=d["v"], scores=sc, positions=pos, block_tables=d["tables"],
             context_lens=d["lens"], token_counts=d["lens"], new_context_lens=new, budget=10, recent_tokens=2)
    for kw in (dict(scores=sc.half()), dict(positions=pos.long()), dict(scores_out=sc[:1]), dict(budget=0),
               dict(budget=1), dict(new_context_lens=d["lens"]), dict(token_counts=d["lens"].cpu()),
               dict(scores=sc[..., :40].contiguous()), dict(positions_out=pos.transpose(1, 2)), dict(recent_tokens=-1)):
        with pytest.raises(L.PkvError):
            E.evict_tokens(**{**e, **kw})
    assert L.pkv_get_device_errors() == 0
    for call in (lambda: E.paged_attention_decode_window(window=8, **a), lambda: E.evict_tokens(**e)):
        call()                                                       # the same calls without the faults
    torch.cuda.synchronize()


@pytest.mark.parametrize("n", [8 * 48 * 1024 + 5000])
def test_evict_rows_longer_than_the_shared_memory_of_a_cluster(n):
    c = evict_case(n, 1, 1, 64, 64, "f16", [n], 20000, again=False)
    check_evict(c, 20000, 1000, 4, in_place=True)
    check_evict(c, 20000, 1000, 4)


@pytest.mark.parametrize("value", [0.0, 1.0, float("nan"), -float("inf"), 1e-40])
def test_evict_equal_scores(value):
    """Nothing but ties, over one CTA and over a cluster."""
    for n, budget in ((300, 299), (300, 1), (9000, 4000)):
        c = evict_case(n, 1, 2, 64, 16, "f16", [n], budget, again=False)
        c["score"][:] = value
        check_evict(c, budget, 0, 0)


# ------------------------------------------------------------ random and extreme
@pytest.mark.parametrize("seed", range(16))
def test_random_shapes(seed):
    rng = np.random.default_rng(900 + seed)
    D, bs = int(rng.choice([64, 128])), int(rng.choice([8, 16, 32, 64]))
    Hkv = int(rng.choice([1, 2, 3, 4, 5, 6, 8, 12]))
    G = int(rng.integers(1, 17))
    S = int(rng.integers(1, 12))
    top = int(rng.choice([20, 200, 2500]))
    lens = rng.integers(0, top + 1, S)
    lens[rng.random(S) < 0.15] = 0
    dtype = ["f16", "bf16"][seed % 2]
    c = make(seed, S, Hkv * G, Hkv, D, bs, dtype, lens, MB=max(1, -(-top // bs)) + int(rng.integers(0, 3)))
    c["scale"] *= float(rng.choice([1.0, 0.1, -1.0, 0.0, 3.0]))
    check_window(c, int(rng.integers(1, top + 10)), int(rng.integers(0, 40)), max_context_len=int(rng.choice([0, top])))
    cap = c["MB"] * bs + int(rng.integers(0, 9))
    check_accumulate(c, cap=cap, seed=seed, max_context_len=int(rng.choice([0, top])))
    budget = int(rng.integers(1, top + 5))
    sinks = int(rng.integers(0, budget + 1)) if seed % 3 else 0
    e = evict_case(seed, S, Hkv, D, bs, dtype, lens, budget, cap=max(cap, -(-top // bs) * bs))
    check_evict(e, budget, int(rng.integers(0, budget - sinks + 1)), sinks, in_place=bool(seed % 2))


def test_the_most_sequences():
    S = 32767
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 4, S)
    c = make(1, S, 2, 1, 64, 8, "f16", lens, MB=1)
    check_window(c, 2, 1)
    check_accumulate(c)
    e = evict_case(2, S, 1, 64, 8, "f16", lens, 2, cap=8)
    check_evict(e, 2, 1, 1)


def test_one_very_long_context():
    c = make(2, 1, 3, 1, 64, 64, "bf16", [300001])
    check_accumulate(c)
    check_window(c, 2 ** 31 - 1, 2 ** 31 - 1)
    check_window(c, 250000, 7)
    check_window(c, 3, 0)


@pytest.mark.parametrize("scores_in_place", [True, False])
def test_evict_with_one_output_in_place(scores_in_place):
    c = evict_case(31, 3, 2, 64, 16, "bf16", [300, 40, 129], 60)
    d = dev(c)
    score, pos = torch.from_numpy(c["score"].copy()).cuda(), torch.from_numpy(c["pos"].copy()).cuda()
    so = score if scores_in_place else torch.full_like(score, 7.0)
    po = torch.full_like(pos, -7) if scores_in_place else pos
    s0, p0 = score.clone(), pos.clone()
    new = torch.empty_like(d["lens"])
    E.evict_tokens(d["k"], d["v"], score, pos, d["tables"], d["lens"], torch.from_numpy(c["seen"]).cuda(), new, 60, 10, 4,
                   scores_out=so, positions_out=po)
    k, v = c["k"].view(torch.int16).numpy().copy(), c["v"].view(torch.int16).numpy().copy()
    ws, wp = c["score"].copy(), c["pos"].copy()
    B.evict(k, v, ws, wp, c["tables"], c["lens"], c["seen"], 60, 10, 4)
    for s, n in enumerate(c["lens"]):
        assert np.array_equal(so[s, :, :n].cpu().numpy(), ws[s, :, :n], equal_nan=True)
        assert np.array_equal(po[s, :, :n].cpu().numpy(), wp[s, :, :n])
    assert np.array_equal(d["k"].view(torch.int16).cpu().numpy(), k)
    other, was = (pos, p0) if scores_in_place else (score, s0)
    assert torch.equal(other.view(torch.int32), was.view(torch.int32)), "an input that is no output stays"


# ------------------------------------------------- every form a call can take
@pytest.mark.parametrize("S,H,Hkv,D,lo,hi", [
    (100, 8, 8, 128, 0, 40),       # waves of direct CTAs
    (140, 16, 8, 64, 100, 250),    # the same, split with scores
    (300, 16, 8, 64, 0, 64),       # split, ranges of two tiles, a warp per head
    (900, 6, 2, 128, 1, 30),       # two warps per head
    (700, 5, 5, 64, 1, 70),        # four
    (1, 64, 4, 128, 220, 220),     # one CTA per head, four threads fold a token
    (2, 40, 5, 64, 600, 700),      # clusters, two threads
    (3, 30, 3, 128, 1900, 2100)])
def test_forms_of_attention(S, H, Hkv, D, lo, hi):
    rng = np.random.default_rng(S + H)
    lens = rng.integers(lo, hi + 1, S)
    c = make(S + D, S, H, Hkv, D, 16, "bf16" if D == 128 else "f16", lens)
    check_window(c, hi, 0)
    check_window(c, max(1, hi // 2), 3)
    check_accumulate(c, cap=c["MB"] * 16 + 4 * (S % 2))


@pytest.mark.parametrize("S,Hkv,D,lo,hi,budget", [
    (100, 7, 64, 300, 420, 200),       # rows that wait for a place
    (110, 7, 128, 200, 300, 90),       # the same with short rows
    (30, 4, 128, 100, 150, 140),       # short rows
    (16, 8, 64, 400, 1000, 480),       # room for larger CTAs, many moves
    (2, 3, 128, 6000, 9000, 3001),     # clusters of them
    (2, 2, 64, 6000, 9000, 8800)])     # clusters, few moves
def test_forms_of_eviction(S, Hkv, D, lo, hi, budget):
    rng = np.random.default_rng(S + hi)
    lens = rng.integers(lo, hi + 1, S)
    lens[0] = hi
    c = evict_case(S + D, S, Hkv, D, 32, "f16", lens, budget)
    check_evict(c, budget, budget // 3, 5, in_place=bool(S % 4))


@pytest.mark.parametrize("S,H,Hkv,D,hi", [(60, 64, 32, 128, 400), (70, 32, 32, 64, 900), (300, 16, 8, 128, 300)])
def test_lengths_far_below_the_bound_on_a_used_workspace(S, H, Hkv, D, hi):
    """Small ranges for the bound, but none for the lengths: a unit's pieces
    are those of its ranges, not what lies between them in the workspace."""
    rng = np.random.default_rng(S)
    c = make(S + D, S, H, Hkv, D, 16, "bf16", rng.integers(0, hi + 1, S), MB=64)
    ws = E.new_window_workspace(S, H, Hkv, D)
    check_window(c, 1024, 0, workspace=ws.fill_(255))
    ws = E.new_accumulate_workspace(S, H, Hkv, D, 1024)
    check_accumulate(c, workspace=ws.fill_(255))
