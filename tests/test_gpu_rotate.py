"""The rotating appends and the gather from a 4-bit cache against their definitions.

A rotated element a c - b s has two products and a sum in fp32, each rounded:
off by at most 2.01 e (|a c| + |b s|), e = 2^-24; then half a step u of the type
it is stored in (or 2^-25, below fp16's normal numbers).  Everything else of
the 16-bit form is a copy.  In the 4-bit form codes, steps and centres have to be
those of the definition evaluated with fp32 operations (bytes equal), and an
element x reads as a value within
    step (1/2 + 2^-18) + 8 u step + u |centre| + 4.02 e (|a c| + |b s|) + 2^-20
of x: half a step; the ends of the 16 values moved by the rounding of step and
centre; the rotation's error in x and in the group's bounds; in fp16 a step below
the normal numbers is off by 2^-25, at up to 8 codes 2^-22, and one rounded to 0
leaves its group at the centre, 7.5 2^-25 away, and the centre's 2^-25.
"""
import numpy as np
import pytest
import torch

import q4_cases as C
from oracle import q4 as Q
from paged_kv_cache_162_gb300 import _lib as L
from paged_kv_cache_162_gb300 import engine as E

pytestmark = pytest.mark.gpu


def call(c, d, q4, k_cache, v_cache, query_out, **kw):
    f = E.rotate_and_cache_q4 if q4 else E.rotate_and_cache
    return f(d["key"], d["value"], k_cache, v_cache, d["tables"], d["seq"], d["pos"], d["slots"], d["table"],
             query=d["query"], query_out=query_out, rotary_pos=d["turn"], interleaved=c["interleaved"], **kw)


def check16(got_bits, ref, mag, dtype):
    got = Q.widen(got_bits, dtype)
    u = C.U[dtype]
    bound = u * np.abs(ref) + (1 + u) * 2.01 * C.E32 * mag + 2.0 ** -25
    bad = np.abs(got - ref) > bound
    assert not bad.any(), np.abs(got - ref)[bad].max()


CASES = [
    dict(S=1, H=1, Hkv=1, D=64, bs=8, dtype="f16", new=[1], R=64),
    dict(S=4, H=4, Hkv=4, D=64, bs=16, dtype="f16", new=[1, 1, 1, 1], before=[0, 7, 15, 99]),
    dict(S=3, H=5, Hkv=5, D=128, bs=8, dtype="bf16", new=[9, 1, 70], before=[3, 0, 8], interleaved=True, fused=True),
    dict(S=3, H=32, Hkv=8, D=128, bs=16, dtype="bf16", new=[33, 1, 16], before=[0, 4095, 1], pad=3, fused=True),
    dict(S=2, H=6, Hkv=2, D=128, bs=32, dtype="f16", new=[65, 2], R=64, fused=True),
    dict(S=2, H=6, Hkv=2, D=128, bs=64, dtype="f16", new=[130, 2], R=16, interleaved=True),
    dict(S=2, H=3, Hkv=3, D=64, bs=16, dtype="bf16", new=[17, 4], R=48, pad=1),
    dict(S=2, H=3, Hkv=1, D=64, bs=16, dtype="bf16", new=[17, 4], R=32, interleaved=True, shift=1000),
    dict(S=2, H=7, Hkv=7, D=128, bs=8, dtype="f16", new=[5, 6], R=0, pad=2),
    dict(S=1, H=100, Hkv=20, D=128, bs=16, dtype="bf16", new=[3], before=[30000], R=112, base=500000.0),
    dict(S=40, H=8, Hkv=2, D=64, bs=8, dtype="f16", new=[1] * 40, before=list(range(0, 80, 2))),
]


@pytest.mark.parametrize("kw", CASES)
def test_append(kw):
    c = C.append_case(1, **kw)
    d = C.append_on_gpu(c)
    live = c["pos"] >= 0
    shape = (c["NB"], c["bs"], c["Hkv"], c["D"])
    rng = np.random.default_rng(5)
    old = [rng.integers(0, 1 << 16, shape, dtype=np.uint16) for _ in range(2)]
    caches = [C.tensor(x, c["dtype"]).cuda() for x in old]
    out_old = rng.integers(0, 1 << 16, (c["T"], c["H"], c["D"]), dtype=np.uint16)
    out = C.tensor(out_old, c["dtype"]).cuda()
    assert call(c, d, False, *caches, out) is out
    slots = Q.slots(c["tables"], c["seq"], c["pos"], c["bs"])
    assert np.array_equal(d["slots"].cpu().numpy(), slots)
    qref, qmag = C.rotated(c, "query", np.float64)
    check16(C.bits_of(out)[live], qref[live], qmag[live], c["dtype"])
    assert np.array_equal(C.bits_of(out)[~live], out_old[~live])
    kref, kmag = C.rotated(c, "key", np.float64)
    kgot, vgot = (C.bits_of(x).reshape(-1, c["Hkv"], c["D"]) for x in caches)
    check16(kgot[slots[live]], kref[live], kmag[live], c["dtype"])
    assert np.array_equal(vgot[slots[live]], c["value"][live])
    rest = np.ones(c["NB"] * c["bs"], bool)
    rest[slots[live]] = False
    for got, was in zip((kgot, vgot), old):
        assert np.array_equal(got[rest], was.reshape(got.shape)[rest])
    assert L.pkv_get_device_errors() == 0


@pytest.mark.parametrize("big", [1.0, 1e-3, 1e3])
@pytest.mark.parametrize("kw", CASES)
def test_append_q4(kw, big):
    c = C.append_case(2, **kw, big=big)
    d = C.append_on_gpu(c)
    D, dtype, live = c["D"], c["dtype"], c["pos"] >= 0
    rng = np.random.default_rng(6)
    shape = (c["NB"], c["Hkv"], c["bs"], Q.row_bytes(D))
    old = [rng.integers(0, 256, shape, dtype=np.uint8) for _ in range(2)]
    caches = [torch.from_numpy(x).cuda() for x in old]
    out = torch.zeros((c["T"], c["H"], D), dtype=C.DT[dtype], device="cuda")
    call(c, d, True, *caches, out)
    slots = Q.slots(c["tables"], c["seq"], c["pos"], c["bs"])
    assert np.array_equal(d["slots"].cpu().numpy(), slots)
    qref, qmag = C.rotated(c, "query", np.float64)
    check16(C.bits_of(out)[live], qref[live], qmag[live], dtype)
    rest = np.ones(c["NB"] * c["bs"], bool)
    rest[slots[live]] = False
    for got, was, name in zip(caches, old, ("key", "value")):
        got = got.cpu().numpy()
        step, centre, code = Q.parts(got, D)
        x32 = C.rotated(c, name, np.float32)[0] if name == "key" else Q.widen(c[name], dtype).astype(np.float32)
        want = Q.quantise(x32[live], dtype, np.float32)
        for have, ref in zip((step, centre, code), want):
            have = have.reshape(-1, *have.shape[2:])
            assert np.array_equal(have[slots[live]], ref), name
        for have, ref in zip((step, centre, code), Q.parts(was, D)):  # the others' bytes as they were
            have, ref = (y.reshape(-1, *y.shape[2:])[rest] for y in (have, ref))
            assert np.array_equal(have, ref)
        if name == "key":
            x, mag = C.rotated(c, name, np.float64)
        else:
            x = Q.widen(c[name], dtype)
            mag = np.abs(x)
        value = Q.values(got, D, dtype).reshape(-1, c["Hkv"], D)[slots[live]]
        s, a = (np.repeat(Q.widen(y, dtype), 64, -1).reshape(-1, c["Hkv"], D)[slots[live]] for y in (step, centre))
        top = mag[live].reshape(-1, c["Hkv"], D // 64, 64).max(-1).repeat(64, -1).reshape(value.shape)
        bound = s * (0.5 + 2.0 ** -18) + C.U[dtype] * (8 * s + np.abs(a)) + 4.02 * C.E32 * top + 2.0 ** -20
        assert (np.abs(value - x[live]) <= bound).all(), name

    # and back: the values, rounded once; rows of negative slots stay
    rows = [torch.full((c["T"], c["Hkv"], D), 7.0, dtype=C.DT[dtype], device="cuda") for _ in range(2)]
    E.gather_cache_q4(*rows, *caches, d["slots"])
    for got, cache in zip(rows, caches):
        got = Q.widen(C.bits_of(got), dtype)
        ref = Q.values(cache.cpu().numpy(), D, dtype).reshape(-1, c["Hkv"], D)[slots[live]]
        assert (np.abs(got[live] - ref) <= C.U[dtype] * (1 + 2.0 ** -12) * np.abs(ref) + 2.0 ** -25).all()
        assert (got[~live] == 7).all()
    assert L.pkv_get_device_errors() == 0


@pytest.mark.parametrize("q4", [False, True])
def test_in_place_and_without_queries(q4):
    """query_out None rotates in place, in the projection itself; no query writes the caches alone."""
    c = C.append_case(3, S=3, H=8, Hkv=4, D=128, bs=16, dtype="bf16", new=[5, 17, 1], pad=2, fused=True)
    a, b, none = (C.append_on_gpu(c) for _ in range(3))
    caches = []
    for d, out in ((a, torch.zeros(c["T"], 8, 128, dtype=torch.bfloat16, device="cuda")), (b, None), (none, None)):
        k, v = (E.new_cache_q4(c["NB"], 16, 4, 128) if q4 else
                torch.zeros(c["NB"], 16, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        if d is none:
            d["query"] = None
        got = call(c, d, q4, k, v, out)
        caches.append((k, v, got))
    live = torch.from_numpy(c["pos"] >= 0).cuda()
    assert caches[1][2] is b["query"] and caches[2][2] is None
    assert torch.equal(caches[0][2][live], b["query"][live])
    assert torch.equal(C.tensor(c["query"], "bf16").cuda()[~live], b["query"][~live])
    for i in (1, 2):
        assert torch.equal(caches[0][0], caches[i][0]) and torch.equal(caches[0][1], caches[i][1])


@pytest.mark.parametrize("q4", [False, True])
def test_fused_equals_separate_calls(q4):
    """Without a rotation: compute_slot_mapping and reshape_and_cache, bit for bit."""
    c = C.append_case(4, S=4, H=4, Hkv=4, D=64, bs=16, dtype="f16", new=[3, 1, 40, 16], R=0, pad=1)
    d = C.append_on_gpu(c)
    slots = torch.empty_like(d["slots"])
    E.compute_slot_mapping(slots, d["tables"], d["seq"], d["pos"], 16)
    if q4:
        k, v = E.new_cache_q4(c["NB"], 16, 4, 64), E.new_cache_q4(c["NB"], 16, 4, 64)
        call(c, d, True, k, v, None)
        assert torch.equal(slots, d["slots"])
        return
    k, v, k2, v2 = (torch.zeros(c["NB"], 16, 4, 64, dtype=torch.float16, device="cuda") for _ in range(4))
    call(c, d, False, k, v, None)
    E.reshape_and_cache(d["key"], d["value"], k2, v2, slots)
    assert torch.equal(slots, d["slots"]) and torch.equal(k, k2) and torch.equal(v, v2)


def test_groups_that_are_not_finite_and_constant_ones():
    """A group with an infinity or a NaN reads as NaN, its neighbours as they should; a constant
    group and zeros read exactly; the widest bf16 range is not lost."""
    D, T = 128, 6
    key = torch.randn(T, 1, D).bfloat16()
    value = torch.randn(T, 1, D).bfloat16()
    key[0, 0, 3], value[1, 0, 70], key[2, 0, 127] = float("nan"), float("inf"), -float("inf")
    value[3, 0, :64] = 0.3
    value[3, 0, 64:] = 0
    big = torch.finfo(torch.bfloat16).max
    value[4, 0, :32], value[4, 0, 32:64] = big, -big
    value[4, 0, 64:] = big
    value[5, 0, :64] = torch.tensor([1e-40, 2e-40]).repeat(32).bfloat16()
    k, v = E.new_cache_q4(2, 8, 1, D), E.new_cache_q4(2, 8, 1, D)
    at = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.empty(T, dtype=torch.int64, device="cuda")
    E.rotate_and_cache_q4(key.cuda(), value.cuda(), k, v, torch.tensor([[1]], dtype=torch.int32, device="cuda"),
                          torch.zeros_like(at), at, slots)
    ko, vo = (torch.empty(T, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    E.gather_cache_q4(ko, vo, k, v, slots)
    ko, vo = ko.cpu()[:, 0], vo.cpu()[:, 0]
    bad_k = torch.zeros(T, D, dtype=torch.bool)
    bad_k[0, :64] = bad_k[2, 64:] = True
    bad_v = torch.zeros(T, D, dtype=torch.bool)
    bad_v[1, 64:] = True
    assert torch.equal(ko.isnan(), bad_k) and torch.equal(vo.isnan(), bad_v)
    assert torch.equal(vo[3], value[3, 0]) and torch.equal(vo[4, 64:], value[4, 0, 64:])
    # ends of the range: 8 u step + u |centre| off at most, step = 2 max / 15, and rounded
    off = (vo[4, :64].double() - value[4, 0, :64].double()).abs().max() / big
    assert off <= 2.0 ** -8 * (8 * 2 / 15 + 1 / 15) * 1.01 + 2.0 ** -8
    assert (vo[5, :64].double() - value[5, 0, :64].double()).abs().max() <= 1e-40
    assert L.pkv_get_device_errors() == 0


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("what,bit", [
    ("position", L.PKV_DEVERR_POSITION), ("sequence", L.PKV_DEVERR_POSITION), ("unmapped", L.PKV_DEVERR_BLOCK_ID),
    ("block", L.PKV_DEVERR_SLOT), ("turn", L.PKV_DEVERR_POSITION), ("turn below", L.PKV_DEVERR_POSITION)])
def test_errors_on_the_device(q4, what, bit):
    """Tokens that cannot be placed write nothing and set their bit; the others are written."""
    c = C.append_case(5, S=2, H=2, Hkv=2, D=64, bs=16, dtype="f16", new=[4, 20], MB=3)
    d = C.append_on_gpu(c)
    tables, seq, pos = d["tables"].clone(), d["seq"].clone(), d["pos"].clone()
    turn = pos.clone()
    t = int(torch.nonzero((seq == 1) & (pos == 19))[0])
    hit = torch.arange(c["T"], device="cuda") == t
    if what in ("unmapped", "block"):
        hit = (seq == 1) & (pos >= 16)
        tables[1, 1] = -1 if what == "unmapped" else c["NB"] + 3
    elif what == "position":
        pos[t] = 48
    elif what == "sequence":
        seq[t] = 2
    else:
        turn[t] = d["table"].shape[0] if what == "turn" else -1
    shape = (c["NB"], 2, 16, 36) if q4 else (c["NB"], 16, 2, 64)
    k, v = (torch.full(shape, 9, dtype=torch.uint8 if q4 else torch.float16, device="cuda") for _ in range(2))
    out = torch.full((c["T"], 2, 64), 5.0, dtype=torch.float16, device="cuda")
    (E.rotate_and_cache_q4 if q4 else E.rotate_and_cache)(
        d["key"], d["value"], k, v, tables, seq, pos, d["slots"], d["table"], query=d["query"], query_out=out,
        rotary_pos=turn)
    torch.cuda.synchronize()
    assert L.pkv_get_device_errors() == bit
    assert (out[hit] == 5).all() and not (out[~hit] == 5).all(-1).any()
    good = d["slots"][~hit]
    assert (good >= 0).all()
    assert (d["slots"][hit] >= c["NB"] * 16).all() if what == "block" else (d["slots"][hit] == -1).all()
    if q4:
        rows = torch.full((c["T"], 2, 64), 5.0, dtype=torch.float16, device="cuda")
        E.gather_cache_q4(rows, torch.empty_like(rows), k, v, d["slots"])
        assert L.pkv_get_device_errors() == (L.PKV_DEVERR_SLOT if what == "block" else 0)
        assert (rows[hit] == 5).all() and not (rows[~hit] == 5).all(-1).any()
    else:
        flat = k.view(-1, 2, 64)
        written = torch.zeros(flat.shape[0], dtype=torch.bool, device="cuda")
        written[good] = True
        assert (flat[~written] == 9).all() and not (flat[written] == 9).all(-1).any()


def test_other_stream_and_graph():
    """On a stream of its own, and captured: a replay takes what the inputs hold then."""
    c = C.append_case(6, S=3, H=8, Hkv=2, D=128, bs=16, dtype="bf16", new=[1, 1, 1], before=[5, 20, 100])
    d = C.append_on_gpu(c)
    k, v = E.new_cache_q4(c["NB"], 16, 2, 128), E.new_cache_q4(c["NB"], 16, 2, 128)
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    out, out2 = torch.empty_like(d["query"]), torch.empty_like(d["query"])
    call(c, d, True, k, v, out)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(c, d, True, k2, v2, out2, stream=side)
    side.synchronize()
    assert torch.equal(k, k2) and torch.equal(v, v2) and torch.equal(out, out2)
    rows = [torch.empty_like(d["key"]) for _ in range(2)]
    g = torch.cuda.CUDAGraph()
    k2.zero_(), v2.zero_(), out2.zero_()
    with torch.cuda.graph(g):
        call(c, d, True, k2, v2, out2)
        E.gather_cache_q4(*rows, k2, v2, d["slots"])
    assert not k2.any()
    d["query"].mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(k, k2) and torch.equal(v, v2) and torch.equal(out2, 2 * out)
    assert L.pkv_get_device_errors() == 0


def test_one_slot_read_twice_and_strided_rows():
    c = C.append_case(7, S=1, H=2, Hkv=2, D=64, bs=8, dtype="f16", new=[20])
    d = C.append_on_gpu(c)
    k, v = E.new_cache_q4(c["NB"], 8, 2, 64), E.new_cache_q4(c["NB"], 8, 2, 64)
    call(c, d, True, k, v, None)
    twice = d["slots"][[3, 3, 7, 0, 3]]
    wide = torch.full((5, 4 * 64), 3.0, dtype=torch.float16, device="cuda")
    ko, vo = (x.unflatten(-1, (2, 64)) for x in wide.split([128, 128], -1))
    E.gather_cache_q4(ko, vo, k, v, twice)
    whole = [torch.empty(20, 2, 64, dtype=torch.float16, device="cuda") for _ in range(2)]
    E.gather_cache_q4(*whole, k, v, d["slots"])
    for got, all_ in zip((ko, vo), whole):
        assert torch.equal(got, all_[[3, 3, 7, 0, 3]])


def test_tokens_in_pinned_host_memory():
    """Token data may lie in pinned host memory, as in the other calls."""
    c = C.append_case(8, S=2, H=2, Hkv=2, D=64, bs=8, dtype="f16", new=[3, 9])
    d = C.append_on_gpu(c)
    h = dict(d, **{k: d[k].cpu().pin_memory() for k in ("key", "value", "query")})
    got = []
    for x in (d, h):
        k, v = E.new_cache_q4(c["NB"], 8, 2, 64), E.new_cache_q4(c["NB"], 8, 2, 64)
        out = torch.empty_like(x["query"]).pin_memory() if x is h else torch.empty_like(x["query"])
        call(c, x, True, k, v, out)
        torch.cuda.synchronize()
        got.append((k, v, out.cuda()))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_rotary_table():
    t = E.new_rotary_table(100001, 64, base=10000.0).double().cpu().numpy()
    angle = np.arange(100001)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    ref = np.concatenate([np.cos(angle), np.sin(angle)], -1)
    # the angle in 64 bits is off by 2^-51 of itself, 2^-34 at 1e5, on either side; fp32 rounds by 2^-25
    assert np.abs(t - ref).max() <= 2.0 ** -25 + 2.0 ** -32


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("kw", [
    dict(S=3, H=3, Hkv=1, D=64, bs=16, dtype="f16", new=[2600, 1, 1000], pad=30),         # two tokens per CTA
    dict(S=2, H=8, Hkv=2, D=128, bs=32, dtype="bf16", new=[5000, 503], R=64, pad=4, fused=True),  # four
    dict(S=1, H=33, Hkv=3, D=128, bs=8, dtype="bf16", new=[4901], interleaved=True),
])
def test_many_tokens_are_as_few_at_a_time(kw, q4):
    """CTAs of several tokens write what CTAs of one write, bit for bit."""
    c = C.append_case(9, **kw)
    got = []
    for step in (c["T"], 700):
        d = C.append_on_gpu(c)
        shape = (c["NB"], c["bs"], c["Hkv"], c["D"])
        k, v = (E.new_cache_q4(c["NB"], c["bs"], c["Hkv"], c["D"]) if q4 else
                torch.zeros(shape, dtype=C.DT[c["dtype"]], device="cuda") for _ in range(2))
        for at in range(0, c["T"], step):
            part = {x: d[x] if d[x] is None or x in ("tables", "table") else d[x][at:at + step] for x in d}
            call(c, part, q4, k, v, None)
        got.append((k, v, d["query"], d["slots"]))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    live = c["pos"] >= 0
    assert np.array_equal(got[0][3].cpu().numpy(), Q.slots(c["tables"], c["seq"], c["pos"], c["bs"]))
    qref, qmag = C.rotated(c, "query", np.float64)
    check16(C.bits_of(got[0][2])[live], qref[live], qmag[live], c["dtype"])
    assert L.pkv_get_device_errors() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_steps_and_centres_beside_the_64_bit_quotients(dtype):
    """Groups whose quotients lie halfway between two 16-bit numbers, or whose ends are far apart in
    size: within what the header says of the rounding, which here knows of no fp32."""
    from test_q4_cpu import check_rounding, ends_apart
    x = ends_apart(np.random.default_rng(9), dtype, 4096).reshape(2048, 1, 128)
    k, v = E.new_cache_q4(128, 16, 1, 128), E.new_cache_q4(128, 16, 1, 128)
    rows = C.tensor(Q.narrow(x, dtype), dtype).cuda()
    at = torch.arange(2048, dtype=torch.int32, device="cuda")
    slots = torch.empty(2048, dtype=torch.int64, device="cuda")
    E.rotate_and_cache_q4(rows, rows, k, v, torch.arange(128, dtype=torch.int32, device="cuda")[None],
                          torch.zeros_like(at), at, slots)
    for cache in (k, v):
        step, centre, code = (y.reshape(2048, 1, -1) for y in Q.parts(cache.cpu().numpy(), 128))
        check_rounding(x, step, centre, code, dtype)
    assert L.pkv_get_device_errors() == 0
