"""The 4-bit cache's oracle against hand-worked values and other routes, and
what the calls around it refuse, without a GPU."""
import math
import os

import numpy as np
import pytest
import torch

import q4_cases as C
from oracle import q4 as Q
from paged_kv_cache_162_gb300 import _lib as L
from paged_kv_cache_162_gb300 import engine as E


# ---------------------------------------------------------------- the oracle
def test_narrow_rounds_once_to_nearest_even():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(50000) * np.exp2(rng.integers(-20, 20, 50000))).astype(np.float32)
    for dtype, t in C.DT.items():
        assert np.array_equal(Q.narrow(x, dtype), C.bits_of(torch.from_numpy(x).to(t)))
    # a tie of the first rounding to fp32 must not become a tie of the second
    one, ulp = 1.0, 2.0 ** -7
    half = one + ulp / 2
    for x, bits in ((half, 0x3f80), (half + 2.0 ** -40, 0x3f81), (half - 2.0 ** -40, 0x3f80),
                    (one + 1.5 * ulp, 0x3f82), (one + 1.5 * ulp - 2.0 ** -40, 0x3f81),
                    (-half - 2.0 ** -40, 0xbf81), (-half + 2.0 ** -40, 0xbf80)):
        assert Q.narrow(np.array([x]), "bf16")[0] == bits, x
    assert Q.narrow(np.array([np.nan]), "bf16")[0] & 0x7fff > 0x7f80
    assert np.array_equal(Q.widen(Q.narrow(np.array([1.5, -2.0, 0.0]), "f16"), "f16"), [1.5, -2.0, 0.0])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_product_of_complex_numbers(interleaved):
    rng = np.random.default_rng(1)
    x, angle = rng.standard_normal((3, 64)), rng.standard_normal(16)
    y = Q.rotate(x, np.cos(angle), np.sin(angle), interleaved)
    a, b = (x[:, 0:32:2], x[:, 1:32:2]) if interleaved else (x[:, :16], x[:, 16:32])
    z = (a + 1j * b) * np.exp(1j * angle)
    re, im = (y[:, 0:32:2], y[:, 1:32:2]) if interleaved else (y[:, :16], y[:, 16:32])
    assert np.allclose(re, z.real, atol=1e-14) and np.allclose(im, z.imag, atol=1e-14)
    assert np.array_equal(y[:, 32:], x[:, 32:])


def test_codes_worked_by_hand():
    # -7.5 .. 7.5: step 1, centre 0.5; halves go to the even code
    x = np.zeros((1, 64))
    x[0, :6] = [-7.5, 7.5, 0.5, 0.0, 1.0, -1.0]
    step, centre, code = Q.quantise(x, "f16")
    assert Q.widen(step, "f16")[0, 0] == 1.0 and Q.widen(centre, "f16")[0, 0] == 0.5
    # (x - 0.5): -8, 7, 0, -0.5 -> 0, 0.5 -> 0, -1.5 -> -2
    assert code[0, :6].tolist() == [0, 15, 8, 8, 8, 6]
    step, centre, code = Q.quantise(np.full((1, 64), 0.25), "bf16")
    assert step[0, 0] == 0 and Q.widen(centre, "bf16")[0, 0] == 0.25 and (code == 8).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_values_are_near_what_was_quantised(dtype):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((500, 128)) * np.exp2(rng.integers(-6, 6, (500, 1))) + rng.integers(-3, 4, (500, 1))
    step, centre, code = Q.quantise(x, dtype)
    s, a = (np.repeat(Q.widen(v, dtype), 64, -1) for v in (step, centre))
    off = np.abs(a + s * (code - 8) - x)
    assert (off <= s * (0.5 + 1e-12) + C.U[dtype] * (8 * s + np.abs(a)) + 2.0 ** -22).all()
    assert code.min() == 0 and code.max() == 15


@pytest.mark.parametrize("D,bs", [(64, 8), (64, 64), (128, 16), (128, 32)])
def test_every_byte_of_a_pool_has_one_place(D, bs):
    """Codes and pairs fill a (block, head)'s run exactly, and come back."""
    places = [Q._byte(D, off, d) for off in range(bs) for d in range(0, D, 2)]
    places += [Q._pair(D, off, g) + i for off in range(bs) for g in range(D // 64) for i in range(4)]
    assert sorted(places) == list(range(bs * Q.row_bytes(D)))
    rng = np.random.default_rng(3)
    code = rng.integers(0, 16, (2, bs, 3, D))
    step, centre = (rng.integers(0, 1 << 16, (2, bs, 3, D // 64)).astype(np.uint16) for _ in range(2))
    for got, want in zip(Q.parts(Q.pack(step, centre, code), D), (step, centre, code)):
        assert np.array_equal(got, want)


def test_bytes_worked_by_hand():
    code = np.zeros((1, 8, 1, 128), np.int64)
    code[0, 3, 0, 32], code[0, 3, 0, 33] = 5, 9       # token 3, chunk 1
    step, centre = np.zeros((1, 8, 1, 2), np.uint16), np.zeros((1, 8, 1, 2), np.uint16)
    step[0, 3, 0, 1], centre[0, 3, 0, 1] = 0x1234, 0xabcd
    run = Q.pack(step, centre, code).reshape(-1)
    # row 3 at 3 * 64, chunk 1 at place 1 ^ (3 / 2) % 4 = 0; pairs after 512 code bytes, 8 per row
    want = {3 * 64: 0x95, 512 + 3 * 8 + 4: 0x34, 512 + 3 * 8 + 5: 0x12, 512 + 3 * 8 + 6: 0xcd, 512 + 3 * 8 + 7: 0xab}
    assert {int(i): int(run[i]) for i in np.flatnonzero(run)} == want


def test_row_bytes_of_the_library():
    assert [L.pkv_cache_q4_row_bytes(d) for d in (64, 128, 0, 96, 256, -64)] == [Q.row_bytes(64), Q.row_bytes(128), 0, 0, 0, 0]


def test_attention_reference_against_torch():
    c = C.attend_case(5, 3, 6, 2, 64, 8, "f16", [17, 0, 40])
    out, bound = C.attend_reference(c)
    k, v = (Q.values(c[x], 64, "f16").reshape(-1, 2, 64) for x in ("k", "v"))
    q = Q.widen(c["q"], "f16")
    for s, n in enumerate(c["lens"]):
        if n == 0:
            assert (out[s] == 0).all()
            continue
        rows = [int(c["tables"][s, j // 8]) * 8 + j % 8 for j in range(n)]
        for h in range(6):
            w = torch.softmax(torch.from_numpy(k[rows, h // 3] @ q[s, h]) * c["scale"], -1).numpy()
            assert np.allclose(out[s, h], w @ v[rows, h // 3], atol=1e-12)
    assert (bound > 0).all()


def test_the_bound_sees_a_mistake():
    """A swap of two chunks, or the centre of the other group, passes no bound."""
    c = C.attend_case(6, 2, 4, 2, 128, 16, "bf16", [30, 50])
    ref, bound = C.attend_reference(c)
    step, centre, code = Q.parts(c["v"], 128)
    other = dict(c, v=Q.pack(step, centre[..., ::-1], code))
    assert (np.abs(C.attend_reference(other)[0] - ref) > bound).any()
    other = dict(c, k=Q.pack(step, centre, np.roll(Q.parts(c["k"], 128)[2], 32, -1)))
    assert (np.abs(C.attend_reference(other)[0] - ref) > bound).any()


# ---------------------------------------------------------------- refusals of the C entry points
def append_args(**kw):
    a = dict(key=1 << 20, key_stride=256, value=2 << 20, value_stride=256, query=3 << 20, query_stride=1024,
             query_out=4 << 20, query_out_stride=1024, k_cache=256, v_cache=512, block_tables=256, seq_idx=256, pos=256,
             rotary_pos=None, table=256, table_rows=10, R=128, interleaved=0, slots=256, T=5, S=2, H=8, Hkv=2, D=128,
             bs=16, NB=8, MB=4, dtype=L.PKV_BF16, stream=0)
    a.update(kw)
    return a


BAD_APPENDS = [
    (dict(key=None), "null"), (dict(value=None), "null"), (dict(query=None), "null"), (dict(query_out=None), "null"),
    (dict(k_cache=None), "null"), (dict(v_cache=None), "null"), (dict(block_tables=None), "null"),
    (dict(seq_idx=None), "null"), (dict(pos=None), "null"), (dict(slots=None), "null"), (dict(table=None), "null"),
    (dict(key=(1 << 20) + 8), "aligned"), (dict(value=(2 << 20) + 2), "aligned"), (dict(query=(3 << 20) + 8), "aligned"),
    (dict(query_out=(4 << 20) + 8), "aligned"), (dict(k_cache=264), "aligned"), (dict(v_cache=520), "aligned"),
    (dict(table=260), "aligned"), (dict(key_stride=255), "strides"), (dict(key_stride=260), "strides"),
    (dict(value_stride=248), "strides"), (dict(query_stride=1000), "strides"), (dict(query_out_stride=1 << 30), "strides"),
    (dict(key_stride=-256), "strides"), (dict(R=8), "rotary_dim"), (dict(R=144), "rotary_dim"), (dict(R=-16), "rotary_dim"),
    (dict(table_rows=0), "no rows"), (dict(table_rows=-1), "no rows"), (dict(T=-1), "size"), (dict(S=0), "size"),
    (dict(S=-1), "size"), (dict(H=-1), "size"), (dict(Hkv=0), "size"), (dict(NB=0), "size"), (dict(MB=0), "size"),
    (dict(dtype=2), "size"), (dict(NB=1 << 28), "31 bits"), (dict(H=(1 << 20) + 1), "heads"),
    (dict(query_out=(3 << 20) + 1024), "overlap"), (dict(query_out=(3 << 20) + 2048), "overlap"),
    (dict(query_out=(3 << 20), query_out_stride=1032), "overlap"), (dict(query_out=1 << 20), "overlap"),
    (dict(query_out=(2 << 20) - 1024), "overlap"),
]


@pytest.mark.parametrize("name", ["pkv_rotate_and_cache", "pkv_rotate_and_cache_q4"])
@pytest.mark.parametrize("bad,word", BAD_APPENDS)
def test_appends_refuse(name, bad, word):
    with pytest.raises(L.PkvError, match=word) as e:
        getattr(L, name)(*list(append_args(**bad).values())[:-1], stream=0)
    assert e.value.status == L.PKV_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["pkv_rotate_and_cache", "pkv_rotate_and_cache_q4"])
@pytest.mark.parametrize("bad", [dict(D=96), dict(D=256), dict(bs=4), dict(bs=24)])
def test_appends_that_are_not_built(name, bad):
    with pytest.raises(L.PkvError) as e:
        getattr(L, name)(*list(append_args(**bad).values())[:-1], stream=0)
    assert e.value.status == L.PKV_ERR_UNSUPPORTED


def test_appends_of_no_tokens_do_nothing():
    for name in ("pkv_rotate_and_cache", "pkv_rotate_and_cache_q4"):
        getattr(L, name)(*list(append_args(T=0, key=None, S=0).values())[:-1], stream=0)


GATHER = dict(key=1 << 20, key_stride=256, value=2 << 20, value_stride=256, k_cache=256, v_cache=512, slots=256, T=5,
              Hkv=2, D=128, bs=16, NB=8, dtype=L.PKV_F16)


@pytest.mark.parametrize("bad,word", [
    (dict(key=None), "null"), (dict(value=None), "null"), (dict(k_cache=None), "null"), (dict(v_cache=None), "null"),
    (dict(slots=None), "null"), (dict(key=(1 << 20) + 4), "aligned"), (dict(v_cache=513), "aligned"),
    (dict(key_stride=128), "strides"), (dict(value_stride=257), "strides"), (dict(T=-1), "size"), (dict(Hkv=0), "size"),
    (dict(NB=0), "size"), (dict(dtype=7), "size"), (dict(NB=1 << 28), "31 bits"), (dict(value=1 << 20), "overlap"),
    (dict(value=(1 << 20) + 512 * 4), "overlap")])
def test_gather_refuses(bad, word):
    with pytest.raises(L.PkvError, match=word) as e:
        L.pkv_gather_cache_q4(*{**GATHER, **bad}.values(), stream=0)
    assert e.value.status == L.PKV_ERR_INVALID_ARG


ATTEND = dict(out=256, q=256, k_cache=256, v_cache=512, tables=256, lens=256, S=2, H=8, Hkv=2, D=128, bs=16, NB=8, MB=4,
              max_context_len=0, scale=1.0, dtype=L.PKV_F16, workspace=256, workspace_bytes=1 << 40)


@pytest.mark.parametrize("bad,word", [
    (dict(out=None), "null"), (dict(q=None), "null"), (dict(k_cache=None), "null"), (dict(v_cache=None), "null"),
    (dict(tables=None), "null"), (dict(lens=None), "null"), (dict(out=258), "aligned"), (dict(q=264), "aligned"),
    (dict(k_cache=264), "aligned"), (dict(workspace=None), "workspace"), (dict(workspace=128), "workspace"),
    (dict(S=-1), "size"), (dict(H=0), "size"), (dict(Hkv=0), "size"), (dict(NB=0), "size"), (dict(MB=0), "size"),
    (dict(dtype=3), "size"), (dict(H=9), "multiple"), (dict(scale=math.inf), "finite"), (dict(scale=math.nan), "finite"),
    (dict(NB=1 << 28), "31 bits"), (dict(NB=1 << 26, Hkv=32, H=32), "34 bits"), (dict(S=32768), "32767"),
    (dict(max_context_len=65), "max_context_len"), (dict(max_context_len=-1), "max_context_len")])
def test_attention_refuses(bad, word):
    with pytest.raises(L.PkvError, match=word) as e:
        L.pkv_paged_attention_decode_q4(*{**ATTEND, **bad}.values(), stream=0)
    assert e.value.status == L.PKV_ERR_INVALID_ARG


@pytest.mark.parametrize("bad,status", [(dict(D=32), L.PKV_ERR_UNSUPPORTED), (dict(bs=128), L.PKV_ERR_UNSUPPORTED),
                                        (dict(H=34), L.PKV_ERR_UNSUPPORTED), (dict(workspace_bytes=1000), L.PKV_ERR_WORKSPACE)])
def test_attention_that_is_not_built_or_has_no_room(bad, status):
    with pytest.raises(L.PkvError) as e:
        L.pkv_paged_attention_decode_q4(*{**ATTEND, **bad}.values(), stream=0)
    assert e.value.status == status


def test_attention_workspace_size():
    assert L.pkv_decode_q4_workspace_size(4, 32, 8, 128) > 0
    for bad in ((-1, 32, 8, 128), (4, 33, 8, 128), (4, 0, 8, 128), (4, 32, 0, 128), (4, 34, 2, 128), (4, 32, 8, 96),
                (1 << 40, 32, 8, 128)):
        assert L.pkv_decode_q4_workspace_size(*bad) == 0, bad


@pytest.mark.parametrize("bad", [dict(P=-1), dict(Hkv=0), dict(NB=-1), dict(k=None), dict(k=8), dict(P=65535 * 64 + 1)])
def test_copies_of_4_bit_blocks_refuse(bad):
    a = {**dict(k=256, v=256, mapping=256, P=1, Hkv=2, D=128, bs=16, NB=4), **bad}
    with pytest.raises(L.PkvError) as e:
        L.pkv_copy_blocks_q4(*a.values(), stream=0)
    assert e.value.status == L.PKV_ERR_INVALID_ARG
    s = {**dict(k=256, v=256, hk=256, hv=256, mapping=256, P=1, Hkv=2, D=128, bs=16, NB=4, NBh=4, d=0), **bad}
    with pytest.raises(L.PkvError) as e:
        L.pkv_swap_blocks_q4(*s.values(), stream=0)
    assert e.value.status == L.PKV_ERR_INVALID_ARG


# ---------------------------------------------------------------- refusals of the tensor calls
def tensors(q4=False, dt=torch.float16):
    T, H, Hkv, D = 3, 4, 2, 64
    cache = torch.zeros(4, Hkv, 16, 36, dtype=torch.uint8) if q4 else torch.zeros(4, 16, Hkv, D, dtype=dt)
    return dict(key=torch.zeros(T, Hkv, D, dtype=dt), value=torch.zeros(T, Hkv, D, dtype=dt), k_cache=cache,
                v_cache=cache.clone(), block_tables=torch.zeros(2, 2, dtype=torch.int32),
                seq_idx=torch.zeros(T, dtype=torch.int32), pos=torch.zeros(T, dtype=torch.int32),
                slot_mapping=torch.zeros(T, dtype=torch.int64), rotary_table=torch.zeros(9, 64),
                query=torch.zeros(T, H, D, dtype=dt))


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("change,status", [
    (dict(key=torch.zeros(3, 2, 64)), L.PKV_ERR_UNSUPPORTED),                 # fp32
    (dict(key=torch.zeros(3, 128, dtype=torch.float16)), L.PKV_ERR_INVALID_ARG),
    (dict(key=torch.zeros(3, 3, 64, dtype=torch.float16)), L.PKV_ERR_INVALID_ARG),   # heads
    (dict(block_tables=torch.zeros(4, dtype=torch.int32)), L.PKV_ERR_INVALID_ARG),
    (dict(query=None, query_out=torch.zeros(3, 4, 64, dtype=torch.float16)), L.PKV_ERR_INVALID_ARG),
    (dict(), L.PKV_ERR_INVALID_ARG),                                          # not on a CUDA device
])
def test_append_calls_refuse(q4, change, status):
    a = {**tensors(q4), **change}
    with pytest.raises(L.PkvError) as e:
        (E.rotate_and_cache_q4 if q4 else E.rotate_and_cache)(**a)
    assert e.value.status == status


def test_a_cache_of_the_other_kind_is_refused():
    with pytest.raises(L.PkvError, match="4-bit caches must be"):
        E.rotate_and_cache_q4(**tensors(False))
    with pytest.raises(L.PkvError):
        E.rotate_and_cache(**tensors(True))
    t = tensors(False)
    with pytest.raises(L.PkvError, match="4-bit caches must be"):
        E.gather_cache_q4(t["key"], t["value"], t["k_cache"], t["v_cache"], t["slot_mapping"])
    with pytest.raises(L.PkvError, match="4-bit caches must be"):
        E.paged_attention_decode_q4(t["query"], t["query"], t["k_cache"], t["v_cache"], t["block_tables"][[0, 0, 0]],
                                    t["pos"])


def test_token_rows():
    """Strides that the calls take, and those that they refuse."""
    dev = torch.device("cpu")
    dt = torch.float16
    whole = torch.zeros(5, 6 * 64, dtype=dt).pin_memory() if torch.cuda.is_available() else torch.zeros(5, 6 * 64, dtype=dt)
    part = whole[:, 64:192].unflatten(-1, (2, 64))
    assert E._token_rows("x", "key", part, dt, (5, 2, 64), dev) == 384
    assert E._token_rows("x", "key", part[:1], dt, (1, 2, 64), dev) == 128
    for bad in (part.transpose(0, 1), part[..., ::2], torch.zeros(5, 64, 2, dtype=dt).transpose(1, 2)):
        with pytest.raises(L.PkvError):
            E._token_rows("x", "key", bad, dt, tuple(bad.shape), dev)


def test_new_caches_and_tables():
    c = E.new_cache_q4(3, 16, 2, 128, device="cpu")
    assert c.shape == (3, 2, 16, 72) and c.dtype == torch.uint8 and not c.any()
    assert (Q.values(c.numpy(), 128, "f16") == 0).all()
    for bad in ((3, 16, 2, 96), (3, 12, 2, 64), (0, 16, 2, 64), (3, 16, 0, 64)):
        with pytest.raises(L.PkvError):
            E.new_cache_q4(*bad, device="cpu")
    t = E.new_rotary_table(50, 32, base=100.0, device="cpu").double().numpy()
    angle = np.arange(50)[:, None] * 100.0 ** (-np.arange(0, 32, 2) / 32)
    assert np.abs(t - np.concatenate([np.cos(angle), np.sin(angle)], -1)).max() <= 2.0 ** -25 + 2.0 ** -40
    for bad in ((0, 32), (5, 0), (5, 33)):
        with pytest.raises(L.PkvError):
            E.new_rotary_table(*bad, device="cpu")


def test_copies_between_caches_of_two_kinds_are_refused():
    a, b = torch.zeros(4, 2, 16, 36, dtype=torch.uint8), torch.zeros(4, 16, 2, 64, dtype=torch.float16)
    pairs = torch.zeros(1, 2, dtype=torch.int64)
    for args in ((a, b), (a, a[:3]), (torch.zeros(4, 2, 16, 40, dtype=torch.uint8),) * 2):
        with pytest.raises(L.PkvError):
            E.copy_blocks(*args, pairs)
    for args in ((a, a, b, b), (a, a, a[:, :1], a[:, :1]), (a, a[:3], a, a), (a, a, a, a[:2])):
        with pytest.raises(L.PkvError):
            E.swap_blocks(*args, pairs, L.PKV_SWAP_OUT)


def test_the_workloads_lay_the_cache_out_alike():
    import importlib.util
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")
    spec = importlib.util.spec_from_file_location("more_operators", path)
    M = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(M)
    for D in (64, 128):
        x = torch.randn(3, 2, 8, D, generator=torch.Generator().manual_seed(D))
        pool = M._pack(x, torch.bfloat16).view(3, 2, 8, Q.row_bytes(D))
        v = Q.values(pool.numpy(), D, "bf16")
        assert np.array_equal(v, M._unpack(pool, D, torch.bfloat16).double().numpy())


# ---------------------------------------------------------------- how step and centre are rounded
def ends_apart(rng, dtype, n):
    """Rows [n, 64] that both 16-bit types hold, with ends far apart in size and, in part, with
    max - min or 8 max + 7 min at 15 times a number halfway between two of the type's."""
    bits = 11 if dtype == "f16" else 8
    x = np.zeros((n, 64))
    half = (2 * rng.integers(1 << (bits - 1), 1 << bits, n) + 1) * 15.0     # times 2^-k below
    hi = np.floor(half * rng.uniform(0.01, 0.99, n) / 2 ** (17 - bits)) * 2 ** (17 - bits)
    x[:, 0], x[:, 1] = hi, hi - half
    wide = np.exp2(rng.integers(-6, 7, n))
    x[::3, 0], x[::3, 1] = rng.integers(1, 200, x[::3].shape[0]) * wide[::3], -rng.integers(1, 200, x[::3].shape[0]) / 64
    x = Q.widen(Q.narrow(x / 512, dtype), dtype)
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    mid = Q.widen(Q.narrow(lo + (hi - lo) * rng.uniform(0, 1, (n, 64)), dtype), dtype)
    mid[:, :2] = x[:, :2]
    return np.clip(mid, lo, hi)


def rounding_bound(step, centre, dtype):
    """What include/pagedkv.h says that an element may be off by."""
    u = C.U[dtype] + 2.0 ** -21
    return step * (0.5 + 2.0 ** -18) + u * (8 * step + np.abs(centre)) + (2.0 ** -21 if dtype == "f16" else 2.0 ** -122)


def check_rounding(x, step, centre, code, dtype):
    """step, centre (bits) and codes of rows x: the 64-bit quotients rounded once, but for those within
    2^-21 of halfway, which may go to either side; values within the bound."""
    g = x.reshape(x.shape[:-1] + (-1, 64))
    hi, lo = g.max(-1), g.min(-1)
    size = np.maximum(np.abs(hi), np.abs(lo))
    for got, exact, slack in ((step, (hi - lo) / 15, (hi - lo) / 15 * 2.0 ** -21),
                              (centre, (8 * hi + 7 * lo) / 15, size * 2.0 ** -21)):
        below, above = (Q.widen(Q.narrow(exact + s, dtype), dtype) for s in (-slack, slack))
        value = Q.widen(got, dtype)
        assert ((below <= value) & (value <= above)).all()
    s, a = (np.repeat(Q.widen(y, dtype), 64, -1).reshape(x.shape) for y in (step, centre))
    assert (np.abs(a + s * (code - 8) - x) <= rounding_bound(s, a, dtype)).all()
    return (step != Q.narrow((hi - lo) / 15, dtype)).sum()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_step_and_centre_are_those_of_fp32_numbers(dtype):
    """A product with fp32's 1/15, rounded again to 16 bits: a quotient halfway between two 16-bit
    numbers may go to either, and every element keeps the stated bound."""
    rng = np.random.default_rng(8)
    x = ends_apart(rng, dtype, 6000)
    assert check_rounding(x, *Q.quantise(x, dtype, np.float32), dtype) > 0
    assert check_rounding(x, *Q.quantise(x, dtype), dtype) == 0
    # steps and centres below fp16's normal numbers, down to a step of 0
    small = rng.standard_normal((3000, 64)) * np.exp2(rng.integers(-24, -12, (3000, 1)))
    small = Q.widen(Q.narrow(small, "f16"), "f16")
    for wide in (np.float32, np.float64):
        step, centre, code = Q.quantise(small, "f16", wide)
        s, a = (np.repeat(Q.widen(y, "f16"), 64, -1) for y in (step, centre))
        assert (step == 0).any()
        assert (np.abs(a + s * (code - 8) - small) <= rounding_bound(s, a, "f16")).all()
