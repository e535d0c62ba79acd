"""The rotating appends, the 4-bit cache and the block allocator together, as a
serving loop uses them, against histories kept token by token on the host."""
import numpy as np
import pytest
import torch

import q4_cases as C
from oracle import bounded as B
from oracle import q4 as Q
from paged_kv_cache_162_gb300 import _lib as L
from paged_kv_cache_162_gb300 import engine as E
from paged_kv_cache_162_gb300.allocator import BlockAllocator

pytestmark = pytest.mark.gpu


class Model:
    """A rotary model's projections of new tokens, on the host and on the device."""

    def __init__(self, dtype, H, Hkv, D, R, positions, seed):
        self.dtype, self.H, self.Hkv, self.D, self.R = dtype, H, Hkv, D, R
        self.rng = np.random.default_rng(seed)
        self.table = E.new_rotary_table(positions, R)
        self.cos, self.sin = np.split(self.table.cpu().numpy(), 2, -1)

    def tokens(self, T):
        """One projection [T, (H + 2 Hkv) D]: its bits, and query, key, value as slices of the device's."""
        bits = Q.narrow(self.rng.standard_normal((T, self.H + 2 * self.Hkv, self.D)), self.dtype)
        dev = C.tensor(bits, self.dtype).cuda().view(T, -1)
        parts = dev.split([self.H * self.D, self.Hkv * self.D, self.Hkv * self.D], -1)
        return bits, [x.unflatten(-1, (-1, self.D)) for x in parts]

    def turned(self, bits, pos):
        """A token's rows in fp32, rotated for position pos as the library rounds."""
        return Q.rotate(Q.widen(bits, self.dtype).astype(np.float32), self.cos[pos], self.sin[pos], False)


def reference(m, histories, q_bits, bs):
    """attend_reference of every sequence's history [(K quantised, V quantised) per token]."""
    S = len(histories)
    lens = np.array([len(h) for h in histories], np.int32)
    MB = max(1, -(-int(lens.max()) // bs))
    tables = np.arange(S * MB, dtype=np.int32).reshape(S, MB)
    c = dict(S=S, H=m.H, Hkv=m.Hkv, D=m.D, bs=bs, dtype=m.dtype, lens=lens, tables=tables, scale=m.D ** -0.5, q=q_bits)
    for i, name in enumerate("kv"):
        step, centre = (np.zeros((S * MB, bs, m.Hkv, m.D // 64), np.uint16) for _ in range(2))
        code = np.zeros((S * MB, bs, m.Hkv, m.D), np.int64)
        for s, h in enumerate(histories):
            for j, tok in enumerate(h):
                at = (tables[s, j // bs], j % bs)
                step[at], centre[at], code[at] = tok[i]
        c[name] = Q.pack(step, centre, code)
    return C.attend_reference(c)


@pytest.mark.parametrize("dtype,H,Hkv,D,R,bs", [("bf16", 8, 2, 128, 128, 16), ("f16", 3, 3, 64, 32, 8)])
def test_serving_loop_over_a_4_bit_cache(dtype, H, Hkv, D, R, bs):
    """Prompts in one padded call, forks that share blocks, copies on write, 14 decode steps, one
    sequence swapped out and back, and in the end moved to a 16-bit cache."""
    m = Model(dtype, H, Hkv, D, R, 200, 4)
    NB, MB, S = 60, 16, 4
    alloc = BlockAllocator(NB)
    k, v = E.new_cache_q4(NB, bs, Hkv, D), E.new_cache_q4(NB, bs, Hkv, D)
    tables, nblocks = np.full((S, MB), -1, np.int32), np.zeros(S, np.int32)
    ctx = np.array([37, 5, 0, 0], np.int32)
    for s in (0, 1):
        nblocks[s], _ = alloc.append_row(tables[s], 0, 0, int(ctx[s]), bs)
    ws = E.new_q4_workspace(S, H, Hkv, D)
    histories = [[] for _ in range(S)]

    def append(seq, pos):
        """The tokens' queries as the device has them [T, H, D], and their slots."""
        bits, (q, key, value) = m.tokens(len(seq))
        slots = torch.empty(len(seq), dtype=torch.int64, device="cuda")
        E.rotate_and_cache_q4(key, value, k, v, torch.from_numpy(tables).cuda(),
                              torch.tensor(seq, dtype=torch.int32, device="cuda"),
                              torch.tensor(pos, dtype=torch.int32, device="cuda"), slots, m.table, query=q)
        for t, (s, at) in enumerate(zip(seq, pos)):
            if at >= 0:
                assert len(histories[s]) == at
                rows = (m.turned(bits[t, H:H + Hkv], at), Q.widen(bits[t, H + Hkv:], dtype).astype(np.float32))
                histories[s].append(tuple(Q.quantise(x, dtype, np.float32) for x in rows))
        assert np.array_equal(slots.cpu().numpy(), Q.slots(tables, seq, pos, bs))
        return q

    append([0] * 37 + [1] * 5 + [0] * 6, list(range(37)) + list(range(5)) + [-1] * 6)
    parents = np.array([0, 1, 0, 1], np.int32)
    alloc.fork(tables, nblocks, parents)
    ctx = ctx[parents]
    histories = [list(histories[p]) for p in parents]
    copies = 0
    for step in range(14):
        if step == 6:  # sequence 2 to the host and back, into other blocks
            host = [torch.zeros((MB, Hkv, bs, k.shape[3]), dtype=torch.uint8).pin_memory() for _ in range(2)]
            mine = tables[2, :nblocks[2]].copy()
            out = torch.tensor([[int(b), i] for i, b in enumerate(mine)], device="cuda")
            E.swap_blocks(k, v, *host, out, L.PKV_SWAP_OUT)
            fresh = alloc.alloc(len(mine))
            alloc.decref(mine)
            tables[2, :len(mine)] = fresh
            E.swap_blocks(k, v, *host, torch.tensor([[i, b] for i, b in enumerate(fresh)], device="cuda"), L.PKV_SWAP_IN)
        pairs = alloc.append_batch(tables, nblocks, ctx, np.ones(S, np.int32), bs)
        copies += len(pairs)
        if len(pairs):
            E.copy_blocks(k, v, torch.from_numpy(np.ascontiguousarray(pairs)).cuda())
        q = append(list(range(S)), ctx.tolist())
        ctx = ctx + 1
        out = torch.empty(S, H, D, dtype=C.DT[dtype], device="cuda")
        E.paged_attention_decode_q4(out, q.contiguous(), k, v, torch.from_numpy(tables).cuda(),
                                    torch.from_numpy(ctx).cuda(), workspace=ws)
        ref, bound = reference(m, histories, C.bits_of(q), bs)
        assert (np.abs(Q.widen(C.bits_of(out), dtype) - ref) <= bound).all(), step
    assert copies > 0  # forks wrote into shared blocks
    # sequence 3 into a 16-bit cache, and on from there
    n = int(ctx[3])
    slots = torch.tensor([int(tables[3, j // bs]) * bs + j % bs for j in range(n)], device="cuda")
    rows = [torch.empty(n, Hkv, D, dtype=C.DT[dtype], device="cuda") for _ in range(2)]
    E.gather_cache_q4(*rows, k, v, slots)
    caches = [torch.zeros(MB, bs, Hkv, D, dtype=C.DT[dtype], device="cuda") for _ in range(2)]
    E.reshape_and_cache(*rows, *caches, torch.arange(n, device="cuda"))
    o16 = torch.empty(1, H, D, dtype=C.DT[dtype], device="cuda")
    E.paged_attention_decode_window(o16, q[3:4].contiguous(), *caches,
                                    torch.arange(MB, dtype=torch.int32, device="cuda")[None],
                                    torch.tensor([n], dtype=torch.int32, device="cuda"), window=n)
    got, ref = (Q.widen(C.bits_of(x), dtype) for x in (o16[0], out[3]))
    # values of up to a few units rounded by u, weights off by u times logits of a few units
    assert np.abs(got - ref).max() <= 40 * C.U[dtype]
    assert L.pkv_get_device_errors() == 0


def test_rotation_by_position_after_an_eviction():
    """16-bit caches: after evict_tokens a token's place in the cache lies below its position."""
    m = Model("f16", 2, 2, 64, 64, 100, 5)
    bs, NB = 8, 20
    k, v = (torch.zeros(NB, bs, 2, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    tables = torch.arange(NB, dtype=torch.int32, device="cuda")[None]
    one = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731

    def append(places, positions):
        bits, (q, key, value) = m.tokens(len(places))
        slots = torch.empty(len(places), dtype=torch.int64, device="cuda")
        E.rotate_and_cache(key, value, k, v, tables, torch.zeros(len(places), dtype=torch.int32, device="cuda"),
                           torch.tensor(places, dtype=torch.int32, device="cuda"), slots, m.table, query=q,
                           rotary_pos=torch.tensor(positions, dtype=torch.int32, device="cuda"))
        return bits, q

    append(list(range(40)), list(range(40)))
    scores = torch.rand(1, 2, NB * bs, device="cuda")
    positions = torch.full((1, 2, NB * bs), -1, dtype=torch.int32, device="cuda")
    lens = one(0)
    E.evict_tokens(k, v, scores, positions, tables, one(40), one(40), lens, budget=16, recent_tokens=4)
    assert int(lens) == 16
    bits, q = append([16], [40])
    got = Q.widen(C.bits_of(k.view(-1, 2, 64)[16]), "f16")
    ref = Q.rotate(Q.widen(bits[0, 2:4], "f16"), m.cos[40].astype(float), m.sin[40].astype(float), False)
    mag = np.abs(Q.widen(bits[0, 2:4], "f16")).max()
    assert np.abs(got - ref).max() <= 2.0 ** -11 * 2 * mag + 2.01 * C.E32 * 2 * mag
    # and the attention over what is left
    out = torch.empty(1, 2, 64, dtype=torch.float16, device="cuda")
    E.paged_attention_decode_window(out, q.contiguous(), k, v, tables, one(17), window=17)
    kk, vv = (x.double().cpu().numpy() for x in (k, v))
    ref, _, _ = B.attend(Q.widen(C.bits_of(q), "f16"), kk, vv, tables.cpu().numpy(), [17], 0.125)
    assert np.abs(Q.widen(C.bits_of(out), "f16") - ref).max() <= 4e-3
    assert L.pkv_get_device_errors() == 0
