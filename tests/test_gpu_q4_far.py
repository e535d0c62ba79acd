"""The rotating appends and the 4-bit cache where bytes lie past 32 bits: pools and
strided tokens of more than 4 GiB, against the same data close together (which the
other tests hold to the definitions)."""
import numpy as np
import pytest
import torch

import q4_cases as C
from paged_kv_cache_162_gb300 import _lib as L
from paged_kv_cache_162_gb300 import engine as E

pytestmark = pytest.mark.gpu

GIB = 1 << 30


def far_ids(n, NB):
    """n block ids of NB: the last, the first, and some around every 2^31 and 2^32 bytes of a pool just past 4 GiB."""
    ids = [NB - 1, 0, NB // 2, NB // 2 - 1, NB - 2, 1, NB * 3 // 4, NB // 4]
    return np.array((ids + [NB // 3 + i for i in range(n)])[:n], np.int32)


def append(c, d, q4, tables, k, v, out):
    (E.rotate_and_cache_q4 if q4 else E.rotate_and_cache)(
        d["key"], d["value"], k, v, tables, d["seq"], d["pos"], d["slots"], d["table"], query=d["query"], query_out=out)
    return d["slots"].clone()


def only(pool, blocks):
    """Nothing but these blocks of a pool of zeros has been written."""
    rest = torch.ones(pool.shape[0], dtype=torch.bool, device="cuda")
    rest[blocks] = False
    for i in range(0, pool.shape[0], 8192):
        part = pool[i:i + 8192].view(min(8192, pool.shape[0] - i), -1).view(torch.int64).ne(0).any(-1)
        if (part & rest[i:i + 8192]).any():
            return False
    return True


@pytest.mark.parametrize("q4,D,dtype", [(True, 128, "bf16"), (True, 64, "f16"), (False, 128, "f16")])
def test_a_pool_past_32_bits(q4, D, dtype):
    Hkv, H, bs = 8, 16, 64
    c = C.append_case(51, S=3, H=H, Hkv=Hkv, D=D, bs=bs, dtype=dtype, new=[300, 1, 129], before=[0, 63, 0], pad=2)
    per = Hkv * bs * (D // 2 + D // 16 if q4 else 2 * D)
    NB = 4 * GIB // per + 200
    near = torch.from_numpy(c["tables"]).cuda()
    ids = torch.from_numpy(far_ids(c["NB"], NB)).cuda()
    assert len(ids.unique()) == c["NB"] and (int(ids.max()) * per) >> 32 and NB * bs < 2 ** 31
    far = torch.where(near >= 0, ids[near.clamp(min=0).long()], near)
    pools, got = [], []
    for n, tables in ((c["NB"], near), (NB, far)):
        shape, t = ((n, Hkv, bs, D // 2 + D // 16), torch.uint8) if q4 else ((n, bs, Hkv, D), C.DT[dtype])
        k, v = (torch.zeros(shape, dtype=t, device="cuda") for _ in range(2))
        d = C.append_on_gpu(c)
        out = torch.zeros_like(d["query"])
        slots = append(c, d, q4, tables, k, v, out)
        pools.append((k, v))
        got.append([out])
        lens = torch.tensor([300, 64, 129], dtype=torch.int32, device="cuda")
        q = torch.randn(3, H, D, generator=torch.Generator("cuda").manual_seed(1), device="cuda", dtype=C.DT[dtype])
        res = torch.empty_like(q)
        if q4:
            rows = [torch.zeros_like(d["key"]) for _ in range(2)]
            E.gather_cache_q4(*rows, k, v, slots)
            got[-1] += rows
            for most in (0, 300):
                E.paged_attention_decode_q4(res, q, k, v, tables, lens, max_context_len=most)
                got[-1].append(res.clone())
            # the split form
            wide = torch.cat([tables, torch.full((3, 4096), -1, dtype=torch.int32, device="cuda")], -1)
            E.paged_attention_decode_q4(res, q, k, v, wide, lens)
        else:
            E.paged_attention_decode_window(res, q, k, v, tables, lens, window=300)
        got[-1].append(res)
    for a, b in zip(*got):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    for a, b in zip(*pools):
        assert torch.equal(a, b[ids.long()]) and only(b, ids.long())
    if q4:  # copies from end to end
        (k, v), last, first = pools[1], int(ids[0]), int(ids[1])
        want = k[last].clone(), v[last].clone(), k[first].clone(), v[first].clone()
        E.copy_blocks(k, v, torch.tensor([[last, 7], [first, NB - 5]], device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip((k[7], v[7], k[NB - 5], v[NB - 5]), want))
    assert L.pkv_get_device_errors() == 0


@pytest.mark.parametrize("q4", [False, True])
def test_tokens_past_32_bits(q4):
    """Tokens 1 MB apart, 4200 of them: rows of queries, keys and values past 2^32 bytes."""
    T, H, Hkv, D, bs, wide = 4200, 4, 2, 64, 16, 1 << 19
    c = C.append_case(52, S=1, H=H, Hkv=Hkv, D=D, bs=bs, dtype="f16", new=[T])
    big = torch.zeros(T, wide, dtype=torch.float16, device="cuda")
    assert (T - 1) * wide * 2 >> 32
    at = {"query": 0, "key": H * D, "value": wide - Hkv * D}
    got = []
    for far in (False, True):
        d = C.append_on_gpu(c)
        if far:
            for name, x in at.items():
                view = big[:, x:x + d[name][0].numel()].unflatten(-1, (-1, D))
                view.copy_(d[name])
                d[name] = view
        shape = (c["NB"], bs, Hkv, D)
        k, v = (E.new_cache_q4(c["NB"], bs, Hkv, D) if q4 else torch.zeros(shape, dtype=torch.float16, device="cuda") for _ in "kv")
        slots = append(c, d, q4, d["tables"], k, v, None)
        got.append([k, v, slots, d["query"].contiguous()])
        if q4:
            rows = [d[name] if far else torch.zeros_like(d[name]) for name in ("key", "value")]
            E.gather_cache_q4(*rows, k, v, slots)
            got[-1] += [x.contiguous() for x in rows]
    assert all(torch.equal(a, b) for a, b in zip(*got))
    # between the rows nothing was written
    assert not big[:, (H + Hkv) * D:wide - Hkv * D].any()
    assert L.pkv_get_device_errors() == 0
