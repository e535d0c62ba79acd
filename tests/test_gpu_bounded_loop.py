"""The bounded-cache calls together, as a serving loop uses them, against the
64-bit definitions after every step."""
import math

import numpy as np
import pytest
import torch

import workloads as W
from oracle import bounded as B
from paged_kv_cache_162_gb300 import _lib as L
from paged_kv_cache_162_gb300 import engine as E
from paged_kv_cache_162_gb300.allocator import BlockAllocator
from tests.gpu_harness import assert_attention_close, device_step
from tests.test_gpu_bounded import DT

pytestmark = pytest.mark.gpu


def close(got, ref, dtype):
    """2e-3 + 1e-2 |ref|, the library's bar for attention."""
    assert_attention_close(got.float().cpu().double().numpy(), ref, dtype)


def appended(alloc, tables, nblocks, ctx, S, H, Hkv, D, bs, dt, g, k, v):
    """Room for one token per sequence, its K and V written; returns device
    tables and lengths, and the new q."""
    for s in range(S):
        nblocks[s], pairs = alloc.append_row(tables[s], int(nblocks[s]), int(ctx[s]), 1, bs)
        assert len(pairs) == 0
    bt = torch.from_numpy(tables).cuda()
    nk = torch.randn(S, Hkv, D, generator=g).to(dt).cuda()
    nv = torch.randn(S, Hkv, D, generator=g).to(dt).cuda()
    q = torch.randn(S, H, D, generator=g).to(dt).cuda()
    slots = torch.empty(S, dtype=torch.int64, device="cuda")
    E.compute_slot_mapping(slots, bt, torch.arange(S, dtype=torch.int32, device="cuda"), torch.from_numpy(ctx).cuda(), bs)
    E.reshape_and_cache(nk, nv, k, v, slots)
    ctx += 1
    return bt, torch.from_numpy(ctx).cuda(), q


@pytest.mark.parametrize("dtype,H,Hkv,D,bs", [("f16", 4, 4, 64, 8), ("bf16", 8, 2, 128, 16)])
def test_decode_with_eviction(dtype, H, Hkv, D, bs):
    """40 decode steps: every sequence keeps at most budget + bs tokens, its
    blocks go back to the pool, scores follow the moved tokens."""
    S, NB, budget, recent, sinks = 3, 64, 48, 12, 2
    MB = (budget + bs) // bs + 8
    dt = DT[dtype]
    g = torch.Generator().manual_seed(3)
    k = torch.full((NB, bs, Hkv, D), float("nan"), dtype=dt, device="cuda")
    v = k.clone()
    alloc = BlockAllocator(NB)
    tables, nblocks = np.full((S, MB), -1, np.int32), np.zeros(S, np.int32)
    ctx = np.array([0, 5, 60], np.int32)
    for s in range(S):  # prompts
        nblocks[s], _ = alloc.append_row(tables[s], 0, 0, int(ctx[s]), bs)
    rows = np.concatenate([B.rows_of(tables[s], range(int(ctx[s])), bs) for s in range(S)])
    prompt = torch.randn(2, len(rows), Hkv, D, generator=g).to(dt).cuda()
    E.reshape_and_cache(prompt[0], prompt[1], k, v, torch.from_numpy(rows).cuda())
    seen, cap, scale = ctx.copy(), MB * bs, 1 / math.sqrt(D)
    scores = torch.zeros(S, Hkv, cap, device="cuda")
    pos = torch.full((S, Hkv, cap), -1, dtype=torch.int32, device="cuda")
    w_scores, w_pos = np.zeros((S, Hkv, cap)), np.full((S, Hkv, cap), -1, np.int32)
    ws = E.new_accumulate_workspace(S, H, Hkv, D, cap)
    evictions = 0
    for step in range(40):
        bt, lens, q = appended(alloc, tables, nblocks, ctx, S, H, Hkv, D, bs, dt, g, k, v)
        seen += 1
        out = torch.empty(S, H, D, dtype=dt, device="cuda")
        E.paged_attention_decode_accumulate(out, scores, q, k, v, bt, lens, scale, workspace=ws)
        kn, vn = k.double().cpu().numpy(), v.double().cpu().numpy()
        ref, weights, _ = B.attend(q.double().cpu().numpy(), kn, vn, tables, ctx, scale)
        close(out, ref, dtype)
        w_scores = B.accumulate(w_scores, weights, Hkv)
        got = scores.double().cpu().numpy()
        # 40 steps of at most G a step, fp32: far inside 1e-4
        assert np.abs(got - w_scores).max() < 1e-4
        if (ctx >= budget + bs).any():
            evictions += 1
            new = torch.empty_like(lens)
            E.evict_tokens(k, v, scores, pos, bt, lens, torch.from_numpy(seen).cuda(), new, budget, recent, sinks)
            # the definition on what the GPU had: scores that agree to rounding may order differently
            w_scores = got.copy()
            ki = kn.copy()
            lens_after = B.evict(ki, vn, w_scores, w_pos, tables, ctx, seen, budget, recent, sinks)
            assert np.array_equal(new.cpu().numpy(), lens_after)
            assert np.array_equal(pos.cpu().numpy(), w_pos)
            assert np.array_equal(scores.double().cpu().numpy(), w_scores)
            assert np.array_equal(k.double().cpu().numpy(), ki, equal_nan=True)
            for s in range(S):
                free = alloc.num_free
                nblocks[s], freed = alloc.truncate(tables[s], int(nblocks[s]), int(lens_after[s]), bs)
                assert alloc.num_free == free + freed and nblocks[s] == -(-int(lens_after[s]) // bs)
                if ctx[s] > budget:  # the newest and the first tokens are still there
                    kept = w_pos[s, :, :budget]
                    assert all(set(range(seen[s] - recent, seen[s])) <= set(r.tolist()) for r in kept)
                    assert all(set(range(sinks)) <= set(r.tolist()) for r in kept)
            ctx[:] = lens_after
    assert evictions >= 3 and ctx.max() <= budget + bs
    assert L.pkv_get_device_errors() == 0


@pytest.mark.parametrize("dtype,H,Hkv,D,bs", [("bf16", 4, 4, 64, 8), ("f16", 16, 4, 128, 16)])
def test_decode_with_a_window(dtype, H, Hkv, D, bs):
    """More decode steps than the pool could hold tokens of: passed blocks are
    released, reused and overwritten by other sequences."""
    S, window, sinks = 3, 21, 3
    NB = S * ((window + 2 * bs) // bs + 3)
    steps = NB * bs // S + 20
    MB = -(-steps // bs)
    dt = DT[dtype]
    g = torch.Generator().manual_seed(4)
    k = torch.full((NB, bs, Hkv, D), float("nan"), dtype=dt, device="cuda")
    v = k.clone()
    alloc = BlockAllocator(NB)
    tables, nblocks, ctx = np.full((S, MB), -1, np.int32), np.zeros(S, np.int32), np.zeros(S, np.int32)
    scale = 1 / math.sqrt(D)
    history = [[[], []] for _ in range(S)]   # every token's K and V, as written
    freed = 0
    for step in range(steps):
        bt, lens, q = appended(alloc, tables, nblocks, ctx, S, H, Hkv, D, bs, dt, g, k, v)
        kn, vn = k.double().cpu().numpy(), v.double().cpu().numpy()
        for s in range(S):
            r = int(B.rows_of(tables[s], [int(ctx[s]) - 1], bs)[0])
            history[s][0].append(kn.reshape(-1, Hkv, D)[r])
            history[s][1].append(vn.reshape(-1, Hkv, D)[r])
        out = torch.empty(S, H, D, dtype=dt, device="cuda")
        E.paged_attention_decode_window(out, q, k, v, bt, lens, window, sinks, scale)
        n = int(ctx[0])
        hk = np.stack([np.stack(h[0]) for h in history])   # [S, n, Hkv, D]: one long block per sequence
        hv = np.stack([np.stack(h[1]) for h in history])
        ref, _, _ = B.attend(q.double().cpu().numpy(), hk, hv, np.arange(S)[:, None], ctx, scale, window, sinks)
        close(out, ref, dtype)
        for s in range(S):
            freed += alloc.release_window(tables[s], int(nblocks[s]), n, window, sinks, bs)
    assert freed > 0 and NB * bs < S * steps
    assert L.pkv_get_device_errors() == 0


def test_decode_step_methods():
    """DecodeStep: accumulate, evict with shared prompt blocks (copied first),
    decode what is left; the other sequences' blocks are unchanged."""
    w = W.shared_prefix(seed=9, prompts=2, samples=3, prefix=160, tail_lo=1, tail_hi=60, H=4, D=64)
    more = np.arange(w.NB, w.NB + 40, dtype=np.int32)      # room to copy the shared blocks
    w.initial_free, w.NB = np.concatenate([more, w.initial_free]), w.NB + 40
    st = device_step(w)
    st.plan()
    st.run()
    S, bs, budget = w.S, w.bs, 96
    ctx = st.context_lens_host.copy()
    full = st.out.clone()
    st.out.zero_()
    st.decode_accumulate()
    close(st.out, full.double().cpu().numpy(), "as decode()")
    assert torch.allclose(st.scores.sum(-1), torch.ones(S, 4, device="cuda"), atol=1e-4)
    kn, vn = st.k_cache.double().cpu().numpy(), st.v_cache.double().cpu().numpy()
    tables = st.tables_host.copy()
    st.decode_window(50, 4)
    ref, _, _ = B.attend(st.q.double().cpu().numpy(), kn, vn, tables, ctx, st.scale, 50, 4)
    close(st.out, ref, "window")
    sc, pos = st.scores.cpu().numpy().copy(), st.positions.cpu().numpy().copy()
    free = st.allocator.num_free
    freed = st.evict(budget, 20, 4)
    assert (st.context_lens_host == np.minimum(ctx, budget)).all()
    assert (st.context_lens.cpu().numpy() == st.context_lens_host).all()
    held = [set(t[:n].tolist()) for t, n in zip(st.tables_host, st.nblocks_host)]
    assert all(len(h) == -(-budget // bs) for h in held)
    assert sum(len(h) for h in held) == len(set().union(*held)), "evicted rows own their blocks"
    assert freed > 0 and st.allocator.num_free + sum(len(h) for h in held) == w.NB
    ref = np.zeros((S, 4, 64))
    q = st.q.double().cpu().numpy()
    for s in range(S):
        n = int(ctx[s])
        for h in range(4):
            r = B.evict_row(sc[s, h], pos[s, h], n, n, budget, 20, 4)
            source = r[0] if r else list(range(n))
            rows = B.rows_of(tables[s], source, bs)
            z = st.scale * (kn.reshape(-1, 4, 64)[rows, h] @ q[s, h])
            p = np.exp(z - z.max())
            ref[s, h] = (p / p.sum()) @ vn.reshape(-1, 4, 64)[rows, h]
    st.decode()
    close(st.out, ref, "after eviction")
    assert L.pkv_get_device_errors() == 0


def test_evict_without_room_for_the_shared_blocks_leaves_a_valid_step():
    """OutOfBlocks from copy-on-write: blocks copied so far are the rows' own,
    with their contents, and decoding gives what it gave."""
    w = W.shared_prefix(seed=9, prompts=2, samples=3, prefix=160, tail_lo=1, tail_hi=60, H=4, D=64)
    st = device_step(w)
    st.plan()
    st.run()
    want = st.out.clone()
    st.decode_accumulate()
    lens = st.context_lens_host.copy()
    with pytest.raises(L.PkvError) as e:
        st.evict(96, 20, 4)
    assert e.value.status == L.PKV_ERR_OOM
    assert np.array_equal(st.context_lens_host, lens)
    st.out.zero_()
    st.decode()
    assert torch.equal(st.out.view(torch.int16), want.view(torch.int16))
    assert np.array_equal(st.block_tables.cpu().numpy(), st.tables_host)
