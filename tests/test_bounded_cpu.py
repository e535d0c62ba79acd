"""The bounded-cache operators without a GPU: the 64-bit oracle against hand
values and the existing decode oracle, the allocator calls that go with
eviction and windows, and refusals before any launch."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import bounded as B
from oracle import kernels as K
from paged_kv_cache_162_gb300 import _lib as L
from paged_kv_cache_162_gb300 import engine as E
from paged_kv_cache_162_gb300.allocator import BlockAllocator, OutOfBlocks


# ------------------------------------------------------------- the oracle
def test_visible_tokens_by_hand():
    assert B.visible(0, 3, 2) == []
    assert B.visible(1, 1, 0) == [0]
    assert B.visible(10, 3, 2) == [0, 1, 7, 8, 9]
    assert B.visible(10, 3, 0) == [7, 8, 9]
    assert B.visible(10, 9, 1) == list(range(10))     # the gap closes
    assert B.visible(10, 8, 1) == [0] + list(range(2, 10))
    assert B.visible(4, 100, 50) == [0, 1, 2, 3]


def test_window_oracle_with_everything_visible_is_the_decode_oracle():
    rng = np.random.default_rng(5)
    S, H, D, bs, NB = 3, 2, 64, 8, 12
    bits = lambda shape: W.normal_bits(np.random.Generator(np.random.SFC64(int(rng.integers(1 << 30)))), shape, W.F16)
    q, k, v = bits((S, H, D)), bits((NB, bs, H, D)), bits((NB, bs, H, D))
    tables = np.array([[3, 7, 1, 0], [5, 2, 9, 8], [11, 4, 6, 10]], np.int32)
    lens = np.array([25, 8, 31], np.int32)
    ref = K.decode(q, k, v, tables, lens, 0.125, False)
    f = lambda x: x.view(np.float16).astype(np.float64)
    for window, sinks in ((None, 0), (31, 0), (1000, 5)):
        out, weights, mag = B.attend(f(q), f(k), f(v), tables, lens, 0.125, window, sinks)
        assert np.abs(out - ref).max() < 1e-12
        assert all(abs(p.sum(1) - 1).max() < 1e-12 for _, p in weights)
        assert (mag >= np.abs(out) - 1e-15).all()


def test_accumulated_weights_add_up_to_the_query_heads():
    rng = np.random.default_rng(6)
    S, Hkv, G, D, bs, NB = 2, 3, 4, 64, 8, 9
    q, k, v = (rng.standard_normal(s) for s in ((S, Hkv * G, D), (NB, bs, Hkv, D), (NB, bs, Hkv, D)))
    tables = np.array([[0, 3, 6], [8, 1, 2]])
    lens = np.array([20, 9])
    _, w, _ = B.attend(q, k, v, tables, lens, 0.2)
    out = B.accumulate(np.zeros((S, Hkv, 24)), w, Hkv)
    assert np.allclose(out.sum(-1), G)
    assert (out[0, :, 20:] == 0).all() and (out[1, :, 9:] == 0).all()


def test_eviction_by_hand():
    # 8 tokens, keep 4: token 0 (sink) and 7 (recent) are safe; of the rest
    # 3 and 5 score highest.  Holes 1, 2; movers 5, 7.
    score = [0.1, 0.2, 0.1, 0.9, 0.3, 0.8, 0.2, 0.0]
    source, pos = B.evict_row(score, [-1] * 8, 8, 8, budget=4, recent=1, sinks=1)
    assert source == [0, 5, 7, 3] and pos == [0, 5, 7, 3]
    # again with 2 more tokens: entries 0..3 hold positions 0, 5, 7, 3 and
    # entries 4, 5 are tokens 8, 9; 9 is recent, 7 no longer is
    score = [0.1, 0.8, 0.05, 0.9, 0.4, 0.0]
    source, pos = B.evict_row(score, [0, 5, 7, 3, -1, -1], 6, 10, budget=4, recent=1, sinks=1)
    assert source == [0, 1, 5, 3] and pos == [0, 5, 9, 3]
    # ties stay from the lowest index; NaN is no better than -inf
    assert B.evict_row([1.0] * 6, [-1] * 6, 6, 6, 3, 0, 0) == ([0, 1, 2], [0, 1, 2])
    assert B.evict_row([np.nan, -np.inf, 0.0], [-1] * 3, 3, 3, 2, 0, 0)[0] == [0, 2]
    assert B.evict_row([0.0, -0.0, 0.0], [-1] * 3, 3, 3, 2, 0, 0)[0] == [0, 1]
    assert B.evict_row([1.0, 2.0], [-1] * 2, 2, 2, 2, 0, 0) is None


# ---------------------------------------------------------- the allocator
def test_unshare_copies_only_shared_blocks_in_order():
    a = BlockAllocator(12)
    row = np.array(a.alloc(5), np.int32)      # 11, 10, 9, 8, 7
    a.incref(row[1:4])
    before = row.copy()
    pairs = a.unshare(row, 3)
    assert pairs.tolist() == [[before[1], 6], [before[2], 5]]
    assert row.tolist() == [11, 6, 5, 8, 7]
    assert [a.refcount(int(b)) for b in before] == [1, 1, 1, 2, 1]
    assert a.refcount(6) == a.refcount(5) == 1
    assert len(a.unshare(row, 3)) == 0 and len(a.unshare(row, 0)) == 0
    with pytest.raises(L.PkvError):
        a.unshare(row, 6)


def test_unshare_without_room_changes_nothing():
    a = BlockAllocator(4)
    row = np.array(a.alloc(3), np.int32)
    a.incref(row)
    before = row.copy()
    with pytest.raises(OutOfBlocks):
        a.unshare(row, 3)
    assert np.array_equal(row, before) and a.num_free == 1
    assert [a.refcount(int(b)) for b in row] == [2, 2, 2]
    bad = np.array([int(row[0]), -1, int(row[1])], np.int32)
    with pytest.raises(L.PkvError):
        a.unshare(bad, 2)


@pytest.mark.parametrize("tokens,keep", [(0, 0), (1, 1), (15, 1), (16, 1), (17, 2), (64, 4), (1000, 5)])
def test_truncate_frees_the_tail_last_first(tokens, keep):
    a = BlockAllocator(8)
    row = np.full(7, -1, np.int32)
    row[:5] = a.alloc(5)
    ids = row[:5].tolist()
    a.incref(ids[4:])                         # the last block has another holder
    nb, freed = a.truncate(row, 5, tokens, 16)
    assert nb == keep and freed == max(0, 5 - keep) - (1 if keep < 5 else 0)
    assert row.tolist() == ids[:keep] + [-1] * (7 - keep)
    gone = [b for b in ids[keep:] if b != ids[4]]
    if gone:                                  # the lowest entry was freed last: handed out first
        assert a.alloc(1) == [gone[0]]


def test_truncate_passes_over_released_entries_and_checks_first():
    a = BlockAllocator(8)
    row = np.array(a.alloc(5), np.int32)
    free_one = int(row[3])
    a.decref([free_one])
    row[3] = -1
    assert a.truncate(row, 5, 20, 16) == (2, 2)
    row = np.array(a.alloc(3), np.int32)
    a.decref([int(row[2])])                   # the row still lists a block it does not hold
    before, free = row.copy(), a.num_free
    with pytest.raises(L.PkvError):
        a.truncate(row, 3, 0, 16)
    assert np.array_equal(row, before) and a.num_free == free
    assert a.refcount(int(row[0])) == 1


def test_release_window_keeps_what_later_queries_see():
    rng = np.random.default_rng(8)
    for _ in range(300):
        bs = int(rng.choice([4, 8, 16]))
        n = int(rng.integers(0, 100))
        window, sinks = int(rng.integers(1, 60)), int(rng.integers(0, 30))
        nb = -(-n // bs) + int(rng.integers(0, 2))
        a = BlockAllocator(nb + 3)
        row = np.array(a.alloc(nb), np.int32) if nb else np.zeros(0, np.int32)
        before = row.copy()
        freed = a.release_window(row, nb, n, window, sinks, bs)
        # tokens any query from context n + 1 on sees, up to token n
        seen = set(B.visible(n + 1, window, sinks)) - {n}
        for lb in range(nb):
            holds = set(range(lb * bs, lb * bs + bs))
            dead = not (holds & seen) and max(holds) < n + 1 - window
            assert (row[lb] == -1) == dead, (n, window, sinks, bs, lb)
            assert row[lb] in (-1, before[lb])
        assert freed == (row == -1).sum() == a.num_free - 3
        assert a.release_window(row, nb, n, window, sinks, bs) == 0   # once is enough
        if nb and row[0] != -1:                                      # appending goes on
            assert a.append_row(np.append(row, -1).astype(np.int32), nb, nb * bs, 1, bs)[0] == nb + 1


def test_release_window_refuses_bad_arguments():
    a = BlockAllocator(4)
    row = np.array(a.alloc(2), np.int32)
    for kw in (dict(context_len=33), dict(window=0), dict(sink_tokens=-1), dict(block_size=0),
               dict(num_blocks=3), dict(context_len=-1)):
        args = dict(num_blocks=2, context_len=32, window=4, sink_tokens=0, block_size=16)
        args.update(kw)
        with pytest.raises(L.PkvError):
            a.release_window(row, **args)
    assert (row >= 0).all()


# --------------------------------------------------------------- refusals
def _window_args(**kw):
    a = dict(out=16, q=16, k_cache=16, v_cache=16, block_tables=16, context_lens=16, S=2, H=8,
             Hkv=4, D=128, bs=16, NB=8, MB=4, max_context_len=0, window=8, sink_tokens=2, scale=0.1,
             dtype=L.PKV_F16, workspace=256, workspace_bytes=1 << 40, stream=0)
    a.update(kw)
    return a


COMMON = [
    (dict(D=96), L.PKV_ERR_UNSUPPORTED), (dict(bs=24), L.PKV_ERR_UNSUPPORTED),
    (dict(dtype=7), L.PKV_ERR_INVALID_ARG), (dict(q=0), L.PKV_ERR_INVALID_ARG),
    (dict(out=18), L.PKV_ERR_INVALID_ARG), (dict(k_cache=24), L.PKV_ERR_INVALID_ARG),
    (dict(workspace=0), L.PKV_ERR_INVALID_ARG), (dict(workspace=272), L.PKV_ERR_INVALID_ARG),
    (dict(workspace_bytes=100), L.PKV_ERR_WORKSPACE), (dict(max_context_len=65), L.PKV_ERR_INVALID_ARG),
    (dict(max_context_len=-1), L.PKV_ERR_INVALID_ARG), (dict(scale=float("nan")), L.PKV_ERR_INVALID_ARG),
    (dict(scale=float("inf")), L.PKV_ERR_INVALID_ARG), (dict(H=9), L.PKV_ERR_INVALID_ARG),
    (dict(H=0), L.PKV_ERR_INVALID_ARG), (dict(Hkv=0), L.PKV_ERR_INVALID_ARG),
    (dict(H=68), L.PKV_ERR_UNSUPPORTED), (dict(NB=0), L.PKV_ERR_INVALID_ARG),
    (dict(NB=1 << 28), L.PKV_ERR_INVALID_ARG), (dict(S=-1), L.PKV_ERR_INVALID_ARG),
    (dict(S=32768), L.PKV_ERR_INVALID_ARG), (dict(block_tables=0), L.PKV_ERR_INVALID_ARG)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(window=0), L.PKV_ERR_INVALID_ARG), (dict(window=-3), L.PKV_ERR_INVALID_ARG),
    (dict(sink_tokens=-1), L.PKV_ERR_INVALID_ARG)])
def test_window_refuses_before_launch(kw, status):
    with pytest.raises(L.PkvError) as e:
        L.pkv_paged_attention_decode_window(**_window_args(**kw))
    assert e.value.status == status and L.pkv_last_error_string()


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(scores=0), L.PKV_ERR_INVALID_ARG), (dict(scores=18), L.PKV_ERR_INVALID_ARG),
    (dict(score_stride=63), L.PKV_ERR_INVALID_ARG)])
def test_accumulate_refuses_before_launch(kw, status):
    a = _window_args(scores=16, score_stride=64)
    del a["window"], a["sink_tokens"]
    a.update(kw)
    with pytest.raises(L.PkvError) as e:
        L.pkv_paged_attention_decode_accumulate(**a)
    assert e.value.status == status


def _evict_args(**kw):
    a = dict(k_cache=16, v_cache=16, scores=16, positions=16, block_tables=16, context_lens=16,
             token_counts=16, scores_out=16, positions_out=16, new_context_lens=32, S=2, Hkv=4, D=128,
             bs=16, NB=8, MB=4, max_context_len=0, score_stride=64, budget=32, recent_tokens=8,
             sink_tokens=4, dtype=L.PKV_BF16, workspace=256, workspace_bytes=1 << 40, stream=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(D=80), L.PKV_ERR_UNSUPPORTED), (dict(bs=4), L.PKV_ERR_UNSUPPORTED),
    (dict(dtype=2), L.PKV_ERR_INVALID_ARG), (dict(budget=0), L.PKV_ERR_INVALID_ARG),
    (dict(budget=11), L.PKV_ERR_INVALID_ARG), (dict(recent_tokens=-1), L.PKV_ERR_INVALID_ARG),
    (dict(sink_tokens=-1), L.PKV_ERR_INVALID_ARG), (dict(k_cache=8), L.PKV_ERR_INVALID_ARG),
    (dict(scores=0), L.PKV_ERR_INVALID_ARG), (dict(token_counts=0), L.PKV_ERR_INVALID_ARG),
    (dict(new_context_lens=16), L.PKV_ERR_INVALID_ARG), (dict(score_stride=63), L.PKV_ERR_INVALID_ARG),
    (dict(max_context_len=65), L.PKV_ERR_INVALID_ARG), (dict(workspace=0), L.PKV_ERR_INVALID_ARG),
    (dict(workspace=128), L.PKV_ERR_INVALID_ARG), (dict(workspace_bytes=10), L.PKV_ERR_WORKSPACE),
    (dict(S=1 << 27), L.PKV_ERR_INVALID_ARG), (dict(NB=1 << 28), L.PKV_ERR_INVALID_ARG)])
def test_evict_refuses_before_launch(kw, status):
    with pytest.raises(L.PkvError) as e:
        L.pkv_evict_tokens(**_evict_args(**kw))
    assert e.value.status == status


def test_an_empty_batch_is_a_noop():
    L.pkv_paged_attention_decode_window(**_window_args(S=0, out=0, q=0, workspace=0))
    a = _window_args(S=0, scores=0, score_stride=64)
    del a["window"], a["sink_tokens"]
    L.pkv_paged_attention_decode_accumulate(**a)
    L.pkv_evict_tokens(**_evict_args(S=0, k_cache=0, workspace=0))


def test_workspace_sizes():
    # pieces of (M, L, out) per range; logits of every head with scores
    assert L.pkv_decode_window_workspace_size(64, 32, 8, 128) > 0
    a = L.pkv_decode_accumulate_workspace_size(64, 32, 8, 128, 1000)
    assert a >= L.pkv_decode_window_workspace_size(64, 32, 8, 128) + 4 * 64 * 32 * 1000
    assert L.pkv_evict_workspace_size(64, 8, 500) >= 2 * 4 * 64 * 8 * 500
    for args in ((64, 32, 7, 128), (64, 32, 8, 96), (-1, 32, 8, 128), (1, 34, 2, 64), (1, 0, 1, 64)):
        assert L.pkv_decode_window_workspace_size(*args) == 0
        assert L.pkv_decode_accumulate_workspace_size(*args, 100) == 0
    assert L.pkv_decode_accumulate_workspace_size(1, 8, 8, 64, -1) == 0
    assert L.pkv_evict_workspace_size(1, 0, 5) == L.pkv_evict_workspace_size(1, 1, 0) == 0


def test_tensor_calls_refuse_host_caches():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.float16)
    q = torch.zeros(1, 2, 64, dtype=torch.float16)
    t = torch.zeros(1, 4, dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    ws = torch.zeros(8, dtype=torch.uint8)
    with pytest.raises(L.PkvError, match="CUDA device"):
        E.paged_attention_decode_window(q.clone(), q, k, k.clone(), t, n, 4, workspace=ws)
    sc = torch.zeros(1, 2, 64)
    with pytest.raises(L.PkvError, match="CUDA device"):
        E.evict_tokens(k, k.clone(), sc, sc.int(), t, n, n, n.clone(), 8, 2, workspace=ws)
    with pytest.raises(L.PkvError, match="head_dim"):
        E.paged_attention_decode_window(q, q[..., :32].contiguous(), k, k, t, n, 4, workspace=ws)
    with pytest.raises(L.PkvError, match="must be \\[S, H, D\\]"):
        E.paged_attention_decode_window(q, q[0], k, k, t, n, 4, workspace=ws)
