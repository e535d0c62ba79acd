"""The host side of the bounded-cache calls without a GPU: which stream their
memory belongs to, what a step keeps between calls, and what is refused."""
import contextlib
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import workloads as W
from oracle import bounded as B
from paged_kv_cache_162_gb300 import _lib as L
from paged_kv_cache_162_gb300 import engine as E
from paged_kv_cache_162_gb300.allocator import BlockAllocator
from tests.bounded_rows import Rows


# ---------------------------------------------------------------- streams
class FakeStream:
    """Stands for a torch stream; remembers which streams it has waited for."""

    def __init__(self, handle):
        self.cuda_stream = handle
        self.waited = []

    def wait_stream(self, other):
        self.waited.append(other.cuda_stream)


class Streams:
    """Torch's streams as far as these calls use them, on the CPU: the handle
    of the current one, and on which each tensor was made or copied."""

    def __init__(self, monkeypatch):
        self.now = FakeStream(0)
        self.made = []
        monkeypatch.setattr(torch.cuda, "stream", self.on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.now)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle))
        self.captured = ()                   # handles of streams that are being captured
        monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
        monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: None)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing",
                            lambda: self.now.cuda_stream in self.captured)
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
        for name in ("empty", "zeros", "full", "empty_like"):
            monkeypatch.setattr(torch, name, self.logged(name, getattr(torch, name)))
        for name in ("clone", "to", "copy_"):
            monkeypatch.setattr(torch.Tensor, name, self.logged(name, getattr(torch.Tensor, name)))

    def logged(self, name, real):
        def call(*args, **kw):
            self.made.append((name, self.now.cuda_stream))
            return real(*args, **kw)
        return call

    @contextlib.contextmanager
    def on(self, stream):
        before, self.now = self.now, stream or self.now
        try:
            yield
        finally:
            self.now = before


@pytest.mark.parametrize("given", [77, FakeStream(77)])
def test_a_call_s_workspace_comes_from_its_own_stream(monkeypatch, given):
    """Memory that the current stream has given back may still be in use
    there: it must not become the scratch of a call on another stream."""
    streams = Streams(monkeypatch)
    E._workspace("call", 1024, torch.device("cpu"), given)
    assert streams.made == [("empty", 77)]
    E._workspace("call", 1024, torch.device("cpu"))
    assert streams.made[1:] == [("empty", 0)]


# ------------------------------------------------------- DecodeStep on the CPU
def cpu_step(**kw):
    """A planned DecodeStep on the CPU: two requests of three sequences that share their prompt's blocks."""
    args = dict(seed=9, prompts=2, samples=3, prefix=160, tail_lo=1, tail_hi=60, H=2, D=64)
    w = W.shared_prefix(**{**args, **kw})
    w.initial_free = np.concatenate([np.arange(w.NB, w.NB + 60, dtype=np.int32), w.initial_free])
    w.NB += 60
    st = E.DecodeStep(dtype=w.dtype, S=w.S, H=w.H, D=w.D, bs=w.bs, NB=w.NB, MB=w.MB, scale=w.scale,
                      ctx_before=w.ctx_before, n_new=w.n_new, tables_pre=w.tables_pre, nblocks_pre=w.nblocks_pre,
                      initial_free=w.initial_free, blocks=w.blocks, k_blocks=w.k_blocks, v_blocks=w.v_blocks, q=w.q,
                      new_k=w.new_k, new_v=w.new_v, seq_idx=w.seq_idx, pos=w.pos, fill_bits=int(W.POISON[w.dtype]),
                      device="cpu")
    st.plan()
    for t in (st.k_cache, st.v_cache):       # as if every row had been written
        t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(1)))
    return st


class FakeKernels:
    """The calls that DecodeStep makes, by the 64-bit definitions on CPU tensors; what each was given."""

    def __init__(self, monkeypatch, streams=None):
        self.calls, self.streams = [], streams
        for name in ("paged_attention_decode_window", "paged_attention_decode_accumulate", "evict_tokens",
                     "copy_blocks"):
            monkeypatch.setattr(E, name, getattr(self, name))

    def note(self, name, stream):
        at = None if self.streams is None else self.streams.now.cuda_stream
        self.calls.append((name, at if stream is None else getattr(stream, "cuda_stream", stream)))

    def paged_attention_decode_window(self, out, *args):
        self.note("window", args[-1])
        return out

    def paged_attention_decode_accumulate(self, out, scores, q, k, v, bt, lens, scale, most, ws, stream=None):
        self.note("accumulate", stream)
        S, Hkv = scores.shape[:2]
        assert ws.numel() >= E.L.pkv_decode_accumulate_workspace_size(S, q.shape[1], Hkv, q.shape[2], most)
        assert int(lens.max()) <= most
        _, weights, _ = B.attend(*(x.double().numpy() for x in (q, k, v)), bt.numpy(), lens.numpy(), scale)
        scores.numpy()[:] = B.accumulate(scores.numpy(), weights, Hkv)
        return out

    def evict_tokens(self, k, v, scores, pos, bt, lens, seen, new, budget, recent, sinks=0, max_context_len=0,
                     stream=None):
        self.note("evict", stream)
        s, p = scores.numpy(), pos.numpy()
        new.numpy()[:] = B.evict(k.view(torch.int16).numpy(), v.view(torch.int16).numpy(), s, p, bt.numpy(),
                                 lens.numpy(), seen.numpy(), budget, recent, sinks)

    def copy_blocks(self, k, v, pairs, stream=None):
        self.note("copy", stream)
        for src, dst in pairs.tolist():
            k[dst], v[dst] = k[src].clone(), v[src].clone()


def test_a_step_s_calls_keep_to_the_stream_they_are_given(monkeypatch):
    """Scores zeroed, tables uploaded and temporary tensors made on another
    stream than the kernels' would race with them."""
    st = cpu_step()
    streams = Streams(monkeypatch)
    kernels = FakeKernels(monkeypatch, streams)
    side = FakeStream(5)
    for call, expect in ((lambda: st.decode_window(30, 4, stream=side), ["window"]),
                         (lambda: st.decode_accumulate(stream=side), ["accumulate"]),
                         (lambda: st.evict(96, 20, 4, stream=side), ["copy", "evict"])):
        streams.made.clear()
        kernels.calls.clear()
        main = streams.now
        main.waited.clear()
        side.waited.clear()
        call()
        assert kernels.calls == [(name, 5) for name in expect]
        assert streams.made and {at for _, at in streams.made} == {5}, streams.made
        assert side.waited == [0] and main.waited == [5]
        assert streams.now is main
    st.evict(80, 20, 4)                       # without one, all on the current stream and nothing to wait for
    assert kernels.calls[-1] == ("evict", 0) and side.waited == [0]


# ------------------------------------------------- what a step keeps between calls
def test_eviction_updates_the_step_s_tensors_in_place(monkeypatch):
    """A graph captured before holds the addresses of the tables and lengths."""
    st = cpu_step()
    FakeKernels(monkeypatch)
    tables, lens = st.block_tables, st.context_lens
    st.decode_accumulate()
    assert st.evict(96, 20, 4) > 0
    assert st.block_tables is tables and st.context_lens is lens
    assert np.array_equal(tables.numpy(), st.tables_host) and np.array_equal(lens.numpy(), st.context_lens_host)
    assert lens.max() == 96 and (tables.numpy()[:, 6:] == -1).all()


# --------------------------------------------------- what a wait that ran out leaves
def test_entries_that_nobody_wrote_name_no_pieces(tmp_path):
    """After a wait that ran out the join finds any contents in the workspace
    and must not look for pieces outside the call's."""
    csrc = os.path.join(os.path.dirname(E.__file__), "csrc")
    src, so = tmp_path / "place.cpp", tmp_path / "place.so"
    src.write_text('#include "bounded_place.h"\n'
                   'extern "C" int pieces(int x, int y, int r) { return pkv::pieces_of(x, y, r); }\n')
    subprocess.run(["g++", "-shared", "-fPIC", "-I", csrc, str(src), "-o", str(so)], check=True)
    pieces = ctypes.CDLL(str(so)).pieces
    for ranges in (1, 304, 1536):
        for x in range(0, ranges, 7):
            assert [pieces(x, y, ranges) for y in (x, ranges - 1)] == [1, ranges - x]
        top, low = 2 ** 31 - 1, -2 ** 31
        for x, y in ((-1, -1), (low, top), (top, low), (low, low), (top, top), (0, ranges), (0, top), (1, 0), (-1, 0),
                     (low, 0), (0x7f7f7f7f, 0x7f7f7f7f), (ranges, ranges), (0, -1)):
            assert pieces(x, y, ranges) == 0, (x, y, ranges)
    # the kernel asks it wherever it reads an entry
    with open(os.path.join(csrc, "bounded.cu")) as f:
        kernel = f.read()
    assert kernel.count("= p.place[") == kernel.count("pkv::pieces_of(") == 3


# ------------------------------------------------------------------ refusals
def evict_args(**kw):
    a = dict(k_cache=256, v_cache=256, scores=256, positions=256, block_tables=256, context_lens=1024,
             token_counts=2048, scores_out=256, positions_out=256, new_context_lens=4096, S=5, Hkv=4, D=128, bs=16,
             NB=8, MB=4, max_context_len=0, score_stride=64, budget=32, recent_tokens=8, sink_tokens=4,
             dtype=L.PKV_BF16, workspace=256, workspace_bytes=1 << 40, stream=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("new", [1024, 2048, 1024 + 16, 2048 + 16, 1024 - 16, 2048 - 16, 2048 + 4])
def test_evict_refuses_lengths_written_over_what_it_reads(new):
    """Heads and CTAs of a row read its length and its token count while one of them writes the new length."""
    with pytest.raises(L.PkvError, match="must not overlap") as e:
        L.pkv_evict_tokens(**evict_args(new_context_lens=new))
    assert e.value.status == L.PKV_ERR_INVALID_ARG


@pytest.mark.parametrize("new", [1024 + 20, 2048 - 20, 2048 + 20])
def test_evict_takes_lengths_next_to_what_it_reads(new):
    with pytest.raises(L.PkvError, match="workspace too small"):  # the next check
        L.pkv_evict_tokens(**evict_args(new_context_lens=new, workspace_bytes=10))


# ------------------------------------------------------------- beam search
class FakeEvent:
    def record(self, stream=None):
        pass

    def synchronize(self):
        pass


def on_cpu(st, monkeypatch):
    """Lets beam_step run on the CPU: its buffers, and the native step by the allocator's own calls."""
    S, MB, H, D, bs = st.S, st.MB, st.H, st.D, st.bs

    class Native:
        def step(self, parents, q, key, value, stream):
            parents = np.ctypeslib.as_array((ctypes.c_int32 * S).from_address(parents)).copy()
            pos = st.beam_ctx[parents]
            st.allocator.fork(st.tables_host, st.nblocks_host, parents)
            pairs = st.allocator.append_batch(st.tables_host, st.nblocks_host, pos, np.ones(S, np.int32), bs)
            k, v = (t.view(torch.int16).numpy() for t in (st.k_cache, st.v_cache))
            for a, b in pairs:
                k[b], v[b] = k[a], v[a]
            tok = st._beam_dev_u16.numpy().reshape(3, S, H, D)
            for s in range(S):
                block = st.tables_host[s, pos[s] // bs]
                k[block, pos[s] % bs], v[block, pos[s] % bs] = tok[1, s], tok[2, s]
            st.beam_ctx[:] = pos + 1
            st._beam_views[0].numpy()[:], st._beam_views[1].numpy()[:] = st.tables_host, st.beam_ctx
            return 0, 0

        def close(self):
            pass

    def buffers():
        st._beam_slots = [dict(stg_np=np.zeros(64, np.uint8), u16=torch.empty(3 * S * H * D, dtype=torch.int16),
                               done=FakeEvent(), used=False) for _ in range(2)]
        st._beam_dev_u16 = torch.empty(3 * S * H * D, dtype=torch.int16)
        st._beam_turn, st._beam_inputs_bytes, st._beam_stg_base = 0, 64, [0, 1 << 40]
        st._beam_views = (torch.empty(S, MB, dtype=torch.int32), torch.empty(S, dtype=torch.int32),
                          torch.empty(S, dtype=torch.int32), torch.empty(S, dtype=torch.int32))
        groups = getattr(st, "beam_groups", None)
        st._beam_G = 0 if groups is None else len(groups)
        st.max_context_len = MB * bs
        st._beam_native = Native()

    monkeypatch.setattr(st, "_beam_buffers", buffers)
    return st


def beam_tokens(st, rng):
    """q, K and V of a step's new tokens: bit patterns, and their values."""
    b = W.normal_bits(np.random.Generator(np.random.SFC64(int(rng.integers(1 << 30)))), (3, st.S, st.H, st.D), W.F16)
    return b, b.view(np.float16).astype(np.float64)


def step_rows(st):
    return Rows(st.k_cache.double().numpy(), st.v_cache.double().numpy(), st.tables_host, st.context_lens_host,
                st.scale)


def test_a_beam_search_goes_on_from_the_evicted_lengths(monkeypatch):
    """The native search has lengths of its own: a token appended past them
    would leave rows that nobody wrote inside the context."""
    rng = np.random.default_rng(3)
    Streams(monkeypatch)
    FakeKernels(monkeypatch)
    st = on_cpu(cpu_step(H=1), monkeypatch)
    for t in (st.k_cache, st.v_cache):
        t.view(-1, 1, st.D)[:] = 0.25                   # whatever a row holds that nobody writes
    step = lambda: st.beam_step(np.arange(st.S), *(beam_tokens(st, rng)[0][i] for i in (1, 2, 0)))  # noqa: E731
    step()
    st.decode_accumulate()
    st.evict(160, 20, 4)
    assert (st.context_lens_host == 160).all() and (st.beam_ctx == 160).all()
    tables = st.tables_host.copy()
    step()
    assert (st.context_lens.numpy() == 161).all() and (st.context_lens_host == 161).all()
    assert (st.nblocks_host == 11).all() and np.array_equal(st.tables_host[:, :10], tables[:, :10])
    assert (st.tables_host[:, 10] >= 0).all()


@pytest.mark.parametrize("start", [0, 2])
def test_scores_positions_and_ages_follow_a_beam_search(monkeypatch, start):
    """Three cycles of beam steps, accumulated weights and eviction, token by
    token: every beam has its parent's rows, and new tokens their true ages."""
    rng = np.random.default_rng(start)
    Streams(monkeypatch)
    FakeKernels(monkeypatch)
    st = on_cpu(cpu_step(), monkeypatch)
    rows, S = step_rows(st), st.S

    def step():
        parents = rng.integers(0, S, S)
        b, x = beam_tokens(st, rng)
        st.beam_step(parents, b[1], b[2], b[0])
        rows.beam_step(parents, x[1], x[2])
        return x[0]
    for _ in range(start):                   # a search that had begun before the first scores
        step()
    q = st.q.double().numpy()
    st.decode_accumulate()
    rows.attend(q, add=True)
    rows.check_state(st, 1e-6)
    for cycle in range(3):
        rows.take_scores(st)
        st.evict(100, 30, 4)
        rows.evict(100, 30, 4)
        rows.check_state(st, 0)
        for _ in range(12 + 5 * cycle):
            q = step()
            st.decode_accumulate()
            rows.attend(q, add=True)
        rows.check_state(st, 1e-4)


def test_prefix_groups_end_with_an_eviction(monkeypatch):
    """Evicted sequences own their blocks and hold other tokens per head: no group reads them through its first member."""
    FakeKernels(monkeypatch)
    seen = []
    monkeypatch.setattr(E, "paged_attention_decode_shared_prefix", lambda *a, **kw: seen.append(a[6].tolist()))
    st = cpu_step()
    groups = [[0, 3, 160], [3, 3, 160]]
    st.prefix_groups, st.beam_groups = torch.tensor(groups, dtype=torch.int32), groups
    st.decode_accumulate()
    st.decode_shared_prefix(groups)
    lens = st.context_lens_host.copy()
    assert st.evict(int(lens.max()), 20, 4) == 0       # nothing over the budget: all as before
    assert st.prefix_groups is not None and st.beam_groups is groups
    st.decode_shared_prefix(groups)
    assert seen == [groups, groups]
    budget = int(lens[:3].max())                       # sequences of the second request alone
    assert (lens[3:] > budget).any() or (lens[:3] > (budget := int(lens[3:].max()))).any()
    st.evict(budget, 20, 4)
    assert st.prefix_groups is None and st.beam_groups is None
    whole = 0 if (lens[:3] <= budget).all() else 1     # the request that kept its blocks
    st.decode_shared_prefix(groups[whole:whole + 1])
    with pytest.raises(L.PkvError, match="no longer share"):
        st.decode_shared_prefix(groups[1 - whole:2 - whole])
    st.decode_shared_prefix(np.empty((0, 3)))
    st.evict(96, 20, 4)
    for i in (0, 1):
        with pytest.raises(L.PkvError, match="no longer share"):
            st.decode_shared_prefix(groups[i:i + 1])
    st.plan()
    st.decode_shared_prefix(groups)
    assert seen[2:] == [groups[whole:whole + 1], [], groups]


def test_a_beam_search_with_groups_is_not_evicted(monkeypatch):
    rng = np.random.default_rng(5)
    Streams(monkeypatch)
    FakeKernels(monkeypatch)
    st = on_cpu(cpu_step(), monkeypatch)
    st.beam_groups = [[0, 3, 160], [3, 3, 160]]
    b, _ = beam_tokens(st, rng)
    st.beam_step(np.arange(st.S), b[1], b[2], b[0])
    st.decode_accumulate()
    tables, lens, free = st.tables_host.copy(), st.context_lens_host.copy(), st.allocator.num_free
    with pytest.raises(L.PkvError, match="prefix groups"):
        st.evict(96, 20, 4)
    assert np.array_equal(st.tables_host, tables) and np.array_equal(st.context_lens_host, lens)
    assert st.allocator.num_free == free


def test_weights_go_on_when_a_beam_search_raises_the_bound(monkeypatch):
    """beam_step allows contexts up to the table's end: a workspace for less is refused."""
    rng = np.random.default_rng(6)
    Streams(monkeypatch)
    FakeKernels(monkeypatch)                 # its accumulate checks the workspace
    st = on_cpu(cpu_step(tail_lo=33, tail_hi=33, bs=32, D=128), monkeypatch)
    st.decode_accumulate()
    ws = st._accumulate_ws
    st.decode_accumulate()
    assert st._accumulate_ws is ws and st.MB * st.bs > st.max_context_len + 16
    b, _ = beam_tokens(st, rng)
    st.beam_step(np.arange(st.S), b[1], b[2], b[0])
    st.decode_accumulate()
    ws = st._accumulate_ws
    st.decode_accumulate()
    assert st._accumulate_ws is ws


def test_a_step_refuses_an_eviction_before_anything_moves(monkeypatch):
    """Without scores, or with arguments that evict_tokens refuses, no block has been copied or freed."""
    kernels = FakeKernels(monkeypatch)
    st = cpu_step()
    tables, free = st.tables_host.copy(), st.allocator.num_free

    def refused(match, *args):
        with pytest.raises(L.PkvError, match=match) as e:
            st.evict(*args)
        assert e.value.status == L.PKV_ERR_INVALID_ARG
        assert np.array_equal(st.tables_host, tables) and st.allocator.num_free == free
    refused("no scores", 96, 20, 4)
    st.decode_accumulate()
    for args in ((0, 0, 0), (-3, 0, 0), (96, -1, 0), (96, 20, -1), (96, 93, 4)):
        refused("budget must be", *args)
    assert kernels.calls == [("accumulate", None)]
    st.evict(96, 92, 4)


def test_a_new_plan_starts_over(monkeypatch):
    """plan() makes the tables from before the step: no lengths, scores, positions or ages of an eviction outlive it."""
    FakeKernels(monkeypatch)
    st = cpu_step()
    lens, tables = st.context_lens_host.copy(), st.tables_host.copy()
    k, v = st.k_cache.clone(), st.v_cache.clone()
    st.decode_accumulate()
    first = st.scores.clone()
    st.plan()                                # no eviction yet
    assert np.array_equal(st.context_lens.numpy(), lens)
    st.decode_accumulate()
    assert torch.equal(st.scores, first)
    held = st.context_lens
    st.evict(96, 20, 4)
    st.plan()
    st.k_cache.copy_(k), st.v_cache.copy_(v)
    assert st.context_lens is held and np.array_equal(held.numpy(), lens)
    assert np.array_equal(st.context_lens_host, lens) and np.array_equal(st.tables_host, tables)
    with pytest.raises(L.PkvError, match="no scores"):
        st.evict(96, 20, 4)
    st.decode_accumulate()
    assert torch.equal(st.scores, first) and np.array_equal(st.token_counts.numpy(), lens)
    assert (st.positions == -1).all()
    st.evict(96, 20, 4)
    assert (st.context_lens_host == 96).all()


def test_a_step_is_not_written_again_after_an_eviction(monkeypatch):
    """Its copy pairs and slots name blocks that have gone back to the pool."""
    kernels = FakeKernels(monkeypatch)
    monkeypatch.setattr(E, "compute_slot_mapping", lambda *a: kernels.calls.append(("slots", None)))
    monkeypatch.setattr(E, "reshape_and_cache", lambda *a: kernels.calls.append(("write", None)))
    monkeypatch.setattr(E.DecodeStep, "decode", lambda st, stream=None: kernels.calls.append(("decode", None)))
    monkeypatch.setattr(E.L, "pkv_decode_step", lambda *a: kernels.calls.append(("step", None)))
    st = cpu_step()
    st.run()
    st.decode_accumulate()
    st.run()
    st.evict(96, 20, 4)
    done = len(kernels.calls)
    for kw in ({}, dict(fused=True), dict(attention=False)):
        with pytest.raises(L.PkvError, match="plan\\(\\) starts over"):
            st.run(**kw)
    assert len(kernels.calls) == done
    st.run(write=False)
    st.run(write=False, fused=True)
    assert kernels.calls[done:] == [("decode", None)] * 2
    st.plan()
    st.run()


@pytest.mark.parametrize("captured,given", [(0, None), (5, 5), (0, 5)])
def test_what_a_graph_would_repeat_is_not_captured(monkeypatch, captured, given):
    """A captured first decode_accumulate would zero the scores on every replay; evict decides on the host."""
    streams = Streams(monkeypatch)
    kernels = FakeKernels(monkeypatch)
    side = None if given is None else FakeStream(given)
    st = cpu_step()
    free, tables = st.allocator.num_free, st.tables_host.copy()
    streams.captured = (captured,)
    with pytest.raises(L.PkvError, match="cannot be captured"):
        st.decode_accumulate(stream=side)
    assert st.scores is None
    streams.captured = ()
    st.decode_accumulate(stream=side)
    streams.captured = (captured,)
    st.decode_accumulate(stream=side)        # this may be
    waited = len(streams.now.waited), 0 if side is None else len(side.waited)
    with pytest.raises(L.PkvError, match="cannot be captured"):
        st.evict(96, 20, 4, stream=side)
    assert np.array_equal(st.tables_host, tables) and st.allocator.num_free == free
    assert (len(streams.now.waited), 0 if side is None else len(side.waited)) == waited
    assert [name for name, _ in kernels.calls] == ["accumulate"] * 2


# ------------------------------------------------------- numbers past 32 bits
FAR = [2 ** 32 + 8, 2 ** 31, -2 ** 31 - 1, 2 ** 40]


def window_args(**kw):
    a = dict(out=16, q=16, k_cache=16, v_cache=16, block_tables=16, context_lens=16, S=2, H=8, Hkv=4, D=128, bs=16,
             NB=8, MB=4, max_context_len=0, window=8, sink_tokens=2, scale=0.1, dtype=L.PKV_F16, workspace=256,
             workspace_bytes=10, stream=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("far", FAR)
def test_numbers_past_32_bits_are_refused_not_cut(far):
    """2**32 + 8 is no window of 8."""
    def refused(call, *args, **kw):
        with pytest.raises(L.PkvError, match="does not fit 32 bits") as e:
            call(*args, **kw)
        assert e.value.status == L.PKV_ERR_INVALID_ARG
    for name in ("window", "sink_tokens", "max_context_len"):
        refused(L.pkv_paged_attention_decode_window, **window_args(**{name: far}))
    a = window_args(scores=16, score_stride=64, max_context_len=far)
    del a["window"], a["sink_tokens"]
    refused(L.pkv_paged_attention_decode_accumulate, **a)
    for name in ("budget", "recent_tokens", "sink_tokens", "max_context_len"):
        refused(L.pkv_evict_tokens, **evict_args(**{name: far}))
    assert L.pkv_decode_window_workspace_size(far, 8, 8, 64) == 0
    assert L.pkv_decode_accumulate_workspace_size(1, 8, 8, 64, far) == 0
    assert L.pkv_evict_workspace_size(1, 8, far) == 0
    # the tensor calls (their own checks come first on the CPU: what they pass on is checked next)
    k, q = torch.zeros(4, 16, 2, 64, dtype=torch.float16), torch.zeros(1, 2, 64, dtype=torch.float16)
    t, n, sc = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, 64)
    huge = torch.zeros(1, 1, dtype=torch.int32).expand(1, 2 ** 31)
    for name, tables in (("window", t), ("sink_tokens", t), ("max_context_len", t), (None, huge)):
        kw = dict(window=4, **({} if name in (None, "window") else {name: far}))
        kw.update({name: far} if name == "window" else {})
        with pytest.MonkeyPatch.context() as m:
            m.setattr(E, "_need", lambda *a: None)
            refused(E.paged_attention_decode_window, q.clone(), q, k, k, tables, n, **kw)
            if name in (None, "max_context_len"):
                kw.pop("window")
                refused(E.paged_attention_decode_accumulate, q.clone(), sc, q, k, k, tables, n, **kw)
    for name in ("budget", "recent_tokens", "sink_tokens", "max_context_len"):
        kw = {**dict(budget=8, recent_tokens=2), name: far}
        refused(E.evict_tokens, k, k, sc, sc.int(), t, n, n, n.clone(), **kw)
    refused(E.evict_tokens, k, k, sc, sc.int(), huge, n, n, n.clone(), 8, 2)


@pytest.mark.parametrize("far", FAR)
def test_the_allocator_does_not_cut_numbers(far):
    a = BlockAllocator(8)
    row = np.array(a.alloc(4), np.int32)
    before = row.copy()
    calls = [lambda: a.truncate(row, 4, far, 16), lambda: a.truncate(row, 4, 16, far)]
    calls += [lambda kw=kw: a.release_window(row, **{**dict(num_blocks=4, context_len=64, window=8, sink_tokens=0,
                                                            block_size=16), **kw})
              for kw in ({"context_len": far}, {"window": far}, {"sink_tokens": far}, {"block_size": far})]
    for call in calls:
        with pytest.raises(L.PkvError, match="does not fit 32 bits"):
            call()
    assert np.array_equal(row, before) and a.num_free == 4
    assert a.truncate(row, np.int64(4), np.int64(33), np.int32(16)) == (3, 1)   # numpy's integers are taken


def test_no_workspace_for_a_context_of_zero():
    """A call takes 0 as MB * bs: a workspace made for 0 would be too small for it."""
    assert L.pkv_decode_accumulate_workspace_size(2, 8, 4, 128, 0) == 0
    assert L.pkv_decode_accumulate_workspace_size(2, 8, 4, 128, 1) > 0
    for n in (0, -1):
        with pytest.raises(L.PkvError, match="MB \\* bs") as e:
            E.new_accumulate_workspace(2, 8, 4, 128, n, device="cpu")
        assert e.value.status == L.PKV_ERR_INVALID_ARG


# ------------------------------------------------------------------ the build
def a_build(tmp_path, monkeypatch, bad=()):
    """The build with its files under tmp_path and its commands recorded, not run; those that name something in
    `bad` fail."""
    from paged_kv_cache_162_gb300 import _build
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        fails = any(b in " ".join(cmd) for b in bad)
        if not fails:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("built")
        return subprocess.CompletedProcess(cmd, int(fails), "", "no such header" if fails else "")
    for name in ("BUILD", "LIB", "BIND", "FLAGS", "BIND_FLAGS"):
        monkeypatch.setattr(_build, name, str(tmp_path / name.lower()), raising=False)
    monkeypatch.setattr(_build.subprocess, "run", run)
    return _build, ran


def test_the_library_is_built_where_the_binding_is_not(tmp_path, monkeypatch, capfd):
    """A C user has nvcc and no torch, or a torch that the binding does not compile against."""
    build, ran = a_build(tmp_path, monkeypatch, bad=["tensor_bind.cpp"])
    (tmp_path / "bind").write_text("of another build")
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.BIND)              # no stale one either
    assert "no such header" in capfd.readouterr().err and not build.up_to_date()
    monkeypatch.setattr(build, "_torch_version", lambda: "")
    assert build.up_to_date()                          # without a torch nothing is missing
    os.remove(build.LIB)
    ran.clear()
    build.build()
    assert os.path.exists(build.LIB) and not any("tensor_bind" in " ".join(c) for c in ran)


def test_the_binding_is_built_again_for_another_torch(tmp_path, monkeypatch):
    build, ran = a_build(tmp_path, monkeypatch)
    build.build()
    assert build.up_to_date() and os.path.exists(build.BIND)
    ran.clear()
    monkeypatch.setattr(build, "_torch_version", lambda: "9.9")
    assert not build.up_to_date()
    build.build()
    assert build.up_to_date() and len(ran) == 2 and not any(".cu" in " ".join(c[:-1]) for c in ran)


def test_a_binding_of_another_torch_is_not_used(monkeypatch):
    monkeypatch.setattr(E, "_bind", None)
    native = E._native()
    assert native.torch_version == torch.__version__   # this tree's is for this torch
    monkeypatch.setattr(E, "_bind", None)
    monkeypatch.setattr(torch, "__version__", "1.0")
    assert E._native().window(1, 2, 3) == E._native().evict() == -1


@pytest.mark.parametrize("most,status", [(2 ** 31 - 1, L.PKV_ERR_INVALID_ARG), (2 ** 31 - 1024, L.PKV_ERR_INVALID_ARG),
                                         (2 ** 31 - 65, L.PKV_ERR_INVALID_ARG), (2 ** 31 - 1025, L.PKV_ERR_WORKSPACE)])
def test_contexts_whose_token_numbers_would_pass_31_bits(most, status):
    """The fold of the weights counts its tokens in stretches of up to 512: the last one must not wrap."""
    a = window_args(MB=1 << 26, bs=64, max_context_len=most)
    with pytest.raises(L.PkvError) as e:
        L.pkv_paged_attention_decode_window(**a)
    assert e.value.status == status
    del a["window"], a["sink_tokens"]
    with pytest.raises(L.PkvError) as e:
        L.pkv_paged_attention_decode_accumulate(**a, scores=16, score_stride=1 << 32)
    assert e.value.status == status
    size = L.pkv_decode_accumulate_workspace_size(1, 2, 1, 64, most)
    assert (size == 0) == (status == L.PKV_ERR_INVALID_ARG)


def test_a_step_without_a_plan_has_no_tables(monkeypatch):
    kernels = FakeKernels(monkeypatch)
    st = cpu_step()
    st.block_tables = None                   # as __init__ leaves it
    for call in (lambda: st.decode_window(8), st.decode_accumulate, lambda: st.evict(8, 2)):
        with pytest.raises(L.PkvError) as e:
            call()
        assert e.value.status == L.PKV_ERR_INVALID_ARG
    assert not kernels.calls and st.scores is None


def test_a_captured_call_s_memory_stays(monkeypatch):
    """A captured decode_accumulate holds the addresses of the scores and of
    its workspace: neither a raised bound nor a new plan may free them."""
    rng = np.random.default_rng(6)
    Streams(monkeypatch)
    FakeKernels(monkeypatch)
    st = on_cpu(cpu_step(tail_lo=33, tail_hi=33, bs=32, D=128), monkeypatch)
    st.decode_accumulate()
    held = [x.data_ptr() for x in (st.scores, st.positions, st.token_counts, st._accumulate_ws)]
    first = st.scores.clone()
    b, _ = beam_tokens(st, rng)
    st.beam_step(rng.integers(0, st.S, st.S), b[1], b[2], b[0])
    st.decode_accumulate()
    st.evict(96, 20, 4)
    k, v = st.k_cache, st.v_cache
    st.plan()
    st.decode_accumulate()
    assert held == [x.data_ptr() for x in (st.scores, st.positions, st.token_counts, st._accumulate_ws)]
    assert (st.positions == -1).all() and torch.equal(st.token_counts, st.context_lens)
    assert (st.scores[:, :, 193:] == 0).all() and torch.allclose(st.scores.sum(-1), first.sum(-1), atol=1e-4)
    assert k is st.k_cache and v is st.v_cache


def test_a_binding_that_names_no_torch_is_not_used(monkeypatch):
    import paged_kv_cache_162_gb300 as P
    monkeypatch.setattr(E, "_bind", None)
    monkeypatch.setitem(__import__("sys").modules, "paged_kv_cache_162_gb300._tensor_bind", object())
    monkeypatch.setattr(P, "_tensor_bind", object(), raising=False)
    assert E._native().window() == -1


def test_a_captured_step_is_not_replayed_after_an_eviction(monkeypatch):
    """The graph holds the step's block copies and writes, like run()."""
    FakeKernels(monkeypatch)
    launched = []
    graph = E.StepGraph.__new__(E.StepGraph)             # capturing needs a GPU
    graph.step, graph._exec, graph._stream = cpu_step(), None, None
    graph._launch = lambda *a: launched.append(a) or 0
    graph.replay()
    graph.step.decode_accumulate()
    graph.replay()
    graph.step.evict(96, 20, 4)
    with pytest.raises(L.PkvError, match="capture it anew"):
        graph.replay()
    assert len(launched) == 2


def test_the_other_calls_scratch_is_their_stream_s_too(monkeypatch):
    """Decode, the fused step and the shared-prefix decode without a workspace, and DecodeStep's groups."""
    st = cpu_step()
    streams = Streams(monkeypatch)
    launched = []
    for name in ("pkv_paged_attention_decode", "pkv_decode_step", "pkv_paged_attention_decode_shared_prefix"):
        monkeypatch.setattr(E.L, name, lambda *a, name=name: launched.append((name, a[-1])))
    side = FakeStream(5)
    a = (st.out, st.q, st.k_cache, st.v_cache, st.block_tables, st.context_lens)
    g = torch.tensor([[0, 3, 160]], dtype=torch.int32)
    E.paged_attention_decode(*a, stream=side)
    E.decode_step(*a[:2], st.new_k, st.new_v, *a[2:], st.seq_idx, st.pos, st.slot_mapping, stream=side)
    E.decode_step(*a[:2], st.new_k, st.new_v, *a[2:], st.seq_idx, st.pos, st.slot_mapping, g, stream=side)
    E.paged_attention_decode_shared_prefix(*a, g, stream=side)
    assert streams.made == [("empty", 5)] * 4 and [s for _, s in launched] == [side] * 4
    streams.made.clear()
    st.decode_shared_prefix([[0, 3, 160]], stream=side)
    assert streams.made == [("to", 5), ("empty", 5)] and side.waited == [0] and streams.now.waited == [5]
    streams.made.clear()
    E.paged_attention_decode(*a)
    assert streams.made == [("empty", 0)]


def test_scratch_is_where_the_caches_are(monkeypatch):
    """Queries may be in pinned host memory; the kernels' scratch may not."""
    st = cpu_step()
    made = []
    monkeypatch.setattr(E, "_scratch", lambda n, device, stream=None: made.append(device) or torch.empty(1))
    for name in ("pkv_paged_attention_decode", "pkv_decode_step", "pkv_paged_attention_decode_shared_prefix"):
        monkeypatch.setattr(E.L, name, lambda *a: None)
    k = st.k_cache.to("meta")                # stands for another device than the queries'
    a = (st.out, st.q, k, k, st.block_tables, st.context_lens)
    g = torch.tensor([[0, 3, 160]], dtype=torch.int32)
    E.paged_attention_decode(*a)
    E.decode_step(*a[:2], st.new_k, st.new_v, *a[2:], st.seq_idx, st.pos, st.slot_mapping)
    E.paged_attention_decode_shared_prefix(*a, g)
    assert made == [torch.device("meta")] * 3
