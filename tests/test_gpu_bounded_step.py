"""Bounded-cache calls on streams of their own, and DecodeStep's over more
than one cycle, against the 64-bit definitions."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import bounded as B
from paged_kv_cache_162_gb300 import _lib as L
from paged_kv_cache_162_gb300 import engine as E
from tests.bounded_rows import Rows
from tests.gpu_harness import assert_attention_close, device_step
from tests.test_gpu_bounded import check_out, dev, f64, make, weight_error

pytestmark = pytest.mark.gpu


def keep_busy(rounds=40):
    """Work of some milliseconds on the current stream."""
    a = torch.randn(4096, 4096, device="cuda")
    for _ in range(rounds):
        a = a @ a * 1e-2
    return a


def test_scratch_is_not_shared_with_another_stream():
    """A call that makes its own scratch on the current stream gives the
    memory back while its kernels wait; a call with stream= right after it
    must not get the same memory."""
    c = [make(31 + i, 6, 8, 4, 128, 16, "f16", [1500, 700, 2000, 1, 0, 999]) for i in range(2)]
    side = torch.cuda.Stream()
    refs = [B.attend(f64(x["q"]), f64(x["k"]), f64(x["v"]), x["tables"], x["lens"], x["scale"]) for x in c]
    for _ in range(4):
        d = [dev(x) for x in c]
        scores = [torch.zeros(6, 4, c[0]["MB"] * 16, device="cuda") for _ in c]
        torch.cuda.synchronize()
        keep_busy()
        for x, y, z, stream in zip(c, d, scores, (None, side)):
            E.paged_attention_decode_accumulate(y["out"], z, y["q"], y["k"], y["v"], y["tables"], y["lens"],
                                                x["scale"], stream=stream)
        torch.cuda.synchronize()
        for x, y, z, (ref, weights, mag) in zip(c, d, scores, refs):
            w = weight_error(x)
            check_out(x, y["out"], ref, mag, w)
            want = B.accumulate(np.zeros(z.shape), weights, 4)
            # two query heads per KV head, from zero: (w + 2 e) of what was added, once rounded
            assert np.all(np.abs(f64(z.cpu()) - want) <= (w + 3 * 2.0 ** -24) * want + 2.0 ** -126)
    assert L.pkv_get_device_errors() == 0


def shared_step(**kw):
    """A step of two requests of three sequences that share their prompt's
    blocks, planned and run, with room in the pool to copy them."""
    args = dict(seed=9, prompts=2, samples=3, prefix=160, tail_lo=1, tail_hi=60, H=4, D=64)
    w = W.shared_prefix(**{**args, **kw})
    w.initial_free = np.concatenate([np.arange(w.NB, w.NB + 80, dtype=np.int32), w.initial_free])
    w.NB += 80
    st = device_step(w)
    st.plan()
    st.run()
    return st


def bits(st):
    torch.cuda.synchronize()
    return [x.view(torch.int16 if x.element_size() == 2 else torch.int32).cpu()
            for x in (st.out, st.k_cache, st.v_cache, st.scores, st.positions, st.block_tables, st.context_lens,
                      st.token_counts)]


def test_step_on_another_stream():
    """Both streams busy before every call, and no synchronisation but the
    calls' own: the results are those of one stream."""
    def cycle(stream):
        st = shared_step()
        torch.cuda.synchronize()
        for _ in range(2):
            if stream is not None:
                with torch.cuda.stream(stream):
                    keep_busy()
            keep_busy()
            st.decode_accumulate(stream=stream)
        freed = st.evict(96, 20, 4, stream=stream)
        junk = [torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
        st.decode()
        after = st.out.clone()
        st.decode_window(30, 4, stream=stream)
        got = bits(st) + [after.view(torch.int16).cpu()]
        del junk
        return freed, got
    freed, want = cycle(None)
    assert freed > 0
    for _ in range(3):
        got_freed, got = cycle(torch.cuda.Stream())
        assert got_freed == freed and all(torch.equal(a, b) for a, b in zip(got, want))
    assert L.pkv_get_device_errors() == 0


def test_captured_decode_follows_an_eviction():
    """A graph captured before evict() decodes what is left after it."""
    st = shared_step()
    st.decode_accumulate()
    st.decode_window(60, 4)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        st.decode_window(60, 4)
    torch.cuda.synchronize()
    st.evict(96, 20, 4)
    junk = [torch.full((1 << 12,), 77, dtype=torch.int32, device="cuda") for _ in range(64)]
    st.decode_window(60, 4)
    want = st.out.clone()
    st.out.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(st.out.view(torch.int16), want.view(torch.int16))
    assert L.pkv_get_device_errors() == 0
    del junk


@pytest.mark.parametrize("dtype,D,streamed", [("f16", 64, False), ("f16", 64, True), ("bf16", 128, False)])
def test_cycles_of_beam_search_and_eviction(dtype, D, streamed):
    """Beam steps, accumulated weights and evictions in turn, token by token:
    caches, positions and lengths exact, attention within the library's bar,
    scores within 1e-4 (24 steps of weights of at most 1, each within 2e-6)."""
    rng = np.random.default_rng(D + streamed)
    st = shared_step(dtype=dtype, D=D)
    S, H = st.S, st.H
    stream = torch.cuda.Stream() if streamed else None
    if streamed:
        torch.cuda.synchronize()
    rows = Rows(st.k_cache.double().cpu().numpy(), st.v_cache.double().cpu().numpy(), st.tables_host,
                st.context_lens_host, st.scale)

    def attended(q):
        torch.cuda.synchronize()
        assert_attention_close(st.out.double().cpu().numpy(), rows.attend(q, add=True), "accumulate")

    q = st.q.double().cpu().numpy()
    st.decode_accumulate(stream=stream)
    attended(q)
    for cycle in range(3):
        rows.take_scores(st)
        st.evict(100, 30, 4, stream=stream)
        rows.evict(100, 30, 4)
        torch.cuda.synchronize()
        rows.check_state(st, 0)
        for _ in range(8 + 5 * cycle):
            parents = rng.integers(0, S, S)
            tok = [torch.from_numpy(rng.standard_normal((S, H, D))).to(st.dtype) for _ in range(3)]
            bits16 = [t.view(torch.int16).numpy().view(np.uint16) for t in tok]
            q, k, v = (t.double().numpy() for t in tok)
            st.beam_step(parents, bits16[1], bits16[2], bits16[0], stream=stream)
            rows.beam_step(parents, k, v)
            torch.cuda.synchronize()
            assert_attention_close(st.out.double().cpu().numpy(), rows.attend(q), "beam step")
            st.decode_accumulate(stream=stream)
            attended(q)
        rows.check_state(st, 1e-4)
    assert L.pkv_get_device_errors() == 0


def test_captured_weights_add_up():
    """decode_accumulate captured after a first call: every replay adds the
    same weights; a first call or an eviction inside a capture is refused."""
    st, side = shared_step(), torch.cuda.Stream()
    with pytest.raises(L.PkvError, match="cannot be captured"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
            st.decode_accumulate()
    assert st.scores is None
    st.decode_accumulate()
    torch.cuda.synchronize()
    once = st.scores.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        st.decode_accumulate()
        with pytest.raises(L.PkvError, match="cannot be captured"):
            st.evict(96, 20, 4)
    for k in (2, 3):
        graph.replay()
        torch.cuda.synchronize()
        # k sums of one weight, each rounded to fp32
        assert torch.allclose(st.scores, k * once, rtol=3 * 2.0 ** -24, atol=0)
    assert L.pkv_get_device_errors() == 0


@pytest.mark.parametrize("D,H,Hkv,n", [(64, 2, 2, 700), (128, 12, 1, 5000), (64, 3, 1, 40000), (128, 20, 4, 20000),
                                       (64, 4, 4, 60000)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_many_small_weights_are_not_lost(dtype, D, H, Hkv, n):
    """One token of logit 0 and V = 0, the others of logit -18 and V = 1000:
    the output is made of weights of 1.5e-8, below half the smallest fp16
    number.  check_out's bound without its term for those: a weight is the
    sum of two 16-bit numbers in units of 2^-15, 2^-40 absolute at most."""
    c = make(n, 1, H, Hkv, D, 16, dtype, [n])
    top = int(B.rows_of(c["tables"][0], [n // 3], 16)[0])
    for name, rest, one in (("k", -18.0, 0.0), ("v", 1000.0, 0.0)):
        c[name][:] = 0
        rows = c[name].view(-1, Hkv, D)
        rows[:, :, slice(0, 1) if name == "k" else slice(None)] = rest
        rows[top] = one
    c["q"][:] = 0
    c["q"][:, :, 0] = 8.0
    c["scale"] = 0.125
    d = dev(c)
    scores = torch.zeros(1, Hkv, c["MB"] * 16, device="cuda")
    ref, weights, mag = B.attend(f64(c["q"]), f64(c["k"]), f64(c["v"]), c["tables"], c["lens"], c["scale"])
    assert ref.min() > 0.9 * n * 1.5e-5
    u = torch.finfo(c["q"].dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0     # a subnormal output's rounding
    tol = u * np.abs(ref) + (1 + u) * (mag * (weight_error(c) + u * u) + n * 2.0 ** -40 * 1000) + tiny
    for call in ("window", "accumulate"):
        d["out"].fill_(float("nan"))
        if call == "window":
            E.paged_attention_decode_window(d["out"], d["q"], d["k"], d["v"], d["tables"], d["lens"], n, 0, c["scale"])
        else:
            E.paged_attention_decode_accumulate(d["out"], scores, d["q"], d["k"], d["v"], d["tables"], d["lens"],
                                                c["scale"])
        err = np.abs(f64(d["out"].cpu()) - ref)
        assert np.all(err <= tol), f"{call}: {err.max():.3g} of {ref.max():.3g}"
    want = B.accumulate(np.zeros(scores.shape), weights, Hkv)
    w = weight_error(c) + (H // Hkv + 1) * 2.0 ** -24
    assert np.all(np.abs(f64(scores.cpu()) - want) <= w * want + 2.0 ** -126)
