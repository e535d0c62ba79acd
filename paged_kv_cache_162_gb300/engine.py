"""Tensor-level calls and one decode step over a paged KV cache.

PyTorch supplies device memory and streams only; every step of the path
runs in libpagedkv.so through the C ABI (see _lib.py).

The step, in the order a serving loop runs it ("3.3 页面级显存管理" 3.3.2;
"vLLM三大核心技术分页内存与共享解码", Copy-on-Write section):
  host   make room for each sequence's new tokens (copy-on-write of shared
         blocks, new blocks as the token count grows) -- `plan_step`
  device copy_blocks -> compute_slot_mapping -> reshape_and_cache ->
         paged_attention_decode
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import time

import numpy as np
import torch

from . import _lib as L
from .allocator import BlockAllocator, check_copy_pairs, plan_step

_DTYPES = {torch.float16: L.PKV_F16, torch.bfloat16: L.PKV_BF16}
_TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


def dtype_code(t: torch.dtype) -> int:
    if t not in _DTYPES:
        raise L.PkvError(L.PKV_ERR_UNSUPPORTED, f"dtype {t} (fp16 and bf16 only)")
    return _DTYPES[t]


def torch_dtype(name: str) -> torch.dtype:
    return _TORCH[name]


def workspace_size(S, H, D, max_context_len, partition_tokens=0) -> int:
    return L.pkv_decode_workspace_size(S, H, D, max_context_len, partition_tokens)


def new_workspace(S, H, D, max_context_len, partition_tokens=0, device="cuda") -> torch.Tensor:
    n = workspace_size(S, H, D, max_context_len, partition_tokens)
    if n == 0:
        raise L.PkvError(L.PKV_ERR_INVALID_ARG, "bad workspace arguments")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _as_stream(stream, device):
    """`stream`, a torch stream or a handle, as a torch stream."""
    return torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream


def _scratch(nbytes, device, stream=None) -> torch.Tensor:
    """Memory for one call on `stream` (None: the current one), out of the
    memory of that stream: what another stream has given back may still be in
    use there, and what this call gives back is its stream's again."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(_as_stream(stream, device)):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _no_q4(who, *caches):
    """Refuses 4-bit caches (new_cache_q4) in a call on 16-bit ones, which would
    reach past their smaller blocks."""
    for c in caches:
        if c.dtype is torch.uint8:
            _refuse(f"{who}: takes 16-bit caches, not 4-bit ones (uint8 {tuple(c.shape)})")


def paged_attention_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale=None,
                           max_context_len=0, partition_tokens=0, workspace=None, stream=None):
    """out[s,h] = softmax(scale q[s,h] K^T) V over each sequence's paged context.

    q, out: [S, H, D]; caches: [NB, bs, H, D]; block_tables [S, MB] int32;
    context_lens [S] int32 (all on the device).
    """
    _no_q4("paged_attention_decode", k_cache, v_cache)
    S, H, D = q.shape
    NB, bs = k_cache.shape[0], k_cache.shape[1]
    MB = block_tables.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if workspace is None:
        n = workspace_size(S, H, D, max_context_len or MB * bs, partition_tokens)
        if n == 0:
            raise L.PkvError(L.PKV_ERR_INVALID_ARG, "bad workspace arguments")
        workspace = _scratch(n, k_cache.device, stream)
    L.pkv_paged_attention_decode(out, q, k_cache, v_cache, block_tables, context_lens, S, H, D, bs,
                                 NB, MB, max_context_len, scale, dtype_code(q.dtype),
                                 partition_tokens, workspace, workspace.numel(), stream)
    return out


def decode_step(out, q, key, value, k_cache, v_cache, block_tables, context_lens, seq_idx, pos,
                slot_mapping, prefix_groups=None, scale=None, max_context_len=0,
                partition_tokens=0, workspace=None, stream=None):
    """compute_slot_mapping + reshape_and_cache + paged_attention_decode (or
    its shared-prefix form, with prefix_groups [G, 3] int32 on the device) in
    fewer kernels (see pkv_decode_step): the new tokens (key/value [T, H, D],
    seq_idx/pos [T] int32) are written into the caches, slot_mapping [T]
    int64 receives their slots, then out = attention over every context."""
    _no_q4("decode_step", k_cache, v_cache)
    S, H, D = q.shape
    NB, bs = k_cache.shape[0], k_cache.shape[1]
    MB = block_tables.shape[1]
    T = int(seq_idx.numel())
    G = 0 if prefix_groups is None else int(prefix_groups.shape[0])
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if workspace is None:
        mc = max_context_len or MB * bs
        n = (L.pkv_decode_shared_prefix_workspace_size(S, H, D, G, mc, partition_tokens) if G
             else workspace_size(S, H, D, mc, partition_tokens))
        workspace = _scratch(n, k_cache.device, stream)
    L.pkv_decode_step(out, q, key, value, k_cache, v_cache, block_tables, context_lens, seq_idx,
                      pos, slot_mapping, prefix_groups, G, T, S, H, D, bs, NB, MB,
                      max_context_len, scale, dtype_code(q.dtype), partition_tokens, workspace,
                      workspace.numel(), stream)
    return out


def paged_attention_decode_shared_prefix(out, q, k_cache, v_cache, block_tables, context_lens,
                                         prefix_groups, scale=None, max_context_len=0,
                                         partition_tokens=0, workspace=None, stream=None):
    """paged_attention_decode where groups of sequences share a prefix
    (prefix_groups [G, 3] int32 on the device: first sequence, members,
    prefix tokens); the prefix is read once per group (tensor cores)."""
    _no_q4("paged_attention_decode_shared_prefix", k_cache, v_cache)
    S, H, D = q.shape
    NB, bs = k_cache.shape[0], k_cache.shape[1]
    MB = block_tables.shape[1]
    G = prefix_groups.shape[0]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if workspace is None:
        mcl = max_context_len or MB * bs
        need = L.pkv_decode_shared_prefix_workspace_size(S, H, D, G, mcl, partition_tokens)
        workspace = _scratch(need, k_cache.device, stream)
    L.pkv_paged_attention_decode_shared_prefix(out, q, k_cache, v_cache, block_tables,
                                               context_lens, prefix_groups, G, S, H, D, bs, NB, MB,
                                               max_context_len, scale, dtype_code(q.dtype),
                                               partition_tokens, workspace, workspace.numel(),
                                               stream)
    return out


class _AskCtypes:
    """Stands for _tensor_bind where there is none for this torch: every call is left to ctypes."""
    window = accumulate = evict = rotate = gather = decode_q4 = staticmethod(lambda *args: -1)


_bind = None


def _native():
    """The module that calls the library with tensors (csrc/tensor_bind.cpp).
    Its functions answer with the call's status, or -1 for arguments that it
    leaves to the checks and the ctypes call below."""
    global _bind
    if _bind is None:
        L.lib()
        try:
            from . import _tensor_bind as found
        except ImportError:  # not built, or for a torch with other symbols
            found = None
        _bind = found if getattr(found, "torch_version", None) == torch.__version__ else _AskCtypes
    return _bind


def _refuse(what: str):
    raise L.PkvError(L.PKV_ERR_INVALID_ARG, what)


def _need(who, tensors, cache):
    """Refuses unless every (name, tensor, dtype, shape) is contiguous, of
    that type and shape (None: any), on the caches' device -- or, for q and
    out, in pinned host memory."""
    dev = cache.device
    if dev.type != "cuda":
        _refuse(f"{who}: the caches must be on a CUDA device, not {dev}")
    for name, t, dtype, shape in tensors:
        if t.dtype != dtype or (shape is not None and t.shape != shape) or not t.is_contiguous():
            _refuse(f"{who}: {name} must be contiguous {dtype} of shape "
                    f"{tuple(shape) if shape is not None else 'any'}, got {t.dtype} {tuple(t.shape)}"
                    f"{'' if t.is_contiguous() else ' (not contiguous)'}")
        if t.device != dev and not (name in ("q", "out") and t.device.type == "cpu" and t.is_pinned()):
            _refuse(f"{who}: {name} is on {t.device}, the caches on {dev}")


def _token_rows(who, name, t, dtype, shape, dev) -> int:
    """Refuses unless t is [T, heads, D] of that type and shape with each
    token's rows contiguous, on device `dev` or in pinned host memory; the
    elements from one token to the next."""
    if t.dtype != dtype or t.shape != shape:
        _refuse(f"{who}: {name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    T, heads, D = shape
    if T * heads * D and (t.stride(2) != 1 or (heads > 1 and t.stride(1) != D)):
        _refuse(f"{who}: {name}: the {heads} x {D} elements of a token must be contiguous, got strides {t.stride()}")
    if t.device != dev and not (t.device.type == "cpu" and t.is_pinned()):
        _refuse(f"{who}: {name} is on {t.device}, the caches on {dev}")
    return t.stride(0) if T > 1 else heads * D


_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8


def _attention_sizes(who, out, q, k_cache, v_cache, block_tables, context_lens):
    """Checks what the two attention calls share; returns the sizes and the
    device.  One expression on the way through: these calls take a few
    microseconds on the GPU, and every attribute counts.  _need then says
    what is wrong."""
    shape, cshape, tshape = q.shape, k_cache.shape, block_tables.shape
    if len(shape) != 3 or len(cshape) != 4 or len(tshape) != 2:
        _refuse(f"{who}: q must be [S, H, D], the caches [NB, bs, Hkv, D], block_tables [S, MB]")
    S, H, D = shape
    NB, bs, Hkv, Dk = cshape
    if Dk != D:
        _refuse(f"{who}: q has head_dim {D}, the caches {Dk}")
    L.int32(max(*shape, *cshape, *tshape), f"{who}: the largest extent")
    dt, dev = k_cache.dtype, k_cache.get_device()
    if not (dev >= 0 and q.dtype is dt and out.dtype is dt and v_cache.dtype is dt
            and block_tables.dtype is _I32 and context_lens.dtype is _I32 and out.shape == shape
            and v_cache.shape == cshape and tshape[0] == S and context_lens.shape == (S,)
            and q.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous()
            and v_cache.is_contiguous() and block_tables.is_contiguous()
            and context_lens.is_contiguous() and q.get_device() == dev
            and out.get_device() == dev and v_cache.get_device() == dev
            and block_tables.get_device() == dev and context_lens.get_device() == dev):
        _need(who, (("k_cache", k_cache, dt, None), ("q", q, dt, None), ("out", out, dt, shape),
                    ("v_cache", v_cache, dt, cshape),
                    ("block_tables", block_tables, _I32, (S, tshape[1])),
                    ("context_lens", context_lens, _I32, (S,))), k_cache)
    return S, H, D, NB, bs, Hkv, tshape[1], dev


@contextlib.contextmanager
def _on(stream, device):
    """Torch's work inside runs on `stream` (None: the current one), after
    what the current stream holds by now; what the current stream gets later
    runs after it."""
    if stream is None:
        yield
        return
    stream, current = _as_stream(stream, device), torch.cuda.current_stream(device)
    stream.wait_stream(current)
    try:
        with torch.cuda.stream(stream):
            yield
    finally:
        current.wait_stream(stream)


def _no_capture(who, stream, device):
    """Refuses while the current stream or `stream` is being captured."""
    if not torch.cuda.is_initialized():
        return
    with torch.cuda.stream(None if stream is None else _as_stream(stream, device)):
        capturing = torch.cuda.is_current_stream_capturing()
    if capturing or torch.cuda.is_current_stream_capturing():
        _refuse(f"{who} cannot be captured in a graph")


def _workspace(who, nbytes, device, stream=None):
    """_scratch for a call of this section."""
    if nbytes == 0:
        _refuse(f"{who}: bad workspace arguments (H a multiple of Hkv, at most 16 per group?)")
    return _scratch(nbytes, device, stream)


def _check_workspace(who, ws, dev):
    if ws.dtype is not _U8 or ws.get_device() != dev or not ws.is_contiguous():
        _refuse(f"{who}: workspace must be a contiguous uint8 tensor on the caches' device")


def new_window_workspace(S, H, Hkv, D, device="cuda") -> torch.Tensor:
    return _workspace("new_window_workspace", L.pkv_decode_window_workspace_size(S, H, Hkv, D),
                      device)


def new_accumulate_workspace(S, H, Hkv, D, max_context_len, device="cuda") -> torch.Tensor:
    """max_context_len: the call's, or MB * bs where the call is given 0."""
    if max_context_len < 1:
        _refuse("new_accumulate_workspace: max_context_len must be at least 1 (MB * bs for a call given 0)")
    return _workspace("new_accumulate_workspace",
                      L.pkv_decode_accumulate_workspace_size(S, H, Hkv, D, max_context_len), device)


def new_evict_workspace(S, Hkv, budget, device="cuda") -> torch.Tensor:
    return _workspace("new_evict_workspace", L.pkv_evict_workspace_size(S, Hkv, budget), device)


def paged_attention_decode_window(out, q, k_cache, v_cache, block_tables, context_lens, window,
                                  sink_tokens=0, scale=None, max_context_len=0, workspace=None,
                                  stream=None):
    """Decode attention of each sequence's newest token over its first
    sink_tokens tokens and its last `window` tokens.

    q, out: [S, H, D]; caches: [NB, bs, Hkv, D] with H a multiple of Hkv (at
    most 16 query heads per KV head); block_tables [S, MB] int32;
    context_lens [S] int32.  Blocks without a visible token are not looked
    up: their table entries may be -1 (BlockAllocator.release_window).
    workspace: new_window_workspace(S, H, Hkv, D), kept between calls.
    """
    who = "paged_attention_decode_window"
    if stream is None and workspace is not None:
        st = _native().window(out, q, k_cache, v_cache, block_tables, context_lens, window,
                              sink_tokens, scale, max_context_len, workspace)
        if st == 0:
            return out
        if st > 0:
            L.check(st, who)
    S, H, D, NB, bs, Hkv, MB, dev = _attention_sizes(who, out, q, k_cache, v_cache, block_tables,
                                                     context_lens)
    window, sink_tokens, max_context_len = (L.int32(window, "window"), L.int32(sink_tokens, "sink_tokens"),
                                            L.int32(max_context_len, "max_context_len"))
    ws = workspace
    if ws is None:
        ws = _workspace(who, L.pkv_decode_window_workspace_size(S, H, Hkv, D), k_cache.device, stream)
    else:
        _check_workspace(who, ws, dev)

    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return paged_attention_decode_window(out, q, k_cache, v_cache, block_tables,
                                                 context_lens, window, sink_tokens, scale,
                                                 max_context_len, ws, stream)
    handle = L.current_stream_handle(dev) if stream is None else L.stream_handle(stream)
    st = L.lib().pkv_paged_attention_decode_window(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        block_tables.data_ptr(), context_lens.data_ptr(), S, H, Hkv, D, bs, NB, MB,
        max_context_len, window, sink_tokens, D ** -0.5 if scale is None else scale,
        dtype_code(k_cache.dtype), ws.data_ptr(), ws.numel(), handle)
    if st:
        L.check(st, who)
    return out


def paged_attention_decode_accumulate(out, scores, q, k_cache, v_cache, block_tables, context_lens,
                                      scale=None, max_context_len=0, workspace=None, stream=None):
    """Decode attention over each whole context that also adds each cached
    token's attention weight, summed over the query heads of its KV head, to
    scores [S, Hkv, cap] fp32 (cap >= max_context_len, or MB * bs when that
    is 0; entries past a context are left alone).  The statistic
    evict_tokens goes by.  Other arguments as in
    paged_attention_decode_window; workspace: new_accumulate_workspace(S, H,
    Hkv, D, max_context_len)."""
    who = "paged_attention_decode_accumulate"
    if stream is None and workspace is not None:
        st = _native().accumulate(out, scores, q, k_cache, v_cache, block_tables, context_lens,
                                  scale, max_context_len, workspace)
        if st == 0:
            return out
        if st > 0:
            L.check(st, who)
    S, H, D, NB, bs, Hkv, MB, dev = _attention_sizes(who, out, q, k_cache, v_cache, block_tables,
                                                     context_lens)
    max_context_len = L.int32(max_context_len, "max_context_len")
    rows = scores.shape
    if not (scores.dtype is _F32 and len(rows) == 3 and rows[0] == S and rows[1] == Hkv
            and scores.is_contiguous() and scores.get_device() == dev):
        _need(who, (("scores", scores, _F32, (S, Hkv, rows[-1] if len(rows) else 0)),), k_cache)
    ws = workspace
    if ws is None:
        ws = _workspace(who, L.pkv_decode_accumulate_workspace_size(
            S, H, Hkv, D, max_context_len or MB * bs), k_cache.device, stream)
    else:
        _check_workspace(who, ws, dev)

    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return paged_attention_decode_accumulate(out, scores, q, k_cache, v_cache,
                                                     block_tables, context_lens, scale,
                                                     max_context_len, ws, stream)
    handle = L.current_stream_handle(dev) if stream is None else L.stream_handle(stream)
    st = L.lib().pkv_paged_attention_decode_accumulate(
        out.data_ptr(), scores.data_ptr(), q.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), S, H, Hkv, D, bs,
        NB, MB, max_context_len, rows[2], D ** -0.5 if scale is None else scale,
        dtype_code(k_cache.dtype), ws.data_ptr(), ws.numel(), handle)
    if st:
        L.check(st, who)
    return out


def evict_tokens(k_cache, v_cache, scores, positions, block_tables, context_lens, token_counts,
                 new_context_lens, budget, recent_tokens, sink_tokens=0, scores_out=None,
                 positions_out=None, max_context_len=0, workspace=None, stream=None):
    """Keeps the `budget` best tokens of every (sequence, KV head) with more
    -- the first sink_tokens positions and the last recent_tokens ones, then
    the highest scores, ties by the lowest index -- and compacts the caches,
    scores and positions to them in place (see pkv_evict_tokens).

    scores [S, Hkv, cap] fp32 (paged_attention_decode_accumulate), positions
    [S, Hkv, cap] int32 (-1: appended since the last eviction; a new
    sequence's row is all -1); context_lens, token_counts [S] int32: tokens
    cached and tokens seen; new_context_lens [S] int32 receives
    min(context_lens, budget).  scores_out / positions_out: other arrays for
    the results (default: in place); max_context_len bounds context_lens (0:
    MB * bs).  The evicted sequences' blocks must be
    their own (BlockAllocator.unshare); afterwards BlockAllocator.truncate
    releases the blocks past the budget."""
    who = "evict_tokens"
    if scores_out is None:
        scores_out = scores
    if positions_out is None:
        positions_out = positions
    if stream is None and workspace is not None:
        st = _native().evict(k_cache, v_cache, scores, positions, block_tables, context_lens,
                             token_counts, new_context_lens, budget, recent_tokens, sink_tokens,
                             scores_out, positions_out, max_context_len, workspace)
        if st == 0:
            return
        if st > 0:
            L.check(st, who)
    if k_cache.dim() != 4 or block_tables.dim() != 2:
        _refuse(f"{who}: the caches must be [NB, bs, Hkv, D], block_tables [S, MB]")
    NB, bs, Hkv, D = k_cache.shape
    S, MB = block_tables.shape
    L.int32(max(*k_cache.shape, S, MB), f"{who}: the largest extent")
    budget, recent_tokens, sink_tokens, max_context_len = (
        L.int32(budget, "budget"), L.int32(recent_tokens, "recent_tokens"),
        L.int32(sink_tokens, "sink_tokens"), L.int32(max_context_len, "max_context_len"))
    dt, dev = k_cache.dtype, k_cache.get_device()
    rows = scores.shape
    if not (dev >= 0 and len(rows) == 3 and rows[0] == S and rows[1] == Hkv and v_cache.dtype is dt
            and scores.dtype is _F32 and scores_out.dtype is _F32 and positions.dtype is _I32
            and positions_out.dtype is _I32 and block_tables.dtype is _I32
            and context_lens.dtype is _I32 and token_counts.dtype is _I32
            and new_context_lens.dtype is _I32 and v_cache.shape == k_cache.shape
            and scores_out.shape == rows and positions.shape == rows and positions_out.shape == rows
            and context_lens.shape == (S,) and token_counts.shape == (S,)
            and new_context_lens.shape == (S,) and k_cache.is_contiguous()
            and v_cache.is_contiguous() and scores.is_contiguous() and scores_out.is_contiguous()
            and positions.is_contiguous() and positions_out.is_contiguous()
            and block_tables.is_contiguous() and context_lens.is_contiguous()
            and token_counts.is_contiguous() and new_context_lens.is_contiguous()
            and v_cache.get_device() == dev and scores.get_device() == dev
            and scores_out.get_device() == dev and positions.get_device() == dev
            and positions_out.get_device() == dev and block_tables.get_device() == dev
            and context_lens.get_device() == dev and token_counts.get_device() == dev
            and new_context_lens.get_device() == dev):
        want = (S, Hkv, rows[-1] if len(rows) else 0)
        _need(who, (("k_cache", k_cache, dt, None), ("v_cache", v_cache, dt, k_cache.shape),
                    ("scores", scores, _F32, want), ("positions", positions, _I32, want),
                    ("scores_out", scores_out, _F32, want),
                    ("positions_out", positions_out, _I32, want),
                    ("block_tables", block_tables, _I32, None),
                    ("context_lens", context_lens, _I32, (S,)),
                    ("token_counts", token_counts, _I32, (S,)),
                    ("new_context_lens", new_context_lens, _I32, (S,))), k_cache)
    ws = workspace
    if ws is None:
        ws = _workspace(who, L.pkv_evict_workspace_size(S, Hkv, budget), k_cache.device, stream)
    else:
        _check_workspace(who, ws, dev)

    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return evict_tokens(k_cache, v_cache, scores, positions, block_tables, context_lens,
                                token_counts, new_context_lens, budget, recent_tokens, sink_tokens,
                                scores_out, positions_out, max_context_len, ws, stream)
    handle = L.current_stream_handle(dev) if stream is None else L.stream_handle(stream)
    st = L.lib().pkv_evict_tokens(
        k_cache.data_ptr(), v_cache.data_ptr(), scores.data_ptr(), positions.data_ptr(),
        block_tables.data_ptr(), context_lens.data_ptr(), token_counts.data_ptr(),
        scores_out.data_ptr(), positions_out.data_ptr(), new_context_lens.data_ptr(), S, Hkv, D,
        bs, NB, MB, max_context_len, rows[2], budget, recent_tokens, sink_tokens,
        dtype_code(dt), ws.data_ptr(), ws.numel(), handle)
    if st:
        L.check(st, who)


def new_rotary_table(positions, rotary_dim, base=10000.0, device="cuda") -> torch.Tensor:
    """The rotary table of rotate_and_cache for positions 0 .. positions - 1:
    [positions, rotary_dim] fp32, the cosines of the rotary_dim / 2 angles
    position * base^(-2i / rotary_dim), then their sines.  The angles are taken
    in 64 bits: in 32 those of far positions are off by whole steps."""
    if positions < 1 or rotary_dim < 2 or rotary_dim % 2:
        _refuse("new_rotary_table: positions >= 1 and an even rotary_dim >= 2")
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * float(base) ** (-i / rotary_dim)
    return torch.cat([angle.cos(), angle.sin()], -1).float()


def rotate_and_cache(key, value, k_cache, v_cache, block_tables, seq_idx, pos, slot_mapping, rotary_table=None,
                     query=None, query_out=None, rotary_pos=None, interleaved=False, stream=None):
    """compute_slot_mapping + the rotary position encoding of a step's queries
    and keys + reshape_and_cache, in one kernel (see pkv_rotate_and_cache).

    key, value: [T, Hkv, D] and query: [T, H, D], each token's rows contiguous,
    tokens any multiple of 8 elements apart (slices of one projection);
    caches: [NB, bs, Hkv, D]; block_tables [S, MB], seq_idx, pos [T] int32
    (pos -1: padding, left alone); slot_mapping [T] int64 receives the slots.
    rotary_table [positions, rotary_dim] fp32 (new_rotary_table; None: no
    rotation) is read at rotary_pos [T] int32 (None: pos).  query_out receives
    the queries (None: in place) and is returned."""
    return _rotate("rotate_and_cache", False, key, value, k_cache, v_cache, block_tables, seq_idx, pos, slot_mapping,
                   rotary_table, query, query_out, rotary_pos, interleaved, stream)


def new_cache_q4(NB, bs, Hkv, D, device="cuda") -> torch.Tensor:
    """A K (or V) pool held in 4 bits, all elements 0: uint8 [NB, Hkv, bs, RB]
    with RB = D/2 + D/16 bytes per (token, KV head).  Written by
    rotate_and_cache_q4, read by paged_attention_decode_q4 and
    gather_cache_q4; its bytes are laid out as include/pagedkv.h says."""
    RB = L.pkv_cache_q4_row_bytes(D)
    if RB == 0 or bs not in (8, 16, 32, 64) or NB < 1 or Hkv < 1:
        _refuse("new_cache_q4: head_dim must be 64/128, block_size 8/16/32/64, NB and Hkv at least 1")
    return torch.zeros((NB, Hkv, bs, RB), dtype=_U8, device=device)


def rotate_and_cache_q4(key, value, k_cache, v_cache, block_tables, seq_idx, pos, slot_mapping, rotary_table=None,
                        query=None, query_out=None, rotary_pos=None, interleaved=False, stream=None):
    """rotate_and_cache into 4-bit caches (new_cache_q4): K is quantised from
    its rotated values in fp32."""
    return _rotate("rotate_and_cache_q4", True, key, value, k_cache, v_cache, block_tables, seq_idx, pos,
                   slot_mapping, rotary_table, query, query_out, rotary_pos, interleaved, stream)


def _cache_sizes(who, cache, D, q4):
    """(NB, bs, Hkv) of a cache for head_dim D."""
    if cache.dim() != 4:
        _refuse(f"{who}: the caches must be [NB, {'Hkv, bs, RB' if q4 else 'bs, Hkv, D'}]")
    if not q4:
        NB, bs, Hkv, Dk = cache.shape
        if Dk != D:
            _refuse(f"{who}: key has head_dim {D}, the caches {Dk}")
        return NB, bs, Hkv
    NB, Hkv, bs, RB = cache.shape
    want = L.pkv_cache_q4_row_bytes(D)
    if want == 0:
        raise L.PkvError(L.PKV_ERR_UNSUPPORTED, f"{who}: head_dim must be 64 or 128, got {D}")
    if RB != want or cache.dtype != _U8:
        _refuse(f"{who}: 4-bit caches must be uint8 [NB, Hkv, bs, {want}] for head_dim {D}, got {cache.dtype} "
                f"{tuple(cache.shape)}")
    return NB, bs, Hkv


def _rotate(who, q4, key, value, k_cache, v_cache, block_tables, seq_idx, pos, slot_mapping, rotary_table, query,
            query_out, rotary_pos, interleaved, stream):
    if query_out is None:
        query_out = query
    if stream is None:
        st = _native().rotate(q4, key, value, k_cache, v_cache, block_tables, seq_idx, pos, slot_mapping, rotary_table,
                              query, query_out, rotary_pos, interleaved)
        if st == 0:
            return query_out
        if st > 0:
            L.check(st, who)
    if key.dim() != 3 or block_tables.dim() != 2 or (query is not None and query.dim() != 3):
        _refuse(f"{who}: key must be [T, Hkv, D], query [T, H, D], block_tables [S, MB]")
    T, Hkv, D = key.shape
    dt, dev = key.dtype, k_cache.device
    code = dtype_code(dt)
    NB, bs, heads = _cache_sizes(who, k_cache, D, q4)
    if heads != Hkv:
        _refuse(f"{who}: key has {Hkv} heads, the caches {heads}")
    if query is None and query_out is not None:
        _refuse(f"{who}: query_out without query")
    cdt = _U8 if q4 else dt
    _need(who, [("k_cache", k_cache, cdt, None), ("v_cache", v_cache, cdt, k_cache.shape),
                ("block_tables", block_tables, _I32, None), ("seq_idx", seq_idx, _I32, (T,)),
                ("pos", pos, _I32, (T,)), ("slot_mapping", slot_mapping, torch.int64, (T,))]
          + ([("rotary_pos", rotary_pos, _I32, (T,))] if rotary_pos is not None else [])
          + ([("rotary_table", rotary_table, _F32, None)] if rotary_table is not None else []), k_cache)
    rows, R = 0, 0
    if rotary_table is not None:
        if rotary_table.dim() != 2:
            _refuse(f"{who}: rotary_table must be [positions, rotary_dim]")
        rows, R = rotary_table.shape
    ks, vs = _token_rows(who, "key", key, dt, key.shape, dev), _token_rows(who, "value", value, dt, key.shape, dev)
    H, qs, qos = 0, 0, 0
    if query is not None:
        H = query.shape[1]
        if H == 0:
            _refuse(f"{who}: query has no heads")
        qs = _token_rows(who, "query", query, dt, (T, H, D), dev)
        qos = _token_rows(who, "query_out", query_out, dt, (T, H, D), dev)
    S, MB = block_tables.shape
    L.int32(max(T, H, S, MB, rows, R, *k_cache.shape), f"{who}: the largest extent")
    with torch.cuda.device(dev):
        (L.pkv_rotate_and_cache_q4 if q4 else L.pkv_rotate_and_cache)(
            key, ks, value, vs, query, qs, query_out, qos, k_cache, v_cache, block_tables, seq_idx, pos, rotary_pos,
            rotary_table, rows, R, bool(interleaved), slot_mapping, T, S, H, Hkv, D, bs, NB, MB, code, stream=stream)
    return query_out


def gather_cache_q4(key, value, k_cache, v_cache, slot_mapping, stream=None):
    """Reads the rows of slot_mapping [T] int64 out of 4-bit caches into key
    and value [T, Hkv, D] (strides as in rotate_and_cache), as the 16-bit
    values that they stand for; rows of negative slots are left as they were.
    For the cached prefix of a prompt's next chunk, or a sequence on its way
    into a 16-bit cache (reshape_and_cache)."""
    who = "gather_cache_q4"
    if stream is None:
        st = _native().gather(key, value, k_cache, v_cache, slot_mapping)
        if st == 0:
            return key, value
        if st > 0:
            L.check(st, who)
    if key.dim() != 3:
        _refuse(f"{who}: key must be [T, Hkv, D]")
    T, Hkv, D = key.shape
    dt, dev = key.dtype, k_cache.device
    code = dtype_code(dt)
    NB, bs, heads = _cache_sizes(who, k_cache, D, True)
    if heads != Hkv:
        _refuse(f"{who}: key has {Hkv} heads, the caches {heads}")
    _need(who, (("k_cache", k_cache, _U8, None), ("v_cache", v_cache, _U8, k_cache.shape),
                ("slot_mapping", slot_mapping, torch.int64, (T,))), k_cache)
    ks, vs = _token_rows(who, "key", key, dt, key.shape, dev), _token_rows(who, "value", value, dt, key.shape, dev)
    L.int32(max(T, *k_cache.shape), f"{who}: the largest extent")
    with torch.cuda.device(dev):
        L.pkv_gather_cache_q4(key, ks, value, vs, k_cache, v_cache, slot_mapping, T, Hkv, D, bs, NB, code, stream)
    return key, value


def new_q4_workspace(S, H, Hkv, D, device="cuda") -> torch.Tensor:
    return _workspace("new_q4_workspace", L.pkv_decode_q4_workspace_size(S, H, Hkv, D), device)


def paged_attention_decode_q4(out, q, k_cache, v_cache, block_tables, context_lens, scale=None, max_context_len=0,
                              workspace=None, stream=None):
    """Decode attention of each sequence's newest token over its whole context
    in 4-bit caches (new_cache_q4).  q, out: [S, H, D] with H a multiple of Hkv
    (at most 16 query heads per KV head), of the type the caches were written
    with; block_tables [S, MB], context_lens [S] int32.  workspace:
    new_q4_workspace(S, H, Hkv, D), kept between calls."""
    who = "paged_attention_decode_q4"
    if stream is None and workspace is not None:
        st = _native().decode_q4(out, q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len,
                                 workspace)
        if st == 0:
            return out
        if st > 0:
            L.check(st, who)
    if q.dim() != 3 or block_tables.dim() != 2:
        _refuse(f"{who}: q must be [S, H, D], block_tables [S, MB]")
    S, H, D = q.shape
    code = dtype_code(q.dtype)
    NB, bs, Hkv = _cache_sizes(who, k_cache, D, True)
    MB = block_tables.shape[1]
    L.int32(max(S, H, MB, *k_cache.shape), f"{who}: the largest extent")
    max_context_len = L.int32(max_context_len, "max_context_len")
    _need(who, (("k_cache", k_cache, _U8, None), ("v_cache", v_cache, _U8, k_cache.shape),
                ("q", q, q.dtype, None), ("out", out, q.dtype, q.shape),
                ("block_tables", block_tables, _I32, (S, MB)), ("context_lens", context_lens, _I32, (S,))), k_cache)
    ws, dev = workspace, k_cache.get_device()
    if ws is None:
        ws = _workspace(who, L.pkv_decode_q4_workspace_size(S, H, Hkv, D), k_cache.device, stream)
    else:
        _check_workspace(who, ws, dev)
    with torch.cuda.device(dev):
        L.pkv_paged_attention_decode_q4(out, q, k_cache, v_cache, block_tables, context_lens, S, H, Hkv, D, bs, NB,
                                        MB, max_context_len, D ** -0.5 if scale is None else scale, code, ws,
                                        ws.numel(), stream)
    return out


def compute_slot_mapping(slot_mapping, block_tables, seq_idx, pos, block_size, stream=None):
    L.pkv_compute_slot_mapping(slot_mapping, block_tables, seq_idx, pos, seq_idx.numel(),
                               block_tables.shape[0], block_tables.shape[1], block_size, stream)
    return slot_mapping


def reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, stream=None):
    _no_q4("reshape_and_cache", k_cache, v_cache)
    T, H, D = key.shape
    NB, bs = k_cache.shape[0], k_cache.shape[1]
    L.pkv_reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, T, H, D, bs, NB,
                            dtype_code(key.dtype), stream)


def _q4_head_dim(who, cache) -> int:
    """head_dim of a 4-bit cache [NB, Hkv, bs, RB]."""
    for D in (64, 128):
        if cache.dim() == 4 and cache.shape[3] == L.pkv_cache_q4_row_bytes(D):
            return D
    _refuse(f"{who}: not a 4-bit cache: uint8 {tuple(cache.shape)}")


def copy_blocks(k_cache, v_cache, block_mapping, stream=None):
    """Block copies (src, dst) [P, 2] int64 within 16-bit caches [NB, bs, H,
    D], or within 4-bit ones (new_cache_q4)."""
    P = block_mapping.shape[0] if block_mapping is not None else 0
    if k_cache.dtype == _U8:
        D = _q4_head_dim("copy_blocks", k_cache)
        NB, Hkv, bs, _ = k_cache.shape
        if v_cache.dtype != _U8 or v_cache.shape != k_cache.shape:
            _refuse("copy_blocks: k_cache and v_cache differ in type or shape")
        if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
            _refuse("copy_blocks: 4-bit caches must be contiguous")
        L.pkv_copy_blocks_q4(k_cache, v_cache, block_mapping, P, Hkv, D, bs, NB, stream)
        return
    _no_q4("copy_blocks", v_cache)
    NB, bs, H, D = k_cache.shape
    L.pkv_copy_blocks(k_cache, v_cache, block_mapping, P, H, D, bs, NB,
                      dtype_code(k_cache.dtype), stream)


def swap_blocks(gpu_k, gpu_v, host_k, host_v, block_mapping, direction, stream=None):
    """GPU <-> pinned-host block copies (CPU swap).  block_mapping [P, 2]
    int64 on the device: (gpu block, host block) pairs for swap-out,
    (host block, gpu block) pairs for swap-in.  16-bit caches, or 4-bit ones on
    both sides."""
    P = block_mapping.shape[0]
    if gpu_k.dtype == _U8:
        D = _q4_head_dim("swap_blocks", gpu_k)
        NBg, Hkv, bs, _ = gpu_k.shape
        if any(x.dtype != _U8 or x.dim() != 4 or x.shape[1:] != gpu_k.shape[1:] for x in (gpu_v, host_k, host_v)) \
                or gpu_v.shape != gpu_k.shape or host_v.shape != host_k.shape:
            _refuse("swap_blocks: the 4-bit caches differ in type or shape")
        if not all(x.is_contiguous() for x in (gpu_k, gpu_v, host_k, host_v)):
            _refuse("swap_blocks: 4-bit caches must be contiguous")
        L.pkv_swap_blocks_q4(gpu_k, gpu_v, host_k, host_v, block_mapping, P, Hkv, D, bs, NBg, host_k.shape[0],
                             direction, stream)
        return
    _no_q4("swap_blocks", gpu_v, host_k, host_v)
    NBg, bs, H, D = gpu_k.shape
    L.pkv_swap_blocks(gpu_k, gpu_v, host_k, host_v, block_mapping, P, H, D, bs, NBg,
                      host_k.shape[0], dtype_code(gpu_k.dtype), direction, stream)


class DecodeStep:
    """Device-resident state of one decode step and the calls that run it.

    Built from plain arrays (16-bit data as uint16 bit patterns):
      caches: pool [NB, bs, H, D]; `blocks` lists the physical blocks whose
              contents `k_blocks`/`v_blocks` give, every other slot is set
              to `fill_bits`;
      tables_pre/nblocks_pre/ctx_before: the sequences before the step;
      n_new, new_k/new_v [T, H, D], seq_idx/pos [T]: the tokens appended;
      initial_free: the free list (last element handed out first).
    `plan()` runs the host allocator; `run()` launches copy_blocks, slot
    mapping, reshape_and_cache and decode on `stream` (`run(fused=True)`:
    copy_blocks and pkv_decode_step).
    """

    def __init__(self, *, dtype: str, S, H, D, bs, NB, MB, scale, ctx_before, n_new, tables_pre,
                 nblocks_pre, initial_free, blocks, k_blocks, v_blocks, q, new_k, new_v, seq_idx,
                 pos, fill_bits: int, partition_tokens: int = 0, device="cuda"):
        self.dtype = torch_dtype(dtype)
        self.S, self.H, self.D, self.bs, self.NB, self.MB = S, H, D, bs, NB, MB
        self.scale = float(scale)
        self.partition_tokens = partition_tokens
        self.device = torch.device(device)
        self.ctx_before = np.asarray(ctx_before, dtype=np.int32)
        self.n_new = np.asarray(n_new, dtype=np.int32)
        self.context_lens_host = (self.ctx_before + self.n_new).astype(np.int32)
        self.tables_pre = np.asarray(tables_pre, dtype=np.int32)
        self.nblocks_pre = np.asarray(nblocks_pre, dtype=np.int32)
        self.initial_free = np.asarray(initial_free, dtype=np.int32)
        self.max_context_len = max(int(self.context_lens_host.max(initial=0)), 1)
        dev = self.device

        def up16(a):
            t = torch.from_numpy(np.ascontiguousarray(a).view(np.int16))
            return t.to(dev).view(self.dtype)

        self.k_cache = torch.empty((NB, bs, H, D), dtype=torch.int16, device=dev)
        self.v_cache = torch.empty((NB, bs, H, D), dtype=torch.int16, device=dev)
        fill = int(np.int16(np.uint16(fill_bits)))
        self.k_cache.fill_(fill)
        self.v_cache.fill_(fill)
        if len(blocks):
            idx = torch.from_numpy(np.asarray(blocks, dtype=np.int64)).to(dev)
            for dst, src in ((self.k_cache, k_blocks), (self.v_cache, v_blocks)):
                chunk = 2048
                for i in range(0, len(blocks), chunk):
                    part = torch.from_numpy(np.ascontiguousarray(src[i:i + chunk]).view(np.int16))
                    dst.index_copy_(0, idx[i:i + chunk], part.to(dev))
        self.k_cache = self.k_cache.view(self.dtype)
        self.v_cache = self.v_cache.view(self.dtype)
        self.q = up16(q)
        self.new_k = up16(new_k)
        self.new_v = up16(new_v)
        self.seq_idx = torch.from_numpy(np.asarray(seq_idx, dtype=np.int32)).to(dev)
        self.pos = torch.from_numpy(np.asarray(pos, dtype=np.int32)).to(dev)
        self.T = int(self.seq_idx.numel())
        self.context_lens = torch.from_numpy(self.context_lens_host).to(dev)
        self.slot_mapping = torch.empty(max(self.T, 1), dtype=torch.int64, device=dev)
        self.out = torch.empty((S, H, D), dtype=self.dtype, device=dev)
        self.workspace = new_workspace(S, H, D, self.max_context_len, partition_tokens, dev)
        self.block_tables = None
        self.pairs = None
        # shared-prefix groups [G, 3] int32 on the device for run(fused=True)
        # (the workspace must then have the shared-prefix size)
        self.prefix_groups = None
        self._evicted = False  # since plan(): rows own their blocks, tokens have moved
        self.scores = self.positions = self.token_counts = None  # of decode_accumulate
        self._scored = False   # since plan(): they hold weights

    def plan(self):
        """Host allocator: tables and copy-on-write pairs for this step.
        A new plan also starts a new beam search (beam_step), and new scores
        (decode_accumulate) over the lengths from before any eviction; the
        caches keep what an eviction has moved."""
        for name in ("beam_ctx", "_beam_native"):
            old = self.__dict__.pop(name, None)
            if name == "_beam_native" and old is not None:
                torch.cuda.synchronize(self.device)  # its staging buffers may still be in flight
                old.close()
        self._forget_scores()
        self.allocator = BlockAllocator(self.NB, self.initial_free)
        ids, counts = np.unique(self.tables_pre[self.tables_pre >= 0], return_counts=True)
        for b, c in zip(ids.tolist(), counts.tolist()):
            if c > 1:
                self.allocator.incref([b] * (c - 1))
        tables, nb, pairs = plan_step(self.allocator, self.tables_pre, self.nblocks_pre,
                                      self.ctx_before, self.n_new, self.bs)
        self.tables_host, self.nblocks_host, self.pairs_host = tables, nb, pairs
        self.block_tables = torch.from_numpy(tables).to(self.device)
        self.pairs = torch.from_numpy(np.ascontiguousarray(pairs)).to(self.device)
        return tables, nb, pairs

    def _forget_scores(self):
        """Ends what decode_accumulate and evict() have begun: a step planned
        anew has no scores, and its lengths are those of its tables."""
        self._scored = False
        if self._evicted:
            self._evicted = False
            self.context_lens_host = (self.ctx_before + self.n_new).astype(np.int32)
            self.context_lens.copy_(torch.from_numpy(self.context_lens_host))

    def run(self, stream=None, attention=True, write=True, fused=False):
        """The device part of the step: copy_blocks, slot mapping, cache
        write, decode.  fused=True runs the last three as pkv_decode_step
        (fewer kernels, the same results), with the shared-prefix decode
        when self.prefix_groups is set.  After evict() the step's copies and
        writes would go to blocks that are other rows' by now: only
        write=False then."""
        if self.block_tables is None:
            self.plan()
        if write and self._evicted:
            _refuse("run: the step was written before an eviction moved it (plan() starts over)")
        if fused and write and attention:
            if self.pairs.shape[0]:
                copy_blocks(self.k_cache, self.v_cache, self.pairs, stream)
            g = self.prefix_groups
            L.pkv_decode_step(self.out, self.q, self.new_k, self.new_v, self.k_cache, self.v_cache,
                              self.block_tables, self.context_lens, self.seq_idx, self.pos,
                              self.slot_mapping, g, 0 if g is None else int(g.shape[0]), self.T,
                              self.S, self.H, self.D, self.bs, self.NB, self.MB,
                              self.max_context_len, self.scale, dtype_code(self.dtype),
                              self.partition_tokens, self.workspace, self.workspace.numel(),
                              stream)
            return self.out
        if write:
            if self.pairs.shape[0]:
                copy_blocks(self.k_cache, self.v_cache, self.pairs, stream)
            if self.T:
                compute_slot_mapping(self.slot_mapping, self.block_tables, self.seq_idx, self.pos,
                                     self.bs, stream)
                reshape_and_cache(self.new_k, self.new_v, self.k_cache, self.v_cache,
                                  self.slot_mapping, stream)
        if attention:
            self.decode(stream)
        return self.out

    def _beam_buffers(self):
        """Buffers of the native beam step: two pinned staging buffers used
        in turn (an event per buffer keeps one from being rewritten while
        its upload may still be in flight), the device twin they upload to,
        a device buffer for host-given tokens, and a workspace sized for
        the longest context the tables allow."""
        S, MB, H, D = self.S, self.MB, self.H, self.D
        dev = self.device
        nb = L.pkv_beam_inputs_bytes(S, MB)
        self._beam_inputs_bytes = nb
        self._beam_slots = []
        for _ in range(2):
            raw = torch.empty(nb + 256, dtype=torch.uint8).pin_memory()
            off = (-raw.data_ptr()) % 256
            stg = raw[off:off + nb]
            self._beam_slots.append({"stg": stg, "stg_np": stg.numpy(),
                                     "u16": torch.empty(3 * S * H * D, dtype=torch.int16).pin_memory(),
                                     "done": torch.cuda.Event(), "used": False})
        self._beam_dev_inputs = torch.empty(nb, dtype=torch.uint8, device=dev)
        self._beam_dev_u16 = torch.empty(3 * S * H * D, dtype=torch.int16, device=dev)
        self._beam_turn = 0
        # prefix groups ([G, 3]: first sequence, members, prefix tokens) set
        # before the first beam_step as `beam_groups`: the beams of a
        # request keep their prompt's full blocks shared, so each group's
        # prefix is read once per step
        groups = getattr(self, "beam_groups", None)
        if groups is not None and len(groups):
            g = np.ascontiguousarray(groups, dtype=np.int32).reshape(-1, 3)
            self._beam_groups_dev = torch.from_numpy(g).to(dev)
            self._beam_G = int(g.shape[0])
            nws = L.pkv_decode_shared_prefix_workspace_size(S, H, D, self._beam_G, MB * self.bs,
                                                            self.partition_tokens)
            self._beam_ws = torch.empty(nws, dtype=torch.uint8, device=dev)
        else:
            self._beam_groups_dev, self._beam_G = None, 0
            self._beam_ws = new_workspace(S, H, D, MB * self.bs, self.partition_tokens, dev)
        # decode() after beam steps: the tables allow contexts up to MB * bs
        self.max_context_len = MB * self.bs
        if self._beam_G == 0:
            self.workspace = self._beam_ws
        else:
            self.workspace = new_workspace(S, H, D, MB * self.bs, self.partition_tokens, dev)
        if self.slot_mapping.numel() < S:
            self.slot_mapping = torch.empty(S, dtype=torch.int64, device=dev)
        # offsets of the staged inputs (the layout pkv_beam_step documents)
        up = lambda x: (x + 255) // 256 * 256
        o_ctx = up(4 * S * MB)
        o_pos = o_ctx + up(4 * S)
        o_seq = o_pos + up(4 * S)
        self._beam_offsets = {"ctx": o_ctx, "pos": o_pos, "seq": o_seq, "pairs": o_seq + up(4 * S)}
        # the step's device inputs, as views of the uploaded buffer
        d = self._beam_dev_inputs
        self._beam_views = (d[:4 * S * MB].view(torch.int32).view(S, MB),
                            d[o_ctx:o_ctx + 4 * S].view(torch.int32),
                            d[o_pos:o_pos + 4 * S].view(torch.int32),
                            d[o_seq:o_seq + 4 * S].view(torch.int32))
        self._beam_stg_base = [sl["stg"].data_ptr() for sl in self._beam_slots]
        # the native side of the search: every argument of pkv_beam_step
        # that stays the same, and the alternation of the staging buffers
        self._beam_native = L.BeamSearch(
            self.allocator._h, self.tables_host, self.nblocks_host, self.beam_ctx, S, MB,
            self._beam_slots[0]["stg"], self._beam_slots[1]["stg"], self._beam_dev_inputs, nb,
            self.out, self.k_cache, self.v_cache, self.slot_mapping, self._beam_groups_dev,
            self._beam_G, self.H, self.D, self.bs, self.NB, self.scale, dtype_code(self.dtype),
            self.partition_tokens, self._beam_ws, self._beam_ws.numel())

    def beam_step(self, parents, new_k, new_v, q, stream=None):
        """One beam-search step after plan(): every sequence b continues from
        sequence parents[b] (fork: share the parent's blocks), appends one
        token (copy-on-write of its shared partial block first), then the
        device copies, writes and attends -- one native call
        (pkv_beam_step).  new_k/new_v/q: [S, H, D] 16-bit values, either
        host arrays of uint16 bit patterns (uploaded first) or device
        tensors (used in place, as a model on the device would produce
        them).  Scores and positions of decode_accumulate follow the parents.
        Returns the (src, dst) copy pairs of the step."""
        S, MB, H, D, bs = self.S, self.MB, self.H, self.D, self.bs
        if not hasattr(self, "beam_ctx"):
            self.beam_ctx = np.ascontiguousarray(self.context_lens_host, dtype=np.int32).copy()
            self.nblocks_host = np.ascontiguousarray(self.nblocks_host, dtype=np.int32)
            self.tables_host = np.ascontiguousarray(self.tables_host, dtype=np.int32)
            self._beam_buffers()
        sh = stream.cuda_stream if stream is not None else torch.cuda.current_stream().cuda_stream
        n = S * H * D
        if (isinstance(q, torch.Tensor) and isinstance(new_k, torch.Tensor)
                and isinstance(new_v, torch.Tensor) and q.is_cuda and new_k.is_cuda and new_v.is_cuda):
            for t in (q, new_k, new_v):
                if t.element_size() != 2 or t.numel() != n or not t.is_contiguous():
                    raise L.PkvError(L.PKV_ERR_INVALID_ARG,
                                     "beam_step: q/new_k/new_v must be contiguous [S, H, D] 16-bit")
            tq, tk, tv = q, new_k, new_v
        else:
            # host arrays: through a pinned buffer (two used in turn, each
            # guarded by an event) into the device token buffer
            slot = self._beam_slots[self._beam_turn]
            self._beam_turn ^= 1
            if slot["used"]:
                slot["done"].synchronize()
            u16 = slot["u16"].numpy().view(np.uint16)
            u16[:n] = np.asarray(q).ravel()
            u16[n:2 * n] = np.asarray(new_k).ravel()
            u16[2 * n:] = np.asarray(new_v).ravel()
            st = stream if stream is not None else torch.cuda.current_stream()
            with torch.cuda.stream(st):
                self._beam_dev_u16.copy_(slot["u16"], non_blocking=True)
            slot["done"].record(st)
            slot["used"] = True
            tok = self._beam_dev_u16.view(self.dtype)
            tq, tk, tv = (tok[:n].view(S, H, D), tok[n:2 * n].view(S, H, D),
                          tok[2 * n:].view(S, H, D))
        par = np.ascontiguousarray(parents, dtype=np.int32)
        t0 = time.perf_counter()
        P, at = self._beam_native.step(par.ctypes.data, tq.data_ptr(), tk.data_ptr(), tv.data_ptr(),
                                       sh)
        self.last_native_seconds = time.perf_counter() - t0
        if self._scored:
            with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
                self._scores_follow(par)
        # the pairs sit in the staging buffer the step used
        k = 0 if 0 <= at - self._beam_stg_base[0] < self._beam_inputs_bytes else 1
        o = at - self._beam_stg_base[k]
        pairs = self._beam_slots[k]["stg_np"][o:o + 16 * P].view(np.int64).reshape(P, 2).copy()
        self.pairs_host = pairs
        self.context_lens_host = self.beam_ctx
        self.T = S
        self.q, self.new_k, self.new_v = tq, tk, tv
        (self.block_tables, self.context_lens, self.pos,
         self.seq_idx) = self._beam_views
        return pairs

    def _scores_follow(self, parents):
        """After a beam step, on the current stream: every sequence has its
        parent's scores and positions, and one more token than its parent."""
        moved = np.flatnonzero(parents != np.arange(self.S))
        if len(moved):
            to = torch.from_numpy(moved).to(self.device)
            of = torch.from_numpy(parents[moved].astype(np.int64)).to(self.device)
            for t in (self.scores, self.positions, self.token_counts):
                t.index_copy_(0, to, t.index_select(0, of))
        self.token_counts.add_(1)

    def pack_inputs(self, on_host=()):
        """Move the step's inputs (q, new K/V, block tables, context lengths,
        token positions, copy pairs) into one buffer, at 256-byte aligned
        offsets, so that one copy uploads all of them.

        on_host: names among "q", "new_k", "new_v" that stay in the pinned
        host buffer, where the kernels read them directly (a GPU can address
        pinned host memory; on GB300 the reads cross the coherent NVLink-C2C
        link to the Grace CPU's memory).  They come first in the buffers and
        are not part of the upload.

        Returns (device buffer, pinned host buffer holding the same bytes,
        (device view, host view) of the bytes to upload each step).  The
        step's tensors become views of the device buffer (of the host buffer
        for `on_host`); a caller writes the next step's inputs into the host
        buffer at the same offsets (`input_offsets`) and uploads."""
        if self.block_tables is None:
            self.plan()
        tokens = ["q", "new_k", "new_v"]
        if any(n not in tokens for n in on_host):
            raise L.PkvError(L.PKV_ERR_INVALID_ARG, "pack_inputs: on_host takes q, new_k, new_v")
        names = [n for n in tokens if n in on_host] + [n for n in tokens if n not in on_host]
        names += ["block_tables", "context_lens", "seq_idx", "pos"]
        if self.pairs.numel():
            names.append("pairs")
        offsets, o = {}, 0
        for n in names:
            t = getattr(self, n)
            offsets[n] = o
            o = (o + t.numel() * t.element_size() + 255) // 256 * 256
        buf = torch.empty(max(o, 256), dtype=torch.uint8, device=self.device)
        views = {}
        for n in names:
            t = getattr(self, n)
            nbytes = t.numel() * t.element_size()
            views[n] = (t, nbytes)
            view = buf[offsets[n]:offsets[n] + nbytes].view(t.dtype).view(t.shape)
            view.copy_(t)
            setattr(self, n, view)
        host = buf.cpu().pin_memory()
        for n in on_host:
            t, nbytes = views[n]
            setattr(self, n, host[offsets[n]:offsets[n] + nbytes].view(t.dtype).view(t.shape))
        self.input_offsets = offsets
        first = offsets[names[len(on_host)]]  # the first uploaded input
        return buf, host, (buf[first:], host[first:])

    def pin_output(self):
        """The step's output goes to a pinned host tensor (returned), which
        becomes `out`: the kernels write it there directly, so no
        device-to-host copy follows the step."""
        host = torch.empty(self.out.shape, dtype=self.out.dtype).pin_memory()
        self.out = host
        return host

    def decode_shared_prefix(self, prefix_groups, stream=None):
        """decode() with the prefix of each group read once (see
        paged_attention_decode_shared_prefix); prefix_groups [G, 3] int32."""
        prefix_groups = np.asarray(prefix_groups, dtype=np.int32)
        if self._evicted:
            for first, n, tokens in prefix_groups.reshape(-1, 3).tolist():
                rows = self.tables_host[max(first, 0):max(first + n, 0), :-(-tokens // self.bs)]
                held = self.context_lens_host[max(first, 0):max(first + n, 0)]
                if (rows != rows[:1]).any() or (held < tokens).any():
                    _refuse("decode_shared_prefix: after evict() the sequences from "
                            f"{first} on no longer share {tokens} tokens")
        with _on(stream, self.device):  # the groups are read, and given back, on that stream
            g = torch.as_tensor(prefix_groups).to(self.device)
        return paged_attention_decode_shared_prefix(
            self.out, self.q, self.k_cache, self.v_cache, self.block_tables, self.context_lens, g,
            self.scale, self.max_context_len, self.partition_tokens, stream=stream)

    def _need_plan(self, who):
        if self.block_tables is None:
            _refuse(f"{who}: the step has no tables yet (plan() makes them)")

    def decode_window(self, window, sink_tokens=0, stream=None):
        """decode() over the first sink_tokens tokens and the last `window`
        of each context (see paged_attention_decode_window)."""
        self._need_plan("decode_window")
        if getattr(self, "_window_ws", None) is None:
            with _on(stream, self.device):
                self._window_ws = new_window_workspace(self.S, self.H, self.H, self.D, self.device)
        return paged_attention_decode_window(
            self.out, self.q, self.k_cache, self.v_cache, self.block_tables, self.context_lens,
            window, sink_tokens, self.scale, self.max_context_len, self._window_ws, stream)

    def decode_accumulate(self, stream=None):
        """decode() that also adds every token's attention weight to
        self.scores ([S, H, MB * bs] fp32, zero before the first call after
        plan(); see paged_attention_decode_accumulate), which evict() goes by.
        May be captured in a graph after a first call outside it."""
        self._need_plan("decode_accumulate")
        if not self._scored:
            # captured, every replay would zero the scores
            _no_capture("the first decode_accumulate, which makes the scores,", stream, self.device)
            with _on(stream, self.device):
                self._begin_scores()
        return paged_attention_decode_accumulate(
            self.out, self.scores, self.q, self.k_cache, self.v_cache, self.block_tables,
            self.context_lens, self.scale, self.max_context_len, self._accumulate_ws, stream)

    def _begin_scores(self):
        """No weights yet, on the current stream.  The tensors stay where they
        are and the workspace is for the longest context that the tables
        allow: a captured graph holds their addresses."""
        rows = (self.S, self.H, self.MB * self.bs)
        if self.scores is None:
            self.scores = torch.zeros(rows, device=self.device)
            self.positions = torch.full(rows, -1, dtype=torch.int32, device=self.device)
            self.token_counts = self.context_lens.clone()
            self._accumulate_ws = new_accumulate_workspace(self.S, self.H, self.H, self.D, rows[2], self.device)
        else:
            self.scores.zero_()
            self.positions.fill_(-1)
            self.token_counts.copy_(self.context_lens)
        self._scored = True

    def evict(self, budget, recent_tokens, sink_tokens=0, stream=None):
        """After decode_accumulate: keeps `budget` tokens of every longer
        sequence (see evict_tokens) and returns the blocks past them to the
        pool.  Blocks that will be written are copied first where they are
        shared (OutOfBlocks if the pool has no room for that: nothing is
        evicted then).  With a stream, the eviction runs there after what the
        current stream holds, and the current stream goes on after it.
        block_tables and context_lens are updated where they are: a captured
        graph reads the new ones.  Evicted rows own their blocks: prefix_groups
        and beam_groups are dropped, and a beam search that has begun with
        groups is refused.  Returns the number of blocks freed."""
        _no_capture("evict, whose tables are the host's,", stream, self.device)
        with _on(stream, self.device):
            return self._evict(budget, recent_tokens, sink_tokens)

    def _evict(self, budget, recent_tokens, sink_tokens):
        """evict() on the current stream, temporary tensors and all."""
        if not self._scored:
            _refuse("evict: there are no scores to go by (decode_accumulate makes them)")
        if budget < 1 or recent_tokens < 0 or sink_tokens < 0 or recent_tokens + sink_tokens > budget:
            _refuse("evict: budget must be >= 1 and hold the sinks and the recent tokens")
        over = [s for s in range(self.S) if self.context_lens_host[s] > budget]
        if over and hasattr(self, "beam_ctx") and self._beam_G:
            _refuse("evict: the beam search reads prefix groups that evicted sequences would no longer share")
        pairs = []
        try:
            for s in over:
                n = min(-(-budget // self.bs), int(self.nblocks_host[s]))
                pairs.append(self.allocator.unshare(self.tables_host[s], n))
        finally:  # rows that own their blocks now need the contents, also when the pool ran out
            pairs = np.concatenate(pairs) if pairs else np.empty((0, 2), dtype=np.int64)
            if len(pairs):
                check_copy_pairs(pairs, self.NB)
                self.block_tables.copy_(torch.from_numpy(self.tables_host))
                copy_blocks(self.k_cache, self.v_cache, torch.from_numpy(pairs).to(self.device))
        new_lens = torch.empty_like(self.context_lens)
        evict_tokens(self.k_cache, self.v_cache, self.scores, self.positions, self.block_tables,
                     self.context_lens, self.token_counts, new_lens, budget, recent_tokens,
                     sink_tokens, max_context_len=self.max_context_len)
        self.context_lens.copy_(new_lens)
        if hasattr(self, "beam_ctx"):  # the native search goes by this array
            self.context_lens_host = np.minimum(self.beam_ctx, budget, out=self.beam_ctx)
        else:
            self.context_lens_host = np.minimum(self.context_lens_host, budget).astype(np.int32)
        freed = 0
        for s in over:
            nb, n = self.allocator.truncate(self.tables_host[s], self.nblocks_host[s], budget, self.bs)
            self.nblocks_host[s] = nb
            freed += n
        if over:
            self._evicted = True
            self.prefix_groups = self.beam_groups = None
        self.block_tables.copy_(torch.from_numpy(self.tables_host))
        return freed

    def decode(self, stream=None):
        L.pkv_paged_attention_decode(self.out, self.q, self.k_cache, self.v_cache,
                                     self.block_tables, self.context_lens, self.S, self.H, self.D,
                                     self.bs, self.NB, self.MB, self.max_context_len, self.scale,
                                     dtype_code(self.dtype), self.partition_tokens, self.workspace,
                                     self.workspace.numel(), stream)
        return self.out


_driver = None


def _cu_graph_launch():
    """The driver's cuGraphLaunch(graph_exec, stream) -> CUresult."""
    global _driver
    if _driver is None:
        lib = ctypes.CDLL("libcuda.so.1")
        lib.cuGraphLaunch.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
        lib.cuGraphLaunch.restype = ctypes.c_int
        _driver = lib
    return _driver.cuGraphLaunch


class StepGraph:
    """One decode step captured in a CUDA graph, optionally with the copies
    of its inputs from pinned host memory and of its output back to it.

    h2d: [(device_tensor, pinned_host_tensor), ...] copied in first;
    d2h: [(pinned_host_tensor, device_tensor), ...] copied out last;
    fused: run the step through pkv_decode_step (DecodeStep.run).
    The step runs once eagerly before capture so that every per-device
    set-up of the library happens outside the capture.  replay() enqueues
    the whole step on the capture stream with one launch, as it was captured:
    block copies, writes and prefix groups included.  Like DecodeStep.run it is
    refused after an eviction; a step planned anew is captured anew.
    """

    def __init__(self, step: DecodeStep, stream: torch.cuda.Stream, h2d=(), d2h=(), fused=False):
        self.step = step
        self.stream = stream
        self._groups = step.prefix_groups  # read by every replay
        with torch.cuda.stream(stream):
            step.run(fused=fused)
        stream.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=stream):
            for dev, host in h2d:
                dev.copy_(host, non_blocking=True)
            step.run(fused=fused)
            for host, dev in d2h:
                host.copy_(dev, non_blocking=True)
        self._exec = ctypes.c_void_p(self.graph.raw_cuda_graph_exec())
        self._stream = ctypes.c_void_p(stream.cuda_stream)
        self._launch = _cu_graph_launch()

    def replay(self):
        """Enqueue the captured step on its stream (not torch's current one).

        One driver call: switching torch's current stream around
        CUDAGraph.replay() costs more host time per step than the launch."""
        if self.step._evicted:
            _refuse("replay: the step was written before an eviction moved it (plan it and capture it anew)")
        r = self._launch(self._exec, self._stream)
        if r != 0:
            raise L.PkvError(L.PKV_ERR_CUDA, f"cuGraphLaunch failed (CUresult {r})")
