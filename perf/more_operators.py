"""Workloads of the rotating appends and of the 4-bit cache, and their plain forms.

Four operators over the paged KV cache (block tables [S, MB], H query heads in
groups of H / Hkv per KV head):

  append   new tokens' slots by address translation, rotary position encoding
           of their queries and keys, keys and values written into the 16-bit
           caches [NB, bs, Hkv, D]
  append4  the same into a cache held in 4 bits; the rows written are then
           read back (gather4's call) as the 16-bit values they stand for
  gather4  the rows of given slots of a 4-bit cache as 16-bit values
  attend4  decode attention over a 4-bit cache

The 4-bit cache: uint8 [NB, Hkv, bs, RB], RB = D/2 + D/16 bytes per (token, KV
head), K and V apart.  A row's D elements go in groups of 64; element i of a
group stands for centre + step * (code - 8), code in 0..15, with one step and
one centre per group in the model's 16-bit type:
  step = (max - min) / 15, centre = (8 max + 7 min) / 15, each rounded once;
  code = round((x - centre) / step) + 8 within 0..15, 8 where step is 0.
Memory order of a (block, head): for every 8 tokens first their codes (8 rows
of D/2 bytes; byte j holds elements 2j, low nibble, and 2j + 1; the 16-byte
chunks of row r are permuted, chunk c at place c ^ (r >> 1) % 4 for D = 128 and
c ^ (r >> 2) % 2 for D = 64), then their (step, centre) pairs, groups in order.

`own` selects what run() calls: False the plain torch forms, True the library
through paged_kv_cache_162_gb300.engine.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 4 requests on a small model; launch latency counts
        dict(name="append_tiny", op="append", S=4, before=100, new_lo=1, new_hi=1, H=4, Hkv=4, D=64, bs=16, dtype="f16",
             rotary=64, interleaved=False, shift=0, pad=0, fused=False),
        # one decode step of continuous batching, grouped heads, q, k and v slices of one projection, the batch padded
        dict(name="append_decode", op="append", S=250, before=4095, new_lo=1, new_hi=1, H=32, Hkv=8, D=128, bs=16,
             dtype="bf16", rotary=128, interleaved=False, shift=0, pad=6, fused=True),
        # prompts of a 7B-like layer, ragged, every head with its own K and V, neighbouring pairs
        dict(name="append_prefill", op="append", S=16, before=0, new_lo=320, new_hi=1727, H=32, Hkv=32, D=128, bs=16,
             dtype="f16", rotary=128, interleaved=True, shift=0, pad=0, fused=True),
        dict(name="append4_tiny", op="append4", S=4, before=100, new_lo=1, new_hi=1, H=4, Hkv=4, D=64, bs=16,
             dtype="f16", rotary=64, interleaved=False, shift=0, pad=0, fused=False),
        dict(name="append4_decode", op="append4", S=250, before=4095, new_lo=1, new_hi=1, H=32, Hkv=8, D=128, bs=16,
             dtype="bf16", rotary=128, interleaved=False, shift=0, pad=6, fused=True),
        # long prompts, grouped heads, half of the dims rotated, large blocks
        dict(name="append4_prefill", op="append4", S=8, before=0, new_lo=1000, new_hi=4001, H=32, Hkv=8, D=128, bs=32,
             dtype="bf16", rotary=64, interleaved=False, shift=0, pad=0, fused=True),
        # the cached prefix of one request, read back for the next chunk of its prompt
        dict(name="gather4_prefix", op="gather4", S=1, lens="uniform", lo=1024, hi=1024, Hkv=8, D=128, bs=16,
             dtype="bf16"),
        # whole contexts on their way into a 16-bit cache
        dict(name="gather4_batch", op="gather4", S=64, lens="uniform", lo=128, hi=2048, Hkv=32, D=128, bs=16,
             dtype="f16"),
        # 4 short requests on a small model
        dict(name="attend4_tiny", op="attend4", S=4, H=4, Hkv=4, D=64, bs=16, dtype="f16", lens="uniform", lo=1, hi=100),
        # one long conversation, grouped heads: few rows, the context has to be split over the card
        dict(name="attend4_one_long", op="attend4", S=1, H=32, Hkv=8, D=128, bs=16, dtype="bf16", lens="uniform",
             lo=32768, hi=32768),
        # continuous batching: 256 requests, lengths spread over a factor of 256, grouped heads
        dict(name="attend4_gqa_mixed", op="attend4", S=256, H=32, Hkv=8, D=128, bs=16, dtype="bf16", lens="lognormal",
             lo=16, hi=4096),
        # a large batch of long contexts of a 7B-like layer, every head with its own K and V
        dict(name="attend4_long_batch", op="attend4", S=32, H=32, Hkv=32, D=128, bs=32, dtype="f16", lens="uniform",
             lo=4001, hi=16384),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append4", "gather4", "attend4", "attend4"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 12, 16) if g * Hkv <= 64])
    c = dict(op=op, Hkv=Hkv, D=D, bs=rng.choice([8, 16, 32, 64]), dtype=rng.choice(["f16", "bf16"]))
    if op in ("append", "append4"):
        new = _log_int(rng, 1, 2048) if rng.random() < 0.5 else 1
        most = max(1, min(256, 2 ** 26 // (new * max(Hkv, 8) * D)))
        c.update(S=_log_int(rng, 1, most), before=_log_int(rng, 1, 4096) - 1, new_lo=max(1, new // 3), new_hi=new,
                 H=Hkv * group, rotary=rng.choice([0, 16, 32, 64, D, D]), interleaved=rng.random() < 0.5,
                 shift=rng.choice([0, 0, 1000]), pad=rng.choice([0, 0, 1, 7]), fused=rng.random() < 0.5)
        return c
    hi = _log_int(rng, 16, 32768)
    # at most 2**28 cached elements of K, 256 requests
    most = max(1, min(256, 2 ** 28 // (hi * Hkv * D)))
    c.update(S=_log_int(rng, 1, most), lens=rng.choice(["uniform", "lognormal"]), hi=hi)
    c["lo"] = rng.choice([1, max(1, hi // 8), hi] if c["lens"] == "lognormal" or op == "gather4"
                         else [0, 1, max(1, hi // 8), hi])
    if op == "attend4":
        c["H"] = Hkv * group
    return c


def _row_bytes(D):
    return D // 2 + D // 16


def _quantiles(lo, hi, S):
    u = (np.arange(S) + 0.5) / S
    return np.clip(np.rint(lo + u * (hi - lo + 1) - 0.5), lo, hi).astype(np.int64)


def _lens(c):
    """The S context lengths, evenly spread quantiles of the case's distribution."""
    if c["lens"] == "uniform":
        return _quantiles(c["lo"], c["hi"], c["S"])
    u = (np.arange(c["S"]) + 0.5) / c["S"]  # median at an eighth of the longest, sigma 1
    z = torch.special.ndtri(torch.from_numpy(u)).numpy()
    return np.clip(np.rint(c["hi"] / 8 * np.exp(z)), c["lo"], c["hi"]).astype(np.int64)


def work(case):
    c = case
    Hkv, D, RB = c["Hkv"], c["D"], _row_bytes(c["D"])
    if c["op"] in ("append", "append4"):
        new = _quantiles(c["new_lo"], c["new_hi"], c["S"])
        T = float(new.sum())
        before = _quantiles(0, c["before"], c["S"])
        places = float(min((before + new).max(), T))  # distinct rows of the rotary table, at most
        row = 2 * D
        nbytes = T * (2 * Hkv * row + (2 * c["H"] * row if c["rotary"] else 0) + 20) + places * 4 * c["rotary"]
        if c["op"] == "append":
            nbytes += T * 2 * Hkv * row
            return {"bytes": nbytes, "flops": 3 * T * (c["H"] + Hkv) * c["rotary"]}
        # the 4-bit rows are written, then read and written as 16-bit values
        nbytes += T * Hkv * (2 * RB + 2 * RB + 2 * row)
        return {"bytes": nbytes, "flops": 3 * T * (c["H"] + Hkv) * c["rotary"] + 6 * T * 2 * Hkv * D}
    tokens = float(_lens(c).sum())
    if c["op"] == "gather4":
        return {"bytes": tokens * (Hkv * (2 * RB + 4 * D) + 8), "flops": 2 * tokens * 2 * Hkv * D}
    S, H = c["S"], c["H"]
    return {"bytes": tokens * Hkv * 2 * RB + 2 * S * H * D * 2 + 4 * tokens / c["bs"] + 4 * S,
            "flops": 4.0 * tokens * H * D}


# ---------------------------------------------------------------- the 4-bit layout
def _chunk_places(D, device):
    """[8, D/32]: where row r's 16-byte chunk c is."""
    r = torch.arange(8, device=device)[:, None]
    c = torch.arange(D // 32, device=device)[None, :]
    return c ^ ((r >> 1) & 3 if D == 128 else (r >> 2) & 1)


def _quantize(x, dt, wide=torch.float32):
    """(step, centre [..., D/64] in dt, codes [..., D] as `wide`) of rows [..., D]."""
    g = x.to(wide).unflatten(-1, (-1, 64))
    hi, lo = g.amax(-1), g.amin(-1)
    step = ((hi - lo) / 15).to(dt)
    centre = ((8 * hi + 7 * lo) / 15).to(dt)
    s, a = step.to(wide)[..., None], centre.to(wide)[..., None]
    code = torch.where(s > 0, torch.round((g - a) / torch.where(s > 0, s, 1.0)).clamp(-8, 7), 0.0) + 8
    return step, centre, code.flatten(-2)


def _pack(x, dt):
    """Rows [n, Hkv, 8, D] (8 tokens) as cache bytes [n, Hkv, 8 * RB]."""
    D = x.shape[-1]
    step, centre, code = _quantize(x, dt)
    code = code.to(torch.uint8)
    rows = (code[..., 0::2] | (code[..., 1::2] << 4)).unflatten(-1, (D // 32, 16))
    places = _chunk_places(D, x.device)[:, :, None].expand(rows.shape)
    rows = torch.zeros_like(rows).scatter_(-2, places, rows)
    pairs = torch.stack([step, centre], -1).contiguous().view(torch.uint8)
    return torch.cat([rows.flatten(-3), pairs.flatten(-3)], -1)


def _unpack(cache, D, dt):
    """A 4-bit cache's values, fp32 [NB, bs, Hkv, D]."""
    NB, Hkv, bs, RB = cache.shape
    unit = cache.view(NB, Hkv, bs // 8, 8 * RB)
    rows = unit[..., :4 * D].unflatten(-1, (8, D // 32, 16))
    places = _chunk_places(D, cache.device)[:, :, None].expand(rows.shape)
    rows = rows.gather(-2, places).flatten(-2)
    code = torch.stack([rows & 15, rows >> 4], -1).flatten(-2).float()
    pairs = unit[..., 4 * D:].contiguous().view(dt).unflatten(-1, (8, D // 64, 2)).float()
    value = pairs[..., 1:] + pairs[..., :1] * (code.unflatten(-1, (D // 64, 64)) - 8)
    return value.flatten(-2).reshape(NB, Hkv, bs, D).transpose(1, 2)


# ---------------------------------------------------------------- inputs
def _tables(rng, blocks, MB):
    """Block tables with `blocks[s]` random blocks each, and the pool's size."""
    NB = int(blocks.sum() * 1.1) + 1
    ids = rng.permutation(NB)
    tables = np.full((len(blocks), MB), -1, np.int32)
    at = 0
    for s, n in enumerate(blocks):
        tables[s, :n] = ids[at:at + n]
        at += n
    return tables, NB


def _filled4(NB, Hkv, bs, D, dt, g):
    """A 4-bit cache of quantised normal values, some blocks at a time."""
    RB = _row_bytes(D)
    cache = torch.empty((NB, Hkv, bs, RB), dtype=torch.uint8, device="cuda")
    n = max(1, 2 ** 26 // (Hkv * bs * D))
    for i in range(0, NB, n):
        m = min(n, NB - i)
        x = torch.randn((m, Hkv, bs // 8, 8, D), generator=g, device="cuda")
        cache[i:i + m] = _pack(x.transpose(1, 2).flatten(0, 1), dt).view(m, bs // 8, Hkv, 8 * RB) \
            .transpose(1, 2).reshape(m, Hkv, bs, RB)
    return cache


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    S, Hkv, D, bs = c["S"], c["Hkv"], c["D"], c["bs"]
    dt = _DT[c["dtype"]]
    if c["op"] in ("append", "append4"):
        return _prepare_append(c, g, rng, dt)
    n = rng.permutation(_lens(c))
    MB = max(1, -(-int(c["hi"]) // bs))
    tables, NB = _tables(rng, -(-n // bs), MB)
    st = dict(case=c, k_cache=_filled4(NB, Hkv, bs, D, dt, g), v_cache=_filled4(NB, Hkv, bs, D, dt, g))
    if c["op"] == "gather4":
        pos = np.concatenate([np.arange(m) for m in n])
        seq = np.repeat(np.arange(S), n)
        slots = tables[seq, pos // bs].astype(np.int64) * bs + pos % bs
        st["slots"] = torch.from_numpy(slots).cuda()
        st["key"] = torch.zeros((len(slots), Hkv, D), dtype=dt, device="cuda")
        st["value"] = torch.zeros_like(st["key"])
        return st
    st.update(scale=1.0 / math.sqrt(D), max_len=max(1, int(c["hi"])), block_tables=torch.from_numpy(tables).cuda(),
              context_lens=torch.from_numpy(n.astype(np.int32)).cuda(),
              q=torch.randn((S, c["H"], D), generator=g, device="cuda", dtype=dt),
              out=torch.empty((S, c["H"], D), dtype=dt, device="cuda"))
    return st


def _prepare_append(c, g, rng, dt):
    S, H, Hkv, D, bs, R = c["S"], c["H"], c["Hkv"], c["D"], c["bs"], c["rotary"]
    new = rng.permutation(_quantiles(c["new_lo"], c["new_hi"], S))
    before = rng.permutation(_quantiles(0, c["before"], S))
    n = before + new
    MB = int(-(-n.max() // bs))
    tables, NB = _tables(rng, -(-n // bs), MB)
    # the batch's tokens sequence by sequence, then padding (position -1)
    seq = np.concatenate([np.repeat(np.arange(S), new), np.zeros(c["pad"], np.int64)])
    pos = np.concatenate([np.arange(b, e) for b, e in zip(before, n)] + [np.full(c["pad"], -1)])
    T = len(seq)
    if c["fused"]:
        qkv = torch.randn((T, (H + 2 * Hkv) * D), generator=g, device="cuda", dtype=dt)
        q, k, v = (x.unflatten(-1, (-1, D)) for x in qkv.split([H * D, Hkv * D, Hkv * D], -1))
    else:
        q, k, v = (torch.randn((T, h, D), generator=g, device="cuda", dtype=dt) for h in (H, Hkv, Hkv))
    st = dict(case=c, query=q, key=k, value=v, query_out=torch.zeros((T, H, D), dtype=dt, device="cuda"),
              block_tables=torch.from_numpy(tables).cuda(),
              seq_idx=torch.from_numpy(seq.astype(np.int32)).cuda(), pos=torch.from_numpy(pos.astype(np.int32)).cuda(),
              slots=torch.zeros(T, dtype=torch.int64, device="cuda"))
    # after an eviction a token's place in the cache is behind its position
    st["rotary_pos"] = torch.where(st["pos"] >= 0, st["pos"] + c["shift"], st["pos"]) if c["shift"] else None
    # cos of the R / 2 angles, then sin
    P = int(n.max()) + c["shift"]
    angle = torch.arange(P, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))[None, :]
    st["table"] = torch.cat([angle.cos(), angle.sin()], -1).float().cuda() if R else None
    for name in ("k_cache", "v_cache"):
        if c["op"] == "append":
            st[name] = torch.randn((NB, bs, Hkv, D), generator=g, device="cuda", dtype=dt)
        else:
            st[name] = _filled4(NB, Hkv, bs, D, dt, g)
            st[name[0] + "_rows"] = torch.zeros((T, Hkv, D), dtype=dt, device="cuda")
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return {"append": _plain_append, "append4": _plain_append4, "gather4": _plain_gather4,
            "attend4": _plain_attend4}[c["op"]](state, c)


def _own(st, c):
    from paged_kv_cache_162_gb300 import engine as E
    if c["op"] == "append":
        E.rotate_and_cache(st["key"], st["value"], st["k_cache"], st["v_cache"], st["block_tables"], st["seq_idx"],
                           st["pos"], st["slots"], st["table"], query=st["query"], query_out=st["query_out"],
                           rotary_pos=st["rotary_pos"], interleaved=c["interleaved"])
        return {"query": st["query_out"], "k": st["k_cache"], "v": st["v_cache"], "slots": st["slots"]}
    if c["op"] == "append4":
        E.rotate_and_cache_q4(st["key"], st["value"], st["k_cache"], st["v_cache"], st["block_tables"], st["seq_idx"],
                              st["pos"], st["slots"], st["table"], query=st["query"], query_out=st["query_out"],
                              rotary_pos=st["rotary_pos"], interleaved=c["interleaved"])
        E.gather_cache_q4(st["k_rows"], st["v_rows"], st["k_cache"], st["v_cache"], st["slots"])
        return {"query": st["query_out"], "k": st["k_rows"], "v": st["v_rows"], "slots": st["slots"]}
    if c["op"] == "gather4":
        E.gather_cache_q4(st["key"], st["value"], st["k_cache"], st["v_cache"], st["slots"])
        return {"key": st["key"], "value": st["value"]}
    if "workspace" not in st:  # kept with the state, as a serving loop keeps it
        st["workspace"] = E.new_q4_workspace(c["S"], c["H"], c["Hkv"], c["D"])
    return E.paged_attention_decode_q4(st["out"], st["q"], st["k_cache"], st["v_cache"], st["block_tables"],
                                       st["context_lens"], st["scale"], max_context_len=st["max_len"],
                                       workspace=st["workspace"])


def _rotate(x, cos, sin, c):
    """Rows [T, heads, D] (fp32) with their first `rotary` dims rotated."""
    R = c["rotary"]
    head, rest = x[..., :R], x[..., R:]
    if c["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)
    a, b = head[..., :R // 2], head[..., R // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _places(st, c):
    """(slots, tokens that are none of the padding, their rotated keys); the queries are done."""
    pos = st["pos"].long()
    live = pos >= 0
    at = pos.clamp(min=0)
    block = st["block_tables"].long()[st["seq_idx"].long(), at // c["bs"]]
    st["slots"].copy_(torch.where(live, block * c["bs"] + at % c["bs"], -1))
    key, query = st["key"].float(), st["query"].float()
    if c["rotary"]:
        turn = st["table"][(at if st["rotary_pos"] is None else st["rotary_pos"].long().clamp(min=0))][:, None, :]
        cos, sin = turn[..., :c["rotary"] // 2], turn[..., c["rotary"] // 2:]
        key, query = _rotate(key, cos, sin, c), _rotate(query, cos, sin, c)
    st["query_out"].copy_(torch.where(live[:, None, None], query, st["query_out"].float()))
    return st["slots"][live], live, key[live]


def _plain_append(st, c):
    slots, live, key = _places(st, c)
    st["k_cache"].view(-1, c["Hkv"], c["D"])[slots] = key.to(st["k_cache"].dtype)
    st["v_cache"].view(-1, c["Hkv"], c["D"])[slots] = st["value"][live]
    return {"query": st["query_out"], "k": st["k_cache"], "v": st["v_cache"], "slots": st["slots"]}


def _plain_append4(st, c):
    slots, live, key = _places(st, c)
    bs, D, Hkv, dt = c["bs"], c["D"], c["Hkv"], _DT[c["dtype"]]
    RB = _row_bytes(D)
    row, block, unit = slots % 8, slots // bs, slots % bs // 8
    places = _chunk_places(D, slots.device)[row]
    for name, x in (("k", key), ("v", st["value"][live].float())):
        step, centre, code = _quantize(x, dt)
        code = code.to(torch.uint8)
        byte = (code[..., 0::2] | (code[..., 1::2] << 4)).unflatten(-1, (D // 32, 16))
        byte = torch.zeros_like(byte).scatter_(-2, places[:, None, :, None].expand(byte.shape), byte).flatten(-2)
        pair = torch.stack([step, centre], -1).contiguous().view(torch.uint8).flatten(-2)
        unit_of = st[name + "_cache"].view(-1, Hkv, bs // 8, 8 * RB)
        at = (torch.arange(D // 2, device=slots.device) + (row * (D // 2))[:, None])[:, None, :]
        heads = torch.arange(Hkv, device=slots.device)[None, :, None]
        unit_of[block[:, None, None], heads, unit[:, None, None], at] = byte
        at = (4 * D + torch.arange(D // 16, device=slots.device) + (row * (D // 16))[:, None])[:, None, :]
        unit_of[block[:, None, None], heads, unit[:, None, None], at] = pair
        s, a = step.float()[..., None], centre.float()[..., None]
        st[name + "_rows"][live] = (a + s * (code.float().unflatten(-1, (-1, 64)) - 8)).flatten(-2).to(dt)
    return {"query": st["query_out"], "k": st["k_rows"], "v": st["v_rows"], "slots": st["slots"]}


def _plain_gather4(st, c):
    for name, out in (("k_cache", "key"), ("v_cache", "value")):
        st[out].copy_(_unpack(st[name], c["D"], _DT[c["dtype"]]).flatten(0, 1)[st["slots"]])
    return {"key": st["key"], "value": st["value"]}


def _plain_attend4(st, c):
    S, H, Hkv, D, bs = c["S"], c["H"], c["Hkv"], c["D"], c["bs"]
    n = st["context_lens"].long()[:, None]
    token = torch.arange(st["max_len"], device=n.device)[None, :]
    seen = token < n
    slot = torch.where(seen, st["block_tables"].long().gather(1, (token // bs).expand(S, -1)) * bs + token % bs, 0)
    k = _unpack(st["k_cache"], D, _DT[c["dtype"]]).flatten(0, 1)[slot]
    z = torch.einsum("sgrd,svgd->sgrv", st["q"].float().view(S, Hkv, H // Hkv, D), k) * st["scale"]
    del k
    z = torch.where(seen[:, None, None, :], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    v = _unpack(st["v_cache"], D, _DT[c["dtype"]]).flatten(0, 1)[slot]
    st["out"].copy_(torch.einsum("sgrv,svgd->sgrd", p, v).reshape(S, H, D))
    return st["out"]


# ---------------------------------------------------------------- in 64 bits
def _read64(cache, slots, D, dt):
    """Rows of slots [n] of a 4-bit cache by the layout's definition: float64 [n, Hkv, D]."""
    NB, Hkv, bs, RB = cache.shape
    flat = cache.view(NB, Hkv, bs * RB)
    block, off = slots // bs, slots % bs
    unit, r = off // 8, off % 8
    d = torch.arange(D, device=slots.device)
    chunk = d // 32
    place = chunk[None] ^ (((r >> 1) & 3) if D == 128 else ((r >> 2) & 1))[:, None]
    byte = (unit * 8 * RB + r * (D // 2))[:, None] + place * 16 + (d % 32 // 2)[None]
    code = (flat[block[:, None], :, byte].long() >> (d % 2 * 4)[None, :, None]) & 15  # [n, D, Hkv]
    par = (unit * 8 * RB + 4 * D + r * (D // 16))[:, None] + (d // 64 * 4)[None]
    pair = torch.stack([flat[block[:, None], :, par + i] for i in range(4)], -1).contiguous().view(dt).double()
    return (pair[..., 1] + pair[..., 0] * (code - 8).double()).transpose(1, 2)


def exact(case, seed):
    """The outputs from the definitions, in 64 bits."""
    c = case
    st = prepare(c, seed)
    Hkv, D, bs, dt = c["Hkv"], c["D"], c["bs"], _DT[c["dtype"]]
    if c["op"] == "gather4":
        return {"key": _read64(st["k_cache"], st["slots"], D, dt), "value": _read64(st["v_cache"], st["slots"], D, dt)}
    if c["op"] == "attend4":
        S, H = c["S"], c["H"]
        out = torch.zeros((S, H, D), dtype=torch.float64)
        tables, lens = st["block_tables"].long(), st["context_lens"].tolist()
        for s, n in enumerate(lens):
            if n == 0:
                continue
            j = torch.arange(n, device="cuda")
            slots = tables[s, j // bs] * bs + j % bs
            k, v = (_read64(st[x], slots, D, dt) for x in ("k_cache", "v_cache"))
            w = torch.softmax(torch.bmm(st["q"][s].double().view(Hkv, H // Hkv, D), k.permute(1, 2, 0)) * st["scale"], -1)
            out[s] = torch.bmm(w, v.permute(1, 0, 2)).reshape(H, D).cpu()
        return out
    live = st["pos"] >= 0
    pos, seq = st["pos"].long()[live], st["seq_idx"].long()[live]
    slots = st["block_tables"].long()[seq, pos // bs] * bs + pos % bs
    R = c["rotary"]

    def turned(x):
        y = x[live].double()
        if R:
            t = st["table"].double()[(pos if st["rotary_pos"] is None else st["rotary_pos"].long()[live])][:, None, :]
            first = torch.arange(0, R, 2, device="cuda") if c["interleaved"] else torch.arange(R // 2, device="cuda")
            second = first + (1 if c["interleaved"] else R // 2)
            a, b = y[..., first].clone(), y[..., second].clone()
            y[..., first] = a * t[..., :R // 2] - b * t[..., R // 2:]
            y[..., second] = a * t[..., R // 2:] + b * t[..., :R // 2]
        return y

    query = torch.zeros((len(live), c["H"], D), dtype=torch.float64, device="cuda")
    query[live] = turned(st["query"])
    where = torch.full((len(live),), -1, dtype=torch.int64, device="cuda")
    where[live] = slots
    if c["op"] == "append":
        k, v = st["k_cache"].double().view(-1, Hkv, D), st["v_cache"].double().view(-1, Hkv, D)
        k[slots], v[slots] = turned(st["key"]), st["value"][live].double()
        shape = st["k_cache"].shape
        return {"query": query, "k": k.view(shape), "v": v.view(shape), "slots": where}
    got = {"query": query, "slots": where}
    for name, x in (("k", turned(st["key"])), ("v", st["value"][live].double())):
        rows = torch.zeros((len(live), Hkv, D), dtype=torch.float64, device="cuda")
        parts = []
        for lo in range(0, D, 64):
            part = x[..., lo:lo + 64]
            top, low = part.max(-1, keepdim=True).values, part.min(-1, keepdim=True).values
            step, centre = ((top - low) / 15).to(dt).double(), ((8 * top + 7 * low) / 15).to(dt).double()
            code = ((part - centre) / step).round().clamp(-8, 7).nan_to_num(0.0)
            parts.append(centre + step * torch.where(step > 0, code, 0.0))
        rows[live] = torch.cat(parts, -1)
        got[name] = rows
    return got
