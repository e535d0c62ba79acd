"""Workloads of the operators that bound a sequence's cache, and their plain forms.

Three operators over the paged KV cache ([NB, bs, Hkv, D] pools, block tables
[S, MB], H query heads in groups of H / Hkv per KV head):

  window      decode attention over the first `sinks` tokens and the last
              `window` tokens of each context
  accumulate  decode attention over the whole context that also adds each
              cached token's attention weight, summed over the query heads
              of its KV head, to a running score
  evict       keeps the `budget` best tokens per (sequence, KV head) -- the
              first `sinks` positions and the last `recent` ones always, then
              the highest scores -- and compacts cache, scores and positions

`own` selects what run() calls: False the plain torch forms (fp32), True the
library through paged_kv_cache_162_gb300.engine.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the smallest calls: 4 short requests on a small model; launch latency counts
        dict(name="window_tiny", op="window", S=4, H=4, Hkv=4, D=64, bs=16, dtype="f16", lens="uniform", lo=1, hi=100,
             window=32, sinks=4),
        # one long conversation, grouped heads: few rows, the context has to be split over the card
        dict(name="window_one_long", op="window", S=1, H=32, Hkv=8, D=128, bs=16, dtype="bf16", lens="uniform", lo=32768,
             hi=32768, window=4096, sinks=4),
        # a 7B-like layer, 64 requests, every head with its own K and V; ragged, a part of them below the window
        dict(name="window_batch64", op="window", S=64, H=32, Hkv=32, D=128, bs=16, dtype="f16", lens="uniform", lo=128,
             hi=2048, window=1000, sinks=4),
        # a large batch of long contexts with grouped heads, a window of odd size that starts inside blocks
        dict(name="window_gqa_batch", op="window", S=96, H=32, Hkv=8, D=128, bs=32, dtype="bf16", lens="uniform", lo=4001,
             hi=16384, window=4093, sinks=7),
        dict(name="accumulate_tiny", op="accumulate", S=4, H=4, Hkv=4, D=64, bs=16, dtype="f16", lens="uniform", lo=1,
             hi=100),
        # the 7B-like layer over whole contexts
        dict(name="accumulate_batch64", op="accumulate", S=64, H=32, Hkv=32, D=128, bs=16, dtype="f16", lens="uniform",
             lo=128, hi=2048),
        # continuous batching: 256 requests, lengths spread over a factor of 256, grouped heads
        dict(name="accumulate_gqa_mixed", op="accumulate", S=256, H=32, Hkv=8, D=128, bs=16, dtype="bf16",
             lens="lognormal", lo=16, hi=4096),
        # long contexts, few requests
        dict(name="accumulate_long", op="accumulate", S=8, H=32, Hkv=32, D=128, bs=16, dtype="f16", lens="uniform",
             lo=32768, hi=32768),
        # the smallest: a few short requests
        dict(name="evict_tiny", op="evict", S=4, H=4, Hkv=4, D=64, bs=16, dtype="f16", lens="uniform", lo=50, hi=100,
             budget=48, sinks=4, recent=16),
        # the steady state of decoding: one block of 16 tokens over the budget, evicted at once
        dict(name="evict_steady", op="evict", S=64, H=32, Hkv=8, D=128, bs=16, dtype="bf16", lens="uniform", lo=2064,
             hi=2064, budget=2048, sinks=4, recent=512),
        # ragged contexts of continuous batching, an odd budget, some already below it
        dict(name="evict_mixed", op="evict", S=256, H=32, Hkv=32, D=128, bs=16, dtype="bf16", lens="lognormal", lo=16,
             hi=4096, budget=500, sinks=4, recent=125),
        # after long prompts: most of the context goes
        dict(name="evict_after_prefill", op="evict", S=8, H=32, Hkv=32, D=128, bs=32, dtype="f16", lens="uniform",
             lo=32768, hi=32768, budget=4096, sinks=4, recent=1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "accumulate", "evict"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 12, 16) if g * Hkv <= 64])
    hi = _log_int(rng, 16, 32768)
    # at most 2**28 cached elements of K (0.5 GB), 256 requests
    most = max(1, min(256, 2 ** 28 // (hi * Hkv * D)))
    c = dict(op=op, S=_log_int(rng, 1, most), H=Hkv * group, Hkv=Hkv, D=D, bs=rng.choice([8, 16, 32, 64]),
             dtype=rng.choice(["f16", "bf16"]), lens=rng.choice(["uniform", "lognormal"]),
             lo=rng.choice([0, 1, max(1, hi // 8), hi]), hi=hi)
    if c["lens"] == "lognormal":
        c["lo"] = max(1, c["lo"])
    if op == "window":
        c.update(window=_log_int(rng, 1, 2 * hi), sinks=rng.choice([0, 1, 4, 5, 16, 33]))
    if op == "evict":
        budget = _log_int(rng, max(8, hi // 16), hi)
        sinks = rng.choice([0, 1, 4, 7])
        c.update(budget=budget, sinks=sinks, recent=rng.randint(1, budget - sinks))
    return c


def _lens(c):
    """The S context lengths, evenly spread quantiles of the case's distribution."""
    S = c["S"]
    u = (np.arange(S) + 0.5) / S
    if c["lens"] == "uniform":
        v = c["lo"] + u * (c["hi"] - c["lo"] + 1) - 0.5
    else:  # median at an eighth of the longest, sigma 1
        z = torch.special.ndtri(torch.from_numpy(u)).numpy()
        v = c["hi"] / 8 * np.exp(z)
    return np.clip(np.rint(v), c["lo"], c["hi"]).astype(np.int64)


def work(case):
    c, n = case, _lens(case)
    S, H, Hkv, D = c["S"], c["H"], c["Hkv"], c["D"]
    row = 2 * D * 2  # K and V of one token and head
    if c["op"] == "window":
        n = np.minimum(n, c["window"] + c["sinks"])
    if c["op"] in ("window", "accumulate"):
        tokens = float(n.sum())
        nbytes = tokens * Hkv * row + 2 * S * H * D * 2 + 4 * tokens / c["bs"] + 4 * S
        if c["op"] == "accumulate":
            nbytes += 8 * tokens * Hkv
        return {"bytes": nbytes, "flops": 4.0 * tokens * H * D}
    over = n > c["budget"]
    b = np.minimum(n, c["budget"])
    # every entry's score and position is read and written (kept or reset)
    entries = float(n.sum()) * Hkv
    # scores are independent of the age: the unprotected tokens past the budget stay with even probability
    tail = (n - b).astype(np.float64)
    recent = np.minimum(c["recent"], tail)
    middle = np.maximum(n - c["sinks"] - c["recent"], 1)
    stay = np.maximum(c["budget"] - c["sinks"] - c["recent"], 0) / middle
    moves = float((over * (recent + (tail - recent) * np.minimum(stay, 1))).sum()) * Hkv
    return {"bytes": 16 * entries + moves * 2 * row + 12 * S, "flops": entries}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    rng = np.random.default_rng(seed)
    S, H, Hkv, D, bs = c["S"], c["H"], c["Hkv"], c["D"], c["bs"]
    dt = _DT[c["dtype"]]
    n = rng.permutation(_lens(c))
    MB = max(1, -(-int(c["hi"]) // bs))
    blocks = -(-n // bs)
    NB = int(blocks.sum() * 1.1) + 1
    ids = rng.permutation(NB)
    tables = np.full((S, MB), -1, np.int32)
    at = 0
    for s in range(S):
        tables[s, :blocks[s]] = ids[at:at + blocks[s]]
        at += blocks[s]
    st = dict(case=c, scale=1.0 / math.sqrt(D), max_len=max(1, int(c["hi"])),
              k_cache=torch.randn((NB, bs, Hkv, D), generator=g, device=dev, dtype=dt),
              v_cache=torch.randn((NB, bs, Hkv, D), generator=g, device=dev, dtype=dt),
              block_tables=torch.from_numpy(tables).to(dev),
              context_lens=torch.from_numpy(n.astype(np.int32)).to(dev))
    if c["op"] in ("window", "accumulate"):
        st["q"] = torch.randn((S, H, D), generator=g, device=dev, dtype=dt)
        st["out"] = torch.empty((S, H, D), device=dev, dtype=dt)
    if c["op"] in ("accumulate", "evict"):
        cap = MB * bs
        live = torch.arange(cap, device=dev) < st["context_lens"][:, None, None]
        st["scores"] = torch.randn((S, Hkv, cap), generator=g, device=dev).exp_() * live
    if c["op"] == "evict":
        # half of the sequences have been evicted before: their older entries hold shuffled positions
        pos = torch.full((S, Hkv, cap), -1, dtype=torch.int32)
        seen = n.copy()
        for s in range(S):
            old = min(int(n[s]), c["budget"])
            if s % 2 and old:
                seen[s] = n[s] + 3 * old
                stored = np.sort(rng.permutation(4 * old)[:old])
                pos[s, :, :old] = torch.from_numpy(rng.permuted(np.tile(stored, (Hkv, 1)), axis=1).astype(np.int32))
        st["positions"] = pos.to(dev)
        st["token_counts"] = torch.from_numpy(seen.astype(np.int32)).to(dev)
        st["scores_out"] = torch.zeros_like(st["scores"])
        st["positions_out"] = torch.full_like(st["positions"], -1)
        st["new_lens"] = torch.zeros_like(st["context_lens"])
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return {"window": _plain_window, "accumulate": _plain_accumulate, "evict": _plain_evict}[c["op"]](state, c)


def _own(st, c):
    from paged_kv_cache_162_gb300 import engine as E
    if "workspace" not in st:  # kept with the state, as a serving loop keeps it
        S, H, Hkv, D = c["S"], c["H"], c["Hkv"], c["D"]
        if c["op"] == "window":
            st["workspace"] = E.new_window_workspace(S, H, Hkv, D)
        elif c["op"] == "accumulate":
            st["workspace"] = E.new_accumulate_workspace(S, H, Hkv, D, st["max_len"])
        else:
            st["workspace"] = E.new_evict_workspace(S, Hkv, c["budget"])
    ws = st["workspace"]
    if c["op"] == "window":
        return E.paged_attention_decode_window(st["out"], st["q"], st["k_cache"], st["v_cache"], st["block_tables"],
                                               st["context_lens"], c["window"], c["sinks"], st["scale"],
                                               max_context_len=st["max_len"], workspace=ws)
    if c["op"] == "accumulate":
        out = E.paged_attention_decode_accumulate(st["out"], st["scores"], st["q"], st["k_cache"], st["v_cache"],
                                                  st["block_tables"], st["context_lens"], st["scale"],
                                                  max_context_len=st["max_len"], workspace=ws)
        return {"out": out, "scores": st["scores"]}
    E.evict_tokens(st["k_cache"], st["v_cache"], st["scores"], st["positions"], st["block_tables"],
                   st["context_lens"], st["token_counts"], st["new_lens"], c["budget"], c["recent"], c["sinks"],
                   scores_out=st["scores_out"], positions_out=st["positions_out"], workspace=ws)
    return _evicted(st)


def _evicted(st):
    return {"k": st["k_cache"], "v": st["v_cache"], "scores": st["scores_out"], "positions": st["positions_out"],
            "lens": st["new_lens"]}


def _attend(st, c, token, valid):
    """Attention of each sequence's query over the tokens token[s, :] where
    valid[s, :]; returns (out fp32 [S, Hkv, G, D], weights [S, Hkv, G, V])."""
    S, H, Hkv, D, bs = c["S"], c["H"], c["Hkv"], c["D"], c["bs"]
    token = torch.where(valid, token, 0)
    slot = torch.where(valid, st["block_tables"].long().gather(1, token // bs) * bs + token % bs, 0)
    k = st["k_cache"].view(-1, Hkv, D)[slot].float()
    v = st["v_cache"].view(-1, Hkv, D)[slot].float()
    q = st["q"].float().view(S, Hkv, H // Hkv, D)
    z = torch.einsum("sgrd,svgd->sgrv", q, k) * st["scale"]
    z = torch.where(valid[:, None, None, :], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    return torch.einsum("sgrv,svgd->sgrd", p, v), p


def _plain_window(st, c):
    n = st["context_lens"].long()[:, None]
    most = min(st["max_len"], c["window"] + c["sinks"])
    v = torch.arange(most, device=n.device)[None, :]
    seen = n.clamp(max=c["window"] + c["sinks"])
    token = torch.where(v < c["sinks"], v, v + (n - seen))
    o, _ = _attend(st, c, token, v < seen)
    st["out"].copy_(o.reshape(st["out"].shape))
    return st["out"]


def _plain_accumulate(st, c):
    n = st["context_lens"].long()[:, None]
    v = torch.arange(st["max_len"], device=n.device)[None, :].expand(c["S"], -1)
    o, p = _attend(st, c, v, v < n)
    st["out"].copy_(o.reshape(st["out"].shape))
    st["scores"][:, :, :st["max_len"]] += p.sum(2)
    return {"out": st["out"], "scores": st["scores"]}


def _plain_evict(st, c):
    Hkv, bs = c["Hkv"], c["bs"]
    n = st["context_lens"].long()[:, None, None]
    seen = st["token_counts"].long()[:, None, None]
    score, stored = st["scores"], st["positions"].long()
    j = torch.arange(score.shape[2], device=n.device).expand(score.shape)
    live = j < n
    pos = torch.where(stored >= 0, stored, seen - n + j)
    kept_always = live & ((pos < c["sinks"]) | (pos >= seen - c["recent"]))
    kind = torch.where(kept_always, 0, torch.where(live, 1, 2))
    # order: protected tokens, the others by falling score, ties by index
    order = torch.sort(torch.where(score.isnan(), -math.inf, score), dim=2, descending=True, stable=True).indices
    order = order.gather(2, torch.sort(kind.gather(2, order), dim=2, stable=True).indices)
    b = n.clamp(max=c["budget"])
    keep = torch.zeros_like(live).scatter_(2, order, j < b)
    holes = torch.nonzero(~keep & (j < b), as_tuple=True)
    movers = torch.nonzero(keep & (j >= b), as_tuple=True)
    table = st["block_tables"].long()
    to = table[holes[0], holes[2] // bs] * bs + holes[2] % bs
    of = table[movers[0], movers[2] // bs] * bs + movers[2] % bs
    for name in ("k_cache", "v_cache"):
        rows = st[name].view(-1, Hkv, c["D"])
        rows[to, holes[1]] = rows[of, movers[1]]
    evicted = n > b
    new_score = score.clone()
    new_score[holes] = score[movers]
    new_pos = torch.where(evicted, pos, stored)
    new_pos[holes] = pos[movers]
    gone = live & (j >= b)
    st["scores_out"].copy_(torch.where(live, new_score.masked_fill(gone, 0.0), st["scores_out"]))
    st["positions_out"].copy_(torch.where(live, new_pos.masked_fill(gone, -1), st["positions_out"].long()))
    st["new_lens"].copy_(b.view(-1))
    return _evicted(st)


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The outputs from the definitions, one sequence at a time in 64 bits."""
    c = case
    st = prepare(c, seed)
    n = st["context_lens"].tolist()
    tables = st["block_tables"].tolist()
    if c["op"] == "evict":
        return _exact_evict(st, c, n, tables)
    S, H, Hkv, D, bs = c["S"], c["H"], c["Hkv"], c["D"], c["bs"]
    out = torch.zeros((S, H, D), dtype=torch.float64)
    scores = st["scores"].double().cpu() if c["op"] == "accumulate" else None
    for s in range(S):
        seen = [t for t in range(n[s]) if t < c["sinks"] or t >= n[s] - c["window"]] if c["op"] == "window" \
            else list(range(n[s]))
        if not seen:
            continue
        rows = torch.tensor([tables[s][t // bs] * bs + t % bs for t in seen], device="cuda")
        k = st["k_cache"].view(-1, Hkv, D).index_select(0, rows).double().permute(1, 2, 0)
        v = st["v_cache"].view(-1, Hkv, D).index_select(0, rows).double().permute(1, 0, 2)
        w = torch.softmax(torch.bmm(st["q"][s].double().view(Hkv, H // Hkv, D), k) * st["scale"], -1)
        out[s] = torch.bmm(w, v).reshape(H, D).cpu()
        if scores is not None:
            scores[s, :, :n[s]] += w.sum(1).cpu()
    return out if scores is None else {"out": out, "scores": scores}


def _exact_evict(st, c, n, tables):
    Hkv, D, bs, budget = c["Hkv"], c["D"], c["bs"], c["budget"]
    score, stored, seen = st["scores"].cpu().numpy(), st["positions"].cpu().numpy(), st["token_counts"].tolist()
    new_score, new_pos = np.zeros_like(score, dtype=np.float64), np.full_like(stored, -1)
    new_lens = np.array([min(x, budget) for x in n], np.int32)
    moves = []  # (source row, target row, head)
    for s, m in enumerate(n):
        table = np.array(tables[s])
        for h in range(Hkv):
            value, pos = score[s, h, :m].astype(np.float64), stored[s, h, :m].astype(np.int64)
            if m <= budget:
                new_score[s, h, :m], new_pos[s, h, :m] = value, pos
                continue
            pos = np.where(pos < 0, seen[s] - m + np.arange(m), pos)
            safe = (pos < c["sinks"]) | (pos >= seen[s] - c["recent"])
            stay = np.lexsort((np.arange(m), -np.nan_to_num(value, nan=-np.inf, posinf=np.inf, neginf=-np.inf),
                               ~safe))[:budget]
            kept = np.zeros(m, bool)
            kept[stay] = True
            source = np.arange(budget)
            source[~kept[:budget]] = budget + np.flatnonzero(kept[budget:])
            new_score[s, h, :budget], new_pos[s, h, :budget] = value[source], pos[source]
            to = np.flatnonzero(source != np.arange(budget))
            row = lambda t: table[t // bs].astype(np.int64) * bs + t % bs  # noqa: E731
            moves.append(np.stack([row(source[to]), row(to), np.full(len(to), h)]))
    k, v = st["k_cache"].view(-1, Hkv, D).clone(), st["v_cache"].view(-1, Hkv, D).clone()
    if moves:
        of, to, head = torch.from_numpy(np.concatenate(moves, 1)).cuda()
        k[to, head], v[to, head] = k[of, head], v[of, head]
    shape = st["k_cache"].shape
    return {"k": k.view(shape).double(), "v": v.view(shape).double(), "scores": torch.from_numpy(new_score),
            "positions": torch.from_numpy(new_pos), "lens": torch.from_numpy(new_lens)}
