"""Inputs and bounds shared by the tests of the rotating appends and the 4-bit cache."""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import q4 as Q

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}   # half a step, relative
E32 = 2.0 ** -24
NAN_BITS = {"f16": 0x7e01, "bf16": 0x7fc1}


def tensor(bits, dtype):
    """uint16 bit patterns as a 16-bit CPU tensor."""
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(DT[dtype])


def bits_of(t) -> np.ndarray:
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def tables_for(rng, lens, bs, extra=3, MB=None):
    need = [-(-int(n) // bs) for n in lens]
    MB = MB or max(1, max(need, default=1))
    NB = sum(need) + extra
    ids = rng.permutation(NB)
    tables = np.full((len(lens), MB), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = ids[at:at + n]
        at += n
    return tables, NB


# ---------------------------------------------------------------- attention
def pool_for(rng, NB, bs, Hkv, D, dtype, live, spread=1.0):
    """A 4-bit pool of quantised normal rows (each group scaled by 2^(spread *
    N(0, 1))); tokens that are not live [NB * bs] have NaN steps and centres
    and random codes."""
    x = rng.standard_normal((NB, bs, Hkv, D // 64, 64))
    x = (x + 0.3 * rng.standard_normal(x.shape[:-1] + (1,))) * np.exp2(spread * rng.standard_normal(x.shape[:-1] + (1,)))
    step, centre, code = Q.quantise(x.reshape(NB, bs, Hkv, D), dtype)
    dead = ~live.reshape(NB, bs)
    step, centre = step.copy(), centre.copy()
    step[dead] = centre[dead] = NAN_BITS[dtype]
    code[dead] = rng.integers(0, 16, code[dead].shape)
    return Q.pack(step, centre, code)


def attend_case(seed, S, H, Hkv, D, bs, dtype, lens, MB=None, spread=1.0):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    tables, NB = tables_for(rng, lens, bs, MB=MB)
    live = np.zeros(NB * bs, bool)
    for s, n in enumerate(lens):
        pos = np.arange(n)
        live[tables[s, pos // bs].astype(np.int64) * bs + pos % bs] = True
    return dict(S=S, H=H, Hkv=Hkv, D=D, bs=bs, dtype=dtype, lens=lens, tables=tables, scale=1 / math.sqrt(D),
                q=Q.narrow(rng.standard_normal((S, H, D)), dtype), k=pool_for(rng, NB, bs, Hkv, D, dtype, live, spread),
                v=pool_for(rng, NB, bs, Hkv, D, dtype, live, spread))


def attend_reference(c, own_units=False):
    """(out, bound) [S, H, D] in 64 bits.  The bound, with u = half a step of the
    output type and e = 2^-24:
     * a logit z_j = scale sum_r (step_r (sum_d q_d code_d - 8 sum_d q_d) + centre_r
       sum_d q_d): the products are exact, the sums of 64 in fp32 with truncation, 2 e
       each, partial sums at most sum_d |q_d| (|code_d - 8| + 16), and a few more
       roundings: 144 e Z, Z = scale max_j sum_d |q_d| (step (|code_d - 8| + 16) + |centre|);
       a q as fp16 loses what is below 2^-24 of the head's largest: e Zq, Zq with
       that largest for every q_d.  A weight errs by twice that (the maximum errs too)
       and 2^-22 of the exponential; the normaliser by as much; n / 8 sums per lane
       and n / 16 products' sums with 4 e each:
         w = 4 (144 e Z + e Zq) + 2^-21 + (n / 8 + 100) 4 e
     * a weight times V's step enters as one fp16 number (bf16 output: rounded by r =
       2^-11) or as two (fp16: r = 2^-22), or 2^-33 of the largest step off where it
       is below 2^-14 in units of 2^-8 (at most 8 codes up).
       With A = sum_j p_j (step_j |code_j - 8| + |centre_j|), A' the same with 16 more codes:
         |out - ref| <= u |ref| + (1 + u) (A r + A' w + n 2^-30 max step) + 2^-25
       own_units, for inputs where that is far too much: the units of the weights are
       each head's and group's own, so that what a weight is small beside is the
       largest p_j step_j of that head and group; Z and Zq are each token's own, with 4 e
       max |z| for the exponent's sum; below the least normal number a rounding is 2^-25
       (fp16) or 2^-134 (bf16):
         |out - ref| <= u |ref| + (1 + u) (A r + sum_j p_j (a_j + A16) w_j + n 2^-30 max_j p_j step_j)
       and that, a_j = step_j (|code_j - 8| + 16) + |centre_j|, A16 = sum_j p_j a_j"""
    S, H, Hkv, D, bs, dtype = (c[x] for x in ("S", "H", "Hkv", "D", "bs", "dtype"))
    G, u = H // Hkv, U[dtype]
    out, bound = np.zeros((S, H, D)), np.zeros((S, H, D))
    q = Q.widen(c["q"], dtype)
    kv = []
    for pool in (c["k"], c["v"]):
        step, centre, code = Q.parts(pool, D)
        s, a = (np.repeat(Q.widen(x, dtype), 64, -1).reshape(-1, Hkv, D) for x in (step, centre))
        kv.append((s, a, code.reshape(-1, Hkv, D) - 8))
    for i in range(S):
        n = int(c["lens"][i])
        if n == 0:
            bound[i] = 2.0 ** -25
            continue
        pos = np.arange(n)
        rows = c["tables"][i, pos // bs].astype(np.int64) * bs + pos % bs
        (ks, ka, kc), (vs, va, vc) = (tuple(y[rows].transpose(1, 0, 2) for y in x) for x in kv)
        k, v = ka + ks * kc, va + vs * vc
        kmag, vmag = np.abs(ka) + ks * (np.abs(kc) + 16), np.abs(va) + vs * np.abs(vc)
        r16 = 2.0 ** -22 if dtype == "f16" else 2.0 ** -11
        qq = q[i].reshape(Hkv, G, D)
        z = c["scale"] * (qq @ k.transpose(0, 2, 1))
        p = np.exp(z - z.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        Z = abs(c["scale"]) * (np.abs(qq) @ kmag.transpose(0, 2, 1)).max(-1)
        Zq = abs(c["scale"]) * (np.abs(qq).max(-1) * kmag.sum(-1).max(-1)[:, None])
        w = 4 * (144 * E32 * Z + E32 * Zq) + 2.0 ** -21 + (n / 8 + 100) * 4 * E32
        A, A16, r = p @ vmag, p @ (vmag + 16 * vs), p @ v
        if own_units:
            Z = abs(c["scale"]) * (np.abs(qq) @ kmag.transpose(0, 2, 1))
            Zq = abs(c["scale"]) * np.abs(qq).max(-1)[..., None] * kmag.sum(-1)[:, None]
            w = 2 * (144 * E32 * Z + E32 * Zq) + 4 * E32 * np.abs(z).max() + 2.0 ** -21 + (n / 8 + 100) * 4 * E32
            off = (p * w) @ (vmag + 16 * vs) + (p * w).sum(-1, keepdims=True) * A16
            small = n * 2.0 ** -30 * np.stack([(p[..., None] * vs[:, None, :, g:g + 64]).max(2) for g in range(0, D, 64)], 2)
            small = small.reshape(Hkv, G, D)
            b = u * np.abs(r) + (1 + u) * (A * r16 + off + small) + (2.0 ** -25 if dtype == "f16" else 2.0 ** -134)
        else:
            b = u * np.abs(r) + (1 + u) * (A * r16 + A16 * w[..., None] + n * 2.0 ** -30 * vs.max()) + 2.0 ** -25
        out[i], bound[i] = r.reshape(H, D), b.reshape(H, D)
    return out, bound


def on_gpu(c):
    d = {k: torch.from_numpy(c[k]).cuda() for k in ("tables", "lens", "k", "v")}
    d["q"] = tensor(c["q"], c["dtype"]).cuda()
    return d


# ---------------------------------------------------------------- appends
def append_case(seed, S, H, Hkv, D, bs, dtype, new, before=None, R=None, interleaved=False, pad=0, fused=False,
                shift=0, MB=None, base=10000.0, big=1.0):
    """Tokens in a shuffled order: sequence s gets new[s] tokens behind before[s]."""
    rng = np.random.default_rng(seed)
    new = np.asarray(new)
    before = np.zeros(S, int) if before is None else np.asarray(before)
    R = D if R is None else R
    lens = before + new
    tables, NB = tables_for(rng, lens, bs, MB=MB)
    seq = np.concatenate([np.repeat(np.arange(S), new), np.zeros(pad, int)]).astype(np.int32)
    pos = np.concatenate([np.arange(b, e) for b, e in zip(before, lens)] + [np.full(pad, -1)]).astype(np.int32)
    order = rng.permutation(len(seq))
    seq, pos = seq[order], pos[order]
    T = len(seq)
    rows = {k: Q.narrow(big * rng.standard_normal((T, h, D)), dtype) for k, h in (("key", Hkv), ("value", Hkv), ("query", H))}
    P = int(lens.max(initial=0)) + shift + 1
    angle = np.arange(P)[:, None] * base ** (-np.arange(0, R, 2) / max(R, 1))
    table = np.concatenate([np.cos(angle), np.sin(angle)], -1).astype(np.float32)
    return dict(S=S, H=H, Hkv=Hkv, D=D, bs=bs, NB=NB, dtype=dtype, R=R, interleaved=interleaved, T=T, tables=tables,
                seq=seq, pos=pos, shift=shift, table=table, fused=fused, **rows)


def rotated(c, name, wide):
    """(rows [T, heads, D] after the rotation in `wide`, the sum of its products' sizes in 64 bits)."""
    x = Q.widen(c[name], c["dtype"]).astype(wide)
    mag = np.abs(x.astype(np.float64))
    if c["R"] == 0:
        return x, mag
    y = x.copy()
    h = c["R"] // 2
    for t in range(c["T"]):
        if c["pos"][t] < 0:
            continue
        row = c["table"][c["pos"][t] + c["shift"]].astype(wide)
        y[t] = Q.rotate(x[t], row[:h], row[h:], c["interleaved"])
        cos, sin = np.abs(row[:h]).astype(np.float64), np.abs(row[h:]).astype(np.float64)
        # a cos + b sin and b cos + a sin of the sizes: the first dims of one turn, the second of the other
        mag[t] = np.maximum(Q.rotate(mag[t], cos, -sin, c["interleaved"]), Q.rotate(mag[t], cos, sin, c["interleaved"]))
    return y, mag


def append_on_gpu(c):
    """Device tensors of the call: fused, key, value and query are slices of one projection."""
    d = {k: tensor(c[k], c["dtype"]).cuda() for k in ("key", "value", "query")}
    if c["fused"]:
        T = c["T"]
        flat = torch.cat([d[k].reshape(T, -1) for k in ("query", "key", "value")], -1)
        parts = flat.split([d[k][0].numel() for k in ("query", "key", "value")], -1)
        d.update({k: x.unflatten(-1, (-1, c["D"])) for k, x in zip(("query", "key", "value"), parts)})
    d["tables"], d["seq"], d["pos"] = (torch.from_numpy(c[k]).cuda() for k in ("tables", "seq", "pos"))
    d["table"] = torch.from_numpy(c["table"]).cuda() if c["R"] else None
    d["turn"] = torch.where(d["pos"] >= 0, d["pos"] + c["shift"], d["pos"]) if c["shift"] else None
    d["slots"] = torch.full((c["T"],), -7, dtype=torch.int64, device="cuda")
    return d
