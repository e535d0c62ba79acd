"""What a step's caches hold, token by token, as the definitions have it: the
rows of every sequence and KV head, followed through beam steps (fork and
append), accumulated weights and evictions.  One query head per KV head."""
from __future__ import annotations

import numpy as np

from oracle import bounded as B


class Rows:
    """rows[s][h]: K [n, D], V [n, D], score [n], position [n] of a cached sequence; seen[s]: tokens so far."""

    def __init__(self, k, v, tables, lens, scale):
        H = k.shape[2]
        self.scale, self.seen = scale, np.array(lens, dtype=np.int64)
        self.rows = []
        for s, n in enumerate(lens):
            at = B.rows_of(tables[s], range(int(n)), k.shape[1])
            kk, vv = k.reshape(-1, H, k.shape[3])[at], v.reshape(-1, H, v.shape[3])[at]
            self.rows.append([dict(k=kk[:, h], v=vv[:, h], score=np.zeros(n), pos=np.arange(n)) for h in range(H)])

    def beam_step(self, parents, k, v):
        """Sequence s continues parents[s] with the token k[s], v[s] [H, D]."""
        old, seen = self.rows, self.seen
        self.rows, self.seen = [], seen[parents] + 1
        for s, p in enumerate(parents):
            self.rows.append([dict(k=np.concatenate([r["k"], k[s, h][None]]), v=np.concatenate([r["v"], v[s, h][None]]),
                                   score=np.append(r["score"], 0.0), pos=np.append(r["pos"], seen[p]))
                              for h, r in enumerate(old[p])])

    def lens(self):
        return [len(r[0]["pos"]) for r in self.rows]

    def attend(self, q, add=False):
        """out [S, H, D] for the queries; add: every token's weight is added to its score."""
        out = np.zeros(q.shape)
        for s, heads in enumerate(self.rows):
            for h, r in enumerate(heads):
                z = self.scale * (r["k"] @ q[s, h])
                p = np.exp(z - z.max(initial=-np.inf))
                p /= p.sum()
                out[s, h] = p @ r["v"]
                if add:
                    r["score"] = r["score"] + p
        return out

    def evict(self, budget, recent, sinks):
        for s, heads in enumerate(self.rows):
            for r in heads:
                n = len(r["pos"])
                kept = B.evict_row(r["score"], r["pos"], n, int(self.seen[s]), budget, recent, sinks)
                if kept is not None:
                    source = np.array(kept[0])
                    assert kept[1] == r["pos"][source].tolist()
                    r.update({name: r[name][source] for name in ("k", "v", "score", "pos")})

    def check_state(self, st, atol):
        """The step's lengths, tables, caches, positions and scores are these rows' (scores to atol)."""
        lens = self.lens()
        assert np.array_equal(st.context_lens.cpu().numpy(), lens) and np.array_equal(st.context_lens_host, lens)
        tables = st.block_tables.cpu().numpy()
        assert np.array_equal(tables, st.tables_host)
        assert np.array_equal(st.nblocks_host, [-(-n // st.bs) for n in lens])
        k, v = st.k_cache.double().cpu().numpy(), st.v_cache.double().cpu().numpy()
        scores, pos = st.scores.double().cpu().numpy(), st.positions.cpu().numpy()
        H, D = k.shape[2:]
        for s, n in enumerate(lens):
            at = B.rows_of(tables[s], range(n), st.bs)
            for h, r in enumerate(self.rows[s]):
                assert np.array_equal(k.reshape(-1, H, D)[at, h], r["k"]), (s, h)
                assert np.array_equal(v.reshape(-1, H, D)[at, h], r["v"]), (s, h)
                stored = np.where(pos[s, h, :n] >= 0, pos[s, h, :n], self.seen[s] - n + np.arange(n))
                assert np.array_equal(stored, r["pos"]), (s, h)
                assert np.abs(scores[s, h, :n] - r["score"]).max(initial=0.0) <= atol
            assert (scores[s, :, n:] == 0).all() and (pos[s, :, n:] == -1).all()
        assert np.array_equal(st.token_counts.cpu().numpy(), self.seen)

    def take_scores(self, st):
        """Goes on from the step's scores, whose rounding may order two tokens the other way."""
        scores = st.scores.double().cpu().numpy()
        for s, heads in enumerate(self.rows):
            for h, r in enumerate(heads):
                r["score"] = scores[s, h, :len(r["pos"])].copy()
