"""Plain 64-bit implementations of the 8-bit cache and of drafted trees (numpy), and
their inputs: test infrastructure only."""
from __future__ import annotations

import numpy as np
import torch

from . import serving_ref as ref

E4M3 = ref.E4M3


# ------------------------------------------------------------------ 8-bit rows
def encode8(x, gs):
    """fp32 values -> e4m3 bytes of x / gs: the quotient rounded to fp32, a NaN held as 0."""
    x = np.asarray(x, np.float32)
    x = np.where(np.isnan(x), np.float32(0), x)
    with np.errstate(over="ignore"):
        y = (x / np.float32(gs)).astype(np.float32)
    mag = ref.nearest_even(np.minimum(np.abs(y).astype(np.float64), 448.0), E4M3)
    return (mag + 128 * np.signbit(y)).astype(np.uint8)


def decode8(b, gs):
    """What bytes stand for, in 64 bits."""
    v = np.append(E4M3, np.nan)[b & 127]
    return np.where(b & 128, -v, v) * float(np.float32(gs))


def as_e4m3(b):
    return torch.from_numpy(np.ascontiguousarray(b)).view(torch.float8_e4m3fn)


# ----------------------------------------------------------------------- trees
def random_tree(rng, T, shape="random"):
    """Parents of T drafted tokens."""
    if shape == "chain":
        return list(range(-1, T - 1))
    if shape == "flat":
        return [-1] * T
    if shape == "star":
        return [-1] + [0] * (T - 1)
    return [-1 if t == 0 or rng.random() < 0.1 else int(rng.integers(max(0, t - 10), t))
            for t in range(T)]


def lineage(parents, t, window=0):
    seen = []
    while t >= 0:
        seen.append(t)
        t = parents[t]
    return (seen[:window] if window else seen), len(seen) - 1


def tree_rows(trees, table, P, S, page, n_rows, words, window=0):
    """masks uint32 [n_rows, words], positions, slots of the drafted rows."""
    masks = np.zeros((n_rows, words), np.uint32)
    positions, slots = np.zeros(n_rows, np.int32), np.full(n_rows, -1, np.int64)
    r = 0
    for b, parents in enumerate(trees):
        for t in range(len(parents)):
            seen, depth = lineage(parents, t, window)
            for u in seen:
                masks[r, u // 32] |= np.uint32(1 << (u % 32))
            key = P + S[b] + t
            positions[r] = P + S[b] + depth
            page_id = int(table[b][key // page])
            slots[r] = -1 if page_id < 0 else page_id * page + key % page
            r += 1
    return masks, positions, slots


def accept(trees, draft, target, first, n_rows):
    path, counts, after = np.full(n_rows, -1, np.int32), [], []
    r = 0
    for b, parents in enumerate(trees):
        at, want, n = -1, int(first[b]), 0
        while True:
            fits = [t for t, p in enumerate(parents) if p == at and int(draft[r + t]) == want]
            if not fits:
                break
            at = fits[0]
            want = int(target[r + at])
            path[r + n] = at
            n += 1
        counts.append(n)
        after.append(want)
        r += len(parents)
    return path, np.array(counts, np.int32), np.array(after, np.int64)


# ------------------------------------------------------------------- attention
class Problem:
    """One attention problem on the host. kind: "bf16", "q4" or "q8" pools. trees None: the
    new tokens in causal order (or all keys); else per branch (S without its tokens, as
    drawn): a list of parents. masks "random": any bits instead of a tree's. Keys that no
    row sees are poisoned; table entries of pages without a seen key are no page."""

    def __init__(self, S, T, P, hq, hkv, page, kind="q8", trees=None, window=0, sinks=0,
                 causal=True, gs=1.0, seed=0, masks="tree", k_amp=1.0, q_amp=1.5, spare=3,
                 extra_words=0):
        rng = np.random.default_rng(seed)
        self.kind, self.P, self.hq, self.hkv, self.page = kind, P, hq, hkv, page
        self.T, self.window, self.sinks, self.causal, self.gs = list(T), window, sinks, causal, gs
        self.tree = trees is not None
        self.S = [s + t for s, t in zip(S, T)] if self.tree else list(S)  # as the call counts
        n_pre = -(-P // page)
        ends = [P + s for s in self.S]
        width = max([n_pre] + [-(-e // page) for e in ends]) + 1
        n_own = sum(max(-(-e // page), n_pre) - P // page for e in ends)
        n = n_pre + n_own + spare
        ids = rng.permutation(n).astype(np.int32)
        self.table, _, _ = ref.fork(ids[:n_pre], P, self.S, page, ids[n_pre:], 0, width)
        self.num_pages, R = n, sum(T)
        bf16 = lambda x: torch.from_numpy(np.asarray(x, np.float32)).bfloat16()  # noqa: E731
        self.q = bf16(rng.standard_normal((R, hq, 128)) * q_amp)
        k = rng.standard_normal((n, hkv, page, 128)) * k_amp
        v = rng.standard_normal((n, hkv, page, 128))
        self.scale = 128 ** -0.5
        # visibility, row by row
        self.masks = self.positions = None
        if self.tree:
            words = -(-max(list(T) + [1]) // 32) + extra_words
            self.masks, self.positions, _ = tree_rows(trees, self.table, P, S, page, R, words, window)
            if masks == "random":
                self.masks = rng.integers(0, 2 ** 32, size=self.masks.shape, dtype=np.uint64
                                          ).astype(np.uint32)
        self.see, r = [], 0
        for b, (s, t) in enumerate(zip(self.S, self.T)):
            n_all = P + s
            j = np.arange(n_all)
            for i in range(t):
                first = n_all - t
                if self.tree:
                    pos = int(self.positions[r])
                    m = np.ones(n_all, bool)
                    if window:
                        m = (j > pos - window) | (j < sinks)
                    bits = [(int(self.masks[r, u // 32]) >> (u % 32)) & 1 for u in range(t)]
                    m[first:] = np.array(bits, bool)
                    m[first + i] = True
                else:
                    pos = first + i
                    m = j <= pos if causal else j >= 0
                    if window:
                        m = m & ((j > pos - window) | (j < sinks))
                self.see.append((b, m))
                r += 1
        seen, used = np.zeros((n, page), bool), np.zeros(self.table.shape, bool)
        for b, m in self.see:
            j = np.nonzero(m)[0]
            seen[self.table[b][j // page], j % page] = True
            used[b, j // page] = True
        if self.tree:  # drafted rows are read whoever sees them, and must be finite
            for b, (s, t) in enumerate(zip(self.S, self.T)):
                j = np.arange(P + s - t, P + s)
                seen[self.table[b][j // page], j % page] = True
        used[:, :P // page] = used[:, :P // page].any(0)
        self.call_table = self.table
        if window:
            junk = np.where(rng.random(used.shape) < 0.5, -1, 1 << 30)
            self.call_table = np.where(used, self.table, junk).astype(np.int32)
        hidden = ~seen
        if kind == "q4":
            kw, kb = ref.encode(k * gs, gs)
            vw, vb = ref.encode(v * gs, gs)
            self.k64, self.v64 = ref.decode(kw, kb, gs), ref.decode(vw, vb, gs)
            for x in (kb, vb):
                x[np.broadcast_to(hidden[:, None, :], x.shape[:3])] = 0x7f
            self.pools = [torch.from_numpy(ref.pool_of(w, x)) for w, x in ((kw, kb), (vw, vb))]
        elif kind == "q8":
            kb, vb = encode8(k * gs, gs), encode8(v * gs, gs)
            self.k64, self.v64 = decode8(kb, gs), decode8(vb, gs)
            for x in (kb, vb):
                x[np.broadcast_to(hidden[:, None, :], x.shape[:3])] = 0x7f
            self.pools = [as_e4m3(kb), as_e4m3(vb)]
        else:
            pools = [bf16(k), bf16(v)]
            self.k64, self.v64 = (x.double().numpy() for x in pools)
            mask = torch.from_numpy(np.broadcast_to(hidden[:, None, :, None], k.shape).copy())
            self.pools = [x.masked_fill(mask, float("nan")) for x in pools]

    def reference(self):
        q, G = self.q.double().numpy(), self.hq // self.hkv
        R = q.shape[0]
        out, A, V = (np.zeros((R, self.hq, 128)) for _ in range(3))
        lse, E = np.full((R, self.hq), -np.inf), np.zeros((R, self.hq))
        K = np.zeros((R, self.hq))  # scale * largest |q| * largest sum |k|
        for r, (b, m) in enumerate(self.see):
            j = np.nonzero(m)[0]
            pages = self.table[b][j // self.page]
            for h in range(self.hkv):
                heads = slice(h * G, (h + 1) * G)
                kk, vv = self.k64[pages, h, j % self.page], self.v64[pages, h, j % self.page]
                x = q[r, heads] @ kk.T * self.scale
                top = x.max(-1, keepdims=True)
                p = np.exp(x - top)
                l = p.sum(-1, keepdims=True)
                out[r, heads] = p @ vv / l
                A[r, heads] = p @ np.abs(vv) / l
                V[r, heads] = np.abs(vv).sum(0)
                E[r, heads] = (np.abs(q[r, heads]) @ np.abs(kk).T).max(-1) * self.scale
                K[r, heads] = np.abs(q[r, heads]).max(-1) * np.abs(kk).sum(-1).max() * self.scale
                lse[r, heads] = (top + np.log(l))[:, 0]
        return out, lse, A, E, V, K

    def check(self, out, lse, what=""):
        """As serving_ref.check_attention; over 8-bit pools a score is a sum of 256 products
        (Q in two parts, whose magnitudes sum to at most 1 + 2^-3 of Q's: the upper part
        is at most 1 + 2^-4, the lower 2^-4 of it), and what the parts leave of a value of Q
        is at most 2^-17 of the row's largest: half of e4m3's smallest step, 2^-10, where
        the largest is 2^7 at least."""
        o64, l64, A, E, V, K = self.reference()
        f16 = self.kind != "bf16"
        if self.kind == "q8":
            e = 256 * 2.0 ** -23 * (1 + 2.0 ** -3) * E + 2.0 ** -17 * K
            e = e / (128 * 2.0 ** -23)  # check_attention multiplies by this
        else:
            e = E
        ref.check_attention(out, lse, (o64, l64, A, e, V), 2.0 ** -11 if f16 else 2.0 ** -8, what)

    def args(self, dev="cuda"):
        if not hasattr(self, "dev"):
            self.dev = [x.to(dev) for x in (self.q, *self.pools)] + \
                       [torch.from_numpy(self.call_table).to(dev)]
            if self.tree:
                self.dev += [torch.from_numpy(self.masks.view(np.int32)).to(dev),
                             torch.from_numpy(self.positions).to(dev)]
        return self.dev

    def run(self, out_dtype="f32", stream=None, **kw):
        from shared_prefix_fan_gb300 import binding
        q, k, v, table, *tree = self.args()
        a = (q, k, v, table, self.P, self.S, self.T, self.hq, self.hkv, self.page, self.scale)
        if self.tree:
            return binding.attn_tree(*a, tree[0], tree[1] if self.window else None, self.window,
                                     self.sinks, self.gs, self.gs, out_dtype=out_dtype,
                                     stream=stream, **kw)
        return binding.attn_q8(*a, self.causal, self.gs, self.gs, self.window, self.sinks,
                               out_dtype=out_dtype, stream=stream, **kw)
