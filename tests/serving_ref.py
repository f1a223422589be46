"""Plain 64-bit implementations of the serving operators (numpy), and their
inputs: test infrastructure only."""
from __future__ import annotations

import numpy as np
import torch

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# e4m3 values of bytes 0x00 .. 0x7e (no infinity; 0x7f is NaN)
E4M3 = np.array([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
                 for e in range(16) for m in range(8)][:127])
# value i of 8 sits in bits 16 (i % 2) + 4 (i / 2) of its word
SHIFT = np.array([16 * (i % 2) + 4 * (i // 2) for i in range(8)], dtype=np.uint32)


def nearest_even(a, grid):
    """Index of the nearest grid value, ties to the even index, clamped at the top."""
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    d = (a - grid[hi - 1]) - (grid[hi] - a)
    return np.where((d > 0) | ((d == 0) & (hi % 2 == 0)), hi, hi - 1)


def encode(x, gs):
    """fp32 rows [..., 128] -> (code words uint32 [..., 16], scale bytes [..., 8]).
    The two quotients and the scale are rounded to fp32, and a NaN is held as 0, as
    defined."""
    x = np.asarray(x, np.float32)
    x = np.where(np.isnan(x), np.float32(0), x)
    gs = np.float32(gs)
    g = x.reshape(*x.shape[:-1], 8, 16)
    top = np.abs(g).max(-1)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        q = np.minimum((top / (np.float32(6) * gs)).astype(np.float64), 448.0)
    byte = nearest_even(q, E4M3)
    den = (E4M3[byte].astype(np.float32) * gs)[..., None]
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        y = np.where(den > 0, g / den, np.float32(0)).astype(np.float32)
    mag = nearest_even(np.minimum(np.abs(y).astype(np.float64), 6.0), LEVELS)
    code = (mag + 8 * np.signbit(y)).astype(np.uint32).reshape(*x.shape[:-1], 16, 8)
    words = np.zeros(code.shape[:-1], np.uint32)
    for i in range(8):
        words |= code[..., i] << SHIFT[i]
    return words, byte.astype(np.uint8)


def decode(words, byte, gs):
    """What they stand for, in 64 bits (the product of scale and gs in fp32)."""
    code = (words[..., None] >> SHIFT) & 15
    v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    den = (np.append(E4M3, np.nan)[byte & 127].astype(np.float32) * np.float32(gs))
    return v.reshape(*words.shape[:-1], 128) * np.repeat(den.astype(np.float64), 16, -1)


def pool_of(words, byte):
    """[pages, H, page, 16] words and [pages, H, page, 8] scales -> pool bytes."""
    n, h, page, _ = words.shape
    return np.concatenate([words.astype("<u4").view(np.uint8).reshape(n, h, page * 64),
                           byte.reshape(n, h, page * 8)], axis=-1)


def parts_of(pool, page):
    n, h, _ = pool.shape
    codes = np.ascontiguousarray(pool[..., :page * 64])
    return (codes.view("<u4").reshape(n, h, page, 16),
            pool[..., page * 64:].reshape(n, h, page, 8))


def fork(prefix, P, S, page, free, used, width):
    table = np.full((len(S), width), -1, np.int32)
    cow = np.full((len(S), 2), -1, np.int32)
    for b, s in enumerate(S):
        need = max(-(-(P + s) // page), -(-P // page))
        table[b, :P // page] = prefix[:P // page]
        n = need - P // page
        table[b, P // page:need] = free[used:used + n]
        if P % page:
            cow[b] = prefix[P // page], table[b, P // page]
        used += n
    return table, cow, used


def extend(table, P, S, A, page, free, used, n_slots):
    table, slots, r = table.copy(), np.full(n_slots, -1, np.int64), 0
    for b, (s, a) in enumerate(zip(S, A)):
        held, need = -(-(P + s) // page), -(-(P + s + a) // page)
        table[b, held:need] = free[used:used + need - held]
        used += need - held
        for t in range(a):
            pos = P + s + t
            slots[r] = int(table[b, pos // page]) * page + pos % page
            r += 1
    return table, slots, used


def attention(q, k, v, table, P, S, T, page, scale, causal=True, window=0, sinks=0):
    """q [R, H_q, 128], k / v [pages, H_kv, page, 128], all float64. Returns (out,
    lse, A, E, V): A = sum p |v| / sum p per output, E = the largest scale * sum
    |q k| of a visible key per (row, head), V = sum |v| over the visible keys: what
    the error bounds scale with."""
    R, hq, d = q.shape
    hkv = k.shape[1]
    G = hq // hkv
    out, A, V = np.zeros((R, hq, d)), np.zeros((R, hq, d)), np.zeros((R, hq, d))
    lse, E = np.full((R, hq), -np.inf), np.zeros((R, hq))
    r = 0
    for b, (s, t) in enumerate(zip(S, T)):
        n = P + s
        for i in range(t):
            pos = n - t + i
            j = np.arange(n)
            see = j <= pos if causal else j >= 0
            if window:
                see = see & ((j > pos - window) | (j < sinks))
            j = j[see]
            pages = table[b][j // page]
            for h in range(hkv):
                kk, vv = k[pages, h, j % page], v[pages, h, j % page]
                x = q[r, h * G:(h + 1) * G] @ kk.T * scale
                E[r, h * G:(h + 1) * G] = (np.abs(q[r, h * G:(h + 1) * G]) @ np.abs(kk).T
                                           ).max(-1) * scale
                m = x.max(-1, keepdims=True)
                p = np.exp(x - m)
                l = p.sum(-1, keepdims=True)
                out[r, h * G:(h + 1) * G] = p @ vv / l
                A[r, h * G:(h + 1) * G] = p @ np.abs(vv) / l
                V[r, h * G:(h + 1) * G] = np.abs(vv).sum(0)
                lse[r, h * G:(h + 1) * G] = (m + np.log(l))[:, 0]
            r += 1
    return out, lse, A, E, V


def check_attention(out, lse, ref, p_step, what=""):
    """|out - ref| and |lse - ref| against bounds derived from the arithmetic:
    - a score is a sum of 128 products accumulated in fp32, off by at most 128 *
      2^-23 * sum |q k| * scale =: e (2^-23: an accumulator may truncate), and its
      scaling, subtraction and ex2 add at most 2^-20 relative to every p while
      |x - m| stays below 64; p and the sum of p each move by that: 2 (e + 2^-20);
    - p is rounded once to p_step for the product with V, relative to A; as f16
      (p_step 2^-11) it carries a factor 2^7 and f16's smallest step is 2^-24, so a
      small p is off by up to 2^-25 / 2^7 = 2^-32 of the row's reference, where the
      sum of p is at least 1 (the key that set the reference has p = 1): 2^-32 V;
    - sums of p and of p v, rescales and the merge of partials: 2^-16 covers
      fewer than 128 fp32 additions per tile and a few per merge;
    - the output's own rounding: half a step of its type, relative to it."""
    o64, l64, A, E, V = ref
    e = 128 * 2.0 ** -23 * E
    rel = 2 * (e + 2.0 ** -20) + p_step + 2.0 ** -16
    tol = A * rel[..., None] + (2.0 ** -32 * V if p_step == 2.0 ** -11 else 0.0)
    step = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[out.dtype]
    tol = tol + step * (np.abs(o64) + tol)
    d = np.abs(out.double().cpu().numpy() - o64)
    assert np.isfinite(d).all(), f"{what}: non-finite output"
    worst = float((d / np.maximum(tol, 1e-30)).max()) if d.size else 0.0
    assert worst <= 1.0, f"{what}: out is {worst:.2f} times its bound off"
    if lse is not None:
        dl = np.abs(lse.double().cpu().numpy() - l64)
        tl = e + 2.0 ** -16 + 2.0 ** -22 * np.abs(l64)
        assert (dl <= tl).all(), f"{what}: lse {float((dl / tl).max()):.2f} times its bound off"


class Problem:
    """Random inputs of one attention problem on the host: permuted pages, page
    tables from the reference fork, pages nobody sees poisoned."""

    def __init__(self, S, T, P, hq, hkv, page, causal=True, window=0, sinks=0, q4=False, gs=1.0,
                 seed=0, k_amp=1.0, spare=3):
        rng = np.random.default_rng(seed)
        self.S, self.T, self.P, self.hq, self.hkv, self.page = list(S), list(T), P, hq, hkv, page
        self.causal, self.window, self.sinks, self.q4, self.gs = causal, window, sinks, q4, gs
        n_pre = -(-P // page)
        width = max([n_pre] + [-(-(P + s) // page) for s in S]) + 1
        n_own = sum(max(-(-(P + s) // page), n_pre) - P // page for s in S)
        n = n_pre + n_own + spare
        ids = rng.permutation(n).astype(np.int32)
        self.table, _, _ = fork(ids[:n_pre], P, S, page, ids[n_pre:], 0, width)
        self.num_pages, R = n, sum(T)
        to_bf16 = lambda x: torch.from_numpy(x.astype(np.float32)).bfloat16()  # noqa: E731
        self.q = to_bf16(rng.standard_normal((R, hq, 128)) * 1.5)
        k = rng.standard_normal((n, hkv, page, 128)) * k_amp
        v = rng.standard_normal((n, hkv, page, 128))
        # slots that no row sees hold NaN; entries whose page nobody sees are no page
        seen = np.zeros((n, page), bool)
        used = np.zeros(self.table.shape, bool)
        for b, (s, t) in enumerate(zip(S, T)):
            for i in range(t):
                pos = P + s - t + i
                j = np.arange(P + s)
                see = j <= pos if causal else j >= 0
                if window:
                    see = see & ((j > pos - window) | (j < sinks))
                j = j[see]
                seen[self.table[b][j // page], j % page] = True
                used[b, j // page] = True
        n_full = P // page
        used[:, :n_full] = used[:, :n_full].any(0)  # row 0 stands for the whole prefix pages
        self.hidden = ~seen
        self.call_table = np.where(used, self.table, np.where(rng.random(used.shape) < 0.5, -1,
                                                              1 << 30)).astype(np.int32)
        if not window:
            self.call_table = self.table
        if q4:
            kw, kb = encode(k * gs, gs)
            vw, vb = encode(v * gs, gs)
            self.k64, self.v64 = decode(kw, kb, gs), decode(vw, vb, gs)
            for b_ in (kb, vb):
                b_[np.broadcast_to(self.hidden[:, None, :], b_.shape[:3])] = 0x7f
            self.k_pool, self.v_pool = (torch.from_numpy(pool_of(w, b_))
                                        for w, b_ in ((kw, kb), (vw, vb)))
        else:
            self.k_pool, self.v_pool = to_bf16(k), to_bf16(v)
            self.k64, self.v64 = self.k_pool.double().numpy(), self.v_pool.double().numpy()
            mask = torch.from_numpy(np.broadcast_to(self.hidden[:, None, :, None], k.shape).copy())
            self.k_pool = self.k_pool.masked_fill(mask, float("nan"))
            self.v_pool = self.v_pool.masked_fill(mask, float("nan"))
        self.scale = 128 ** -0.5

    def reference(self):
        return attention(self.q.double().numpy(), self.k64, self.v64, self.table, self.P, self.S,
                         self.T, self.page, self.scale, self.causal, self.window, self.sinks)

    def run(self, out_dtype="f32", stream=None, **kw):
        from shared_prefix_fan_gb300 import binding
        if not hasattr(self, "dev"):
            self.dev = [x.cuda() for x in (self.q, self.k_pool, self.v_pool)] + \
                       [torch.from_numpy(self.call_table).cuda()]
        a = (*self.dev, self.P, self.S, self.T, self.hq, self.hkv, self.page, self.scale)
        if self.q4:
            return binding.attn_q4(*a, self.causal, self.gs, self.gs, self.window, self.sinks,
                                   out_dtype=out_dtype, stream=stream, **kw)
        return binding.attn_window(*a, self.window, self.sinks, out_dtype=out_dtype,
                                   stream=stream, **kw)
