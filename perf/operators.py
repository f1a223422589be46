"""The serving operators of a shared-prefix fan-out, in plain torch and through
the library: page tables and slot maps built on the GPU, rows into a 4-bit KV
cache and back, attention over that cache, and attention with a sliding window
and first tokens that stay visible.

  listed()  the cases that are timed;   draw(rng)  one more of the same ranges
  prepare(case, seed)  what a caller holds before the call (on the GPU)
  run(state)  one pass: plain torch in 32 bits where `own` is false, the
              library's calls where it is true
  work(case)  the bytes and operations one pass cannot do without
  exact(case, seed)  the same outputs from the definition in 64 bits

Definitions. Branch b holds prefix_len shared tokens and suffix_lens[b] of its
own; token t of its q_rows[b] new ones sits at pos = prefix_len + suffix_lens[b]
- q_rows[b] + t. Key j is visible iff j <= pos and (no window, or j > pos -
window, or j < sinks). A 4-bit row of 128 values is 8 groups of 16: value =
e2m1(code) * e4m3(group scale) * pool scale, group scale = e4m3(max|x| / (6 *
pool scale)), code = e2m1(x / (group scale * pool scale)), each rounded to
nearest, ties to even.
"""
import math
import random

import torch

own = False

GROUP, ROW_BYTES, D = 16, 72, 128  # values a scale covers; bytes of a 4-bit row; head dimension
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # A decode step's bookkeeping: 8 branches, one new token each, a 32k prefix.
        dict(name="tables-step", op="extend", B=8, P=32768, s_lo=512, s_hi=512, t_lo=1, t_hi=1,
             page=64, sizes=1),
        # Forking a wide, ragged fan-out: 1024 branches over a 64k prefix in small pages.
        dict(name="tables-wide", op="fork", B=1024, P=65536, s_lo=64, s_hi=4096, t_lo=0, t_hi=0,
             page=16, sizes=2),
        # The rows of one decode step go into the 4-bit cache and are read back.
        dict(name="rows-step", op="rows", R=8, hkv=8, page=64, gs=1.0),
        # The rows of a long prefill.
        dict(name="rows-prefill", op="rows", R=8192, hkv=8, page=64, gs=0.5),
        # 4-bit attention: one KV head, three branches of four tokens, a 256-token prefix.
        dict(name="q4-tiny", op="q4", B=3, P=256, s_lo=16, s_hi=16, t_lo=4, t_hi=4, hq=8, hkv=1,
             page=16, causal=True, window=0, sinks=0, gs=1.0, sizes=3),
        # 4-bit decode: 8 branches x 1 token over a 32k shared prefix.
        dict(name="q4-decode", op="q4", B=8, P=32768, s_lo=512, s_hi=512, t_lo=1, t_hi=1, hq=64,
             hkv=8, page=64, causal=True, window=0, sinks=0, gs=1.0, sizes=4),
        # 4-bit ragged fan-out: 32 branches of 1..32 tokens over a 64k prefix, small pages.
        dict(name="q4-wide", op="q4", B=32, P=65536, s_lo=64, s_hi=4096, t_lo=1, t_hi=32, hq=64,
             hkv=8, page=16, causal=True, window=0, sinks=0, gs=0.5, sizes=5),
        # 4-bit prefill of 2048 new tokens behind 30720 cached ones.
        dict(name="q4-prefill", op="q4", B=1, P=30720, s_lo=2048, s_hi=2048, t_lo=2048, t_hi=2048,
             hq=64, hkv=8, page=64, causal=True, window=0, sinks=0, gs=1.0, sizes=6),
        # Windowed decode: 8 branches x 1 token, the last 4096 keys and 4 first ones.
        dict(name="window-decode", op="window", B=8, P=32768, s_lo=512, s_hi=512, t_lo=1, t_hi=1,
             hq=64, hkv=8, page=64, window=4096, sinks=4, sizes=7),
        # Windowed ragged fan-out whose windows end in the shared prefix or in a suffix.
        dict(name="window-wide", op="window", B=32, P=16384, s_lo=64, s_hi=4096, t_lo=1, t_hi=32,
             hq=64, hkv=8, page=16, window=2048, sinks=16, sizes=8),
        # Windowed prefill: 4096 new tokens, each seeing 1024 keys.
        dict(name="window-prefill", op="window", B=1, P=4096, s_lo=4096, s_hi=4096, t_lo=4096,
             t_hi=4096, hq=64, hkv=8, page=64, window=1024, sinks=4, sizes=9),
        # A whole decode step on the 4-bit cache: grow the tables, append, attend.
        dict(name="q4-step", op="step", B=8, P=16384, s_lo=100, s_hi=900, t_lo=1, t_hi=1, hq=64,
             hkv=8, page=64, causal=True, window=8192, sinks=4, gs=1.0, sizes=10),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _heads(rng):
    return rng.choice([(8, 1), (16, 2), (32, 8), (64, 8), (28, 4), (40, 8), (16, 16), (12, 4)])


def draw(rng):
    op = rng.choice(["extend", "fork", "rows", "q4", "q4", "window", "window", "step"])
    sizes, page = rng.randrange(1 << 30), rng.choice([16, 32, 64, 128])
    if op == "rows":
        return dict(op=op, R=_log_int(rng, 1, 8192), hkv=rng.choice([1, 2, 4, 8]), page=page,
                    gs=rng.choice([1.0, 0.25, 0.07]))
    if op in ("fork", "extend"):
        t_hi = _log_int(rng, 1, 512)
        return dict(op=op, B=_log_int(rng, 1, 1024), P=_log_int(rng, 1, 65536), s_lo=0,
                    s_hi=_log_int(rng, 16, 4096), t_lo=0, t_hi=t_hi, page=page, sizes=sizes)
    hq, hkv = _heads(rng)
    kind = rng.choice(["decode", "ragged", "chunk"])
    if kind == "chunk":  # one sequence, many new tokens
        t = _log_int(rng, 33, 1024)
        B, t_lo, t_hi, s_lo, s_hi = 1, t, t, t, t + rng.randrange(0, 300)
    else:
        B = _log_int(rng, 1, 24)
        t_lo, t_hi = (1, 1) if kind == "decode" else (1, rng.randrange(2, 33))
        s_lo = t_hi
        s_hi = s_lo + _log_int(rng, 1, 2048)
    c = dict(op=op, B=B, P=_log_int(rng, 1, 16384), s_lo=s_lo, s_hi=s_hi, t_lo=t_lo, t_hi=t_hi,
             hq=hq, hkv=hkv, page=page, sizes=sizes)
    window, sinks = _log_int(rng, 1, 8192), rng.choice([0, 1, 4, 16, 100])
    if op == "window":
        return dict(c, window=window, sinks=sinks)
    full = rng.random() < 0.5
    return dict(c, causal=True, window=0 if full else window, sinks=0 if full else sinks,
                gs=rng.choice([1.0, 0.25]))


def _sizes(case):
    """Suffix lengths and new tokens of every branch; in a table or step case the
    suffix lengths are those before the new tokens."""
    r = random.Random(case["sizes"])
    S = [r.randint(case["s_lo"], case["s_hi"]) for _ in range(case["B"])]
    T = [r.randint(case["t_lo"], case["t_hi"]) for _ in range(case["B"])]
    return S, T


def _pages(tokens, page):
    return -(-tokens // page)


# ----------------------------------------------------------- 4-bit rows, plain
def _encode(x, gs):
    """fp32 rows [..., 128] -> (codes [..., 128] int32, scales [..., 8] e4m3)."""
    g = x.unflatten(-1, (D // GROUP, GROUP))
    top = g.abs().amax(-1)
    c6 = torch.full((), 6.0, device=x.device) * gs
    scale = (top / c6).clamp(max=448.0).to(torch.float8_e4m3fn)
    den = (scale.float() * gs).unsqueeze(-1)
    y = torch.where(den > 0, g / den, torch.zeros((), device=x.device))
    a = y.abs()
    mag = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() +
           (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    return (mag + 8 * (y < 0).int()).flatten(-2), scale


def _pack(codes):
    """codes [..., 128] -> bytes [..., 64]: of each 8 values, 32 bits hold values 0,
    2, 4, 6 in the low half (4 bits each, from bit 0) and 1, 3, 5, 7 in the high."""
    w = codes.unflatten(-1, (16, 2, 2, 2))  # (word, byte of the half, nibble, half)
    return (w[..., 0, :] + 16 * w[..., 1, :]).transpose(-1, -2).flatten(-3).to(torch.uint8)


def _unpack(b):
    n = torch.stack((b & 15, b >> 4), -1).unflatten(-2, (16, 2, 2))  # (word, half, byte, nibble)
    return n.permute(*range(n.dim() - 3), -2, -1, -3).flatten(-4)


def _parts(pool, page):
    """Views of a pool [pages, H, page * 72]: codes [pages, H, page, 64], scales [.., page, 8]."""
    c = pool[..., :page * 64].unflatten(-1, (page, 64))
    return c, pool[..., page * 64:].unflatten(-1, (page, 8))


def _decode(codes, scales, gs):
    lut = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    v = lut[_unpack(codes).int()].unflatten(-1, (D // GROUP, GROUP))
    return (v * (scales.view(torch.float8_e4m3fn).float() * gs).unsqueeze(-1)).flatten(-2)


def _write_rows(pool, rows, slots, page, gs):
    codes, scales = _encode(rows.float(), gs)
    c, s = _parts(pool, page)
    c[slots // page, :, slots % page] = _pack(codes)
    s[slots // page, :, slots % page] = scales.view(torch.uint8)


def _read_rows(pool, slots, page, gs):
    c, s = _parts(pool, page)
    return _decode(c[slots // page, :, slots % page], s[slots // page, :, slots % page], gs)


# --------------------------------------------------------- page tables, plain
def _fork(prefix, P, S, page, free, width):
    n_full = P // page
    need = torch.maximum((P + S + page - 1) // page, torch.full_like(S, _pages(P, page)))
    start = torch.cumsum(need - n_full, 0) - (need - n_full)
    i = torch.arange(width, device=S.device, dtype=torch.int64)[None, :]
    at = (start[:, None] + i - n_full).clamp(0, free.numel() - 1)
    own_pages = torch.where(i < need[:, None], free[at], torch.full((), -1, device=S.device,
                                                                   dtype=torch.int32))
    if n_full == 0:
        return own_pages, (need - n_full).sum().to(torch.int32)
    return (torch.where(i < n_full, prefix[i.clamp(max=n_full - 1)], own_pages),
            (need - n_full).sum().to(torch.int32))


def _extend(table, P, S, T, page, free, R):
    held, need = (P + S + page - 1) // page, (P + S + T + page - 1) // page
    start = torch.cumsum(need - held, 0) - (need - held)
    i = torch.arange(table.shape[1], device=S.device)[None, :]
    new = (i >= held[:, None]) & (i < need[:, None])
    at = (start[:, None] + i - held[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(new, free[at], table))
    b = torch.repeat_interleave(torch.arange(S.numel(), device=S.device), T, output_size=R)
    t = torch.arange(R, device=S.device) - (torch.cumsum(T, 0) - T)[b]
    pos = P + S[b] + t
    slots = table[b, pos // page].long() * page + pos % page
    return slots, (need - held).sum().to(torch.int32)


# ------------------------------------------------------------ attention, plain
def _attention(q, k, v, table, st):
    """q [R, H_q, d]; k, v [pages, H_kv, page, d] fp32; every branch's keys are
    gathered through its table row, padded to the longest branch."""
    c = st["case"]
    page, hkv, P = c["page"], c["hkv"], c["P"]
    S, T = st["S_dev"], st["T_dev"]
    n, Tm, G = _pages(P + st["S_max"], page), st["T_max"], c["hq"] // hkv
    ids = table[:, :n].clamp(min=0).long()
    k, v = (x[ids].transpose(1, 2).flatten(2, 3) for x in (k, v))  # [B, H_kv, keys, d]
    t = torch.arange(Tm, device=q.device)
    rows = ((torch.cumsum(T, 0) - T)[:, None] + t).clamp(max=q.shape[0] - 1)
    qb = q.float()[rows].unflatten(2, (hkv, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = torch.matmul(qb, k.transpose(-1, -2)) * c["scale"]  # [B, H_kv, Tm * G, keys]
    j = torch.arange(n * page, device=q.device)
    pos = P + (S - T)[:, None, None] + t[None, :, None]
    see = (j < P + S[:, None, None]).expand(-1, Tm, -1)
    if c.get("causal", True):
        see = see & (j <= pos)
    if c["window"]:
        see = see & ((j > pos - c["window"]) | (j < c["sinks"]))
    see = see.repeat_interleave(G, 1)[:, None]
    s = torch.where(see, s, torch.full((), -math.inf, device=q.device))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / total
    lse = (m + torch.log(total)).squeeze(-1)
    b = torch.repeat_interleave(torch.arange(S.numel(), device=q.device), T,
                                output_size=q.shape[0])
    at = torch.arange(q.shape[0], device=q.device) - (torch.cumsum(T, 0) - T)[b]
    o = o.unflatten(2, (Tm, G)).transpose(1, 2)[b, at].flatten(1, 2)
    return o.to(torch.bfloat16), lse.unflatten(2, (Tm, G)).transpose(1, 2)[b, at].flatten(1, 2)


# ------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda")

    def normal(*shape):
        return torch.randn(shape, generator=g, **dev)

    if case["op"] == "rows":
        R, hkv, page, gs = case["R"], case["hkv"], case["page"], case["gs"]
        pages = _pages(R, page) + 3
        slots = torch.randperm(pages * page, generator=g, **dev)[:R].contiguous()
        # K channels differ in size, as post-RoPE keys do; V does not
        amp = gs * torch.exp(0.7 * normal(hkv, D))
        pool = torch.zeros((2, pages, hkv, page * ROW_BYTES), dtype=torch.uint8, **dev)
        return dict(case=case, k_new=(amp * normal(R, hkv, D)).bfloat16(),
                    v_new=(gs * normal(R, hkv, D)).bfloat16(), k_pool=pool[0], v_pool=pool[1],
                    slots=slots)
    S, T = _sizes(case)
    P, page, B = case["P"], case["page"], case["B"]
    n_pre, grow = _pages(P, page), case["op"] in ("extend", "step")
    ends = [P + s + (t if grow else 0) for s, t in zip(S, T)]
    width = max(n_pre, max(_pages(e, page) for e in ends))
    # two pages to spare, so that the free list is never empty
    pages = n_pre + sum(max(_pages(e, page), n_pre) - P // page for e in ends) + 2
    ids = torch.randperm(pages, generator=g, **dev).to(torch.int32)
    st = dict(case=case, S=S, T=T, R=sum(T), S_dev=torch.tensor(S, **dev),
              T_dev=torch.tensor(T, **dev), S_i32=torch.tensor(S, dtype=torch.int32, **dev),
              T_i32=torch.tensor(T, dtype=torch.int32, **dev), prefix=ids[:n_pre].contiguous(),
              free=ids[n_pre:].contiguous(), width=width)
    if case["op"] == "fork":
        return st
    st["table"], taken = _fork(st["prefix"], P, st["S_dev"], page, st["free"], width)
    if grow:
        st["free"] = st["free"][int(taken):].contiguous()
        if case["op"] == "extend":
            return st
    hq, hkv = case["hq"], case["hkv"]
    case = st["case"] = dict(case, scale=D ** -0.5)
    q = (2.0 * normal(st["R"], hq, D)).bfloat16()  # scores spread over several units
    amp = torch.exp(0.5 * normal(hkv, 1, D))
    k, v = amp * normal(pages, hkv, page, D), normal(pages, hkv, page, D)
    if case["op"] == "window":
        return dict(st, q=q, k_pool=k.bfloat16(), v_pool=v.bfloat16(), S_max=max(S), T_max=max(T))
    pool = torch.empty((2, pages, hkv, page * ROW_BYTES), dtype=torch.uint8, **dev)
    gs = case["gs"]
    for one, x in ((pool[0], k), (pool[1], v)):
        codes, scales = _encode(x, gs)
        _parts(one, page)[0].copy_(_pack(codes))
        _parts(one, page)[1].copy_(scales.view(torch.uint8))
    st.update(q=q, k_pool=pool[0], v_pool=pool[1], S_max=max(S), T_max=max(T))
    if case["op"] == "step":
        st.update(S_after=[s + t for s, t in zip(S, T)],
                  k_new=(amp[:, 0] * normal(st["R"], hkv, D)).bfloat16(),
                  v_new=normal(st["R"], hkv, D).bfloat16())
    return st


# --------------------------------------------------------------------- run
def run(st):
    c = st["case"]
    op, page = c["op"], c["page"]
    if own:
        from shared_prefix_fan_gb300 import binding
        if op == "fork":
            table, _, used = binding.fork_device(st["prefix"], c["P"], st["S_i32"], page,
                                                 st["free"], st["width"])
            return {"table": table, "used": used}
        if op == "extend":
            slots, used = binding.extend_device(st["table"], c["P"], st["S_i32"], st["T_i32"],
                                                page, st["free"], st["R"])
            return {"table": st["table"], "slots": slots, "used": used}
        if op == "rows":
            binding.kv_append_q4(st["k_new"], st["v_new"], st["k_pool"], st["v_pool"],
                                 st["slots"], page, c["gs"], c["gs"])
            k, v = binding.kv_read_q4(st["k_pool"], st["v_pool"], st["slots"], page, c["gs"],
                                      c["gs"])
            return {"k": k, "v": v}
        if op == "q4":
            out, lse = binding.attn_q4(st["q"], st["k_pool"], st["v_pool"], st["table"], c["P"],
                                       st["S"], st["T"], c["hq"], c["hkv"], page, c["scale"],
                                       c["causal"], c["gs"], c["gs"], c["window"], c["sinks"],
                                       out_dtype="bf16")
            return {"out": out, "lse": lse}
        if op == "window":
            out, lse = binding.attn_window(st["q"], st["k_pool"], st["v_pool"], st["table"],
                                           c["P"], st["S"], st["T"], c["hq"], c["hkv"], page,
                                           c["scale"], c["window"], c["sinks"], out_dtype="bf16")
            return {"out": out, "lse": lse}
        slots, used = binding.extend_device(st["table"], c["P"], st["S_i32"], st["T_i32"], page,
                                            st["free"], st["R"])
        binding.kv_append_q4(st["k_new"], st["v_new"], st["k_pool"], st["v_pool"], slots, page,
                             c["gs"], c["gs"])
        out, lse = binding.attn_q4(st["q"], st["k_pool"], st["v_pool"], st["table"], c["P"],
                                   st["S_after"], st["T"], c["hq"], c["hkv"], page, c["scale"],
                                   c["causal"], c["gs"], c["gs"], c["window"], c["sinks"],
                                   out_dtype="bf16")
        return {"table": st["table"], "slots": slots, "used": used, "out": out, "lse": lse}
    if op == "fork":
        table, used = _fork(st["prefix"], c["P"], st["S_dev"], page, st["free"], st["width"])
        return {"table": table, "used": used.reshape(1)}
    if op == "extend":
        slots, used = _extend(st["table"], c["P"], st["S_dev"], st["T_dev"], page, st["free"],
                              st["R"])
        return {"table": st["table"], "slots": slots, "used": used.reshape(1)}
    if op == "rows":
        _write_rows(st["k_pool"], st["k_new"], st["slots"], page, c["gs"])
        _write_rows(st["v_pool"], st["v_new"], st["slots"], page, c["gs"])
        return {"k": _read_rows(st["k_pool"], st["slots"], page, c["gs"]).bfloat16(),
                "v": _read_rows(st["v_pool"], st["slots"], page, c["gs"]).bfloat16()}
    if op == "window":
        out, lse = _attention(st["q"], st["k_pool"].float(), st["v_pool"].float(), st["table"], st)
        return {"out": out, "lse": lse}
    if op == "q4":
        out, lse = _attention(st["q"], _decode(*_parts(st["k_pool"], page), c["gs"]),
                              _decode(*_parts(st["v_pool"], page), c["gs"]), st["table"], st)
        return {"out": out, "lse": lse}
    slots, used = _extend(st["table"], c["P"], st["S_dev"], st["T_dev"], page, st["free"], st["R"])
    _write_rows(st["k_pool"], st["k_new"], slots, page, c["gs"])
    _write_rows(st["v_pool"], st["v_new"], slots, page, c["gs"])
    after = dict(st, S_dev=st["S_dev"] + st["T_dev"], S_max=max(st["S_after"]))
    out, lse = _attention(st["q"], _decode(*_parts(st["k_pool"], page), c["gs"]),
                          _decode(*_parts(st["v_pool"], page), c["gs"]), st["table"], after)
    return {"table": st["table"], "slots": slots, "used": used.reshape(1), "out": out, "lse": lse}


# -------------------------------------------------------------------- work
def _key_work(case, S, T):
    """(distinct cached tokens that some row sees, visible (row, key) pairs)."""
    P, W, sinks, causal = case["P"], case["window"], case["sinks"], case.get("causal", True)
    pairs, prefix, private = 0, [], 0
    for s, t in zip(S, T):
        if t == 0:
            continue
        end = P + s
        for i in range(t):
            last = end - t + i + 1 if causal else end
            lo = max(0, last - W) if W else 0
            pairs += last - lo + min(sinks, lo)
        lo = max(0, end - t + 1 - W) if W else 0
        prefix.append(min(lo, P))
        kept = min(sinks, lo)
        private += end - max(lo, P) + max(0, kept - P)
    if not prefix:
        return 0, 0
    low = min(prefix)
    return P - low + min(sinks, low, P) + private, pairs


def work(case):
    if case["op"] == "rows":
        # bf16 rows in and the 4-bit rows out, then the 4-bit rows in and bf16 out
        n = 2 * case["R"] * case["hkv"]
        return {"bytes": n * (2 * D * 2 + 2 * ROW_BYTES) + 8 * case["R"], "flops": 4 * n * D}
    S, T = _sizes(case)
    P, page, R = case["P"], case["page"], sum(T)
    if case["op"] == "fork":
        width = max(_pages(P, page), max(_pages(P + s, page) for s in S))
        taken = sum(max(_pages(P + s, page), _pages(P, page)) - P // page for s in S)
        return {"bytes": 4 * (len(S) * width + taken + P // page + len(S)), "flops": len(S)}
    grown = sum(_pages(P + s + t, page) - _pages(P + s, page) for s, t in zip(S, T))
    tables = 4 * (2 * len(S) + 2 * grown) + 4 * len(S) + 8 * R
    if case["op"] == "extend":
        return {"bytes": tables, "flops": R}
    after = [s + t for s, t in zip(S, T)] if case["op"] == "step" else S
    tokens, pairs = _key_work(case, after, T)
    row = 2 * D if case["op"] == "window" else ROW_BYTES
    bytes_ = 2 * tokens * case["hkv"] * row + R * case["hq"] * (2 * D + 2 * D + 4)
    if case["op"] == "step":
        bytes_ += tables + 2 * R * case["hkv"] * (2 * D + ROW_BYTES)
    return {"bytes": bytes_, "flops": 4 * D * pairs * case["hq"]}


# -------------------------------------------------------------------- exact
_VALUES64 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest64(a, grid):
    """Index of the grid value nearest to a >= 0, ties to the even index."""
    grid = torch.tensor(grid, dtype=torch.float64, device=a.device)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, len(grid) - 1)
    d = (a - grid[hi - 1]) - (grid[hi] - a)
    up = (d > 0) | ((d == 0) & (hi % 2 == 0))
    return torch.where(up, hi, hi - 1)


def _scales64():
    return [(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
            for e in range(16) for m in range(8)][:127]  # byte 127 is no number


def _round64(x, gs):
    """What the cache holds for rows x [..., 128], in 64 bits."""
    groups = x.double().reshape(*x.shape[:-1], 8, 16)
    grid = torch.tensor(_scales64(), dtype=torch.float64, device=x.device)
    scale = grid[_nearest64(groups.abs().amax(-1) / (6.0 * gs), _scales64())] * gs
    scale = scale[..., None]
    y = torch.where(scale > 0, groups / torch.where(scale > 0, scale, 1.0), 0.0)
    level = torch.tensor(_VALUES64, dtype=torch.float64, device=x.device)
    return (torch.sign(y) * level[_nearest64(y.abs(), _VALUES64)] * scale).reshape(x.shape)


def _pool64(pool, page, gs):
    """Every row a pool holds, [pages, H, page, 128] in 64 bits, from its bytes."""
    n, h, _ = pool.shape
    words = pool[:, :, :page * 64].contiguous().view(torch.int32).reshape(n, h, page, 16)
    scale = torch.tensor(_scales64() + [math.nan], dtype=torch.float64, device=pool.device)
    scale = scale[pool[:, :, page * 64:].reshape(n, h, page, 8).long()] * gs
    level = torch.tensor(_VALUES64 + tuple(-a for a in _VALUES64), dtype=torch.float64,
                         device=pool.device)
    got = torch.empty((n, h, page, 16, 8), dtype=torch.float64, device=pool.device)
    for e in range(8):  # value e of a word: bits 4 (e / 2) of its half e % 2
        got[..., e] = level[((words >> (16 * (e % 2) + 4 * (e // 2))) & 15).long()]
    return got.reshape(n, h, page, 128) * scale.repeat_interleave(16, -1)


def _attention64(q, k, v, table, case, S, T):
    P, page, hkv, G = case["P"], case["page"], case["hkv"], case["hq"] // case["hkv"]
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    first = 0
    for b, (s, t) in enumerate(zip(S, T)):
        if t == 0:
            continue
        n = P + s
        ids = table[b, :_pages(n, page)].long()
        keys = k[ids].transpose(0, 1).reshape(hkv, -1, D)[:, :n]
        vals = v[ids].transpose(0, 1).reshape(hkv, -1, D)[:, :n]
        j = torch.arange(n, device=q.device)
        for i in range(0, t, 256):
            m = min(256, t - i)
            pos = torch.arange(n - t + i, n - t + i + m, device=q.device)[:, None]
            hide = j > pos if case.get("causal", True) else torch.zeros_like(j > pos)
            if case["window"]:
                hide = hide | ((j <= pos - case["window"]) & (j >= case["sinks"]))
            for h in range(hkv):
                rows = slice(first + i, first + i + m)
                x = q[rows, h * G:(h + 1) * G].double() @ keys[h].double().T * case["scale"]
                x = x.masked_fill(hide[:, None], -math.inf)
                lse[rows, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                out[rows, h * G:(h + 1) * G] = torch.softmax(x, -1) @ vals[h].double()
        first += t
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    op, page = case["op"], case["page"]
    if op == "rows":
        return {"k": _round64(st["k_new"], case["gs"]), "v": _round64(st["v_new"], case["gs"])}
    S, T, P = st["S"], st["T"], case["P"]
    free, taken = st["free"].tolist(), 0
    if op == "fork":
        prefix, rows = st["prefix"].tolist(), []
        for s in S:
            need = max(_pages(P + s, page), _pages(P, page)) - P // page
            rows.append((prefix[:P // page] + free[taken:taken + need] +
                         [-1] * st["width"])[:st["width"]])
            taken += need
        return {"table": torch.tensor(rows, dtype=torch.int32),
                "used": torch.tensor([taken], dtype=torch.int32)}
    case = dict(case, scale=D ** -0.5)
    if op in ("extend", "step"):
        rows, slots = st["table"].tolist(), []
        for row, s, t in zip(rows, S, T):
            for i in range(P + s, P + s + t):
                if i % page == 0:
                    row[i // page] = free[taken]
                    taken += 1
                slots.append(row[i // page] * page + i % page)
        done = {"table": torch.tensor(rows, dtype=torch.int32),
                "slots": torch.tensor(slots, dtype=torch.int64),
                "used": torch.tensor([taken], dtype=torch.int32)}
        if op == "extend":
            return done
    if op == "window":
        out, lse = _attention64(st["q"], st["k_pool"], st["v_pool"], st["table"], case, S, T)
        return {"out": out, "lse": lse}
    k, v = (_pool64(st[n], page, case["gs"]) for n in ("k_pool", "v_pool"))
    if op == "q4":
        out, lse = _attention64(st["q"], k, v, st["table"], case, S, T)
        return {"out": out, "lse": lse}
    at = done["slots"].to(k.device)
    k[at // page, :, at % page] = _round64(st["k_new"], case["gs"])
    v[at // page, :, at % page] = _round64(st["v_new"], case["gs"])
    out, lse = _attention64(st["q"], k, v, done["table"].to(k.device), case, st["S_after"], T)
    return dict(done, out=out, lse=lse)
