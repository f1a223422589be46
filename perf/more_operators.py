"""Drafted tokens over the paged cache, and the 8-bit cache, in plain torch and
through the library: rows into an 8-bit KV cache and back, attention over that
cache, attention for trees of drafted tokens, and what a drafting step does around
it (masks, positions and slots of the drafted rows; the accepted path; the
accepted rows moved together in the cache).

  listed()  the cases that are timed;   draw(rng)  one more of the same ranges
  prepare(case, seed)  what a caller holds before the call (on the GPU)
  run(state)  one pass: plain torch in 32 bits where `own` is false, the
              library's calls where it is true
  work(case)  the bytes and operations one pass cannot do without
  exact(case, seed)  the same outputs from the definition in 64 bits

Definitions. An 8-bit value is e4m3(x / scale) * scale: the quotient in fp32, then
nearest, ties to even, saturating at 448. Branch b holds n = prefix_len +
suffix_lens[b] cached tokens; its drafted token t has key n + t, a parent below t
(or -1) and a depth (0 without a parent), and sits at position n + depth. It sees key
j < n iff there is no window, j > position - window or j < sinks, and drafted key n + u
iff u is t or one of its ancestors less than `window` levels above it. Accepted are,
from the roots on, the first child whose drafted token is the one the model picked
at its parent; in the cache the accepted rows then follow the branch's n tokens.
"""
import math
import random

import torch

own = False

D = 128  # head dimension
VOCAB = 32000


# ----------------------------------------------------------------- the cases
# s_lo .. s_hi: private tokens of a branch (for op "q8" with its new ones, else without the
# drafted ones); t_lo .. t_hi: new or drafted tokens; depth: levels of a drafted tree.
def listed():
    return [
        # The rows of one decode step go into the 8-bit cache and are read back.
        dict(name="rows8-step", op="rows", R=8, hkv=8, page=64, gs=1.0),
        # The rows of a long prefill, with a calibrated scale.
        dict(name="rows8-prefill", op="rows", R=8192, hkv=8, page=64, gs=0.07),
        # 8-bit decode: 8 branches x 1 token over a 32k shared prefix.
        dict(name="q8-decode", op="q8", B=8, P=32768, s_lo=512, s_hi=512, t_lo=1, t_hi=1, hq=64,
             hkv=8, page=64, window=0, sinks=0, gs=1.0, sizes=1),
        # 8-bit ragged fan-out in a sliding window with first tokens, small pages.
        dict(name="q8-window", op="q8", B=32, P=16384, s_lo=64, s_hi=4096, t_lo=1, t_hi=32,
             hq=64, hkv=8, page=16, window=2048, sinks=16, gs=0.25, sizes=2),
        # 8-bit prefill of 2048 new tokens behind 30720 cached ones.
        dict(name="q8-prefill", op="q8", B=1, P=30720, s_lo=2048, s_hi=2048, t_lo=2048,
             t_hi=2048, hq=64, hkv=8, page=64, window=0, sinks=0, gs=1.0, sizes=3),
        # The smallest drafts: 8 tokens each for three branches of one KV head.
        dict(name="tree-tiny", op="tree", kv="bf16", B=3, P=256, s_lo=16, s_hi=16, t_lo=8, t_hi=8,
             depth=4, hq=8, hkv=1, page=16, window=0, sinks=0, gs=1.0, sizes=4),
        # A decode step with drafts: 8 branches x 32 drafted tokens over a 32k prefix.
        dict(name="tree-decode", op="tree", kv="bf16", B=8, P=32768, s_lo=480, s_hi=480, t_lo=32,
             t_hi=32, depth=6, hq=64, hkv=8, page=64, window=0, sinks=0, gs=1.0, sizes=5),
        # Drafts of every size for a ragged fan-out over a 64k prefix in 8 bits, small pages.
        dict(name="tree-wide", op="tree", kv="q8", B=32, P=65536, s_lo=64, s_hi=4096, t_lo=1,
             t_hi=64, depth=8, hq=64, hkv=8, page=16, window=0, sinks=0, gs=0.25, sizes=6),
        # Drafts in a layer with a sliding window and first tokens.
        dict(name="tree-window", op="tree", kv="bf16", B=8, P=32768, s_lo=100, s_hi=900, t_lo=64,
             t_hi=64, depth=8, hq=64, hkv=8, page=64, window=4096, sinks=4, gs=1.0, sizes=7),
        # The bookkeeping of a drafting step: masks, slots, rows in, path, kept rows.
        dict(name="draft-step", op="draft", B=8, P=32768, s_lo=480, s_hi=480, t_lo=32, t_hi=32,
             depth=6, hkv=8, page=64, window=0, gs=1.0, sizes=8),
        # The same for a wide batch of ragged drafts.
        dict(name="draft-wide", op="draft", B=512, P=1024, s_lo=0, s_hi=2048, t_lo=1, t_hi=64,
             depth=8, hkv=8, page=16, window=0, gs=1.0, sizes=9),
        # A whole drafting step on the 8-bit cache: tables, rows, attention, path, kept rows.
        dict(name="tree-step", op="step", kv="q8", B=8, P=16384, s_lo=100, s_hi=900, t_lo=32,
             t_hi=32, depth=6, hq=64, hkv=8, page=64, window=8192, sinks=4, gs=1.0, sizes=10),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _heads(rng):
    return rng.choice([(8, 1), (16, 2), (32, 8), (64, 8), (28, 4), (40, 8), (16, 16), (12, 4)])


def draw(rng):
    op = rng.choice(["rows", "q8", "q8", "tree", "tree", "tree", "draft", "step"])
    sizes, page = rng.randrange(1 << 30), rng.choice([16, 32, 64, 128])
    gs = rng.choice([1.0, 0.25, 0.07])
    if op == "rows":
        return dict(op=op, R=_log_int(rng, 1, 8192), hkv=rng.choice([1, 2, 4, 8]), page=page,
                    gs=gs)
    window, sinks = _log_int(rng, 1, 8192), rng.choice([0, 1, 4, 16, 100])
    if rng.random() < 0.5:
        window = sinks = 0
    hq, hkv = _heads(rng)
    kind = rng.choice(["one", "ragged", "chunk"])
    if op == "q8" and kind == "chunk":  # one sequence, many new tokens
        t = _log_int(rng, 33, 1024)
        B, t_lo, t_hi, s_lo, s_hi = 1, t, t, t, t + rng.randrange(0, 300)
    else:
        B = _log_int(rng, 1, 24)
        t_hi = 1 if kind == "one" else rng.randrange(2, 33 if op == "q8" else 65)
        t_lo = 1
        s_lo = t_hi if op == "q8" else 0
        s_hi = s_lo + _log_int(rng, 1, 2048)
    c = dict(op=op, B=B, P=_log_int(rng, 1, 16384), s_lo=s_lo, s_hi=s_hi, t_lo=t_lo, t_hi=t_hi,
             hkv=hkv, page=page, window=window, gs=gs, sizes=sizes)
    if op != "q8":
        c["depth"] = _log_int(rng, 1, min(16, t_hi))
    if op == "draft":
        return dict(c, B=_log_int(rng, 1, 256))
    c = dict(c, hq=hq, sinks=sinks)
    if op == "q8":
        return c
    return dict(c, kv="q8" if op == "step" else rng.choice(["bf16", "q8"]))


def _sizes(case):
    """Private tokens and new or drafted tokens of every branch."""
    r = random.Random(case["sizes"])
    S = [r.randint(case["s_lo"], case["s_hi"]) for _ in range(case["B"])]
    T = [r.randint(case["t_lo"], case["t_hi"]) for _ in range(case["B"])]
    return S, T


def _pages(tokens, page):
    return -(-tokens // page)


# ------------------------------------------------------------ 8-bit rows, plain
def _encode(x, gs):
    scale = torch.full((), gs, device=x.device)
    return (x.float() / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _write_rows(pool, rows, slots, page, gs):
    pool.view(torch.uint8)[slots // page, :, slots % page] = _encode(rows, gs).view(torch.uint8)


def _read_rows(pool, slots, page, gs):
    b = pool.view(torch.uint8)[slots // page, :, slots % page]
    return b.view(torch.float8_e4m3fn).float() * gs


def _held(pool, ids, gs):
    """The fp32 values of pages `ids`: [H, tokens, d]."""
    if pool.dtype == torch.bfloat16:
        x = pool[ids].float()
    else:
        x = pool.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * gs
    return x.transpose(0, 1).flatten(1, 2)


# ---------------------------------------------------------------- trees, plain
def _rows_of(T, R):
    """Branch and index in it of every row."""
    b = torch.repeat_interleave(torch.arange(T.numel(), device=T.device), T, output_size=R)
    return b, torch.arange(R, device=T.device) - (torch.cumsum(T, 0) - T)[b]


def _tree_rows(st):
    """masks int32 [R, words], positions int32 [R], slots int64 [R]."""
    c, T, R, t_max = st["case"], st["T_dev"], st["R"], st["T_max"]
    b, t = _rows_of(T, R)
    up = torch.zeros((T.numel(), t_max, t_max), device=T.device)  # one level up, or itself
    up[b, t, torch.where(st["parents"] < 0, t, st["parents"].long())] = 1.0
    up[b, t, t] = 1.0
    for _ in range(max(1, (c["depth"] - 1).bit_length())):
        up = (torch.matmul(up, up) > 0).float()
    depth = up.sum(-1) - 1
    see = up > 0
    if c["window"]:
        see = see & (depth[:, :, None] - depth[:, None, :] < c["window"])
    words = _pages(t_max, 32)
    bits = torch.zeros((R, words * 32), dtype=torch.int64, device=T.device)
    bits[:, :t_max] = see[b, t].long()
    w = (bits.unflatten(1, (words, 32)) << torch.arange(32, device=T.device)).sum(-1)
    before = c["P"] + st["S_dev"][b]
    key = before + t
    slots = st["table"][b, key // c["page"]].long() * c["page"] + key % c["page"]
    return w.to(torch.int32), (before + depth[b, t].long()).to(torch.int32), slots


def _accept(st):
    """path int32 [R] (each branch's accepted drafts, then -1), counts, next tokens."""
    c, T, R, t_max = st["case"], st["T_dev"], st["R"], st["T_max"]
    b, t = _rows_of(T, R)
    dev = T.device
    # children of node p (0: of no node) in columns, by the token each was drafted as
    parent = torch.full((T.numel(), t_max), -2, dtype=torch.int64, device=dev)
    draft, target = (torch.full((T.numel(), t_max), -1, dtype=torch.int64, device=dev)
                     for _ in range(2))
    parent[b, t], draft[b, t], target[b, t] = st["parents"].long(), st["draft"], st["target"]
    at = torch.full((T.numel(),), -1, dtype=torch.int64, device=dev)
    want, count = st["first"], torch.zeros_like(at)
    index = torch.arange(t_max, device=dev)
    path = torch.full((T.numel(), t_max), -1, dtype=torch.int64, device=dev)
    for i in range(min(c["depth"], t_max)):
        fits = (parent == at[:, None]) & (draft == want[:, None]) & (at > -2)[:, None]
        child = torch.where(fits, index, t_max).amin(1)
        found = child < t_max
        child = child.clamp(max=t_max - 1)
        path[:, i] = torch.where(found, child, path[:, i])
        count = count + found
        want = torch.where(found, target.gather(1, child[:, None])[:, 0], want)
        at = torch.where(found, child, -3)
    return path[b, t].to(torch.int32), count.to(torch.int32), want


def _keep(st, path, slots):
    """Drafted row i of a branch becomes row path[i] where it is given."""
    b, t = _rows_of(st["T_dev"], st["R"])
    from_row = (torch.cumsum(st["T_dev"], 0) - st["T_dev"])[b] + torch.where(path < 0, t, path.long())
    page = st["case"]["page"]
    for pool in (st["k_pool"], st["v_pool"]):
        bytes_ = pool.view(torch.uint8)
        moved = bytes_[slots[from_row] // page, :, slots[from_row] % page]
        bytes_[slots // page, :, slots % page] = moved


def _extend(st):
    """The table's entries for the drafted tokens; the free pages taken."""
    c, table = st["case"], st["table"]
    before = c["P"] + st["S_dev"]
    held, need = (before + c["page"] - 1) // c["page"], (before + st["T_dev"] + c["page"] - 1) // c["page"]
    start = torch.cumsum(need - held, 0) - (need - held)
    i = torch.arange(table.shape[1], device=table.device)[None, :]
    new = (i >= held[:, None]) & (i < need[:, None])
    at = (start[:, None] + i - held[:, None]).clamp(0, st["free"].numel() - 1)
    table.copy_(torch.where(new, st["free"][at], table))
    return (need - held).sum().to(torch.int32)


# ------------------------------------------------------------ attention, plain
def _attention(st, masks=None, positions=None):
    """One branch after the other. masks None: the new tokens in causal order."""
    c, q = st["case"], st["q"]
    page, hkv, G = c["page"], c["hkv"], c["hq"] // c["hkv"]
    out = torch.empty(q.shape, device=q.device)
    lse = torch.empty(q.shape[:2], device=q.device)
    first = 0
    for b, (s, t) in enumerate(zip(st["S"], st["T"])):
        n = c["P"] + (s - t if masks is None else s)  # keys before the new ones
        ids = st["table"][b, :_pages(n + t, page)].long()
        k, v = (_held(st[x], ids, c["gs"])[:, :n + t] for x in ("k_pool", "v_pool"))
        j = torch.arange(n + t, device=q.device)[None, :]
        if masks is None:
            pos = torch.arange(n, n + t, device=q.device)[:, None]
            see = j <= pos
            if c["window"]:
                see = see & ((j > pos - c["window"]) | (j < c["sinks"]))
        else:
            pos = positions[first:first + t, None]
            see = (j < n).expand(t, -1)
            if c["window"]:
                see = see & ((j > pos - c["window"]) | (j < c["sinks"]))
            u = torch.arange(t, device=q.device)
            bit = (masks[first:first + t, u // 32] >> (u % 32)) & 1
            see = torch.cat((see[:, :n], bit > 0), 1)
        qb = q[first:first + t].float().unflatten(1, (hkv, G)).permute(1, 0, 2, 3).flatten(1, 2)
        x = torch.matmul(qb, k.transpose(-1, -2)) * c["scale"]
        x = torch.where(see.repeat_interleave(G, 0), x, -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, v) / total
        out[first:first + t] = o.unflatten(1, (t, G)).transpose(0, 1).flatten(1, 2)
        l = (m + torch.log(total))[..., 0]
        lse[first:first + t] = l.unflatten(1, (t, G)).transpose(0, 1).flatten(1, 2)
        first += t
    return out.to(torch.bfloat16), lse


# ------------------------------------------------------------------- inputs
def _tree(r, T, depth):
    """Parents of T drafted tokens in at most `depth` levels, and what the model picks."""
    parents, level, children = [], [], [[] for _ in range(T + 1)]
    for t in range(T):
        p = -1
        if t and r.random() < 0.9:  # mostly below one of the last few
            p = r.randrange(max(0, t - 8), t)
            if level[p] + 1 >= depth:
                p = parents[p]
        parents.append(p)
        level.append(0 if p < 0 else level[p] + 1)
        children[p].append(t)
    draft = [r.randrange(VOCAB) for _ in range(T)]

    def pick(p):
        if children[p] and r.random() < 0.8:
            return draft[r.choice(children[p])]
        return r.randrange(VOCAB)
    return parents, draft, [pick(t) for t in range(T)], pick(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda")

    def normal(*shape):
        return torch.randn(shape, generator=g, **dev)

    def pools(pages, hkv, page):
        return [torch.zeros((pages, hkv, page, D), dtype=torch.uint8, **dev).view(
            torch.float8_e4m3fn) for _ in range(2)]

    if case["op"] == "rows":
        R, hkv, page = case["R"], case["hkv"], case["page"]
        pages = _pages(R, page) + 3
        slots = torch.randperm(pages * page, generator=g, **dev)[:R].contiguous()
        # K channels differ in size, as post-RoPE keys do; V does not
        amp = torch.exp(0.7 * normal(hkv, D))
        k_pool, v_pool = pools(pages, hkv, page)
        return dict(case=case, k_new=(amp * normal(R, hkv, D)).bfloat16(),
                    v_new=normal(R, hkv, D).bfloat16(), k_pool=k_pool, v_pool=v_pool, slots=slots)
    S, T = _sizes(case)
    P, page, B, hkv = case["P"], case["page"], case["B"], case["hkv"]
    tree = case["op"] != "q8"
    ends = [P + s + (t if tree else 0) for s, t in zip(S, T)]
    n_full, n_pre = P // page, _pages(P, page)
    width = max(_pages(e, page) for e in ends) + 1
    # two pages to spare, so that the free list is never empty
    pages = n_full + sum(max(_pages(e, page), n_pre) - n_full for e in ends) + 2
    ids = torch.randperm(pages, generator=g, **dev).tolist()
    free, rows = ids[n_full:], []
    for s, e in zip(S, ends):  # the pages a branch holds before the call
        need = max(_pages(P + s if case["op"] == "step" else e, page), n_pre) - n_full
        rows.append((ids[:n_full] + free[:need] + [-1] * width)[:width])
        free = free[need:]
    i32 = dict(dtype=torch.int32, **dev)
    st = dict(case=dict(case, scale=D ** -0.5), S=S, T=T, R=sum(T), T_max=max(T),
              S_dev=torch.tensor(S, **dev), T_dev=torch.tensor(T, **dev),
              S_i32=torch.tensor(S, **i32), T_i32=torch.tensor(T, **i32),
              table=torch.tensor(rows, **i32), free=torch.tensor(free, **i32))
    if tree:
        r = random.Random(seed)
        trees = [_tree(r, t, case["depth"]) for t in T]
        st.update(parents=torch.tensor(sum((x[0] for x in trees), []), **i32),
                  draft=torch.tensor(sum((x[1] for x in trees), []), **dev),
                  target=torch.tensor(sum((x[2] for x in trees), []), **dev),
                  first=torch.tensor([x[3] for x in trees], **dev),
                  S_after=[s + t for s, t in zip(S, T)])
    amp = torch.exp(0.5 * normal(hkv, 1, D))
    if case["op"] == "draft":  # only the drafted rows are touched
        st["k_pool"], st["v_pool"] = pools(pages, hkv, page)
    else:
        st["q"] = (2.0 * normal(st["R"], case["hq"], D)).bfloat16()  # scores over several units
        k, v = amp * normal(pages, hkv, page, D), normal(pages, hkv, page, D)
        if case.get("kv") == "bf16":
            st.update(k_pool=k.bfloat16(), v_pool=v.bfloat16())
        else:
            st.update(k_pool=_encode(k, case["gs"]), v_pool=_encode(v, case["gs"]))
    if case["op"] in ("draft", "step"):
        st.update(k_new=(amp[:, 0] * normal(st["R"], hkv, D)).bfloat16(),
                  v_new=normal(st["R"], hkv, D).bfloat16())
    if case["op"] == "tree":
        st["masks"], st["positions"], _ = _tree_rows(st)
    return st


# --------------------------------------------------------------------- run
def _run_own(st):
    from shared_prefix_fan_gb300 import binding
    c = st["case"]
    op, page, gs = c["op"], c["page"], c["gs"]
    if op == "rows":
        binding.kv_append_q8(st["k_new"], st["v_new"], st["k_pool"], st["v_pool"], st["slots"], gs,
                             gs)
        k, v = binding.kv_read_q8(st["k_pool"], st["v_pool"], st["slots"], gs, gs)
        return {"k": k, "v": v}
    if op == "q8":
        out, lse = binding.attn_q8(st["q"], st["k_pool"], st["v_pool"], st["table"], c["P"],
                                   st["S"], st["T"], c["hq"], c["hkv"], page, c["scale"], True,
                                   gs, gs, c["window"], c["sinks"], out_dtype="bf16")
        return {"out": out, "lse": lse}
    done = {}
    masks, positions = st.get("masks"), st.get("positions")
    if op == "step":
        _, done["used"] = binding.extend_device(st["table"], c["P"], st["S_i32"], st["T_i32"],
                                                page, st["free"], 0)
    if op != "tree":
        masks, positions, slots = binding.tree_rows(st["parents"], st["table"], c["P"],
                                                    st["S_i32"], st["T_i32"], page, st["T_max"],
                                                    c["window"])
        done.update(masks=masks, positions=positions, slots=slots)
        binding.kv_append_q8(st["k_new"], st["v_new"], st["k_pool"], st["v_pool"], slots, gs, gs)
    if op != "draft":
        done["out"], done["lse"] = binding.attn_tree(
            st["q"], st["k_pool"], st["v_pool"], st["table"], c["P"], st["S_after"], st["T"],
            c["hq"], c["hkv"], page, c["scale"], masks, positions, c["window"], c["sinks"], gs, gs,
            out_dtype="bf16")
    if op != "tree":
        path, counts, after = binding.tree_accept(st["parents"], st["draft"], st["target"],
                                                  st["first"], st["T_i32"])
        binding.kv_keep(st["k_pool"], st["v_pool"], st["table"], c["P"], st["S_i32"], st["T_i32"],
                        path, counts, page)
        done["k"], done["v"] = binding.kv_read_q8(st["k_pool"], st["v_pool"], slots, gs, gs)
        done.update(path=path, counts=counts, next=after)
    if op == "step":
        done["table"] = st["table"]
    return done


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    op, page, gs = c["op"], c["page"], c["gs"]
    if op == "rows":
        _write_rows(st["k_pool"], st["k_new"], st["slots"], page, gs)
        _write_rows(st["v_pool"], st["v_new"], st["slots"], page, gs)
        return {"k": _read_rows(st["k_pool"], st["slots"], page, gs).bfloat16(),
                "v": _read_rows(st["v_pool"], st["slots"], page, gs).bfloat16()}
    if op == "q8":
        out, lse = _attention(st)
        return {"out": out, "lse": lse}
    done = {}
    masks, positions = st.get("masks"), st.get("positions")
    if op == "step":
        done["used"] = _extend(st).reshape(1)
    if op != "tree":
        masks, positions, slots = _tree_rows(st)
        done.update(masks=masks, positions=positions, slots=slots)
        _write_rows(st["k_pool"], st["k_new"], slots, page, gs)
        _write_rows(st["v_pool"], st["v_new"], slots, page, gs)
    if op != "draft":
        done["out"], done["lse"] = _attention(st, masks, positions)
    if op != "tree":
        path, counts, after = _accept(st)
        _keep(st, path, slots)
        done["k"] = _read_rows(st["k_pool"], slots, page, gs).bfloat16()
        done["v"] = _read_rows(st["v_pool"], slots, page, gs).bfloat16()
        done.update(path=path, counts=counts, next=after)
    if op == "step":
        done["table"] = st["table"]
    return done


# -------------------------------------------------------------------- work
def _key_work(case, S, T):
    """(distinct cached tokens that some row sees, visible (row, key) pairs), without
    the drafted ones, and taking every drafted row as one at depth 0."""
    P, W, sinks, tree = case["P"], case["window"], case["sinks"], case["op"] != "q8"
    pairs, low, kept, private = 0, P, 0, 0
    for s, t in zip(S, T):
        n = P + s if tree else P + s - t
        for i in range(t):
            last = n if tree else n + i + 1
            lo = max(0, (n + (0 if tree else i) + 1) - W) if W else 0
            pairs += last - lo + min(sinks, lo)
        lo = max(0, n + 1 - W) if W else 0
        low, kept = min(low, lo), min(sinks, lo)
        private += n + (0 if tree else t) - max(lo, P) + max(0, kept - P)
    return P - low + min(sinks, low, P) + private, pairs


def work(case):
    if case["op"] == "rows":
        # bf16 rows in and the 8-bit rows out, then the 8-bit rows in and bf16 out
        n = 2 * case["R"] * case["hkv"]
        return {"bytes": n * (2 * D * 2 + 2 * D) + 8 * case["R"], "flops": 4 * n * D}
    S, T = _sizes(case)
    R, B = sum(T), case["B"]
    words = _pages(max(T), 32)
    # parents in, masks, positions and slots out; rows in and out; tokens, path, counts
    step = R * (4 + 4 * words + 12) + 8 * B + 2 * R * case["hkv"] * (3 * D) + R * (20 + 4) + 20 * B
    step += 2 * R * case["hkv"] * 3 * D  # reading the rows back
    if case["op"] == "draft":
        return {"bytes": step, "flops": R}
    row = 2 * D if case.get("kv") == "bf16" else D
    tokens, pairs = _key_work(case, S, T)
    bytes_ = 2 * tokens * case["hkv"] * row + R * case["hq"] * (2 * D + 2 * D + 4)
    if case["op"] != "q8":  # a drafted row sees itself at least
        bytes_ += 2 * R * case["hkv"] * row + R * 4 * words
        pairs += R
    if case["op"] == "step":
        bytes_ += step + 4 * B
    return {"bytes": bytes_, "flops": 4 * D * pairs * case["hq"]}


# -------------------------------------------------------------------- exact
def _levels64():
    return [(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
            for e in range(16) for m in range(8)][:127]  # byte 127 is no number


def _round64(x, gs):
    """What the cache holds for rows x, in 64 bits (the quotient is one of 32 bits)."""
    a = (x.float() / torch.tensor(gs, dtype=torch.float32, device=x.device)).double()
    grid = torch.tensor(_levels64(), dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(grid, a.abs().contiguous()).clamp(1, 126)
    d = (a.abs() - grid[hi - 1]) - (grid[hi] - a.abs())
    at = torch.where((d > 0) | ((d == 0) & (hi % 2 == 0)), hi, hi - 1)
    return torch.sign(a) * grid[at] * _fp32(gs)


def _fp32(gs):
    return float(torch.tensor(gs, dtype=torch.float32))


def _pool64(pool, gs):
    if pool.dtype == torch.bfloat16:
        return pool.double()
    grid = _levels64() + [math.nan]
    grid = torch.tensor(grid + [-x for x in grid], dtype=torch.float64, device=pool.device)
    return grid[pool.view(torch.uint8).long()] * _fp32(gs)


def _branch64(q, k, v, rows, keys, hide, case, out, lse):
    """Attention of `rows` over the cached rows at `keys`; hide [rows, keys]."""
    page, G = case["page"], case["hq"] // case["hkv"]
    for h in range(case["hkv"]):
        heads = slice(h * G, (h + 1) * G)
        kk, vv = k[keys // page, h, keys % page], v[keys // page, h, keys % page]
        x = q[rows, heads].double() @ kk.T * D ** -0.5
        x = x.masked_fill(hide[:, None], -math.inf)
        lse[rows, heads] = torch.logsumexp(x, -1)
        out[rows, heads] = torch.softmax(x, -1) @ vv


def _attention64(st, case, k, v, table, lineage):
    """lineage: for every row the drafted tokens it sees (None: causal order), its depth."""
    q, dev = st["q"], st["q"].device
    out = torch.empty(q.shape, dtype=torch.float64, device=dev)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=dev)
    first, page = 0, case["page"]
    for b, (s, t) in enumerate(zip(st["S"], st["T"])):
        n = case["P"] + s - (t if lineage is None else 0)
        at = torch.arange(n + t, device=dev)
        keys = torch.tensor(table[b], device=dev)[at // page] * page + at % page
        for i in range(0, t, 256):
            m = min(256, t - i)
            if lineage is None:
                pos = torch.arange(n + i, n + i + m, device=dev)[:, None]
                hide = at > pos
            else:
                mine = lineage[first + i:first + i + m]
                pos = torch.tensor([n + d for _, d in mine], device=dev)[:, None]
                hide = (at >= n).repeat(m, 1)
                for r, (seen, _) in enumerate(mine):
                    hide[r, [n + u for u in seen]] = False
            if case["window"]:
                out_of = (at <= pos - case["window"]) & (at >= case["sinks"])
                hide = hide | (out_of if lineage is None else out_of & (at < n))
            _branch64(q, k, v, slice(first + i, first + i + m), keys, hide, case, out, lse)
        first += t
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    op, page, gs = case["op"], case["page"], case["gs"]
    if op == "rows":
        return {"k": _round64(st["k_new"], gs), "v": _round64(st["v_new"], gs)}
    table = st["table"].tolist()
    if op == "q8":
        out, lse = _attention64(st, case, _pool64(st["k_pool"], gs), _pool64(st["v_pool"], gs),
                                table, None)
        return {"out": out, "lse": lse}
    S, T, P = st["S"], st["T"], case["P"]
    parents, draft, target, picked = (st[x].tolist() for x in ("parents", "draft", "target",
                                                              "first"))
    free, taken = st["free"].tolist(), 0
    lineage, slots, masks, positions, path, counts, after, source = ([] for _ in range(8))
    first, words = 0, _pages(st["T_max"], 32)
    for b, (s, t) in enumerate(zip(S, T)):
        n = P + s
        for i in range(n, n + t):
            if table[b][i // page] < 0:
                table[b][i // page] = free[taken]
                taken += 1
            slots.append(table[b][i // page] * page + i % page)
        up, tokens = parents[first:first + t], draft[first:first + t]
        for i in range(t):
            seen, u = [], i
            while u >= 0:
                seen.append(u)
                u = up[u]
            depth = len(seen) - 1
            seen = seen[:case["window"]] if case["window"] else seen
            lineage.append((seen, depth))
            bits = sum(1 << u for u in seen)
            masks.append([(bits >> (32 * w)) & 0xffffffff for w in range(words)])
            positions.append(n + depth)
        at, want, mine = -1, picked[b], []
        while True:
            fits = [u for u in range(t) if up[u] == at and tokens[u] == want]
            if not fits:
                break
            at = fits[0]
            mine.append(at)
            want = target[first + at]
        path += mine + [-1] * (t - len(mine))
        source += [first + u for u in mine] + list(range(first + len(mine), first + t))
        counts.append(len(mine))
        after.append(want)
        first += t
    done = {}
    if op != "draft":
        k, v = _pool64(st["k_pool"], gs), _pool64(st["v_pool"], gs)
    if op != "tree":
        masks = torch.tensor(masks, dtype=torch.int64)
        done = {"masks": torch.where(masks >= 1 << 31, masks - (1 << 32), masks).to(torch.int32),
                "positions": torch.tensor(positions, dtype=torch.int32),
                "slots": torch.tensor(slots, dtype=torch.int64)}
        k_new, v_new = _round64(st["k_new"], gs), _round64(st["v_new"], gs)
    if op == "step":
        where = done["slots"].to(k.device)
        k[where // page, :, where % page] = k_new
        v[where // page, :, where % page] = v_new
        done["used"] = torch.tensor([taken], dtype=torch.int32)
    if op != "draft":
        done["out"], done["lse"] = _attention64(st, case, k, v, table, lineage)
    if op != "tree":
        done.update(k=k_new[source], v=v_new[source], path=torch.tensor(path, dtype=torch.int32),
                    counts=torch.tensor(counts, dtype=torch.int32),
                    next=torch.tensor(after, dtype=torch.int64))
    if op == "step":
        done["table"] = torch.tensor(table, dtype=torch.int32)
    return done
