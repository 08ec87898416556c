"""Performance cases of the operators around a cache held in 8 bits: block tables, lengths and
slot maps built on the GPU, the append of rotated keys and values in 8 bits with a scale for
each block of tokens and head, attention over such a cache, and attention for batches whose
sequences share a prefix of it.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU, ``run`` is one
pass: the plain form in 32-bit torch operations, or with ``own`` set the library's calls.
``exact`` gives the same outputs in 64 bits from the definition.  Values of the cache are its
codes (e4m3), the scales beside them bytes b that stand for 2^(b - 127).

The lengths of a case's sequences follow from its values alone, the data from the seed.
"""
import math
import random

import torch

own = False

BLOCK = 16  # tokens that share a scale (a page of 8 is one block)

# ------------------------------------------------------------------ cases

_SHAPE = dict(seqs=1, ctx_min=0, ctx_max=0, q_min=1, q_max=1, q_heads=32, kv_heads=8, head_dim=128,
              page=16)


def _plan(name, **kw):
    return dict(dict(op="plan", name=name, seqs=1, ctx_min=0, ctx_max=0, q_min=1, q_max=1, page=16, ended=0, pad=0),
                **kw)


def _append(name, **kw):
    return dict(_SHAPE, name=name, op="append", rot=kw.get("head_dim", 128), axes=1,
                interleaved=False, **kw)


def _attend(name, **kw):
    return dict(_SHAPE, name=name, op="attend", **{"window": 0, "sinks": 0, **kw})


def _prefix(name, **kw):
    return dict(_SHAPE, name=name, op="prefix", **kw)


def listed():
    return [
        # the plan of one decode step: latency counts
        _plan("plan, 64 single tokens", seqs=64, ctx_min=100, ctx_max=8000),
        # thousands of requests: short prompts, single tokens, idle ones, every ninth just ended
        _plan("plan, 3000 requests", seqs=3000, ctx_max=4000, q_min=0, q_max=60, ended=9, pad=37),
        # one decode step of 64 requests, the heads of an 8B-class layer: latency counts
        _append("append, 64 single tokens", seqs=64, ctx_min=100, ctx_max=8000),
        # a prompt of 8192 tokens: bandwidth counts
        _append("append, prompt of 8192", q_min=8192, q_max=8192, page=64),
        # prompts with images: three position axes, odd lengths, seven query heads to a key head
        dict(_append("append, image prompts", seqs=3, ctx_max=40, q_min=900, q_max=2100, q_heads=28,
                     kv_heads=4, page=32), axes=3),
        # one user's decode step on a short context: the smallest call
        _attend("attend, 1 token on 500", ctx_min=499, ctx_max=499),
        # a decode batch in ordinary service
        _attend("attend, 64 tokens on 8K", seqs=64, ctx_min=500, ctx_max=8000),
        # few requests on very long contexts: the work has to be split over the keys
        _attend("attend, 3 tokens on 128K", seqs=3, ctx_min=90000, ctx_max=131000, page=64),
        # a whole prompt: tensor throughput counts
        _attend("attend, prompt of 8192", q_min=8192, q_max=8192, page=64),
        # chunks of prompts and single tokens in one batch, with a window behind which pages are freed
        _attend("attend, window, mixed chunks", seqs=9, ctx_max=9000, q_min=0, q_max=1500, q_heads=64,
                head_dim=64, page=32, window=1024, sinks=16),
        # one system prompt for all 64 requests of a decode step
        _prefix("prefix of 8K, 64 tokens", seqs=64, ctx_max=500, groups=1, prefix_min=8192, prefix_max=8192),
        # requests of four adapters, each with its own prefix
        _prefix("4 prefixes, 150 tokens", seqs=150, ctx_min=10, ctx_max=900, groups=4, prefix_min=1000,
                prefix_max=5000, q_heads=16, kv_heads=2, page=64),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    return min(hi, max(lo, n))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attend", "attend", "attend", "prefix"])
    if op == "plan":
        seqs = _log_int(rng, 1, 3000)
        return dict(op="plan", seqs=seqs, ctx_min=0, ctx_max=_log_int(rng, 10, 4000), q_min=rng.randint(0, 1),
                    q_max=_log_int(rng, 1, max(2, min(8000, 90000 // seqs))), page=rng.choice([8, 16, 32, 64, 128]),
                    ended=rng.choice([0, 2, 5, 11]), pad=rng.choice([0, 1, 50]))
    heads, kv_heads, dim = rng.choice([(32, 8, 128), (28, 4, 128), (16, 2, 128), (10, 10, 128), (40, 8, 128),
                                       (64, 8, 64), (8, 8, 64), (12, 4, 64), (15, 5, 64), (32, 4, 64)])
    case = dict(op=op, q_heads=heads, kv_heads=kv_heads, head_dim=dim, page=rng.choice([8, 16, 32, 64, 128]))
    if op == "append":
        if rng.random() < 0.5:
            case.update(seqs=_log_int(rng, 1, 300), ctx_min=0, ctx_max=_log_int(rng, 20, 9000), q_min=1, q_max=1)
        else:
            seqs = _log_int(rng, 1, 8)
            case.update(seqs=seqs, ctx_min=0, ctx_max=_log_int(rng, 1, 2000), q_min=1,
                        q_max=_log_int(rng, 2, 8000 // seqs))
        return dict(case, rot=rng.choice([dim, dim, dim // 2]), axes=rng.choice([1, 1, 3]),
                    interleaved=rng.random() < 0.4)
    if op == "prefix":
        seqs = _log_int(rng, 2, 150)
        return dict(case, seqs=seqs, ctx_min=0, ctx_max=_log_int(rng, 1, 900), q_min=1, q_max=1,
                    groups=rng.randint(1, min(4, seqs)), prefix_min=50, prefix_max=_log_int(rng, 100, 6000))
    window, sinks = rng.choice([(0, 0), (0, 0), (_log_int(rng, 60, 4096), rng.randint(0, 40))])
    if rng.random() < 0.6:  # single tokens
        seqs = _log_int(rng, 1, 100)
        case.update(seqs=seqs, ctx_min=0, ctx_max=_log_int(rng, 30, min(100000, 600000 // seqs)), q_min=1, q_max=1)
    else:  # prompts and chunks
        seqs = _log_int(rng, 1, 6)
        q = _log_int(rng, 2, 4000 // seqs)
        case.update(seqs=seqs, ctx_min=0, ctx_max=_log_int(rng, 1, 5000), q_min=rng.randint(0, 1), q_max=q)
    return dict(case, window=window, sinks=sinks)


def _lengths(case):
    """New tokens and cached tokens before them of each sequence, prefix lengths and first
    sequences of the groups: functions of the case's values alone.  In a plan -1 new tokens
    mark a request that has ended."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["seqs"]
    q = [r.randint(case["q_min"], case["q_max"]) for _ in range(n)]
    q[0] = max(q[0], case["q_max"])
    ctx = [r.randint(case["ctx_min"], case["ctx_max"]) for _ in range(n)]
    if case["op"] == "plan":
        if case["ended"]:
            q = [-1 if i % case["ended"] == 1 else x for i, x in enumerate(q)]
        return q, ctx, [], []
    if case["op"] == "attend" and n > 4 and case["q_max"] > 1:
        q[1], q[2] = 1, 1  # single tokens among the chunks
    if case["op"] != "prefix":
        return q, ctx, [], []
    g = case["groups"]
    prefix = [r.randint(case["prefix_min"], case["prefix_max"]) for _ in range(g)]
    cuts = sorted(r.sample(range(1, n), g - 1)) if g > 1 else []
    first = [0] + cuts + [n]
    for i in range(g):
        for s in range(first[i], first[i + 1]):
            ctx[s] += prefix[i]
    return q, ctx, prefix, first


def _axis_pairs(case):
    """Rotated pairs of each position axis: the first axis gets a quarter, the others the rest."""
    pairs = case["rot"] // 2
    if case["axes"] == 1:
        return [pairs]
    a = pairs // 4
    return [a, (pairs - a) // 2, pairs - a - (pairs - a) // 2]


# ------------------------------------------------------------------ inputs

def _exponent(top):
    """The least e with top <= 448 * 2^e, at least -126, as the byte e + 127."""
    frac, exp = torch.frexp(top)
    return (exp - 9 + (frac > 0.875).int() + 127).clamp(1, 254)


def _quantized(x, page):
    """Codes and scale bytes of x [pages, heads, page, d], block by block."""
    block = min(BLOCK, page)
    y = x.view(*x.shape[:2], page // block, block, x.shape[3])
    byte = _exponent(y.abs().amax((3, 4)).float())
    codes = torch.ldexp(y.float(), (127 - byte)[..., None, None]).to(torch.float8_e4m3fn)
    return codes.view(x.shape), byte.to(torch.uint8)


def _prepare_plan(case, seed):
    q, ctx, _, _ = _lengths(case)
    pick = random.Random(seed)
    page = case["page"]
    have = [-(-c // page) for c in ctx]
    need = [-(-(c + max(x, 0)) // page) for c, x in zip(ctx, q)]
    max_pages = max(max(have), max(need)) + 1
    taken = sum(b - a for a, b, x in zip(have, need, q) if x > 0)
    n_pages = sum(have) + taken + 50
    gen = torch.Generator("cuda").manual_seed(seed)
    order = torch.randperm(n_pages, device="cuda", generator=gen).to(torch.int32)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    held = torch.arange(max_pages, device="cuda") < i32(have)[:, None]
    table = torch.full((case["seqs"], max_pages), -1, dtype=torch.int32, device="cuda")
    table[held] = order[:sum(have)]
    # the rest is free; room for what ended requests give back
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    free[:n_pages - sum(have)] = order[sum(have):]
    shared = [min(h, pick.randint(0, 3)) for h in have]  # pages in front that others hold too
    return dict(case=case, table=table, n_cached=i32(ctx), n_new=i32(q), n_shared=i32(shared), free=free,
                n_free=i32([n_pages - sum(have)]), n_pages=n_pages, T=sum(max(x, 0) for x in q) + case["pad"])


def prepare(case, seed):
    if case["op"] == "plan":
        return _prepare_plan(case, seed)
    q_lens, ctx, prefix, first = _lengths(case)
    kv_lens = [a + b for a, b in zip(q_lens, ctx)]
    gen = torch.Generator("cuda").manual_seed(seed)
    pick = random.Random(seed)
    T, page, hq, hkv, d = sum(q_lens), case["page"], case["q_heads"], case["kv_heads"], case["head_dim"]
    max_pages = max(-(-n // page) for n in kv_lens) + 1

    # pages: what the window left behind is freed (-1), a group's prefix is held once
    window = case.get("window", 0)
    n_pages = 0
    table = [[-1] * max_pages for _ in kv_lens]
    shared = {}
    for s, n in enumerate(kv_lens):
        g = next((i for i in range(len(prefix)) if first[i] <= s < first[i + 1]), None)
        for p in range(-(-n // page)):
            if case["op"] == "append" and p < ctx[s] // page:
                continue  # only pages that are written have to be there
            if window and p * page >= case["sinks"] and (p + 1) * page <= ctx[s] - window + 1:
                continue
            if g is not None and (p + 1) * page <= prefix[g]:
                if (g, p) not in shared:
                    shared[g, p] = n_pages
                    n_pages += 1
                table[s][p] = shared[g, p]
                continue
            table[s][p] = n_pages
            n_pages += 1
    n_pages += 3
    order = list(range(n_pages))
    pick.shuffle(order)
    table = [[order[p] if p >= 0 else -1 for p in row] for row in table]
    table = torch.tensor(table, dtype=torch.int32, device="cuda")

    def normal(*shape):
        return torch.randn(*shape, device="cuda", dtype=torch.bfloat16, generator=gen)

    # heads with a common direction, which the first token's key has most of: real caches
    # hold such a first token, and scores with a mean; pages of different loudness
    mean = torch.randn(hkv, 1, d, device="cuda", generator=gen)
    k = normal(n_pages, hkv, page, d)
    k += (0.4 * mean).to(torch.bfloat16)
    first_pages = table[:, 0].clamp(min=0).long().unique()
    k[first_pages, :, 0] += (0.6 * mean[:, 0]).to(torch.bfloat16)
    k_cache, k_scale = _quantized(k, page)
    k = normal(n_pages, hkv, page, d)
    k *= torch.exp2(2 * torch.rand(n_pages, hkv, 1, 1, device="cuda", generator=gen) - 1).to(torch.bfloat16)
    v_cache, v_scale = _quantized(k, page)
    del k
    # the last page of a prefix can be the sequences' own copies of it
    for i in range(len(prefix)):
        p = prefix[i] // page
        if prefix[i] % page:
            at = table[first[i]:first[i + 1], p].long()
            for c in (k_cache.view(torch.uint8), v_cache.view(torch.uint8), k_scale, v_scale):
                c[at] = c[at[0]].clone()

    # q, k and v as one projection writes them
    qkv = normal(T, (hq + 2 * hkv) * d)
    q = qkv[:, :hq * d].view(T, hq, d)
    k = qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
    v = qkv[:, (hq + hkv) * d:].view(T, hkv, d)
    q += (0.6 * mean).expand(hkv, hq // hkv, d).reshape(hq, d).to(torch.bfloat16)

    off = [0]
    for n in q_lens:
        off.append(off[-1] + n)
    state = dict(case=case, q=q, k=k, v=v, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
                 table=table, T=T, max_q=max(q_lens), max_kv=max(kv_lens),
                 q_off=torch.tensor(off, dtype=torch.int32, device="cuda"),
                 kv_len=torch.tensor(kv_lens, dtype=torch.int32, device="cuda"))
    if case["op"] == "append":
        n_pos, rot = max(kv_lens) + 8, case["rot"]
        freq = 500000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        angle = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * freq
        state["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        state["axis_pairs"] = _axis_pairs(case)
        if case["axes"] > 1:  # images: time stands still over a frame, height and width run over it
            state["pos"] = torch.randint(0, n_pos, (case["axes"], T), device="cuda", dtype=torch.int32,
                                         generator=gen)
    if prefix:
        state["group_off"] = torch.tensor(first, dtype=torch.int32, device="cuda")
        state["prefix_len"] = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "plan":
        return _plain_plan(state)
    if op == "append":
        return _plain_append(state)
    return _plain_attend(state)


def _own(state, op):
    from lora_serving_device_gb300 import lora as L
    case = state["case"]
    if op == "plan":
        if "ws" not in state:  # what a serving loop keeps: the workspace and the plan's arrays
            state["ws"] = L.batch_plan_workspace(case["seqs"])
            state["plan"] = L.BatchPlan.empty(case["seqs"], state["T"])
        plan = L.batch_plan_t(state["table"], state["n_cached"], state["n_new"], state["free"], state["n_free"],
                              case["page"], state["n_pages"], state["ws"], n_shared=state["n_shared"],
                              out=state["plan"])
        return {"table": state["table"], "free": state["free"], "n_free": plan.n_free, "q_off": plan.q_off,
                "kv_len": plan.kv_len, "slots": plan.slots, "pos": plan.pos}
    if "kv" not in state:  # what a serving loop keeps: the cache's description and the workspace
        state["kv"] = L.PagedKV8bit(state["k_cache"], state["v_cache"], state["k_scale"], state["v_scale"],
                                    state["table"], state["q_off"], state["kv_len"], state["T"],
                                    max_q_len=state["max_q"])
        state["ws"] = L.attn_workspace(state["kv"], case["q_heads"], n_groups=case.get("groups", 0))
    kv, ws = state["kv"], state["ws"]
    if op == "append":
        q = L.kv_append_8bit_t(kv, state["q"], state["k"], state["v"], state["cos_sin"], ws, pos=state.get("pos"),
                               axis_pairs=state["axis_pairs"] if case["axes"] > 1 else None,
                               interleaved=case["interleaved"])
        return _append_outputs(state, q)
    if op == "prefix":
        return L.attn_prefix_8bit_t(kv, state["q"], state["group_off"], state["prefix_len"], ws)
    return L.attn_paged_8bit_t(kv, state["q"], ws, window=case["window"], n_sink=case["sinks"])


def _append_outputs(state, q):
    return {"q": q, "k_cache": state["k_cache"], "v_cache": state["v_cache"], "k_scale": state["k_scale"],
            "v_scale": state["v_scale"]}


def _plain_plan(state):
    """Pages that ended requests held go on top of the stack of free ones, then new pages are
    taken from its top, request by request."""
    case, table, free = state["case"], state["table"], state["free"]
    page, n_new, n_cached = case["page"], state["n_new"], state["n_cached"]
    rows = n_new.clamp(min=0)
    q_off = torch.cat([torch.zeros_like(rows[:1]), rows.cumsum(0, dtype=torch.int32)])
    have, need = (n_cached + page - 1) // page, (n_cached + rows + page - 1) // page
    col = torch.arange(table.shape[1], device="cuda", dtype=torch.int32)
    given = table[(n_new < 0)[:, None] & (col >= state["n_shared"][:, None]) & (col < have[:, None])]
    top = state["n_free"] + given.numel()
    free[state["n_free"] + torch.arange(given.numel(), device="cuda")] = given
    new = (n_new > 0)[:, None] & (col >= have[:, None]) & (col < need[:, None])
    number = new.flatten().cumsum(0).view(new.shape)[new]
    table[new] = free[top - number]
    kv_len = torch.where(n_new < 0, 0, n_cached + rows).to(torch.int32)
    n = state["T"] - case["pad"]
    seq = torch.repeat_interleave(torch.arange(case["seqs"], device="cuda"), rows, output_size=n)
    pos = n_cached[seq] + torch.arange(n, device="cuda", dtype=torch.int32) - q_off[seq]
    slots = table[seq, pos // page].long() * page + pos % page
    rest = torch.full((case["pad"],), -1, device="cuda")
    return {"table": table, "free": free, "n_free": (top - new.sum()).to(torch.int32), "q_off": q_off,
            "kv_len": kv_len, "slots": torch.cat([slots, rest]), "pos": torch.cat([pos, rest.to(torch.int32)])}


def _rows(state):
    """Sequence and cache position of every new token."""
    q_len = (state["q_off"][1:] - state["q_off"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(q_len.numel(), device="cuda"), q_len, output_size=state["T"])
    at = torch.arange(state["T"], device="cuda") - state["q_off"][:-1].long()[seq]
    return seq, state["kv_len"].long()[seq] - q_len[seq] + at


def _rotate(x, cos, sin, rot, interleaved):
    """x [T, heads, d] with its first `rot` values rotated, in the type of cos; cos, sin [T, rot / 2]."""
    x = x.to(cos.dtype)
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    c, s = cos[:, None], sin[:, None]
    a, b = a * c - b * s, b * c + a * s
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _angles(state, pos, table):
    """cos and sin [T, rot / 2] of every token, each pair from its axis' position."""
    half = state["case"]["rot"] // 2
    if "pos" not in state:
        return table[pos, :half], table[pos, half:]
    axis = torch.repeat_interleave(torch.arange(len(state["axis_pairs"]), device="cuda"),
                                   torch.tensor(state["axis_pairs"], device="cuda"), output_size=half)
    at = state["pos"].long()[axis].t()  # [T, half]
    pair = torch.arange(half, device="cuda")
    return table[at, pair], table[at, pair + half]


def _plain_append(state):
    case = state["case"]
    seq, pos = _rows(state)
    page, d = case["page"], case["head_dim"]
    block = min(BLOCK, page)
    cos, sin = _angles(state, pos, state["cos_sin"])
    q = _rotate(state["q"], cos, sin, case["rot"], case["interleaved"]).to(torch.bfloat16)
    k = _rotate(state["k"], cos, sin, case["rot"], case["interleaved"])
    # the blocks that get rows, and the first row that each gets
    place = state["table"][seq, pos // page].long() * page + pos % page
    touched, of_row = (place // block).unique(return_inverse=True)
    start = torch.full_like(touched, block).scatter_reduce_(0, of_row, place % block, "amin")
    before = (torch.arange(block, device="cuda") < start[:, None])[:, None, :, None]
    at_page, at_block = touched * block // page, touched % (page // block)
    for x, cache, scale in ((k, state["k_cache"], state["k_scale"]), (state["v"].float(), state["v_cache"],
                                                                      state["v_scale"])):
        top = torch.zeros(touched.numel(), x.shape[1], device="cuda")
        top.scatter_reduce_(0, of_row[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        byte, old = _exponent(top), scale[at_page, :, at_block].int()
        byte = torch.where((start > 0)[:, None], torch.maximum(byte, old), byte)
        blocks = cache.view(torch.uint8).view(-1, case["kv_heads"], page // block, block, d)
        held = blocks[at_page, :, at_block]  # [blocks, heads, tokens, d]
        moved = torch.ldexp(held.view(torch.float8_e4m3fn).float(), (old - byte)[..., None, None])
        blocks[at_page, :, at_block] = torch.where(before, moved.to(torch.float8_e4m3fn).view(torch.uint8), held)
        scale[at_page, :, at_block] = byte.to(torch.uint8)
        codes = torch.ldexp(x, (127 - byte)[of_row][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        cache.view(torch.uint8)[place // page, :, place % page] = codes
    return _append_outputs(state, q)


def _plain_attend(state):
    """All sequences padded to the longest, the scores of a key head's queries as one product."""
    case = state["case"]
    hkv, d, page = case["kv_heads"], case["head_dim"], case["page"]
    group = case["q_heads"] // hkv
    n, max_q, pages = case["seqs"], state["max_q"], -(-state["max_kv"] // page)
    q_len = (state["q_off"][1:] - state["q_off"][:-1]).long()
    at = torch.arange(max_q, device="cuda")
    token = (state["q_off"][:-1].long()[:, None] + at).clamp(max=state["T"] - 1)  # [n, max_q]
    pos = (state["kv_len"].long() - q_len)[:, None] + at
    block = min(BLOCK, page)

    def rows(cache, scale):
        which = state["table"][:, :pages].clamp(min=0).long()
        x = cache.view(torch.uint8)[which].view(torch.float8_e4m3fn).float()  # [n, pages, hkv, page, d]
        x = x.view(n, pages, hkv, page // block, block, d).mul_(
            torch.exp2(scale[which].float() - 127)[..., None, None])
        return x.view(n, pages, hkv, page, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, pages * page, d)

    q = state["q"][token].view(n, max_q, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * max_q, d)
    score = (q.float() @ rows(state["k_cache"], state["k_scale"]).transpose(2, 3)).mul_(1 / math.sqrt(d))
    score = score.view(n, hkv, group, max_q, pages * page)
    key = torch.arange(pages * page, device="cuda")
    seen = key <= pos[..., None]
    if case.get("window"):
        seen &= (key > pos[..., None] - case["window"]) | (key < case["sinks"])
    seen = seen[:, None, None]
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp_(min=-1e30)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = (score.view(n, hkv, group * max_q, -1) @ rows(state["v_cache"], state["v_scale"]))
    out = (out.view(n, hkv, group, max_q, d) / total.clamp(min=1e-30)).permute(0, 3, 1, 2, 4)
    return out.reshape(n, max_q, hkv * group, d)[at < q_len[:, None]].to(torch.bfloat16)


# ------------------------------------------------------------------ size and value

def _seen_pairs(case):
    """(row, key) pairs that the mask leaves, and the distinct keys of each sequence."""
    q_lens, ctx, prefix, first = _lengths(case)
    window, sinks = case.get("window", 0), case.get("sinks", 0)
    pairs = keys = 0
    for n, c in zip(q_lens, ctx):
        if not n:
            continue
        if not window:
            pairs += n * c + n * (n + 1) // 2
            keys += c + n
            continue
        low = [max(0, p - window + 1) for p in range(c, c + n)]
        pairs += sum(p + 1 - lo + min(sinks, lo) for p, lo in zip(range(c, c + n), low))
        keys += c + n - low[0] + min(sinks, low[0])
    for i, p in enumerate(prefix):
        keys -= p * (first[i + 1] - first[i] - 1)
    return pairs, keys


def work(case):
    q_lens, ctx, _, _ = _lengths(case)
    T, page = sum(max(x, 0) for x in q_lens), case["page"]
    block = min(BLOCK, page)
    if case["op"] == "plan":
        # lengths in and out; a page id in and out; slot and position of a row
        pages = sum(-(-(c + x) // page) + -(-c // page) * -1 for x, c in zip(q_lens, ctx) if x > 0)
        pages += sum(-(-c // page) for x, c in zip(q_lens, ctx) if x < 0)
        rows = T + case["pad"]
        return {"bytes": case["seqs"] * 20 + pages * 8 + rows * 12, "flops": case["seqs"] * 8 + rows * 6}
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "append":
        blocks = sum((c + x - 1) // block - c // block + 1 for x, c in zip(q_lens, ctx))
        return {"bytes": T * d * (hq * 4 + hkv * 2 * 3) + blocks * hkv * 2 +
                T * (case["rot"] * 4 + 4 * (case["axes"] if case["axes"] > 1 else 0)),
                "flops": T * (3 * (hq + hkv) * case["rot"] + 2 * 2 * hkv * d)}
    pairs, keys = _seen_pairs(case)
    return {"bytes": 2 * T * hq * d * 2 + keys * hkv * 2 * (d + 1 / block), "flops": 4 * pairs * hq * d}


def _exact_append(case, state, rows):
    table = state["cos_sin"].double()
    half, page = case["rot"] // 2, case["page"]
    block = min(BLOCK, page)
    pair = 0
    new_q, new_k = state["q"].double(), state["k"].double()
    old_q, old_k = new_q.clone(), new_k.clone()
    at = torch.tensor(rows, device="cuda")
    for axis, count in enumerate(state["axis_pairs"]):
        pos = state["pos"][axis].long() if "pos" in state else at[:, 1]
        for i in range(pair, pair + count):
            c, s = table[pos, i][:, None], table[pos, half + i][:, None]
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, half + i)
            for old, new in ((old_q, new_q), (old_k, new_k)):
                new[..., a] = c * old[..., a] - s * old[..., b]
                new[..., b] = s * old[..., a] + c * old[..., b]
        pair += count
    ids = state["table"].tolist()
    runs = [i for i, (s, p) in enumerate(rows) if i == 0 or rows[i - 1][0] != s or p % block == 0] + [len(rows)]
    out = {"q": new_q, "k_scale": None, "v_scale": None}
    for name, x in (("k", new_k), ("v", state["v"].double())):
        cache, scale = state[name + "_cache"].double(), state[name + "_scale"].double()
        tops = x.abs().amax(-1)
        for i, j in zip(runs, runs[1:]):
            s, p = rows[i]
            where, row = ids[s][p // page], p % page
            top = tops[i:j].amax(0)
            # the least power of two, by logarithm, then held against the border
            e = torch.ceil(torch.log2(top / 448))
            e = torch.where(top > 448 * torch.exp2(e), e + 1, torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e))
            first = row // block * block
            if row > first:
                was = scale[where, :, row // block] - 127
                e = torch.maximum(e, was)
                cache[where, :, first:row] *= torch.exp2(was - e)[:, None, None]
            cache[where, :, row:row + j - i] = x[i:j].transpose(0, 1) * torch.exp2(-e)[:, None, None]
        out[name + "_cache"] = cache
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    state = prepare(case, seed)
    q_lens, ctx, _, _ = _lengths(case)
    hkv, d, page = case["kv_heads"], case["head_dim"], case["page"]
    if case["op"] == "append":
        return _exact_append(case, state, [(s, c + i) for s, (n, c) in enumerate(zip(q_lens, ctx)) for i in range(n)])
    window, sinks = case.get("window", 0), case.get("sinks", 0)
    outs, t = [], 0
    group, block = case["q_heads"] // hkv, min(BLOCK, page)
    for s, (n, c) in enumerate(zip(q_lens, ctx)):
        if not n:
            continue
        key = torch.arange(c + n, device="cuda")
        at, row = state["table"][s].long()[key // page].clamp(min=0), key % page
        k, v = ((state[x + "_cache"].view(torch.uint8)[at, :, row].view(torch.float8_e4m3fn).double() *
                 2.0 ** (state[x + "_scale"][at, :, row // block].double() - 127)[..., None]).transpose(0, 1)
                for x in "kv")  # [hkv, keys, d]
        for a in range(0, n, 1024):
            b = min(n, a + 1024)
            hi = c + b  # keys after the last row's position are seen by none
            pos = torch.arange(c + a, hi, device="cuda")[:, None]
            seen = key[:hi] <= pos
            if window:
                seen &= (key[:hi] > pos - window) | (key[:hi] < sinks)
            q = state["q"][t + a:t + b].double().view(b - a, hkv, group, d).permute(1, 2, 0, 3)
            w = torch.where(seen, (q @ k[:, None, :hi].transpose(2, 3)) / math.sqrt(d), -math.inf)
            w = torch.exp(w - w.amax(-1, keepdim=True))
            o = (w @ v[:, None, :hi]) / w.sum(-1, keepdim=True)
            outs.append(o.permute(2, 0, 1, 3).reshape(b - a, hkv * group, d))
        t += n
    return torch.cat(outs)
