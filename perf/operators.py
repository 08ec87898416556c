"""Performance cases of the paged-cache operators: appending rotated keys and values,
attention over the cache (causal, with a sliding window and first tokens that stay
visible), and attention for batches whose sequences share a prefix.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU, ``run`` is one
pass: the plain form in 32-bit torch operations, or with ``own`` set the library's calls.
``exact`` gives the same outputs in 64 bits from the definition.

The lengths of a case's sequences follow from its values alone, the data from the seed.
"""
import math
import random

import torch

own = False

# ------------------------------------------------------------------ cases

_SHAPE = dict(seqs=1, ctx_min=0, ctx_max=0, q_min=1, q_max=1, q_heads=32, kv_heads=8, head_dim=128,
              page=16)


def _append(name, **kw):
    return dict(_SHAPE, name=name, op="append", rot=kw.get("head_dim", 128), axes=1,
                interleaved=False, **kw)


def _attend(name, **kw):
    return dict(_SHAPE, name=name, op="attend", **{"window": 0, "sinks": 0, **kw})


def _prefix(name, **kw):
    return dict(_SHAPE, name=name, op="prefix", **kw)


def listed():
    return [
        # one decode step of 64 requests, the heads of an 8B-class layer: latency counts
        _append("append, 64 single tokens", seqs=64, ctx_min=100, ctx_max=8000),
        # a prompt of 8192 tokens: bandwidth counts
        _append("append, prompt of 8192", q_min=8192, q_max=8192, page=64),
        # prompts with images: three position axes, odd lengths, seven query heads to a key head
        dict(_append("append, image prompts", seqs=3, q_min=900, q_max=2100, q_heads=28, kv_heads=4,
                     page=32), axes=3),
        # a few single tokens after images; a quarter of the head is rotated, neighbours paired
        dict(_append("append, 7 tokens, 3 axes", seqs=7, ctx_min=50, ctx_max=5000, q_heads=8, kv_heads=8,
                     head_dim=64), rot=32, axes=3, interleaved=True),
        # one user's decode step on a short context: the smallest call
        _attend("attend, 1 token on 500", ctx_min=499, ctx_max=499),
        # a decode batch in ordinary service
        _attend("attend, 64 tokens on 8K", seqs=64, ctx_min=500, ctx_max=8000),
        # few requests on very long contexts: the work has to be split over the keys
        _attend("attend, 3 tokens on 128K", seqs=3, ctx_min=90000, ctx_max=131000, page=64),
        # decode with a window: old pages are already freed, the first four tokens stay
        _attend("attend, window, 96 tokens", seqs=96, ctx_min=200, ctx_max=16000, q_heads=64, head_dim=64,
                page=32, window=4096, sinks=4),
        # a whole prompt: tensor throughput counts
        _attend("attend, prompt of 8192", q_min=8192, q_max=8192, page=64),
        # chunks of prompts and single tokens in one batch, with a window
        _attend("attend, window, mixed chunks", seqs=9, ctx_min=0, ctx_max=9000, q_min=0, q_max=1500,
                window=1024, sinks=16),
        # one system prompt for all 64 requests of a decode step
        _prefix("prefix of 8K, 64 tokens", seqs=64, ctx_min=0, ctx_max=500, groups=1, prefix_min=8192,
                prefix_max=8192),
        # requests of four adapters, each with its own prefix
        _prefix("4 prefixes, 150 tokens", seqs=150, ctx_min=10, ctx_max=900, groups=4, prefix_min=1000,
                prefix_max=5000, q_heads=16, kv_heads=2, head_dim=128, page=64),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    n = min(hi, max(lo, n))
    return n + 1 if n == 3072 else n


def draw(rng):
    heads, kv_heads, dim = rng.choice([(32, 8, 128), (28, 4, 128), (16, 2, 128), (10, 10, 128), (40, 8, 128),
                                       (64, 8, 64), (8, 8, 64), (12, 4, 64), (15, 5, 64), (32, 4, 64)])
    case = dict(q_heads=heads, kv_heads=kv_heads, head_dim=dim, page=rng.choice([16, 32, 64, 128]))
    op = rng.choice(["append", "attend", "attend", "prefix"])
    if op == "append":
        if rng.random() < 0.5:
            case.update(seqs=_log_int(rng, 1, 300), ctx_min=0, ctx_max=_log_int(rng, 20, 9000), q_min=1, q_max=1)
        else:
            seqs = _log_int(rng, 1, 8)
            case.update(seqs=seqs, ctx_min=0, ctx_max=_log_int(rng, 1, 2000), q_min=1,
                        q_max=_log_int(rng, 2, 8000 // seqs))
        return dict(case, op="append", rot=rng.choice([dim, dim, dim // 2]), axes=rng.choice([1, 1, 3]),
                    interleaved=rng.random() < 0.4)
    if op == "prefix":
        seqs = _log_int(rng, 2, 150)
        return dict(case, op="prefix", seqs=seqs, ctx_min=0, ctx_max=_log_int(rng, 1, 900), q_min=1, q_max=1,
                    groups=rng.randint(1, min(4, seqs)), prefix_min=50, prefix_max=_log_int(rng, 100, 6000))
    window, sinks = rng.choice([(0, 0), (0, 0), (_log_int(rng, 60, 4096), rng.randint(0, 40))])
    if rng.random() < 0.6:  # single tokens
        seqs = _log_int(rng, 1, 100)
        case.update(seqs=seqs, ctx_min=0, ctx_max=_log_int(rng, 30, min(100000, 600000 // seqs)), q_min=1, q_max=1)
    else:  # prompts and chunks
        seqs = _log_int(rng, 1, 6)
        q = _log_int(rng, 2, 4000 // seqs)
        case.update(seqs=seqs, ctx_min=0, ctx_max=_log_int(rng, 1, 5000), q_min=rng.randint(0, 1), q_max=q)
    return dict(case, op="attend", window=window, sinks=sinks)


def _lengths(case):
    """New tokens and cached tokens before them of each sequence, prefix lengths and first
    sequences of the groups: functions of the case's values alone."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["seqs"]
    q = [r.randint(case["q_min"], case["q_max"]) for _ in range(n)]
    if case["op"] == "attend" and n > 4 and case["q_max"] > 1:
        q[1], q[2] = 1, 1  # single tokens among the chunks
    q[0] = max(q[0], case["q_max"])
    ctx = [r.randint(case["ctx_min"], case["ctx_max"]) for _ in range(n)]
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

def prepare(case, seed):
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
    # hold such a first token, and scores with a mean
    mean = torch.randn(hkv, 1, d, device="cuda", generator=gen)
    k_cache, v_cache = normal(n_pages, hkv, page, d), normal(n_pages, hkv, page, d)
    k_cache += (0.4 * mean).to(torch.bfloat16)
    first_pages = table[:, 0].clamp(min=0).long().unique()
    k_cache[first_pages, :, 0] += (0.6 * mean[:, 0]).to(torch.bfloat16)
    # the last page of a prefix can be the sequences' own copies of it
    for i in range(len(prefix)):
        rest, p = prefix[i] % page, prefix[i] // page
        if rest:
            at = table[first[i]:first[i + 1], p].long()
            k_cache[at, :, :rest] = k_cache[at[0], :, :rest].clone()
            v_cache[at, :, :rest] = v_cache[at[0], :, :rest].clone()

    # q, k and v as one projection writes them
    qkv = normal(T, (hq + 2 * hkv) * d)
    q = qkv[:, :hq * d].view(T, hq, d)
    k = qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
    v = qkv[:, (hq + hkv) * d:].view(T, hkv, d)
    q += (0.6 * mean).expand(hkv, hq // hkv, d).reshape(hq, d).to(torch.bfloat16)

    off = [0]
    for n in q_lens:
        off.append(off[-1] + n)
    state = dict(case=case, q=q, k=k, v=v, k_cache=k_cache, v_cache=v_cache, table=table, T=T,
                 max_q=max(q_lens), max_kv=max(kv_lens),
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
    if op == "append":
        return _plain_append(state)
    return _plain_attend(state)


def _own(state, op):
    from lora_serving_device_gb300 import lora as L
    case = state["case"]
    if "kv" not in state:  # what a serving loop keeps: the cache's description and the workspace
        state["kv"] = L.PagedKV(state["k_cache"], state["v_cache"], state["table"], state["q_off"],
                                state["kv_len"], state["T"], max_q_len=state["max_q"])
        state["ws"] = L.attn_workspace(state["kv"], case["q_heads"], n_groups=case.get("groups", 0))
    kv, ws = state["kv"], state["ws"]
    if op == "append":
        q = L.kv_append_t(kv, state["q"], state["k"], state["v"], state["cos_sin"], ws, pos=state.get("pos"),
                          axis_pairs=state["axis_pairs"] if case["axes"] > 1 else None,
                          interleaved=case["interleaved"])
        return {"q": q, "k_cache": state["k_cache"], "v_cache": state["v_cache"]}
    if op == "prefix":
        return L.attn_prefix_t(kv, state["q"], state["group_off"], state["prefix_len"], ws)
    return L.attn_paged_t(kv, state["q"], ws, window=case["window"], n_sink=case["sinks"])


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
    cos, sin = _angles(state, pos, state["cos_sin"])
    q = _rotate(state["q"], cos, sin, case["rot"], case["interleaved"]).to(torch.bfloat16)
    k = _rotate(state["k"], cos, sin, case["rot"], case["interleaved"]).to(torch.bfloat16)
    page = state["table"][seq, pos // case["page"]].long()
    state["k_cache"][page, :, pos % case["page"]] = k
    state["v_cache"][page, :, pos % case["page"]] = state["v"]
    return {"q": q, "k_cache": state["k_cache"], "v_cache": state["v_cache"]}


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

    def rows(cache):
        x = cache[state["table"][:, :pages].clamp(min=0).long()]  # [n, pages, hkv, page, d]
        return x.permute(0, 2, 1, 3, 4).reshape(n, hkv, pages * page, d).float()

    q = state["q"][token].view(n, max_q, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * max_q, d)
    score = (q.float() @ rows(state["k_cache"]).transpose(2, 3)).mul_(1 / math.sqrt(d))
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
    out = (score.view(n, hkv, group * max_q, -1) @ rows(state["v_cache"])).view(n, hkv, group, max_q, d)
    out = (out / total.clamp(min=1e-30)).permute(0, 3, 1, 2, 4).reshape(n, max_q, hkv * group, d)
    return out[at < q_len[:, None]].to(torch.bfloat16)


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
    T = sum(_lengths(case)[0])
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "append":
        moved = T * (hq + 2 * hkv) * d * 2
        return {"bytes": 2 * moved + T * (case["rot"] * 4 + 4 * (case["axes"] if case["axes"] > 1 else 0)),
                "flops": 3 * T * (hq + hkv) * case["rot"]}
    pairs, keys = _seen_pairs(case)
    return {"bytes": 2 * T * hq * d * 2 + keys * hkv * d * 2 * 2, "flops": 4 * pairs * hq * d}


def exact(case, seed):
    state = prepare(case, seed)
    q_lens, ctx, _, _ = _lengths(case)
    hkv, d, page = case["kv_heads"], case["head_dim"], case["page"]
    if case["op"] == "append":
        table = state["cos_sin"].double()
        out = {"q": state["q"].double(), "k_cache": state["k_cache"].double(), "v_cache": state["v_cache"].double()}
        rows = torch.tensor([[s, c + i] for s, (n, c) in enumerate(zip(q_lens, ctx)) for i in range(n)],
                            device="cuda")
        half = case["rot"] // 2
        pair = 0
        new_q, new_k = out["q"].clone(), state["k"].double()
        old_q, old_k = out["q"], new_k.clone()
        for axis, count in enumerate(state["axis_pairs"]):
            pos = state["pos"][axis].long() if "pos" in state else rows[:, 1]
            for i in range(pair, pair + count):
                c, s = table[pos, i][:, None], table[pos, half + i][:, None]
                a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, half + i)
                for old, new in ((old_q, new_q), (old_k, new_k)):
                    new[..., a] = c * old[..., a] - s * old[..., b]
                    new[..., b] = s * old[..., a] + c * old[..., b]
            pair += count
        out["q"] = new_q
        at = state["table"][rows[:, 0], rows[:, 1] // page].long()
        out["k_cache"][at, :, rows[:, 1] % page] = new_k
        out["v_cache"][at, :, rows[:, 1] % page] = state["v"].double()
        return out
    window, sinks = case.get("window", 0), case.get("sinks", 0)
    outs, t = [], 0
    group = case["q_heads"] // hkv
    for s, (n, c) in enumerate(zip(q_lens, ctx)):
        if not n:
            continue
        key = torch.arange(c + n, device="cuda")
        at = state["table"][s].long()[key // page].clamp(min=0)
        k = state["k_cache"][at, :, key % page].double().transpose(0, 1)  # [hkv, keys, d]
        v = state["v_cache"][at, :, key % page].double().transpose(0, 1)
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
