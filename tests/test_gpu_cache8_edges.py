"""Edges of the 8-bit cache's operators on the GPU: items of one key tile by the hundred, batches of
all sizes over one workspace, graphs that share one, how far weights and q are off, many groups, and
appends that meet others' rows.

Tolerances are those of test_gpu_cache8.py, derived there, unless a test derives its own.
"""
import numpy as np
import pytest

from oracle import attn_ref as R
from oracle import cache8_ref as C
from tests.test_gpu_cache8 import (Case8, L, U, attend, check_rows, dequantize_t, prefix_attend,  # noqa: F401
                                   random_cache)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d,rows", [(8, 2, 128, 1), (8, 2, 64, 1), (16, 2, 64, 1), (32, 2, 128, 1), (8, 2, 128, 33),
                                           (16, 2, 64, 40)])
@pytest.mark.parametrize("page", [8, 16])
def test_items_of_one_tile_repeat_bit_for_bit(L, hq, hkv, d, rows, page):
    """Every item is one key tile or two, some with rows for one half only: values against fp64, and
    the same bits from every call."""
    import torch
    torch.manual_seed(d + hq)
    n = 304 if rows > 1 else 608
    q_lens = torch.randint(1, rows + 1, (n,))
    kv_len = (q_lens + torch.randint(0, 170, (n,))).int()
    pages = -(-int(kv_len.max()) // page)
    table = torch.randperm(n * pages, device="cuda").to(torch.int32).view(n, pages)
    cache = random_cache(torch, n * pages, hkv, page, d)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), q_lens.cumsum(0)])
    T = int(off[-1])
    q = (0.1 * torch.randn(T, hq, d, device="cuda")).to(torch.bfloat16)
    kv = L.PagedKV8bit(*cache, table, off.int().cuda(), kv_len.cuda(), T, max_q_len=rows)
    ws = L.attn_workspace(kv, hq)
    first = L.attn_paged_8bit_t(kv, q, ws).clone()
    for s in range(0, n, 7):
        m, a, b = int(kv_len[s]), int(off[s]), int(off[s + 1])
        k, v = (dequantize_t(torch, cache[i][table[s].long()], cache[i + 2][table[s].long()]).transpose(1, 2)
                .reshape(-1, hkv, d)[:m].repeat_interleave(hq // hkv, 1) for i in (0, 1))
        check_rows(torch, first[a:b], q[a:b], k, v, m - (b - a))
    out = torch.empty_like(q)
    for _ in range(200):
        assert torch.equal(L.attn_paged_8bit_t(kv, q, ws, out=out).view(torch.int16), first.view(torch.int16))
    assert L.get_error_t(ws) == 0


def test_one_workspace_for_batches_of_all_sizes_and_both_caches(L):
    import torch
    from tests.test_gpu_attn import Case
    cases = [Case8([1], [900], 8, 1, 64, 16, seed=1), Case8([300], [200], 8, 2, 128, 16, seed=2),
             Case8([1] * 70, [9 * i for i in range(70)], 4, 2, 64, 32, seed=3), Case([1, 40], [700, 90], 8, 2, 128, 16),
             Case8([3, 50], [700, 100], 16, 2, 128, 16, seed=4, window=60, n_sink=3)]
    groups = ([0, 40], [300])
    shared = Case8([1] * 40, [300 + i for i in range(40)], 8, 2, 128, 16, seed=5, groups=groups)
    off, pl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in groups)
    ws = torch.zeros(max([L.attn_workspace(shared.kv(L), 8, 1).numel()] +
                         [L.attn_workspace(c.kv(L), c.hq).numel() for c in cases]), dtype=torch.uint8, device="cuda")
    ws[4096:].fill_(0xFF)     # whatever earlier calls left behind the counters
    for _ in range(2):
        for c in cases + [shared] + cases[::-1]:
            if c is shared:
                L.attn_prefix_8bit_t(c.kv(L), c.q, off, pl, ws, out=c.out)
            else:
                call = L.attn_paged_8bit_t if isinstance(c, Case8) else L.attn_paged_t
                call(c.kv(L), c.q, ws, window=c.window, n_sink=c.n_sink, out=c.out)
            c.check(c.out)
    assert L.get_error_t(ws) == 0


def test_two_captured_graphs_share_a_workspace(L):
    import torch
    a, b = Case8([1, 1], [3000, 90], 8, 2, 128, 16, seed=1), Case8([60, 1], [500, 2000], 8, 2, 64, 16, seed=2)
    kvs = [c.kv(L) for c in (a, b)]
    ws = torch.zeros(max(L.attn_workspace(kv, 8).numel() for kv in kvs), dtype=torch.uint8, device="cuda")
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for c, kv in zip((a, b), kvs):
        with torch.cuda.stream(side):
            L.attn_paged_8bit_t(kv, c.q, ws, out=c.out)
            side.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                L.attn_paged_8bit_t(kv, c.q, ws, out=c.out)
    for i in (0, 1, 1, 0, 1, 0):
        c = (a, b)[i]
        c.out.fill_(7.0)
        graphs[i].replay()
        c.check(c.out)
    assert L.get_error_t(ws) == 0


@pytest.mark.parametrize("q_lens,hq,hkv,d", [([1] * 9, 8, 2, 128), ([1] * 9, 8, 8, 64), ([1] * 9, 32, 2, 128),
                                             ([4, 2, 4], 8, 2, 64), ([2, 1], 144, 1, 64), ([60, 3], 8, 2, 128),
                                             ([150], 4, 4, 64)])
def test_how_far_weights_and_q_are_off(L, q_lens, hq, hkv, d):
    """Against a bound that one bf16 a weight would not keep.  A weight's three terms leave 2^-12 of it
    or 2^-23 of the row's largest, one f16 2^-11; the exponential and the sums 2^-20; q's terms and the
    scores' sums what test_gpu_cache8.py derives.  The oracle with weights rounded to bf16 exceeds it."""
    import torch
    c = Case8(q_lens, [3 * i + 20 for i in range(len(q_lens))], hq, hkv, d, 16, seed=hq)
    kv = c.kv(L)
    ws = L.attn_workspace(kv, hq)
    got = L.attn_paged_8bit_t(kv, c.q, ws, out=c.out).double().cpu().numpy()
    assert L.get_error_t(ws) == 0
    k, v = ([x.double().numpy() for x in rows] for rows in (c.rows_k, c.rows_v))
    ref, wv = R.attention(c.q_host, k, v, c.q_off, c.kv_len, d ** -0.5)
    few = max(q_lens) * (hq // hkv) <= 16 or hq // hkv > 128
    bound = U * np.abs(ref)
    for s in range(len(q_lens)):
        a, b = c.q_off[s], c.q_off[s + 1]
        score = d ** -0.5 * 2.0 ** -17 * np.abs(c.q_host[a:b]).max() * np.abs(k[s]).sum(-1).max()
        bound[a:b] += (1 + U) * ((2.0 ** -12 if few else 2.0 ** -11) + 4 * score + 2.0 ** -20) * wv[a:b]
        bound[a:b] += len(k[s]) * 2.0 ** -23 * np.abs(v[s]).max()
    assert np.all(np.abs(got - ref) <= bound)
    once = np.empty_like(ref)
    for t, s, p in R.positions(c.q_off, c.kv_len):
        for h in range(hq):
            g = h // (hq // hkv)
            x = d ** -0.5 * (k[s][:p + 1, g] @ c.q_host[t, h])
            w = np.exp(x - x.max())
            once[t, h] = torch.from_numpy(w).bfloat16().double().numpy() @ v[s][:p + 1, g] / w.sum()
    assert np.linalg.norm(got - ref) < np.linalg.norm(once - ref) + np.linalg.norm(U * ref)


@pytest.mark.parametrize("n_groups", [2, 17, 40])
def test_many_groups(L, n_groups):
    sizes = [[2, 1, 0, 3][i % 4] for i in range(n_groups)]
    sizes[0] = sizes[-1] = 0
    first = [0] + [int(x) for x in np.cumsum(sizes)]
    prefix = [0 if i % 5 == 4 else 15 + 20 * (i % 6) for i in range(n_groups)]
    group = [g for g in range(n_groups) for _ in range(sizes[g])]
    ctx = [prefix[g] + 3 * (i % 4) for i, g in enumerate(group)] + [50, 0]
    q = [1 + (7 if i % 9 == 3 else 0) for i in range(len(ctx))]
    groups = (first, prefix)
    prefix_attend(L, Case8(q, ctx, 8, 2, 64, 16, seed=n_groups, groups=groups, pad_rows=2), groups)


def test_more_sequences_and_groups_than_are_sized_ahead(L):
    rng = np.random.default_rng(4)
    n = 2200
    prefix = [int(x) for x in rng.integers(0, 20, n)]
    groups = (list(range(n + 1)), prefix)
    q = [1] * n
    q[2100] = 40
    prefix_attend(L, Case8(q, [p + int(x) for p, x in zip(prefix, rng.integers(0, 5, n))], 2, 1, 64, 16, seed=12,
                           groups=groups), groups)


@pytest.mark.parametrize("page", [8, 16, 64])
@pytest.mark.parametrize("max_q", [1, 64])
def test_appends_beside_others_blocks(L, page, max_q):
    """Requests whose runs begin and end anywhere, in one call: every block gets its own rows, codes of others
    and of rows behind the run stay, whatever the kernel (max_q_len is a hint)."""
    import torch
    rng = np.random.default_rng(page)
    hkv, d, n = 3, 64, 40
    block = min(16, page)
    ctx = rng.integers(0, 100, n)
    new = rng.integers(0, 50, n)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T, pages = int(off[-1]) + 1, -(-150 // page)
    table = rng.permutation(n * pages).reshape(n, pages).astype(np.int32)
    codes = [rng.integers(0, 127, (n * pages, hkv, page, d)).astype(np.uint8) for _ in range(2)]
    scales = [rng.integers(100, 130, (n * pages, hkv, page // block)).astype(np.uint8) for _ in range(2)]
    dev = [torch.from_numpy(x.copy()).cuda() for x in codes + scales]
    x = [torch.from_numpy((rng.standard_normal((T, hkv, d)) * 2.0 ** rng.integers(-5, 5, (T, 1, 1))).astype(np.float32))
         .bfloat16() for _ in range(2)]
    kv = L.PagedKV8bit(*dev, torch.from_numpy(table).cuda(), torch.from_numpy(off).cuda(),
                       torch.from_numpy((ctx + new).astype(np.int32)).cuda(), T, max_q_len=max_q)
    ws = L.attn_workspace(kv, 3)
    L.kv_append_8bit_t(kv, None, x[0].cuda(), x[1].cuda(), None, ws)
    assert L.get_error_t(ws) == 0
    for s in range(n):
        places = [(int(table[s, p // page]), p % page) for p in range(ctx[s], ctx[s] + new[s])]
        for i in (0, 1):
            C.append(codes[i], scales[i], x[i][off[s]:off[s + 1]].double().numpy(), places)
    for got, want in zip(dev, codes + scales):
        assert np.array_equal(got.cpu().numpy(), want)


def test_append_of_a_long_prompt_past_the_first_blocks(L):
    """More rows than one wave of blocks of warps holds, against torch."""
    import torch
    torch.manual_seed(0)
    n, hq, hkv, d, page = 20011, 4, 2, 128, 32
    cache = L.PagedKV8bit.empty_cache(-(-n // page), hkv, page, d)
    table = torch.randperm(-(-n // page), device="cuda").to(torch.int32)[None]
    q, k, v = (torch.randn(n, h, d, device="cuda").bfloat16() for h in (hq, hkv, hkv))
    kv = L.PagedKV8bit(*cache, table, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                       torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    ws = L.attn_workspace(kv, hq)
    got = L.kv_append_8bit_t(kv, q, k, v, None, ws)
    assert torch.equal(got, q) and L.get_error_t(ws) == 0
    for x, i in ((k, 0), (v, 1)):
        y = dequantize_t(torch, cache[i], cache[i + 2])[table[0].long()].transpose(1, 2).reshape(-1, hkv, d)[:n]
        step = torch.exp2(cache[i + 2][table[0].long()].repeat_interleave(16, -1).transpose(1, 2)
                          .reshape(-1, hkv)[:n].double() - 137)[..., None]
        assert ((x.double() - y).abs() <= 2.0 ** -4 * x.double().abs() + step).all()


def test_two_streams_at_once(L):
    """Calls over one cache on two streams with workspaces of their own: the bits of the calls alone."""
    import torch
    torch.manual_seed(0)
    hq, hkv, d, page, n = 8, 2, 128, 16, 30
    codes, scales = random_cache_t(torch, n * 80, hkv, page, d)
    table = torch.randperm(n * 80, device="cuda").int().view(n, 80)
    jobs = []
    for q_lens in ([1] * n, [40 + i for i in range(n)]):
        off = torch.tensor([0] + q_lens, device="cuda").cumsum(0).int()
        lens = torch.randint(200, 80 * page, (n,), device="cuda", dtype=torch.int32)
        kv = L.PagedKV8bit(*codes, *scales, table, off, lens, sum(q_lens), max_q_len=max(q_lens))
        q = torch.randn(kv.T, hq, d, device="cuda").bfloat16()
        ws = L.attn_workspace(kv, hq)
        want = L.attn_paged_8bit_t(kv, q, ws)
        jobs.append((kv, q, L.attn_workspace(kv, hq), want, torch.empty_like(q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for kv, q, ws, want, out, st in jobs:
            L.attn_paged_8bit_t(kv, q, ws, out=out, stream=st)
    torch.cuda.synchronize()
    for kv, q, ws, want, out, st in jobs:
        assert torch.equal(out, want) and L.get_error_t(ws) == 0


def random_cache_t(torch, n_pages, hkv, page, d):
    codes = [torch.randint(0, 127, (n_pages, hkv, page, d), dtype=torch.uint8, device="cuda") ^
             torch.randint(0, 2, (n_pages, hkv, page, d), dtype=torch.uint8, device="cuda") * 128 for _ in range(2)]
    scales = [torch.randint(116, 120, (n_pages, hkv, page // min(16, page)), dtype=torch.uint8, device="cuda")
              for _ in range(2)]
    return codes, scales


def test_workspaces_elsewhere_are_refused(L):
    """A workspace in host memory, or not contiguous, reaches no kernel."""
    import torch
    hq, hkv, d, page = 4, 2, 64, 16
    cache = L.PagedKV8bit.empty_cache(2, hkv, page, d)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, off, lens = i32([[0, 1]]), i32([0, 1]), i32([1])
    kv = L.PagedKV8bit(*cache, table, off, lens, 1)
    q, k = (torch.zeros(1, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv))
    bad = [torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(1 << 21, dtype=torch.uint8, device="cuda")[::2]]
    for ws in bad:
        for call in (lambda: L.kv_append_8bit_t(kv, q, k, k, None, ws), lambda: L.attn_paged_8bit_t(kv, q, ws),
                     lambda: L.attn_prefix_8bit_t(kv, q, i32([0, 1]), i32([0]), ws),
                     lambda: L.batch_plan_t(table, lens, i32([0]), i32([0]), i32([1]), page, 2, ws, T=1)):
            with pytest.raises(TypeError, match="ws"):
                call()
