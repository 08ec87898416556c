"""Edges of the paged-cache operators on the GPU: items of one key tile by the hundred, windows
and positions at the types' ends, block-table entries of any value, other streams, empty
batches, many sequences and groups, and head counts of every route.

Tolerances are those of test_gpu_attn.py, derived there, unless a test derives its own.
"""
import numpy as np
import pytest

from tests.test_gpu_attn import HEADS, U, Case, L, attend, prefix_attend  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 2, 64), (16, 2, 64), (32, 2, 128)])
def test_items_of_one_tile_repeat_bit_for_bit(L, hq, hkv, d):
    """Every item is one key tile or two, so that each moves its maxima in the tile that its
    sums follow: values against fp64, and the same bits from every call."""
    import torch
    torch.manual_seed(d + hq)
    n, page = 608, 16
    kv_len = torch.randint(1, 200, (n,), dtype=torch.int32, device="cuda")
    pages = -(-200 // page)
    table = torch.randperm(n * pages, device="cuda").to(torch.int32).view(n, pages)
    kc, vc = (torch.randn(n * pages, hkv, page, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = (3 * torch.randn(n, hq, d, device="cuda")).to(torch.bfloat16)
    kv = L.PagedKV(kc, vc, table, torch.arange(n + 1, dtype=torch.int32, device="cuda"), kv_len, n, max_q_len=1)
    ws = L.attn_workspace(kv, hq)
    first = L.attn_paged_t(kv, q, ws).clone()
    k, v = (c[table.long()].transpose(2, 3).reshape(n, -1, hkv, d).double().repeat_interleave(hq // hkv, 2)
            for c in (kc, vc))
    x = torch.einsum("thd,tnhd->thn", q.double(), k) * d ** -0.5
    x = x.masked_fill(torch.arange(pages * page, device="cuda") >= kv_len[:, None, None], -float("inf"))
    w = x.softmax(-1)
    ref, wv = (torch.einsum("thn,tnhd->thd", w, y) for y in (v, v.abs()))
    # (scores three times as large: their error's share of the bound is, too)
    assert ((first.double() - ref).abs() <= U * ref.abs() + (U + 3 * 2.0 ** -12) * wv).all()
    out = torch.empty_like(q)
    for _ in range(200):
        assert torch.equal(L.attn_paged_t(kv, q, ws, out=out).view(torch.int16), first.view(torch.int16))
    assert L.get_error_t(ws) == 0


@pytest.mark.parametrize("window,n_sink", [(2 ** 31 - 1, 0), (2 ** 31 - 2, 2 ** 31 - 1), (2 ** 31 - 20, 3), (1, 0),
                                           (30, 2), (130, 0)])
def test_windows_with_rows_before_the_first_position(L, window, n_sink):
    # the first row's position is -20 or lower where the window may be the type's largest
    attend(L, Case([140], [-20], 4, 2, 64, 16, seed=5, window=window, n_sink=n_sink))
    attend(L, Case([3, 30, 1, 400], [-2, -21, -1, -130], 4, 2, 128, 32, seed=6, window=window, n_sink=n_sink))
    attend(L, Case([4, 4, 1, 1], [-3, -4, 300, 5], 8, 4, 64, 16, seed=7, window=window, n_sink=n_sink))


@pytest.mark.parametrize("wild", [-2 ** 31, -2 ** 31 + 1, -1, 2 ** 31 - 1])
@pytest.mark.parametrize("d", [64, 128])
def test_a_missing_page_may_have_any_id_outside_the_cache(L, wild, d):
    """Missing pages in the first, a middle and the last tile of single tokens and of a chunk.
    The batch of whole pages before leaves its keys and values in the shared memory."""
    for q_lens, ctx in (([1, 1, 1], [100, 700, 20]), ([1, 20, 150], [100, 60, 400])):
        missing = {(0, 2), (0, 6), (1, 0), (1, 3), (2, 1)}
        attend(L, Case(q_lens, ctx, 4, 2, d, 16, seed=9))
        c = Case(q_lens, ctx, 4, 2, d, 16, seed=9, missing=missing)
        for s, p in missing:
            c.table[s, p] = wild
        attend(L, c, err=L.DEVERR_BAD_PAGE)


@pytest.mark.parametrize("op", ["append", "paged", "prefix"])
def test_results_of_a_call_on_another_stream_are_made_there(L, op):
    """The current stream is behind: a tensor of the result's size that it has still to write is
    let go on the host.  The call's result must not be in that memory."""
    import torch
    groups = ([0, 2], [40])
    c = Case([1, 1], [300, 40], 4, 2, 64, 16, seed=4, groups=groups)
    kv = c.kv(L)
    ws = L.attn_workspace(kv, c.hq, n_groups=1)
    off, plen = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in groups)
    k = torch.zeros(c.T, c.hkv, c.d, dtype=torch.bfloat16, device="cuda")

    def call(stream=None):
        if op == "append":
            return L.kv_append_t(kv, c.q, k, k, None, ws, stream=stream)
        if op == "prefix":
            return L.attn_prefix_t(kv, c.q, off, plen, ws, stream=stream)
        return L.attn_paged_t(kv, c.q, ws, stream=stream)

    want = call().clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    late = torch.full_like(want, 7.0)
    where = late.data_ptr()
    del late
    got = call(side)
    torch.cuda.synchronize()
    assert got.data_ptr() != where and torch.equal(got, want)


def test_empty_batches(L):
    import torch
    c = Case([0, 0, 0], [5, 0, 40], 4, 2, 64, 16, seed=1, groups=([0, 3], [2]))
    kv = c.kv(L)
    ws = L.attn_workspace(kv, 4, n_groups=1)
    q, k = (torch.empty(0, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    pos = torch.empty(3, 0, dtype=torch.int32, device="cuda")
    off, plen = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 3], [2]))
    cs = L.rope_table(64, 64)
    assert L.kv_append_t(kv, q, k, k, cs, ws).shape == q.shape
    assert L.kv_append_t(kv, q, k, k, cs, ws, pos=pos, axis_pairs=(8, 12, 12)).shape == q.shape
    assert L.kv_append_t(kv, None, k, k, cs, ws) is None
    assert L.attn_paged_t(kv, q, ws).shape == q.shape
    assert L.attn_prefix_t(kv, q, off, plen, ws).shape == q.shape
    assert L.get_error_t(ws) == 0


@pytest.mark.parametrize("n_groups", [2, 16, 17, 40])
def test_sequences_before_the_first_group_share_nothing(L, n_groups):
    # (many groups are searched another way than few)
    import torch
    first = [3 + 2 * i for i in range(n_groups + 1)]
    prefix = [20 + 5 * (i % 7) for i in range(n_groups)]
    ctx = [9, 100, 30] + [prefix[i // 2] + i % 3 for i in range(2 * n_groups)] + [70]
    groups = (first, prefix)
    c = Case([1] * len(ctx), ctx, 4, 2, 64, 16, seed=n_groups, groups=groups)
    kv = c.kv(L)
    ws = L.attn_workspace(kv, 4, n_groups=n_groups)
    ws[4096:].fill_(0x7F)      # a prefix part that nothing wrote would show
    off, plen = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in groups)
    c.check(L.attn_prefix_t(kv, c.q, off, plen, ws, out=c.out))
    assert L.get_error_t(ws) == 0


# ------------------------------------------------------------------ branches by size

@pytest.mark.parametrize("max_q", [1, None])
def test_more_sequences_than_are_sized_ahead(L, max_q):
    """2300 sequences, with prompts and empty ones past the first 2048, by both routes."""
    rng = np.random.default_rng(3)
    q = [int(x) for x in rng.integers(0, 2, 2300)]
    ctx = [int(x) for x in rng.integers(0, 40, 2300)]
    for s, n in ((2047, 9), (2048, 33), (2049, 0), (2100, 70), (2299, 12)):
        q[s] = n
    attend(L, Case(q, ctx, 2, 1, 64, 16, seed=11), max_q=max_q)


def test_more_groups_than_are_sized_ahead(L):
    rng = np.random.default_rng(4)
    n = 2200
    prefix = [int(x) for x in rng.integers(0, 20, n)]
    groups = (list(range(n + 1)), prefix)
    q = [1] * n
    q[2100] = 40
    prefix_attend(L, Case(q, [p + int(x) for p, x in zip(prefix, rng.integers(0, 5, n))], 2, 1, 64, 16, seed=12,
                          groups=groups), groups)


@pytest.mark.parametrize("n_groups", [16, 17, 33])
def test_many_groups(L, n_groups):
    # empty groups at the ends and in the middle, prefixes of nothing, sequences after the last
    sizes = [[2, 1, 0, 3][i % 4] for i in range(n_groups)]
    sizes[0] = sizes[-1] = sizes[n_groups // 2] = 0
    first = [0] + [int(x) for x in np.cumsum(sizes)]
    prefix = [0 if i % 5 == 4 else 15 + 20 * (i % 6) for i in range(n_groups)]
    group = [g for g in range(n_groups) for _ in range(sizes[g])]
    ctx = [prefix[g] + 3 * (i % 4) for i, g in enumerate(group)] + [50, 0]
    q = [1 + (7 if i % 9 == 3 else 0) for i in range(len(ctx))]
    groups = (first, prefix)
    prefix_attend(L, Case(q, ctx, 8, 2, 64, 16, seed=n_groups, groups=groups, pad_rows=2), groups)


@pytest.mark.parametrize("group", [16, 17, 64, 65, 100, 128, 129, 144])
@pytest.mark.parametrize("d", [64, 128])
def test_query_heads_of_one_key_head(L, group, d):
    """Up to 16: rows in N; to 128: whole tokens in a half (one from 65 on); above: cut into
    tiles of 16 rows across tokens."""
    attend(L, Case([1, 1, 1], [0, 150, 300], 2 * group, 2, d, 16, seed=group))
    attend(L, Case([9, 1, 0, 3], [140, 37, 4, 0], group, 1, d, 32, seed=group, window=60, n_sink=3, pad_rows=1))
    groups = ([0, 3], [150])
    prefix_attend(L, Case([1, 5, 1], [150, 160, 300], group, 1, d, 16, seed=group, groups=groups), groups)


# ------------------------------------------------------------------ weights as a pair of bf16

@pytest.mark.parametrize("q_len,hq,hkv,d", [(1, 8, 2, 128), (1, 8, 8, 64), (1, 16, 2, 64), (1, 32, 2, 128),
                                            (4, 8, 2, 64), (2, 144, 1, 64)])
@pytest.mark.parametrize("prefix", [0, 3])
def test_few_rows_take_the_weights_as_a_pair(L, q_len, hq, hkv, d, prefix):
    """Against a bound that one bf16 a weight would not keep.  The value and its rest leave 2^-16
    of a weight, the product adds 16 keys at a time in fp32 (below 2^-17 over these lengths), the
    exponential and the sum 2^-20: below 2^-15 sum_j w_j |v_j|, beside the scores' 2^-12 and the
    rounding of the result (2^-8 of it).  The oracle with weights rounded once exceeds it."""
    import torch
    from oracle import attn_ref as R
    group = hq // hkv
    n = 9 if not prefix or group > 128 else max(1, 16 // (q_len * group))
    ctx = [prefix + 3 * i for i in range(n)]
    groups = ([0, n], [prefix]) if prefix else None
    c = Case([q_len] * n, ctx, hq, hkv, d, 16, seed=hq, groups=groups)
    kv = c.kv(L)
    ws = L.attn_workspace(kv, hq, n_groups=1 if prefix else 0)
    if prefix:
        off, plen = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in groups)
        got = L.attn_prefix_t(kv, c.q, off, plen, ws, out=c.out)
    else:
        got = L.attn_paged_t(kv, c.q, ws, out=c.out)
    assert L.get_error_t(ws) == 0
    k, v = ([x.double().numpy() for x in rows] for rows in (c.rows_k, c.rows_v))
    ref, wv = R.attention(c.q_host, k, v, c.q_off, c.kv_len, d ** -0.5)
    bound = U * np.abs(ref) + (1 + U) * (2.0 ** -15 + 2.0 ** -12) * wv
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= bound)
    once = np.empty_like(ref)
    for t, s, p in R.positions(c.q_off, c.kv_len):
        for h in range(hq):
            g = h // group
            x = d ** -0.5 * (k[s][:p + 1, g] @ c.q_host[t, h])
            w = np.exp(x - x.max())
            once[t, h] = torch.from_numpy(w).bfloat16().double().numpy() @ v[s][:p + 1, g] / w.sum()
    assert np.any(np.abs(once - ref) > bound)
