"""The 8-bit cache and the batch plan on the GPU against their references in 64 bits
(oracle/cache8_ref.py, oracle/attn_ref.py), at the lengths, masks, scales and layouts where they
can go wrong.

Tolerances.  Append: without rotation codes and scales are exact.  A rotated value is an fp32
expression of two products (error below 2^-22 max|x| over the head) rounded once to e4m3: half a
step is 2^-4 of the value, or 2^-10 of the scale where the code is subnormal.

Attention, with the cache's values as given: the result is rounded once (2^-8 |ref|); a weight
enters its product as bf16, off by at most 2^-8 of itself, or as three e4m3 terms, off by 2^-12
of itself and 2^-23 of the row's largest, so (U wv + n 2^-23 max|v|) over n keys, wv = sum_j w_j
|v_j|.  q as two e4m3 terms is off by at most 2^-17 of its row's largest value, so a score by
scale 2^-17 max|q| max_j |k_j|_1; fp32 sums of at most 128 products add 2^-17 of the same sum.  A
weight changes by twice that, counted against numerator and sum:
    |err| <= 2^-8 |ref| + (2^-8 + 4 scale 2^-17 max|q| max_j |k_j|_1 + 2^-20) wv + n 2^-23 max|v|.
"""
import numpy as np
import pytest

from oracle import attn_ref as R
from oracle import cache8_ref as C
from tests.test_gpu_attn import HEADS, U, Case, L, table_rows  # noqa: F401

pytestmark = pytest.mark.gpu


def quantized(x, page, rng, spread=0):
    """Codes and scales of x [pages, heads, page, d] (fp64; NaN: nothing there).  A block's scale
    is the least that fits, up to 2^spread times that; where nothing is, NaN codes and 255."""
    block = min(16, page)
    y = x.reshape(*x.shape[:2], page // block, block, x.shape[3])
    top = np.nanmax(np.where(np.isnan(y), 0, np.abs(y)), (3, 4))
    byte = np.maximum(np.ceil(np.log2(np.maximum(top, 1e-30) / 448)).astype(int) + 127, 1)
    byte = np.minimum(byte + (rng.integers(0, spread + 1, byte.shape) if spread else 0), 253)
    codes = C.encode(y * 2.0 ** (127.0 - byte)[..., None, None])
    byte = np.where(np.isnan(y).all((3, 4)), 255, byte)
    return codes.reshape(x.shape), byte.astype(np.uint8)


class Case8(Case):
    """Case over a cache in 8 bits: what no row may see has NaN codes and scale byte 255."""

    def __init__(self, *args, loud=0, spread_scales=0, groups=None, seed=0, **kw):
        super().__init__(*args, groups=groups, seed=seed, **kw)
        torch = self.torch
        rng = np.random.default_rng(seed + 100)
        sides = []
        for cache, rows in ((self.kc, self.rows_k), (self.vc, self.rows_v)):
            x = cache.double().cpu().numpy()
            if loud:   # blocks of very different size
                block = min(16, self.page)
                f = 2.0 ** rng.integers(-loud, loud + 1, (*x.shape[:2], self.page // block))
                x = x * np.repeat(f, block, -1)[..., None]
            codes, byte = quantized(x, self.page, rng, spread_scales)
            value = C.dequantize(codes, byte)
            sides += [torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(byte).cuda()]
            table = self.table.cpu().numpy()
            for s in range(len(rows)):
                rows[s] = rows[s].double()
                for j in range(len(rows[s])):
                    i = table[s, j // self.page]
                    if 0 <= i < len(codes) and not np.isnan(value[i, :, j % self.page]).any():
                        rows[s][j] = torch.from_numpy(value[i, :, j % self.page])
            for g in range(len(groups[1]) if groups else 0):
                first = groups[0][g]
                for s in range(first + 1, groups[0][g + 1]):
                    n = min(groups[1][g], len(rows[s]))
                    rows[s][:n] = rows[first][:n]
        self.kc, self.k_scale, self.vc, self.v_scale = sides

    def kv(self, L, max_q=None):
        return L.PagedKV8bit(self.kc, self.vc, self.k_scale, self.v_scale, self.table, self.dq_off, self.dkv_len,
                             self.T, max_q_len=max(self.q_lens) if max_q is None else max_q)

    def check(self, got, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        k, v = ([x.double().numpy() for x in rows] for rows in (self.rows_k, self.rows_v))
        ref, wv = R.attention(self.q_host, k, v, self.q_off, self.kv_len, scale, self.window, self.n_sink)
        got = got.double().cpu().numpy()
        n = int(self.q_off[-1])
        assert np.all(got[n:] == 7.0), "rows of no sequence were written"
        ref, wv, got = ref[:n], wv[:n], got[:n]
        assert np.all(np.isfinite(got))
        assert np.all(got[wv.sum(-1) == 0] == 0), "rows that see nothing are zeros"
        bound = U * np.abs(ref)
        for s in range(len(self.q_lens)):
            a, b = self.q_off[s], self.q_off[s + 1]
            if a == b or not len(k[s]):
                continue
            score = scale * 2.0 ** -17 * np.abs(self.q_host[a:b]).max() * np.abs(k[s]).sum(-1).max()
            bound[a:b] += (U + 4 * score + 2.0 ** -20) * wv[a:b] + len(k[s]) * 2.0 ** -23 * np.abs(v[s]).max()
        excess = np.abs(got - ref) / (bound + 1e-30)
        assert excess.size == 0 or excess.max() <= 1, f"{excess.max()} at {np.unravel_index(excess.argmax(), excess.shape)}"
        if ref.size > 500:
            assert np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref)


def attend(L, c, err=0, max_q=None, scale=None):
    kv = c.kv(L, max_q)
    ws = L.attn_workspace(kv, c.hq)
    got = L.attn_paged_8bit_t(kv, c.q, ws, window=c.window, n_sink=c.n_sink, out=c.out, scale=scale)
    assert L.get_error_t(ws) == err
    c.check(got, scale)
    first = got.clone()
    again = L.attn_paged_8bit_t(kv, c.q, ws, window=c.window, n_sink=c.n_sink, out=c.out, scale=scale)
    assert c.torch.equal(first.view(c.torch.int16), again.view(c.torch.int16)), "the workspace is not left clean"


def prefix_attend(L, c, groups, err=0, max_q=None):
    torch = c.torch
    kv = c.kv(L, max_q)
    off, pl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in groups)
    ws = L.attn_workspace(kv, c.hq, n_groups=len(groups[1]))
    got = L.attn_prefix_8bit_t(kv, c.q, off, pl, ws, out=c.out)
    assert L.get_error_t(ws) == err
    c.check(got)
    before = got.clone()
    again = L.attn_prefix_8bit_t(kv, c.q, off, pl, ws, out=c.out)
    assert torch.equal(before.view(torch.int16), again.view(torch.int16))


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("page", [8, 64])
def test_single_tokens(L, hq, hkv, d, page):
    ctx = [0, 1, 14, 15, 16, 63, 126, 127, 128, 129, 255, 500, 700]
    attend(L, Case8([1] * len(ctx), ctx, hq, hkv, d, page, seed=hq + page))


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_page_sizes(L, page, d):
    attend(L, Case8([1, 5, 200], [300, 3, 77], 4, 2, d, page, seed=page))
    attend(L, Case8([1, 1, 2], [300, 3, 577], 4, 2, d, page, seed=page))


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_chunks_and_single_tokens_in_one_batch(L, hq, hkv, d):
    attend(L, Case8([130, 1, 0, 17, 1, 64], [0, 200, 90, 140, 0, 255], hq, hkv, d, 16, seed=3, pad_rows=3))


@pytest.mark.parametrize("n", [1, 2, 3, 8, 15, 16, 17, 33, 64, 65, 127, 128, 129, 257])
def test_prompt_lengths(L, n):
    attend(L, Case8([n], [0], 4, 2, 128, 16, seed=n))
    attend(L, Case8([n], [70], 4, 1, 64, 32, seed=n))


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 3), (2, 0), (40, 4), (128, 0), (128, 130), (129, 1), (300, 16),
                                           (100000, 5), (64, 1000), (2 ** 31 - 1, 0), (2 ** 31 - 20, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_windows_and_first_tokens(L, window, n_sink, d):
    attend(L, Case8([1, 1, 1, 1, 1], [0, 39, 128, 500, 641], 4, 2, d, 16, seed=window % 1000, window=window,
                    n_sink=n_sink))
    attend(L, Case8([150, 1, 30, 0, 4], [0, 450, 333, 8, -3], 4, 2, d, 16, seed=window % 1000, window=window,
                    n_sink=n_sink))


@pytest.mark.parametrize("d,page,n_sink", [(128, 32, 33), (64, 64, 4), (128, 128, 128), (64, 256, 5), (128, 8, 9)])
def test_windows_that_move_over_pages(L, d, page, n_sink):
    n = [150, 159, 160, 161, 287, 288, 289, 415, 416, 417, 543, 545]
    attend(L, Case8([1] * len(n), [x - 1 for x in n], 8, 1, d, page, seed=page, window=32, n_sink=n_sink))
    attend(L, Case8([40, 1, 200, 3], [x - 40 for x in (289, 545, 700, 161)], 8, 1, d, page, seed=n_sink, window=129,
                    n_sink=n_sink))


def test_rows_that_see_nothing(L):
    attend(L, Case8([3, 1, 2, 140], [0, -1, -2, -20], 4, 2, 64, 16, seed=5))
    attend(L, Case8([2], [-2], 4, 2, 128, 16, seed=5))
    attend(L, Case8([0, 0], [5, 0], 4, 2, 128, 16, seed=5, pad_rows=2))


def test_max_q_len_is_a_hint(L):
    for max_q in (0, 1, 1000):
        attend(L, Case8([1, 90, 3], [100, 50, 7], 8, 2, 64, 16, seed=6), max_q=max_q)


def test_large_scores_and_scale(L):
    attend(L, Case8([1, 40], [600, 300], 4, 2, 64, 16, seed=7, spread=6.0), scale=0.02)
    attend(L, Case8([1, 1], [600, 300], 4, 2, 64, 16, seed=7, spread=6.0), scale=0.02)
    attend(L, Case8([1, 40], [600, 300], 4, 2, 64, 16, seed=8), scale=1.0)
    attend(L, Case8([1, 3], [600, 300], 4, 2, 128, 16, seed=8), scale=1.0)


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [60, 1, 5]])
@pytest.mark.parametrize("d,page", [(64, 8), (128, 64)])
def test_blocks_of_very_different_scales(L, q_lens, d, page):
    # values that differ by 2^6 from block to block, and scales larger than they need be
    attend(L, Case8(q_lens, [500, 20, 777], 8, 2, d, page, seed=d, loud=3), scale=0.01)
    attend(L, Case8(q_lens, [500, 20, 777], 8, 2, d, page, seed=d, spread_scales=3))


@pytest.mark.parametrize("q_len", [1, 40])
def test_scales_at_the_ends_of_their_range(L, q_len):
    """Values far from 1: keys scaled by 2^60 with queries by 2^-60 give the same scores, and values
    scaled by 2^100 and by 2^-100 the same results times that."""
    import torch
    c = Case8([q_len], [300], 4, 2, 128, 16, seed=1)
    kv = c.kv(L)
    ws = L.attn_workspace(kv, 4)
    want = L.attn_paged_8bit_t(kv, c.q, ws).clone()
    q = (c.q.double() * 2.0 ** -60).bfloat16()
    c.k_scale += 60
    assert torch.equal(L.attn_paged_8bit_t(kv, q, ws), want)
    for e in (-100, 200):
        c.v_scale += e % 256
        got = L.attn_paged_8bit_t(kv, q, ws).double()
        assert torch.equal(got, want.double() * 2.0 ** (e if e < 0 else 100))
    c.v_scale.zero_()      # as 1
    tiny = L.attn_paged_8bit_t(kv, q, ws)
    c.v_scale.fill_(1)
    assert torch.equal(L.attn_paged_8bit_t(kv, q, ws), tiny)
    assert L.get_error_t(ws) == 0


def test_a_zero_filled_cache(L):
    import torch
    caches = L.PagedKV8bit.empty_cache(4, 2, 16, 64)
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None].contiguous()
    for rows in (1, 33):
        kv = L.PagedKV8bit(*caches, table, torch.tensor([0, rows], dtype=torch.int32, device="cuda"),
                           torch.tensor([50], dtype=torch.int32, device="cuda"), rows)
        q = torch.randn(rows, 4, 64, device="cuda").bfloat16()
        assert not L.attn_paged_8bit_t(kv, q, L.attn_workspace(kv, 4)).any()


def test_long_runs_of_light_weights(L):
    """One key takes most of the weight, 30000 others share the rest: the terms of a weight reach
    far enough down (the bound's share for what lies below them is 2^-8 of the largest value
    here; the tail carries a seventh of the result)."""
    import torch
    n, d, page = 30000, 64, 64
    k, v = np.zeros((n, 1, d)), np.zeros((n, 1, d))
    k[0, 0, 0] = 12.0                # its score; the others' are 0
    v[:, 0, 0], v[0, 0, 1] = 0.5, 1.0
    pages = -(-n // page)
    kc, vc = (np.zeros((pages, 1, page, d)) for _ in range(2))
    for c, x in ((kc, k), (vc, v)):
        c.reshape(pages * page, d)[:n] = x[:, 0]
    rng = np.random.default_rng(0)
    sides = [quantized(x, page, rng) for x in (kc, vc)]
    (kq, ks), (vq, vs) = [(torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda()) for a, b in sides]
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = 1.0
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    kv = L.PagedKV8bit(kq, vq, ks, vs, table, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                       torch.tensor([n], dtype=torch.int32, device="cuda"), 1)
    got = L.attn_paged_8bit_t(kv, q, L.attn_workspace(kv, 1), scale=1.0)[0, 0].double().cpu().numpy()
    w = np.exp(C.dequantize(*sides[0]).reshape(-1, d)[:n, 0])
    want = (w / w.sum()) @ C.dequantize(*sides[1]).reshape(-1, d)[:n]
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * want + (2.0 ** -12 + 2.0 ** -16) * want + n * 2.0 ** -23)


@pytest.mark.parametrize("wild", [None, -2 ** 31, -1, 2 ** 31 - 1])
def test_missing_pages_read_as_zeros_and_are_reported(L, wild):
    for q_lens, ctx in (([1, 1, 1], [100, 700, 20]), ([1, 20, 150], [100, 60, 400])):
        missing = {(0, 2), (0, 6), (1, 0), (1, 3), (2, 1)}
        attend(L, Case8(q_lens, ctx, 4, 2, 128, 16, seed=9))
        c = Case8(q_lens, ctx, 4, 2, 128, 16, seed=9, missing=missing)
        if wild is not None:
            for s, p in missing:
                c.table[s, p] = wild
        attend(L, c, err=L.DEVERR_BAD_PAGE)


@pytest.mark.parametrize("max_q", [1, None])
def test_many_sequences(L, max_q):
    rng = np.random.default_rng(1)
    q = [int(x) for x in rng.integers(0, 2, 2200)]
    ctx = [int(x) for x in rng.integers(0, 40, 2200)]
    q[2100] = 33
    attend(L, Case8(q, ctx, 2, 1, 64, 16, seed=10), max_q=max_q)


@pytest.mark.parametrize("group", [3, 16, 17, 64, 65, 128, 129, 144])
@pytest.mark.parametrize("d", [64, 128])
def test_query_heads_of_one_key_head(L, group, d):
    attend(L, Case8([1, 1, 1], [0, 150, 300], 2 * group, 2, d, 16, seed=group))
    attend(L, Case8([9, 1, 0, 3], [140, 37, 4, 0], group, 1, d, 32, seed=group, window=60, n_sink=3, pad_rows=1))
    groups = ([0, 3], [150])
    prefix_attend(L, Case8([1, 5, 1], [150, 160, 300], group, 1, d, 16, seed=group, groups=groups), groups)


def dequantize_t(torch, codes, scale):
    """Values of codes [.., page, d] at scales [.., page / B], fp64 on the GPU."""
    n = codes.shape[-2] // scale.shape[-1]
    return codes.view(torch.float8_e4m3fn).double() * torch.exp2(
        scale.double().clamp(1, 253) - 127).repeat_interleave(n, -1)[..., None]


def random_cache(torch, n_pages, hkv, page, d):
    codes = [torch.randint(0, 256, (n_pages, hkv, page, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    for c in codes:
        c[(c & 127) > 118] = 60          # up to 240, no NaN
    scales = [torch.randint(118, 123, (n_pages, hkv, max(1, page // 16)), dtype=torch.uint8, device="cuda")
              for _ in range(2)]
    return (*codes, *scales)


def check_rows(torch, got, q, k, v, first_pos, window=0, n_sink=0):
    """Rows got, q [rows, hq, d] at positions first_pos .. over keys k, v [n, hq, d] (fp64)."""
    rows, n, d = q.shape[0], k.shape[0], q.shape[2]
    x = torch.einsum("thd,nhd->htn", q.double(), k) * d ** -0.5
    pos = torch.arange(first_pos, first_pos + rows, device="cuda")[:, None]
    key = torch.arange(n, device="cuda")
    seen = key <= pos
    if window:
        seen &= (key > pos - window) | (key < n_sink)
    w = x.masked_fill(~seen, -float("inf")).softmax(-1)
    ref, wv = (torch.einsum("htn,nhd->thd", w, y) for y in (v, v.abs()))
    score = d ** -0.5 * 2.0 ** -17 * q.abs().max().double() * k.abs().sum(-1).max()
    err = (got.double() - ref).abs()
    assert (err <= U * ref.abs() + (U + 4 * score + 2.0 ** -20) * wv + n * 2.0 ** -23 * v.abs().max()).all()
    assert err.norm() <= 5e-3 * ref.norm()


def test_long_context_of_few_rows(L):
    import torch
    torch.manual_seed(0)
    n, hq, hkv, d, page = 30011, 8, 2, 128, 64
    pages = -(-n // page)
    cache = random_cache(torch, pages, hkv, page, d)
    table = torch.randperm(pages, device="cuda").to(torch.int32)[None]
    k, v = (dequantize_t(torch, cache[i], cache[i + 2])[table[0].long()].transpose(1, 2).reshape(-1, hkv, d)[:n]
            .repeat_interleave(hq // hkv, 1) for i in (0, 1))
    for rows in (1, 3, 100):
        q = (0.05 * torch.randn(rows, hq, d, device="cuda")).to(torch.bfloat16)
        kv = L.PagedKV8bit(*cache, table, torch.tensor([0, rows], dtype=torch.int32, device="cuda"),
                           torch.tensor([n], dtype=torch.int32, device="cuda"), rows)
        ws = L.attn_workspace(kv, hq)
        check_rows(torch, L.attn_paged_8bit_t(kv, q, ws), q, k, v, n - rows)
        assert L.get_error_t(ws) == 0


@pytest.mark.parametrize("hq,hkv,d,window", [(64, 8, 64, 1024), (32, 8, 128, 0), (12, 12, 64, 0), (32, 2, 128, 300),
                                             (24, 1, 64, 0)])
@pytest.mark.parametrize("rows", [1, 70])
def test_ordinary_batches(L, hq, hkv, d, window, rows):
    """Shares of many segments and tiles, on every SM; equal calls give equal bits."""
    import torch
    rng = np.random.default_rng(hq + window + rows)
    n, page, n_sink = 60, 32, 4
    ctx = rng.integers(0, 4000, n)
    q_lens = rng.integers(1, rows + 1, n)
    kv_len = ctx + q_lens
    max_pages = -(-int(kv_len.max()) // page)
    table = torch.randperm(n * max_pages, device="cuda").to(torch.int32).view(n, max_pages)
    torch.manual_seed(hq)
    cache = random_cache(torch, n * max_pages, hkv, page, d)
    off = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    T = int(off[-1])
    q = (0.05 * torch.randn(T, hq, d, device="cuda")).to(torch.bfloat16)
    kv = L.PagedKV8bit(*cache, table, torch.from_numpy(off).cuda(), torch.from_numpy(kv_len.astype(np.int32)).cuda(),
                       T, max_q_len=int(q_lens.max()))
    ws = L.attn_workspace(kv, hq)
    got = L.attn_paged_8bit_t(kv, q, ws, window=window, n_sink=n_sink)
    assert L.get_error_t(ws) == 0
    for s in range(n):
        m = int(kv_len[s])
        k, v = (dequantize_t(torch, cache[i][table[s].long()], cache[i + 2][table[s].long()]).transpose(1, 2)
                .reshape(-1, hkv, d)[:m].repeat_interleave(hq // hkv, 1) for i in (0, 1))
        a, b = int(off[s]), int(off[s + 1])
        check_rows(torch, got[a:b], q[a:b], k, v, m - (b - a), window, n_sink)
    for _ in range(20):
        assert torch.equal(got, L.attn_paged_8bit_t(kv, q, ws, window=window, n_sink=n_sink))


def test_cache_past_32_bit_offsets(L):
    """A cache of more than 2^32 codes, used at its end."""
    import torch
    hkv, page, d = 8, 256, 128
    n_pages = (1 << 32) // (hkv * page * d) + 40
    cache = [torch.empty(n_pages, hkv, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.zeros(n_pages, hkv, page // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.manual_seed(1)
    n, hq = 700, 8
    ids = torch.tensor([n_pages - 1, 0, n_pages - 3], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(n, hkv, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(n, hq, d, device="cuda").to(torch.bfloat16)
    kv = L.PagedKV8bit(*cache, ids[None].contiguous(), torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                       torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    ws = L.attn_workspace(kv, hq)
    L.kv_append_8bit_t(kv, None, k, v, None, ws)
    kd, vd = (dequantize_t(torch, cache[i][ids.long()], cache[i + 2][ids.long()]).transpose(1, 2)
              .reshape(-1, hkv, d)[:n] for i in (0, 1))
    for x, y in ((k, kd), (v, vd)):
        assert ((x.double() - y).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -16).all()
    check_rows(torch, L.attn_paged_8bit_t(kv, q, ws), q, kd, vd, 0)
    last = L.PagedKV8bit(*cache, ids[None].contiguous(), torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                         torch.tensor([n], dtype=torch.int32, device="cuda"), 1)
    check_rows(torch, L.attn_paged_8bit_t(last, q[-1:], L.attn_workspace(last, hq)), q[-1:], kd, vd, n - 1)
    assert L.get_error_t(ws) == 0


# ------------------------------------------------------------------ shared prefixes

@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("prefix", [1, 17, 128, 300])
def test_shared_prefix(L, hq, hkv, d, prefix):
    n = 9
    groups = ([0, n], [prefix])
    prefix_attend(L, Case8([1] * n, [prefix + 11 * i for i in range(n)], hq, hkv, d, 16, seed=prefix, groups=groups),
                  groups)


@pytest.mark.parametrize("page", [8, 32, 128])
def test_prefix_groups(L, page):
    groups = ([0, 1, 1, 4, 6, 40], [40, 9, 0, 200, 131])
    q = [1, 2, 0, 30, 1, 1] + [1] * 34 + [1, 5]
    ctx = [50, 60, 10, 3, 200, 260] + [131 + 7 * (i % 9) for i in range(34)] + [20, 90]
    prefix_attend(L, Case8(q, ctx, 8, 2, 64, page, seed=page, groups=groups), groups)


def test_prefix_of_many_rows(L):
    groups = ([0, 3], [260])
    prefix_attend(L, Case8([100, 33, 64], [260, 261, 300], 8, 2, 128, 16, seed=2, groups=groups, pad_rows=1), groups)
    groups = ([0, 90, 100], [270, 30])
    prefix_attend(L, Case8([1] * 100, [270 + i % 5 for i in range(90)] + [30] * 10, 8, 2, 128, 16, seed=2,
                           groups=groups), groups)


def test_prefix_longer_than_a_context_is_reported(L):
    import torch
    groups = ([0, 3], [50])
    c = Case8([1, 1, 1], [60, 50, 20], 4, 2, 64, 16, seed=3, groups=groups)
    kv = c.kv(L)
    ws = L.attn_workspace(kv, c.hq, n_groups=1)
    off, pl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in groups)
    L.attn_prefix_8bit_t(kv, c.q, off, pl, ws, out=c.out)
    assert L.get_error_t(ws) == L.DEVERR_BAD_LEN


# ------------------------------------------------------------------ append

def cache_of(torch, rng, n_pages, hkv, page, d):
    codes = [rng.integers(0, 256, (n_pages, hkv, page, d)).astype(np.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 127) == 127] = 3
    scales = [rng.integers(116, 128, (n_pages, hkv, page // min(16, page))).astype(np.uint8) for _ in range(2)]
    return codes, scales


@pytest.mark.parametrize("hq,hkv,d,rot", [(8, 2, 128, 128), (28, 4, 128, 64), (5, 5, 64, 64), (6, 2, 64, 16),
                                          (0, 3, 64, 64), (40, 8, 128, 128), (4, 4, 128, 0), (33, 11, 64, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes,page,few", [(0, 16, False), (0, 8, True), (1, 32, False), (3, 64, True), (4, 256, False)])
def test_append(L, hq, hkv, d, rot, interleaved, axes, page, few):
    import torch
    rng = np.random.default_rng(hq + rot + axes)
    q_lens, ctx = ([1, 0, 3, 1, 3], [20, 5, 14, 0, -2]) if few else ([1, 0, 77, 1, 3, 16], [20, 5, 11, 0, -2, 32])
    n = len(q_lens)
    q_off = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    kv_len = np.asarray([a + b for a, b in zip(q_lens, ctx)], np.int32)
    T = int(q_off[-1]) + 2
    max_pages, n_pos = -(-90 // page), 100
    n_pages = n * max_pages + 5
    table = rng.permutation(n_pages)[:n * max_pages].reshape(n, max_pages).astype(np.int32)
    size = 2.0 ** rng.integers(-3, 4, (T, 1))      # rows of different size: scales grow
    wide = torch.from_numpy((rng.standard_normal((T, (hq + 2 * hkv + 1) * d)) * size).astype(np.float32)).bfloat16()
    parts = [wide[:, a * d:b * d].reshape(T, b - a, d).double().numpy() for a, b in
             ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv))]
    dev = wide.cuda()
    dq, dk, dv = (dev[:, a * d:b * d].view(T, b - a, d) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    (kc, vc), (ks, vs) = cache_of(torch, rng, n_pages, hkv, page, d)
    dev_cache = [torch.from_numpy(x.copy()).cuda() for x in (kc, vc, ks, vs)]
    cs = table_rows(torch, rng, n_pos, rot) if rot else None
    half = rot // 2
    pairs = {0: [half], 1: [half], 3: [half // 4, half // 2 - 1, half - half // 4 - half // 2 + 1],
             4: [0, half // 2, 3, half - half // 2 - 3]}[axes]
    if min(pairs) < 0:
        pytest.skip("too few pairs for these axes")
    pos = rng.integers(0, n_pos, (max(axes, 1), T)).astype(np.int32)
    kv = L.PagedKV8bit(*dev_cache, torch.from_numpy(table).cuda(), torch.from_numpy(q_off).cuda(),
                       torch.from_numpy(kv_len).cuda(), T, max_q_len=max(q_lens))
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    q_out = torch.full((T, max(hq, 1), d), 7.0, dtype=torch.bfloat16, device="cuda")
    kw = dict(pos=torch.from_numpy(pos).cuda() if axes else None, axis_pairs=pairs if axes > 1 else None,
              interleaved=interleaved)
    dcs = None if cs is None else torch.from_numpy(cs).cuda()
    got = L.kv_append_8bit_t(kv, dq if hq else None, dk, dv, dcs, ws, q_out=q_out if hq else None, **kw)
    assert L.get_error_t(ws) == (L.DEVERR_BAD_POS if axes == 0 and rot else 0)
    axis = np.repeat(np.arange(len(pairs)), pairs)
    want_q = np.full((T, max(hq, 1), d), 7.0)
    tol_q = np.zeros_like(want_q)
    turned = np.zeros((T, hkv, d))
    for t, s, p in R.positions(q_off, kv_len):
        at = [int(pos[axis[i], t]) if axes else p for i in range(half)]
        turn = (lambda x: R.rotate(x, cs, at, interleaved)) if rot else (lambda x: x)
        for h in range(hq):
            want_q[t, h] = turn(parts[0][t, h])
            tol_q[t, h] = U * np.abs(want_q[t, h]) * (rot > 0) + 2.0 ** -22 * np.abs(parts[0][t, h]).max()
        for h in range(hkv):
            turned[t, h] = turn(parts[1][t, h])
    old_k = kc.copy(), ks.copy()
    written = np.zeros(kc.shape[:3], bool)
    noise = np.zeros(kc.shape[:3])
    for s in range(n):
        rows = [(t, p) for t, s2, p in R.positions(q_off, kv_len) if s2 == s and p >= 0]
        places = [(int(table[s, p // page]), p % page) for _, p in rows]
        ts = [t for t, _ in rows]
        C.append(kc, ks, turned[ts], places)
        C.append(vc, vs, parts[2][ts], places)
        for t, (a, b) in zip(ts, places):
            written[a, :, b] = True
            noise[a, :, b] = 2.0 ** -22 * np.abs(parts[1][t]).max(-1)
    g_kc, g_vc, g_ks, g_vs = (x.cpu().numpy() for x in dev_cache)
    assert np.array_equal(g_vc, vc) and np.array_equal(g_vs, vs)
    assert np.array_equal(g_ks, ks)
    if not rot:
        assert np.array_equal(g_kc, kc)
    else:
        # earlier rows exactly, new ones within half a step of the rotated value
        assert np.array_equal(g_kc[~written], kc[~written])
        exact, exact_s = old_k
        value = C.dequantize(g_kc, g_ks)
        for s in range(n):
            for t, s2, p in R.positions(q_off, kv_len):
                if s2 != s or p < 0:
                    continue
                a, b = int(table[s, p // page]), p % page
                step = 2.0 ** (C.scale_read(g_ks[a, :, b // min(16, page)]) - 127.0 - 10)
                tol = 2.0 ** -4 * np.abs(turned[t]) + step[:, None] + noise[a, :, b][:, None]
                assert np.all(np.abs(value[a, :, b] - turned[t]) <= tol)
        differ = (g_kc != kc) & written[..., None]
        assert differ.mean() < 1e-3      # (only where the fp32 value falls on the other side of a tie)
    if hq:
        assert np.all(np.abs(got.double().cpu().numpy() - want_q) <= tol_q)
        in_place = L.kv_append_8bit_t(kv, dq, dk, dv, dcs, ws, q_out=dq, **kw)
        m = int(q_off[-1])
        assert torch.equal(in_place[:m], got[:m])
        assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(dev_cache, (g_kc, g_vc, g_ks, g_vs)))


def test_append_token_by_token_and_at_once(L):
    """The scales do not depend on how the tokens are divided over calls, and the values by less than a
    subnormal step."""
    import torch
    torch.manual_seed(0)
    n, hkv, d, page = 100, 3, 64, 32
    size = torch.exp2(torch.randint(-4, 5, (n, 1, 1), device="cuda").float())
    k, v = ((torch.randn(n, hkv, d, device="cuda") * size).to(torch.bfloat16) for _ in range(2))
    table = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device="cuda")
    made = []
    for step in (n, 1, 7, 33):
        cache = L.PagedKV8bit.empty_cache(4, hkv, page, d)
        for a in range(0, n, step):
            m = min(step, n - a)
            kv = L.PagedKV8bit(*cache, table, torch.tensor([0, m], dtype=torch.int32, device="cuda"),
                               torch.tensor([a + m], dtype=torch.int32, device="cuda"), m)
            ws = L.attn_workspace(kv, 3)
            L.kv_append_8bit_t(kv, None, k[a:a + m], v[a:a + m], None, ws)
            assert L.get_error_t(ws) == 0
        made.append(cache)
    for cache in made[1:]:
        for i in (0, 1):
            assert torch.equal(cache[i + 2], made[0][i + 2])
            step = torch.exp2(cache[i + 2].double().clamp(min=1) - 127 - 9).repeat_interleave(16, -1)[..., None]
            x, y = (dequantize_t(torch, c[i], c[i + 2]) for c in (cache, made[0]))
            assert ((x - y).abs() <= step).all()


def test_append_of_values_at_the_ends(L):
    """Zeros, the type's largest and smallest values, borders of a scale, infinities and NaN."""
    import torch
    top = torch.finfo(torch.bfloat16).max
    rows = [[0.0], [448.0, -448.0], [450.0], [2.0 ** -133], [top, 1.0], [-top], [float("inf"), 5.0], [float("nan"), 3.0],
            [1.75, -0.0, 2.0 ** -9 * 1.75 / 448], [2.0 ** -126]]
    x = torch.zeros(len(rows), 1, 64, dtype=torch.bfloat16, device="cuda")
    for i, r in enumerate(rows):
        x[i, 0, :len(r)] = torch.tensor(r, dtype=torch.float64).bfloat16().cuda()
    n = len(rows)
    cache = L.PagedKV8bit.empty_cache(n, 1, 16, 64)
    kv = L.PagedKV8bit(*cache, torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous(),
                       torch.arange(n + 1, dtype=torch.int32, device="cuda"),
                       torch.ones(n, dtype=torch.int32, device="cuda"), n)
    ws = L.attn_workspace(kv, 1)
    L.kv_append_8bit_t(kv, None, x, x, None, ws)
    assert L.get_error_t(ws) == 0
    host = x[:, 0].double().cpu().numpy()
    for codes, scale in ((cache[0], cache[2]), (cache[1], cache[3])):
        for i in range(n):
            fine = host[i][~np.isnan(host[i])]
            b = C.scale_byte(min(np.abs(fine).max(), 3.4028234e38))
            assert int(scale[i, 0, 0]) == b
            want = C.encode(np.clip(host[i], -1e300, 1e300) * 2.0 ** (127 - b))
            got = codes.view(torch.uint8)[i, 0, 0].cpu().numpy()
            nan = np.isnan(host[i])
            assert np.array_equal(got[~nan], want[~nan]) and np.all(got[nan] & 127 == 127)


def test_append_reports_missing_pages_and_writes_nothing_there(L):
    import torch
    torch.manual_seed(0)
    cache = L.PagedKV8bit.empty_cache(4, 1, 16, 64)
    tab = torch.tensor([[0, -1], [99, 2]], dtype=torch.int32, device="cuda")
    kv = L.PagedKV8bit(*cache, tab, torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda"),
                       torch.tensor([18, 40], dtype=torch.int32, device="cuda"), 4)
    x = torch.randn(4, 1, 64, device="cuda").to(torch.bfloat16)
    ws = L.attn_workspace(kv, 1)
    L.kv_append_8bit_t(kv, None, x, x, None, ws)
    assert L.get_error_t(ws) == L.DEVERR_BAD_PAGE
    assert int((cache[0].view(torch.uint8) != 0).any(-1).sum()) == 1 and int((cache[2] != 0).sum()) == 1


# ------------------------------------------------------------------ plans

def run_plan(L, rng, n, page, max_pages, T, n_cached, n_new, n_shared=None, free=None, n_free=None, cap=None, err=0,
             wild=False, in_place=False, spare=40):
    """A plan of sequences with these lengths against the reference, twice."""
    import torch
    have = [min(-(-max(c, 0) // page), max_pages) for c in n_cached]
    n_pages = sum(have) + spare
    order = rng.permutation(n_pages).astype(np.int32)
    table = np.full((n, max_pages), -7, np.int32)
    at = 0
    for s in range(n):
        table[s, :have[s]] = order[at:at + have[s]]
        at += have[s]
    if wild:   # pages that a window left behind
        table[rng.random(table.shape) < 0.3] = -1
    cap = n_pages if cap is None else cap
    stack = np.full(cap, -9, np.int32)
    rest = order[at:][:cap] if free is None else np.asarray(free, np.int32)
    n_free = len(rest) if n_free is None else n_free
    stack[:len(rest)] = rest

    def up(x, t=torch.int32):
        return torch.tensor(np.asarray(x), dtype=t, device="cuda")

    d_table, d_free = up(table), up(stack)
    shared = np.zeros(n, int) if n_shared is None else n_shared
    want = C.plan(table, n_cached, n_new, shared, stack, n_free, page, n_pages, T)
    cached, count = up(n_cached), up([n_free])
    out = L.BatchPlan.empty(n, T)
    if in_place:
        out = out._replace(kv_len=cached, n_free=count)
    ws = L.batch_plan_workspace(n)
    ws[16:].fill_(0x5A)
    for _ in range(1 if in_place else 2):
        got = L.batch_plan_t(d_table, cached, up(n_new), d_free, count, page, n_pages, ws,
                             n_shared=None if n_shared is None else up(n_shared), out=out)
        assert L.get_error_t(ws) == err
        for name, a, b in zip(("q_off", "kv_len", "slots", "pos", "n_free"), got, want):
            assert np.array_equal(a.cpu().numpy(), np.atleast_1d(b)), name
        assert np.array_equal(d_table.cpu().numpy(), table)
        assert np.array_equal(d_free.cpu().numpy(), stack)
    return got


@pytest.mark.parametrize("n", [1, 2, 33, 1023, 1024, 1025, 2500])
@pytest.mark.parametrize("page", [8, 64])
def test_plans(L, n, page):
    rng = np.random.default_rng(n + page)
    for most in (1, 4, 60):
        cached = rng.integers(0, 300, n)
        new = rng.integers(-1, most + 1, n)
        new[rng.integers(0, n)] = most
        rows = int(np.maximum(new, 0).sum())
        shared = np.minimum(rng.integers(0, 4, n), -(-cached // page))
        need = sum(max(-(-(c + x) // page) - -(-c // page), 0) for c, x in zip(cached, np.maximum(new, 0)))
        for T in {rows, rows + 5}:
            got = run_plan(L, rng, n, page, -(-400 // page), T, cached, new, shared, spare=need + 3)
        assert int(got.n_free[0]) >= 3


@pytest.mark.parametrize("in_place", [False, True])
def test_plan_of_long_rows(L, in_place):
    rng = np.random.default_rng(5)
    # a prompt of many pages, requests that end with pages missing in their rows, idle ones
    run_plan(L, rng, 5, 16, 700, 10010, [0, 9000, 5, 0, 37], [500, -1, 0, 100, -1], [0, 3, 0, 0, 1], wild=True,
             in_place=in_place)


def test_plan_takes_pages_that_were_just_given_back(L):
    rng = np.random.default_rng(6)
    got = run_plan(L, rng, 3, 16, 10, 40, [0, 100, 3], [33, -1, 1], free=[], cap=9)
    assert int(got.n_free[0]) == 7 - 3


def test_plan_reports_what_does_not_fit(L):
    rng = np.random.default_rng(7)
    both = L.DEVERR_NO_PAGE | L.DEVERR_BAD_PAGE
    run_plan(L, rng, 3, 16, 10, 70, [0, 5, 16], [33, 12, 20], free=[3], err=both)          # no page left
    run_plan(L, rng, 3, 16, 10, 20, [0, 5, 16], [13, 12, 20], err=L.DEVERR_BAD_LEN)         # more rows than T
    run_plan(L, rng, 2, 16, 2, 50, [20, 3], [40, 1], err=L.DEVERR_BAD_LEN)                  # more pages than the table has
    run_plan(L, rng, 2, 16, 4, 50, [60, 3], [-1, 1], free=[1, 2], cap=4, err=L.DEVERR_BAD_LEN)   # no room on the stack
    for n_free in (-3, 99):
        import torch
        ws = L.batch_plan_workspace(1)
        one = torch.ones(1, dtype=torch.int32, device="cuda")
        table = torch.full((1, 2), -1, dtype=torch.int32, device="cuda")
        stack = torch.arange(3, dtype=torch.int32, device="cuda")
        got = L.batch_plan_t(table, one - 1, one, stack, one * n_free, 16, 3, ws, T=1)
        err = L.get_error_t(ws)
        assert err & L.DEVERR_BAD_LEN and int(got.n_free[0]) == (0 if n_free < 0 else 2)
        got = L.batch_plan_t(table, one * -5, one, stack, one * 3, 16, 3, ws, T=1)
        assert L.get_error_t(ws) == L.DEVERR_BAD_LEN and int(got.kv_len[0]) == 1


def test_plan_without_rows(L):
    rng = np.random.default_rng(8)
    run_plan(L, rng, 4, 16, 4, 0, [5, 0, 60, 1], [0, 0, -1, 0])
    import torch
    out = L.BatchPlan.empty(1, 0)._replace(slots=None, pos=None)
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    got = L.batch_plan_t(torch.zeros(1, 2, dtype=torch.int32, device="cuda"), one, one, one.clone(), one, 16, 3,
                         L.batch_plan_workspace(1), T=4, out=out)
    assert got.q_off.tolist() == [0, 1] and got.kv_len.tolist() == [2]


# ------------------------------------------------------------------ together, streams and graphs

@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("max_q", [1, 64])
def test_a_captured_loop_takes_up_and_drops_requests(L, prefix, max_q):
    """Plan, append and attention as one captured step over many steps: requests begin with a
    prompt, cross page borders, end, and their pages go to others, without the host planning anything.
    Every step against fp64 over all that was appended to each request."""
    import torch
    torch.manual_seed(0)
    n, hq, hkv, d, page, T, max_pages, n_pages = 6, 8, 2, 64, 16, 64, 12, 60
    cache = L.PagedKV8bit.empty_cache(n_pages, hkv, page, d)
    table = torch.full((n, max_pages), -1, dtype=torch.int32, device="cuda")
    common = 32 if prefix else 0
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    free[:n_pages - 2] = torch.randperm(n_pages - 2, device="cuda").to(torch.int32)
    n_free = torch.tensor([n_pages - 2], dtype=torch.int32, device="cuda")
    kv_len, n_new, shared = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(3))
    plan = L.BatchPlan.empty(n, T)._replace(kv_len=kv_len, n_free=n_free)
    kv = L.PagedKV8bit(*cache, table, plan.q_off, kv_len, T, max_q_len=max_q)
    ws = L.attn_workspace(kv, hq, n_groups=1 if prefix else 0)
    plan_ws = L.batch_plan_workspace(n)
    q, k, v = (torch.randn(T, h, d, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    cs = L.rope_table(256, d)
    goff, plen = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [common]))
    if prefix:   # the two last pages hold what all share, written once
        table[:, :2] = torch.tensor([n_pages - 2, n_pages - 1], dtype=torch.int32, device="cuda")
        shared.fill_(2)
        x = torch.randn(common, hkv, d, device="cuda").to(torch.bfloat16)
        first = L.PagedKV8bit(*cache, table, torch.tensor([0] + [common] * n, dtype=torch.int32, device="cuda"),
                              torch.full((n,), common, dtype=torch.int32, device="cuda"), common)
        L.kv_append_8bit_t(first, None, x, x, cs, ws)
        kv_len.fill_(common)

    def step():
        L.batch_plan_t(table, kv_len, n_new, free, n_free, page, n_pages, plan_ws, n_shared=shared, out=plan)
        r = L.kv_append_8bit_t(kv, q, k, v, cs, ws)
        return r, L.attn_prefix_8bit_t(kv, r, goff, plen, ws) if prefix else L.attn_paged_8bit_t(kv, r, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()        # (no new tokens: nothing happens)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            rotated, out = step()
    torch.cuda.synchronize()
    assert L.get_error_t(ws) == 0 and not plan.slots.ne(-1).any()
    rng = np.random.default_rng(2)
    length = [common] * n
    ended = 0
    for turn in range(30):
        new = [int(x) for x in rng.integers(0, 3, n)]
        for s in range(n):
            if length[s] == common and rng.random() < 0.5:
                new[s] = 20 if sum(new) < 40 else 1
            elif rng.random() < 0.12 or length[s] > 120:
                new[s] = -1
        n_new.copy_(torch.tensor(new, dtype=torch.int32))
        for x in (q, k, v):
            x.copy_(torch.randn_like(x) * float(2.0 ** rng.integers(-2, 3)))
        graph.replay()
        torch.cuda.synchronize()
        assert L.get_error_t(plan_ws) == 0 and L.get_error_t(ws) == 0
        off, pos, slots = plan.q_off.tolist(), plan.pos.tolist(), plan.slots.tolist()
        tab = table.tolist()
        for s in range(n):
            assert off[s + 1] - off[s] == max(new[s], 0)
            if new[s] < 0:
                ended += 1
                length[s] = common
                continue
            length[s] += new[s]
            rows = range(off[s], off[s + 1])
            assert [pos[t] for t in rows] == list(range(length[s] - new[s], length[s]))
            assert [slots[t] for t in rows] == [tab[s][pos[t] // page] * page + pos[t] % page for t in rows]
            if not new[s]:
                continue
            m = length[s]
            ids = table[s, :-(-m // page)].long()
            kd, vd = (dequantize_t(torch, cache[i][ids], cache[i + 2][ids]).transpose(1, 2).reshape(-1, hkv, d)[:m]
                      .repeat_interleave(hq // hkv, 1) for i in (0, 1))
            check_rows(torch, out[off[s]:off[s + 1]], rotated[off[s]:off[s + 1]], kd, vd, m - new[s])
            # the new rows' values are in the cache, up to the rounding to a code
            part = vd[-new[s]:, ::hq // hkv]
            x = v[off[s]:off[s + 1]].double()
            byte = cache[3][ids].repeat_interleave(16, -1).transpose(1, 2).reshape(-1, hkv)[m - new[s]:m].double()
            assert ((part - x).abs() <= 2.0 ** -4 * x.abs() + torch.exp2(byte - 137)[..., None]).all()
        held = [x for s in range(n) if length[s] > common for x in tab[s][common // page:-(-length[s] // page)]]
        stack = free[:int(n_free)].tolist()
        assert sorted(held + stack) == list(range(n_pages - 2)), "every page is held once or free"
        # a request that has ended starts over with the shared pages
        kv_len.copy_(torch.tensor(length, dtype=torch.int32))
    assert ended > 3


@pytest.mark.parametrize("op", ["append", "paged", "prefix", "plan"])
def test_results_of_a_call_on_another_stream_are_made_there(L, op):
    import torch
    groups = ([0, 2], [40])
    c = Case8([1, 1], [300, 40], 4, 2, 64, 16, seed=4, groups=groups)
    kv = c.kv(L)
    ws = L.attn_workspace(kv, c.hq, n_groups=1)
    off, plen = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in groups)
    k = torch.zeros(c.T, c.hkv, c.d, dtype=torch.bfloat16, device="cuda")
    lens, new = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([7, 8], [200, 300]))
    table = torch.full((2, 40), 5, dtype=torch.int32, device="cuda")
    free, count = torch.arange(50, dtype=torch.int32, device="cuda"), torch.tensor([50], dtype=torch.int32, device="cuda")
    plan_ws = L.batch_plan_workspace(2)

    def call(stream=None):
        if op == "append":
            return L.kv_append_8bit_t(kv, c.q, k, k, None, ws, stream=stream)
        if op == "prefix":
            return L.attn_prefix_8bit_t(kv, c.q, off, plen, ws, stream=stream)
        if op == "plan":
            return L.batch_plan_t(table, lens, new, free, count, 16, 50, plan_ws, T=512, stream=stream).slots
        return L.attn_paged_8bit_t(kv, c.q, ws, stream=stream)

    want = call().clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    late = torch.full_like(want, 7)
    where = late.data_ptr()
    del late
    got = call(side)
    torch.cuda.synchronize()
    assert got.data_ptr() != where and torch.equal(got, want)


def test_empty_batches(L):
    import torch
    c = Case8([0, 0, 0], [5, 0, 40], 4, 2, 64, 16, seed=1, groups=([0, 3], [2]))
    kv = c.kv(L)
    ws = L.attn_workspace(kv, 4, n_groups=1)
    q, k = (torch.empty(0, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    off, plen = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 3], [2]))
    assert L.kv_append_8bit_t(kv, q, k, k, L.rope_table(64, 64), ws).shape == q.shape
    assert L.attn_paged_8bit_t(kv, q, ws).shape == q.shape
    assert L.attn_prefix_8bit_t(kv, q, off, plen, ws).shape == q.shape
    assert L.get_error_t(ws) == 0
