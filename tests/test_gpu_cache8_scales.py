"""Scales of the 8-bit cache on the GPU: long segments in pages of 8, blocks of very different size,
and how far results may be off, part by part.

Tolerances (tight: one bf16 a weight would not keep them).  With the cache's values as given, w the
weights before their sum, w_max a row's largest and 2^R the largest scale of a block of values
that some row of the call sees:
  result     one rounding to bf16: U |ref|, or half of a step of 2^-133 below 2^-126, where bf16's steps stay
             as they are (a test of scales of 2^-126 comes there: a row that sees one key has its code
             times that, and codes go down to 2^-9); in front of it products in fp32, below 2^-126 in steps
             of 2^-149: 2^-145 for all of them
  weights    three e4m3 terms (keys in M): the first leaves 2^-4 of a value, the others 2^-4 of what is left,
             so 2^-12 w_j, or where the last is subnormal half its step, 2^-10 / 16^2 = 2^-18 of P 2^(vb - R), whose
             largest P is at least 2^5: 2^-23 w_max 2^(R - vb);
             one f16 (rows in M): 2^-11 w_j, or below 2^-14 half of 2^-24, where the largest is at least
             2^6: 2^-31 w_max
  values     e4m3 codes (keys in M) exactly; f16 (rows in M) of code x 2^(vb - R): lost where vb - R < -24, half
             of 2^-24 where that is below -15, else exactly
  scores     q as two terms is off by 2^-17 of the row's largest, the fp32 sums by as much: a weight by
             scale 2^-17 max|q| max_j |k_j|_1 twice, against numerator and sum: four times that
  the rest   exponentials and fp32 sums: 2^-20 of the weights
"""
import numpy as np
import pytest

from tests.test_gpu_cache8 import dequantize_t, random_cache
from tests.test_gpu_attn import U, L  # noqa: F401

pytestmark = pytest.mark.gpu


def check_tight(torch, got, q, k, v, vb, top, first_pos, few, window=0, n_sink=0, scale=None):
    """Rows got, q [rows, hq, d] at positions first_pos .. over keys k, v [n, hq, d] (fp64), vb [n, hq] the
    exponents of the values' blocks, top the largest that is seen."""
    rows, n, d = q.shape[0], k.shape[0], q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    x = torch.einsum("thd,nhd->htn", q.double(), k) * scale
    pos = torch.arange(first_pos, first_pos + rows, device="cuda")[:, None]
    key = torch.arange(n, device="cuda")
    seen = key <= pos
    if window:
        seen &= (key > pos - window) | (key < n_sink)
    w = x.masked_fill(~seen, -float("inf")).softmax(-1)
    w_max = w.amax(-1, keepdim=True) * seen
    size, down = v.abs(), (top - vb).double()
    if few:
        err = torch.maximum(2.0 ** -12 * w, 2.0 ** -23 * w_max * torch.exp2(down.clamp(max=900)).t()[:, None])
        err = torch.einsum("htn,nhd->thd", torch.minimum(err, w + 2.0 ** -12 * w), size)
    else:
        rounding = torch.where(down > 24, size.amax(-1), torch.where(down > 15, 2.0 ** -25 * 2.0 ** top, 0.0))
        err = torch.einsum("htn,nhd->thd", 2.0 ** -11 * w + 2.0 ** -31 * w_max, size) + \
            torch.einsum("htn,nh->th", w, rounding)[..., None]
    ref, wv = (torch.einsum("htn,nhd->thd", w, y) for y in (v, size))
    score = scale * 2.0 ** -17 * q.abs().max().double() * k.abs().sum(-1).max()
    bound = U * ref.abs() + 2.0 ** -134 + 2.0 ** -145 + (1 + U) * (err + (4 * score + 2.0 ** -20) * wv)
    assert bool(torch.isfinite(got).all())
    worst = float(((got.double() - ref).abs() / bound).max())
    assert worst <= 1


def sequence(torch, cache, row, n, group):
    """k, v [n, hq, d] and the values' exponents [n, hq] of the pages in `row`."""
    ids = row.long()
    hkv, d, page = cache[0].shape[1], cache[0].shape[3], cache[0].shape[2]
    k, v = (dequantize_t(torch, cache[i][ids], cache[i + 2][ids]).transpose(1, 2).reshape(-1, hkv, d)[:n]
            .repeat_interleave(group, 1) for i in (0, 1))
    vb = (cache[3][ids].int().clamp(1, 253) - 127).repeat_interleave(min(16, page), -1).transpose(1, 2)
    return k, v, vb.reshape(-1, hkv)[:n].repeat_interleave(group, 1)


def batch(L, torch, cache, q_lens, kv_len, hq, seed=0, size=0.05, window=0, n_sink=0, repeats=2):
    """A batch over the cache: every sequence against check_tight, and equal bits from equal calls."""
    n_pages, hkv, page, d = cache[0].shape
    n, group = len(q_lens), hq // hkv
    pages = n_pages // n
    torch.manual_seed(seed)
    table = torch.randperm(n_pages, device="cuda")[:n * pages].to(torch.int32).view(n, pages)
    off = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    T = int(off[-1])
    q = (size * torch.randn(T, hq, d, device="cuda")).to(torch.bfloat16)
    kv = L.PagedKV8bit(*cache, table, torch.from_numpy(off).cuda(),
                       torch.from_numpy(np.asarray(kv_len, np.int32)).cuda(), T, max_q_len=int(max(q_lens)))
    ws = L.attn_workspace(kv, hq)
    got = L.attn_paged_8bit_t(kv, q, ws, window=window, n_sink=n_sink)
    assert L.get_error_t(ws) == 0
    few = max(q_lens) * group <= 16 or group > 128
    for s in range(n):
        m, a, b = int(kv_len[s]), int(off[s]), int(off[s + 1])
        if a == b:
            continue
        k, v, vb = sequence(torch, cache, table[s], m, group)
        check_tight(torch, got[a:b], q[a:b], k, v, vb, int(vb.max()), m - (b - a), few, window, n_sink)
    for _ in range(repeats):
        assert torch.equal(L.attn_paged_8bit_t(kv, q, ws, window=window, n_sink=n_sink).view(torch.int16),
                           got.view(torch.int16))
    assert L.get_error_t(ws) == 0
    return got


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 64), (8, 8, 64), (64, 8, 64), (16, 1, 64), (32, 8, 128), (32, 2, 128)])
@pytest.mark.parametrize("page", [8, 16])
def test_long_segments_of_single_tokens(L, hq, hkv, d, page):
    """Shares of several segments of many key tiles: in pages of 8 a batch of scales is two tiles, and a
    warpgroup comes for its own while the other's of up to twelve tiles may be on their way."""
    import torch
    rng = np.random.default_rng(hq + page)
    n = 60
    kv_len = rng.integers(1000, 4000, n)
    torch.manual_seed(hq)
    cache = random_cache(torch, n * -(-4000 // page), hkv, page, d)
    # exponents all over, so that another block's would show
    for c in cache[2:]:
        c.copy_(torch.randint(112, 123, c.shape, device="cuda", dtype=torch.uint8))
    batch(L, torch, cache, [1] * n, kv_len, hq, seed=hq, repeats=30)


def test_append_with_offsets_out_of_order(L):
    """Rows whose sequence the offsets do not give are reported and not cached (a run from them would have
    fewer rows than none)."""
    import torch
    hq, hkv, d, page = 4, 2, 64, 16
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = L.PagedKV8bit.empty_cache(6, hkv, page, d)
    for c in cache[2:]:
        c.fill_(77)
    # rows 2 and 3 look like sequence 1's, which ends in front of them
    off, lens, table = i32([0, 50, 2, 4]), i32([50, 15, 0]), i32([[0, 1, 2, 3], [4, 5, -1, -1], [-1] * 4])
    q, k = (torch.ones(4, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv))
    for max_q in (1, 64):
        kv = L.PagedKV8bit(*cache, table, off, lens, 4, max_q_len=max_q)
        ws = L.attn_workspace(kv, hq)
        L.kv_append_8bit_t(kv, q, k, k, None, ws)
        if max_q == 1:
            assert L.get_error_t(ws) == L.DEVERR_BAD_LEN
        for c, s in ((cache[0], cache[2]), (cache[1], cache[3])):
            assert not c.view(torch.uint8)[1:].any() and (s[1:] == 77).all()


@pytest.mark.parametrize("byte", [1, 4, 12])
@pytest.mark.parametrize("rows,n,hkv", [(1, 3000, 2), (40, 3000, 2), (200, 200, 2), (40, 60000, 1), (700, 3000, 8), (2000, 3000, 8)])
def test_values_at_the_small_end(L, byte, rows, n, hkv):
    """Scales of 2^-126 and a little more, thousands of equal weights: results are normal numbers, and the
    sum of the weights must not push a factor of theirs below those."""
    import torch
    hq, d, page = 4 * hkv, 64, 16
    torch.manual_seed(byte + rows)
    cache = random_cache(torch, -(-n // page), hkv, page, d)
    cache[1].bitwise_and_(127)     # (values of one sign, so that the mean is no smaller than they are)
    cache[3].fill_(byte)
    cache[3][0] = byte + 1
    batch(L, torch, cache, [rows], [n], hq, seed=rows, size=0.0)


def test_a_shared_prefix_of_small_values(L):
    import torch
    hq, hkv, d, page, n, prefix, own = 8, 2, 64, 16, 30, 2000, 48
    torch.manual_seed(3)
    pages = prefix // page
    cache = random_cache(torch, pages + n * 3, hkv, page, d)
    cache[1].bitwise_and_(127)
    cache[3].fill_(3)
    table = torch.cat([torch.arange(pages, device="cuda").expand(n, -1),
                       pages + torch.arange(3 * n, device="cuda").view(n, 3)], 1).int().contiguous()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kv = L.PagedKV8bit(*cache, table, torch.arange(n + 1, dtype=torch.int32, device="cuda"), i32([prefix + own] * n), n,
                       max_q_len=1)
    q = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    ws = L.attn_workspace(kv, hq, n_groups=1)
    got = L.attn_prefix_8bit_t(kv, q, i32([0, n]), i32([prefix]), ws)
    assert L.get_error_t(ws) == 0
    for s in range(n):
        k, v, vb = sequence(torch, cache, table[s], prefix + own, hq // hkv)
        check_tight(torch, got[s:s + 1], q[s:s + 1], k, v, vb, 3 - 127, prefix + own - 1, False)


# ------------------------------------------------------------------ blocks of very different size

def spread(torch, cache, low, high):
    """The values' scales anywhere between two bytes, a tenth of them at either end."""
    vs = cache[3]
    x = torch.randint(low, high + 1, vs.shape, device="cuda")
    pick = torch.rand(vs.shape, device="cuda")
    x = torch.where(pick < 0.1, low, torch.where(pick > 0.9, high, x))
    vs.copy_(x.to(torch.uint8))


@pytest.mark.parametrize("low,high", [(110, 123), (100, 125), (95, 135), (20, 240)])
@pytest.mark.parametrize("hq,hkv,d,rows", [(8, 2, 64, 1), (8, 2, 128, 4), (32, 2, 128, 1), (16, 4, 64, 70), (8, 2, 128, 200)])
@pytest.mark.parametrize("page", [8, 32])
def test_value_blocks_of_very_different_size(L, low, high, hq, hkv, d, rows, page):
    """Ratios at which an f16 of a value is exact, rounded, and lost, and a weight's terms leave the range of
    their type; past 2^127 a factor between blocks is no number of fp32's exponents."""
    import torch
    rng = np.random.default_rng(low + rows)
    n = 12
    q_lens = rng.integers(1, rows + 1, n)
    q_lens[0] = rows
    kv_len = q_lens + rng.integers(0, 900, n)
    torch.manual_seed(high + page)
    cache = random_cache(torch, n * -(-1200 // page), hkv, page, d)
    spread(torch, cache, low, high)
    batch(L, torch, cache, list(q_lens), kv_len, hq, seed=low)


@pytest.mark.parametrize("more", [8, 13, 16, 20, 25, 40, 130])
@pytest.mark.parametrize("hq,hkv,d,rows", [(8, 2, 64, 4), (4, 2, 128, 8), (8, 2, 64, 64), (8, 2, 128, 300)])
def test_a_later_token_with_much_larger_values(L, more, hq, hkv, d, rows):
    """The last block of a prompt has values 2^more times the others': rows in front of it do not see them,
    but are rounded against their scale, within the bound of that."""
    import torch
    page, n = 16, 320
    torch.manual_seed(more)
    cache = random_cache(torch, n // page, hkv, page, d)
    table = torch.randperm(n // page, device="cuda").int()[None]
    cache[3].fill_(100)
    cache[3][table[0, -1].long()] = 100 + more
    kv = L.PagedKV8bit(*cache, table, torch.tensor([0, rows], dtype=torch.int32, device="cuda"),
                       torch.tensor([n], dtype=torch.int32, device="cuda"), rows)
    q = (0.05 * torch.randn(rows, hq, d, device="cuda")).to(torch.bfloat16)
    ws = L.attn_workspace(kv, hq)
    got = L.attn_paged_8bit_t(kv, q, ws)
    assert L.get_error_t(ws) == 0
    k, v, vb = sequence(torch, cache, table[0], n, hq // hkv)
    check_tight(torch, got, q, k, v, vb, int(vb.max()), n - rows, rows * hq // hkv <= 16)


# ------------------------------------------------------------------ windows, pages, parts and prefixes

@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 8, 64), (64, 8, 64), (16, 1, 128), (24, 1, 64)])
@pytest.mark.parametrize("rows", [1, 90])
@pytest.mark.parametrize("page,window,n_sink", [(8, 0, 0), (16, 700, 4), (256, 0, 0), (64, 130, 40)])
def test_batches_part_by_part(L, hq, hkv, d, rows, page, window, n_sink):
    import torch
    rng = np.random.default_rng(hq + rows + page)
    n = 24
    q_lens = rng.integers(1, rows + 1, n)
    kv_len = q_lens + rng.integers(0, 2500, n)
    torch.manual_seed(hq)
    cache = random_cache(torch, n * -(-2700 // page), hkv, page, d)
    batch(L, torch, cache, list(q_lens), kv_len, hq, seed=rows, window=window, n_sink=n_sink)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 8, 64), (16, 1, 128)])
@pytest.mark.parametrize("rows", [1, 60])
@pytest.mark.parametrize("n", [1, 2, 40])
def test_prefixes_part_by_part(L, hq, hkv, d, rows, n):
    """The two phases apart: each is rounded against the largest scale of its own keys."""
    import torch
    page, prefix, own = 16, 1500, 200
    rng = np.random.default_rng(n + rows)
    q_lens = [int(x) for x in rng.integers(1, rows + 1, n)]
    torch.manual_seed(n + hq)
    shared = -(-prefix // page)
    mine = -(-(prefix + own) // page) - prefix // page
    cache = random_cache(torch, shared + n * mine, hkv, page, d)
    spread(torch, cache, 112, 122)
    table = torch.full((n, prefix // page + mine), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    table[0, :shared] = torch.arange(shared, device="cuda")
    for s in range(n):
        at = shared + s * mine + torch.arange(mine, device="cuda")
        table[s, prefix // page:] = at
        for c in cache:     # the prefix' last page, a copy each
            c.view(torch.uint8)[at[0]] = c.view(torch.uint8)[shared - 1]
    off = torch.tensor([0] + q_lens, device="cuda").cumsum(0).int()
    T = int(off[-1])
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kv = L.PagedKV8bit(*cache, table, off, i32([prefix + own] * n), T, max_q_len=max(q_lens))
    q = (0.05 * torch.randn(T, hq, d, device="cuda")).to(torch.bfloat16)
    ws = L.attn_workspace(kv, hq, n_groups=1)
    got = L.attn_prefix_8bit_t(kv, q, i32([0, n]), i32([prefix]), ws)
    assert L.get_error_t(ws) == 0
    few = T * (hq // hkv) <= 16 and max(q_lens) * (hq // hkv) <= 16
    a = 0
    for s, m in enumerate(q_lens):
        row = torch.cat([table[0, :prefix // page], table[s, prefix // page:]])
        k, v, vb = sequence(torch, cache, row, prefix + own, hq // hkv)
        check_tight(torch, got[a:a + m], q[a:a + m], k, v, vb, int(vb.max()), prefix + own - m, few)
        a += m
