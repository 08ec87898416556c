"""The paged-cache operators on the GPU against the fp64 reference (oracle/attn_ref.py), at
the lengths, masks, layouts and strides where they can go wrong.

Tolerances.  Append: v is copied bit for bit; a rotated value is an fp32 expression of two
products, rounded once to bf16, so |err| <= 2^-8 |ref| + 2^-22 max|x| over the head.

Attention: the result is rounded once (2^-8 |ref|); each weight enters its product as bf16
(or a more exact pair), an error of at most 2^-8 w_j |v_j| a key, so 2^-8 sum_j w_j |v_j|
over the row; scores in fp32 over at most 128 products of |q_i k_i| < 40 have errors below
128 * 40 * 2^-24 < 2^-11 before scaling by 1/8 or less, so below 2^-14, which moves every
weight by less than 2^-12 of itself, counted against numerator and sum:
    |err| <= 2^-8 |ref| + (2^-8 + 2^-12) sum_j w_j |v_j|.
"""
import numpy as np
import pytest

from oracle import attn_ref as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module")
def L():
    from lora_serving_device_gb300 import build, lora
    build.build()
    lora.load()
    return lora


def bf16(torch, rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


class Case:
    """A batch over a paged cache.  Everything no row may see is NaN (cache) or a wild number
    (block table); page ids are shuffled; q and out are parts of wider rows."""

    def __init__(self, q_lens, ctx, hq, hkv, d, page, seed=0, window=0, n_sink=0, pad_rows=0, groups=None,
                 extra_pages=3, missing=(), spread=1.0):
        import torch
        self.torch = torch
        rng = np.random.default_rng(seed)
        self.q_lens, self.hq, self.hkv, self.d, self.page = q_lens, hq, hkv, d, page
        self.window, self.n_sink = window, n_sink
        self.q_off = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.kv_len = np.asarray([c + n for c, n in zip(ctx, q_lens)], np.int32)
        self.T = int(self.q_off[-1]) + pad_rows
        n = len(q_lens)
        self.rows_k, self.rows_v = [], []
        group_of = {}
        if groups:
            first, plen = groups
            for g in range(len(plen)):
                for s in range(first[g], first[g + 1]):
                    group_of[s] = g
        max_pages = max(1, max(-(-int(x) // page) for x in self.kv_len)) + 2
        table = rng.integers(-(1 << 30), 1 << 30, (n, max_pages)).astype(np.int64)
        table[table >= 0] += 1 << 20           # no wild entry is a page that exists
        pages = []
        for s in range(n):
            length = max(int(self.kv_len[s]), 0)
            k, v = (bf16(torch, rng, length, hkv, d) * spread if length else
                    torch.zeros(0, hkv, d, dtype=torch.bfloat16) for _ in range(2))
            if s in group_of:
                g = group_of[s]
                f, p = groups[0][g], groups[1][g]
                if s > f:
                    p = min(p, length)
                    k[:p], v[:p] = self.rows_k[f][:p], self.rows_v[f][:p]
            self.rows_k.append(k)
            self.rows_v.append(v)
            lo = length
            if q_lens[s]:
                first_row = int(self.kv_len[s]) - q_lens[s]
                lo = max(0, first_row - window + 1) if window else 0
            for p in range(-(-length // page)):
                a, b = p * page, min((p + 1) * page, length)
                if b <= lo and not (window and a < n_sink):
                    continue                       # nobody sees it: freed
                if s in group_of and s > groups[0][group_of[s]] and (p + 1) * page <= groups[1][group_of[s]]:
                    continue                       # wholly inside the prefix: read through the first row
                if (s, p) in missing:
                    k[a:b], v[a:b] = 0, 0
                    continue
                table[s, p] = len(pages)
                pages.append((s, a, b))
        n_pages = len(pages) + extra_pages
        order = rng.permutation(n_pages)
        kc = torch.full((n_pages, hkv, page, d), float("nan"), dtype=torch.bfloat16)
        vc = kc.clone()
        for i, (s, a, b) in enumerate(pages):
            lo = 0
            if window and q_lens[s]:
                lo = max(0, int(self.kv_len[s]) - q_lens[s] - window + 1)
            for j in range(a, b):
                if j >= lo or j < n_sink:
                    kc[order[i], :, j - a] = self.rows_k[s][j]
                    vc[order[i], :, j - a] = self.rows_v[s][j]
        ok = (table >= 0) & (table < len(pages))
        table[ok] = order[table[ok]]
        self.kc, self.vc = kc.cuda(), vc.cuda()
        self.table = torch.from_numpy(table.astype(np.int32)).cuda()
        wide = bf16(torch, rng, self.T, (hq + 2) * d) * spread
        self.q_host = wide[:, d:(hq + 1) * d].reshape(self.T, hq, d).double().numpy()
        self.q = wide.cuda()[:, d:(hq + 1) * d].view(self.T, hq, d)
        self.out = torch.full((self.T, (hq + 1) * d), 7.0, dtype=torch.bfloat16, device="cuda")
        self.out = self.out[:, d:].view(self.T, hq, d)
        self.dq_off = torch.from_numpy(self.q_off).cuda()
        self.dkv_len = torch.from_numpy(self.kv_len).cuda()

    def kv(self, L, max_q=None):
        return L.PagedKV(self.kc, self.vc, self.table, self.dq_off, self.dkv_len, self.T,
                         max_q_len=max(self.q_lens) if max_q is None else max_q)

    def check(self, got, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        ref, wv = R.attention(self.q_host, [k.double().numpy() for k in self.rows_k],
                              [v.double().numpy() for v in self.rows_v], self.q_off, self.kv_len, scale,
                              self.window, self.n_sink)
        got = got.double().cpu().numpy()
        n = int(self.q_off[-1])
        assert np.all(got[n:] == 7.0), "rows of no sequence were written"
        ref, wv, got = ref[:n], wv[:n], got[:n]
        assert np.all(np.isfinite(got))
        assert np.all(got[wv.sum(-1) == 0] == 0), "rows that see nothing are zeros"
        excess = np.abs(got - ref) / (U * np.abs(ref) + (U + 2.0 ** -12) * wv + 1e-30)
        assert excess.size == 0 or excess.max() <= 1, f"{excess.max()} at {np.unravel_index(excess.argmax(), excess.shape)}"
        if ref.size > 500:
            assert np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref)


def attend(L, c, err=0, max_q=None, scale=None):
    kv = c.kv(L, max_q)
    ws = L.attn_workspace(kv, c.hq)
    got = L.attn_paged_t(kv, c.q, ws, window=c.window, n_sink=c.n_sink, out=c.out, scale=scale)
    assert L.get_error_t(ws) == err
    c.check(got, scale)
    first = got.clone()
    again = L.attn_paged_t(kv, c.q, ws, window=c.window, n_sink=c.n_sink, out=c.out, scale=scale)
    assert c.torch.equal(first.view(c.torch.int16), again.view(c.torch.int16)), "the workspace is not left clean"


HEADS = [(8, 2, 128), (8, 8, 64), (7, 1, 128), (15, 5, 64), (20, 1, 64), (32, 2, 128)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("page", [8, 64])
def test_single_tokens(L, hq, hkv, d, page):
    ctx = [0, 1, 14, 15, 16, 63, 126, 127, 128, 129, 255, 500, 700]
    attend(L, Case([1] * len(ctx), ctx, hq, hkv, d, page, seed=hq + page))


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_page_sizes(L, page, d):
    attend(L, Case([1, 5, 200], [300, 3, 77], 4, 2, d, page, seed=page))


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_chunks_and_single_tokens_in_one_batch(L, hq, hkv, d):
    attend(L, Case([130, 1, 0, 17, 1, 64], [0, 200, 90, 140, 0, 255], hq, hkv, d, 16, seed=3, pad_rows=3))


@pytest.mark.parametrize("n", [1, 2, 3, 8, 15, 16, 17, 33, 64, 65, 127, 128, 129, 257])
def test_prompt_lengths(L, n):
    attend(L, Case([n], [0], 4, 2, 128, 16, seed=n))
    attend(L, Case([n], [70], 4, 1, 64, 32, seed=n))


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 3), (2, 0), (40, 4), (128, 0), (128, 130), (129, 1),
                                           (300, 16), (100000, 5), (64, 1000)])
@pytest.mark.parametrize("d", [64, 128])
def test_windows_and_first_tokens(L, window, n_sink, d):
    attend(L, Case([1, 1, 1, 1, 1], [0, 39, 128, 500, 641], 4, 2, d, 16, seed=window, window=window,
                   n_sink=n_sink))
    attend(L, Case([150, 1, 30, 0], [0, 450, 333, 8], 4, 2, d, 16, seed=window, window=window, n_sink=n_sink))


@pytest.mark.parametrize("d,page,n_sink", [(128, 32, 33), (64, 64, 4), (128, 128, 128), (64, 256, 5)])
def test_windows_that_move_over_pages(L, d, page, n_sink):
    # the window's first key at, before and after a page's first, and where its
    # pages reach those of the first tokens
    n = [150, 159, 160, 161, 287, 288, 289, 415, 416, 417, 543, 545]
    attend(L, Case([1] * len(n), [x - 1 for x in n], 8, 1, d, page, seed=page, window=32, n_sink=n_sink))
    attend(L, Case([40, 1, 200, 3], [x - 40 for x in (289, 545, 700, 161)], 8, 1, d, page, seed=n_sink,
                   window=129, n_sink=n_sink))


def test_rows_that_see_nothing(L):
    # kv_len below the number of new tokens: the first rows lie before position 0
    c = Case([3, 1, 2, 140], [0, -1, -2, -20], 4, 2, 64, 16, seed=5)
    attend(L, c)
    attend(L, Case([2], [-2], 4, 2, 128, 16, seed=5))
    attend(L, Case([0, 0], [5, 0], 4, 2, 128, 16, seed=5, pad_rows=2))


def test_max_q_len_is_a_hint(L):
    for max_q in (0, 1, 1000):
        attend(L, Case([1, 90, 3], [100, 50, 7], 8, 2, 64, 16, seed=6), max_q=max_q)


def test_large_scores_and_scale(L):
    # scores of hundreds: the running maximum moves far, most weights vanish
    attend(L, Case([1, 40], [600, 300], 4, 2, 64, 16, seed=7, spread=6.0), scale=0.02)
    attend(L, Case([1, 40], [600, 300], 4, 2, 64, 16, seed=8), scale=1.0)


def test_missing_pages_read_as_zeros_and_are_reported(L):
    attend(L, Case([1, 20], [100, 60], 4, 2, 64, 16, seed=9, missing={(0, 2), (1, 0)}), err=L.DEVERR_BAD_PAGE)


def test_many_sequences(L):
    rng = np.random.default_rng(1)
    ctx = [int(x) for x in rng.integers(0, 60, 1500)]
    q = [int(x) for x in rng.integers(0, 2, 1500)]
    attend(L, Case(q, ctx, 2, 1, 64, 16, seed=10))


def test_long_context_of_few_rows(L):
    """Split over the keys: 30000 of them, against fp64 on the GPU."""
    import torch
    torch.manual_seed(0)
    n, hq, hkv, d, page = 30011, 8, 2, 128, 64
    pages = -(-n // page)
    kc, vc = (torch.randn(pages, hkv, page, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.randperm(pages, device="cuda").to(torch.int32)[None]
    for rows in (1, 3, 100):
        q = torch.randn(rows, hq, d, device="cuda").to(torch.bfloat16)
        kv = L.PagedKV(kc, vc, table, torch.tensor([0, rows], dtype=torch.int32, device="cuda"),
                       torch.tensor([n], dtype=torch.int32, device="cuda"), rows)
        ws = L.attn_workspace(kv, hq)
        got = L.attn_paged_t(kv, q, ws).double()
        assert L.get_error_t(ws) == 0
        k, v = (c[table[0].long()].transpose(1, 2).reshape(-1, hkv, d)[:n].double().repeat_interleave(hq // hkv, 1)
                for c in (kc, vc))
        x = torch.einsum("thd,nhd->htn", q.double(), k) * d ** -0.5
        pos = torch.arange(n - rows, n, device="cuda")
        x = x.masked_fill(torch.arange(n, device="cuda") > pos[:, None], -float("inf"))
        w = x.softmax(-1)
        ref, wv = (torch.einsum("htn,nhd->thd", w, y) for y in (v, v.abs()))
        assert ((got - ref).abs() <= U * ref.abs() + (U + 2.0 ** -12) * wv).all()
        assert (got - ref).norm() <= 5e-3 * ref.norm()


@pytest.mark.parametrize("hq,hkv,d,window", [(64, 8, 64, 1024), (32, 8, 128, 0), (12, 12, 64, 0), (32, 2, 128, 300),
                                             (24, 1, 64, 0)])
@pytest.mark.parametrize("rows", [1, 70])
def test_ordinary_batches(L, hq, hkv, d, window, rows):
    """Shares of many segments and tiles, on every SM: 60 sequences of 1 or up to 70 new rows,
    against fp64 on the GPU."""
    import torch
    rng = np.random.default_rng(hq + window + rows)
    n, page, n_sink = 60, 32, 4
    ctx = rng.integers(0, 4000, n)
    q_lens = rng.integers(1, rows + 1, n)
    kv_len = ctx + q_lens
    max_pages = -(-int(kv_len.max()) // page)
    table = torch.randperm(n * max_pages, device="cuda").to(torch.int32).view(n, max_pages)
    torch.manual_seed(hq)
    kc, vc = (torch.randn(n * max_pages, hkv, page, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    off = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    T = int(off[-1])
    q = torch.randn(T, hq, d, device="cuda").to(torch.bfloat16)
    kv = L.PagedKV(kc, vc, table, torch.from_numpy(off).cuda(), torch.from_numpy(kv_len.astype(np.int32)).cuda(), T,
                   max_q_len=int(q_lens.max()))
    ws = L.attn_workspace(kv, hq)
    got = L.attn_paged_t(kv, q, ws, window=window, n_sink=n_sink)
    assert L.get_error_t(ws) == 0
    for s in range(n):
        m = int(kv_len[s])
        k, v = (c[table[s].long()].transpose(1, 2).reshape(-1, hkv, d)[:m].double().repeat_interleave(hq // hkv, 1)
                for c in (kc, vc))
        a, b = int(off[s]), int(off[s + 1])
        x = torch.einsum("thd,nhd->htn", q[a:b].double(), k) * d ** -0.5
        pos = torch.arange(m - (b - a), m, device="cuda")[:, None]
        key = torch.arange(m, device="cuda")
        seen = key <= pos
        if window:
            seen &= (key > pos - window) | (key < n_sink)
        w = x.masked_fill(~seen, -float("inf")).softmax(-1)
        ref, wv = (torch.einsum("htn,nhd->thd", w, y) for y in (v, v.abs()))
        err = (got[a:b].double() - ref).abs()
        assert (err <= U * ref.abs() + (U + 2.0 ** -12) * wv).all(), s
        assert err.norm() <= 5e-3 * ref.norm()
    assert torch.equal(got, L.attn_paged_t(kv, q, ws, window=window, n_sink=n_sink))


def test_cache_past_32_bit_offsets(L):
    """A cache of more than 2^32 elements, used at its end."""
    import torch
    hkv, page, d = 8, 256, 128
    n_pages = (1 << 32) // (hkv * page * d) + 40
    kc = torch.empty(n_pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    torch.manual_seed(1)
    n, hq = 700, 8
    ids = torch.tensor([n_pages - 1, 0, n_pages - 3], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(n, hkv, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(n, hq, d, device="cuda").to(torch.bfloat16)
    kv = L.PagedKV(kc, vc, ids[None].contiguous(), torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                   torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    ws = L.attn_workspace(kv, hq)
    L.kv_append_t(kv, None, k, v, None, ws)
    for x, c in ((k, kc), (v, vc)):
        assert torch.equal(c[ids.long()].transpose(1, 2).reshape(-1, hkv, d)[:n], x)
    got = L.attn_paged_t(kv, q, ws).double()
    x = torch.einsum("thd,nhd->htn", q.double(), k.double()) * d ** -0.5
    w = x.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -float("inf")).softmax(-1)
    ref, wv = (torch.einsum("htn,nhd->thd", w, y) for y in (v.double(), v.double().abs()))
    assert ((got - ref).abs() <= U * ref.abs() + (U + 2.0 ** -12) * wv).all()
    last = L.PagedKV(kc, vc, ids[None].contiguous(), torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                     torch.tensor([n], dtype=torch.int32, device="cuda"), 1)
    one = L.attn_paged_t(last, q[-1:], L.attn_workspace(last, hq)).double()
    assert ((one - ref[-1:]).abs() <= U * ref[-1:].abs() + (U + 2.0 ** -12) * wv[-1:]).all()
    assert L.get_error_t(ws) == 0


# ------------------------------------------------------------------ shared prefixes

def prefix_attend(L, c, groups, err=0, max_q=None):
    torch = c.torch
    kv = c.kv(L, max_q)
    first, plen = groups
    off, pl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (first, plen))
    ws = L.attn_workspace(kv, c.hq, n_groups=len(plen))
    got = L.attn_prefix_t(kv, c.q, off, pl, ws, out=c.out)
    assert L.get_error_t(ws) == err
    c.check(got)
    before = got.clone()
    again = L.attn_prefix_t(kv, c.q, off, pl, ws, out=c.out)
    assert torch.equal(before.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("prefix", [1, 17, 128, 300])
def test_shared_prefix(L, hq, hkv, d, prefix):
    n = 9
    groups = ([0, n], [prefix])
    prefix_attend(L, Case([1] * n, [prefix + 11 * i for i in range(n)], hq, hkv, d, 16, seed=prefix,
                          groups=groups), groups)


@pytest.mark.parametrize("page", [8, 32, 128])
def test_prefix_groups(L, page):
    # a group of one, an empty group, a prefix of nothing, chunks, sequences without rows and
    # sequences after the last group
    groups = ([0, 1, 1, 4, 6, 40], [40, 9, 0, 200, 131])
    q = [1, 2, 0, 30, 1, 1] + [1] * 34 + [1, 5]
    ctx = [50, 60, 10, 3, 200, 260] + [131 + 7 * (i % 9) for i in range(34)] + [20, 90]
    prefix_attend(L, Case(q, ctx, 8, 2, 64, page, seed=page, groups=groups), groups)


def test_prefix_of_many_rows(L):
    groups = ([0, 3], [260])
    prefix_attend(L, Case([100, 33, 64], [260, 261, 300], 8, 2, 128, 16, seed=2, groups=groups, pad_rows=1), groups)
    groups = ([0, 90, 100], [270, 30])
    prefix_attend(L, Case([1] * 100, [270 + i % 5 for i in range(90)] + [30] * 10, 8, 2, 128, 16, seed=2,
                          groups=groups), groups)


def test_prefix_longer_than_a_context_is_reported(L):
    import torch
    groups = ([0, 3], [50])
    c = Case([1, 1, 1], [60, 50, 20], 4, 2, 64, 16, seed=3, groups=groups)
    kv = c.kv(L)
    ws = L.attn_workspace(kv, c.hq, n_groups=1)
    off, pl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in groups)
    got = L.attn_prefix_t(kv, c.q, off, pl, ws, out=c.out).double().cpu().numpy()
    assert L.get_error_t(ws) == L.DEVERR_BAD_LEN
    ref, wv = R.attention(c.q_host, [k.double().numpy() for k in c.rows_k],
                          [v.double().numpy() for v in c.rows_v], c.q_off, c.kv_len, c.d ** -0.5)
    assert np.all(np.abs(got - ref)[:2] <= U * np.abs(ref[:2]) + (U + 2.0 ** -12) * wv[:2])


def test_one_workspace_for_batches_of_all_sizes(L):
    import torch
    cases = [Case([1], [900], 8, 1, 64, 16, seed=1), Case([300], [200], 8, 2, 128, 16, seed=2),
             Case([1] * 70, [9 * i for i in range(70)], 4, 2, 64, 32, seed=3),
             Case([3, 50], [700, 100], 16, 2, 128, 16, seed=4, window=60, n_sink=3)]
    groups = ([0, 40], [300])
    shared = Case([1] * 40, [300 + i for i in range(40)], 8, 2, 128, 16, seed=5, groups=groups)
    off, pl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in groups)
    ws = torch.zeros(max([L.attn_workspace(shared.kv(L), 8, 1).numel()] +
                         [L.attn_workspace(c.kv(L), c.hq).numel() for c in cases]), dtype=torch.uint8, device="cuda")
    ws[4096:].fill_(0xFF)     # whatever earlier calls left behind the counters
    for _ in range(2):
        for c in cases + [shared] + cases[::-1]:
            if c is shared:
                L.attn_prefix_t(c.kv(L), c.q, off, pl, ws, out=c.out)
            else:
                L.attn_paged_t(c.kv(L), c.q, ws, window=c.window, n_sink=c.n_sink, out=c.out)
            c.check(c.out)
    assert L.get_error_t(ws) == 0


# ------------------------------------------------------------------ append

def table_rows(torch, rng, n_pos, rot):
    freq = 1000.0 ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(n_pos)[:, None] * freq
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


@pytest.mark.parametrize("hq,hkv,d,rot", [(8, 2, 128, 128), (28, 4, 128, 64), (5, 5, 64, 64), (6, 2, 64, 16),
                                          (0, 3, 64, 64), (40, 8, 128, 128), (4, 4, 128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [0, 1, 3, 4])
def test_append(L, hq, hkv, d, rot, interleaved, axes):
    import torch
    rng = np.random.default_rng(hq + rot + axes)
    page = 16
    q_lens, ctx = [1, 0, 37, 1, 3], [20, 5, 11, 0, -2]
    q_off = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    kv_len = np.asarray([a + b for a, b in zip(q_lens, ctx)], np.int32)
    T = int(q_off[-1]) + 2
    n_pages, max_pages, n_pos = 30, 5, 64
    table = rng.permutation(n_pages)[:25].reshape(5, 5).astype(np.int32)
    wide = bf16(torch, rng, T, (hq + 2 * hkv + 1) * d)
    parts = [wide[:, a * d:b * d].reshape(T, b - a, d) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv))]
    dev = wide.cuda()
    dq, dk, dv = (dev[:, a * d:b * d].view(T, b - a, d) for a, b in ((0, hq), (hq, hq + hkv),
                                                                      (hq + hkv, hq + 2 * hkv)))
    kc, vc = (bf16(torch, rng, n_pages, hkv, page, d).cuda() for _ in range(2))
    old_k, old_v = kc.clone(), vc.clone()
    cs = table_rows(torch, rng, n_pos, rot) if rot else None
    half = rot // 2
    pairs = {0: [half], 1: [half], 3: [half // 4, half // 2 - 1, half - half // 4 - half // 2 + 1],
             4: [0, half // 2, 3, half - half // 2 - 3]}[axes]
    if min(pairs) < 0:
        pytest.skip("too few pairs for these axes")
    pos = rng.integers(0, n_pos, (max(axes, 1), T)).astype(np.int32)
    kv = L.PagedKV(kc, vc, torch.from_numpy(table).cuda(), torch.from_numpy(q_off).cuda(),
                   torch.from_numpy(kv_len).cuda(), T)
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    q_out = torch.full((T, max(hq, 1), d), 7.0, dtype=torch.bfloat16, device="cuda")
    got = L.kv_append_t(kv, dq if hq else None, dk, dv, None if cs is None else torch.from_numpy(cs).cuda(), ws,
                        pos=torch.from_numpy(pos).cuda() if axes else None, axis_pairs=pairs if axes > 1 else None,
                        interleaved=interleaved, q_out=q_out if hq else None)
    err = L.get_error_t(ws)
    # positions in the cache: rows before position 0 are outside the rotation's table
    assert err == (L.DEVERR_BAD_POS if axes == 0 and rot else 0)
    want_k, want_v = old_k.double().cpu().numpy(), old_v.double().cpu().numpy()
    tol_k = np.zeros_like(want_k)
    want_q = np.full((T, max(hq, 1), d), 7.0)
    tol_q = np.zeros_like(want_q)
    axis = np.repeat(np.arange(len(pairs)), pairs)
    for t, s, p in R.positions(q_off, kv_len):
        at = [int(pos[axis[i], t]) if axes else p for i in range(half)]
        turn = (lambda x: R.rotate(x, cs, at, interleaved)) if rot else (lambda x: x)
        for h in range(hq):
            x = parts[0][t, h].double().numpy()
            want_q[t, h] = turn(x)
            tol_q[t, h] = U * np.abs(want_q[t, h]) * (rot > 0) + 2.0 ** -22 * np.abs(x).max()
        if p < 0:
            continue
        for h in range(hkv):
            x = parts[1][t, h].double().numpy()
            place = (table[s, p // page], h, p % page)
            want_k[place] = turn(x)
            tol_k[place] = U * np.abs(want_k[place]) * (rot > 0) + 2.0 ** -22 * np.abs(x).max()
            want_v[place] = parts[2][t, h].double().numpy()
    assert np.array_equal(vc.double().cpu().numpy(), want_v)
    assert np.all(np.abs(kc.double().cpu().numpy() - want_k) <= tol_k)
    if hq:
        assert np.all(np.abs(got.double().cpu().numpy() - want_q) <= tol_q)
        in_place = L.kv_append_t(kv, dq, dk, dv, None if cs is None else torch.from_numpy(cs).cuda(), ws,
                                 pos=torch.from_numpy(pos).cuda() if axes else None,
                                 axis_pairs=pairs if axes > 1 else None, interleaved=interleaved, q_out=dq)
        n = int(q_off[-1])
        assert torch.equal(in_place[:n], got[:n])


def test_append_reports_missing_pages_and_writes_nothing_there(L):
    import torch
    torch.manual_seed(0)
    kc = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    tab = torch.tensor([[0, -1], [99, 2]], dtype=torch.int32, device="cuda")
    kv = L.PagedKV(kc, vc, tab, torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda"),
                   torch.tensor([18, 40], dtype=torch.int32, device="cuda"), 4)
    x = torch.randn(4, 1, 64, device="cuda").to(torch.bfloat16)
    ws = L.attn_workspace(kv, 1)
    L.kv_append_t(kv, None, x, x, None, ws)
    assert L.get_error_t(ws) == L.DEVERR_BAD_PAGE
    assert torch.equal(kc[0, 0, 15], x[0, 0]) and int((kc != 0).any(-1).sum()) == 1


# ------------------------------------------------------------------ streams and graphs

@pytest.mark.parametrize("prefix", [False, True])
def test_a_captured_step_follows_lengths_that_grow(L, prefix):
    import torch
    torch.manual_seed(0)
    n, hq, hkv, d, page = 5, 8, 2, 64, 16
    kc, vc = (torch.randn(60, hkv, page, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.randperm(60, device="cuda").to(torch.int32)[:60].view(n, 12).contiguous()
    if prefix:
        table[1:, :2] = table[0, :2]
    kv_len = torch.tensor([33, 47, 100, 64, 34], dtype=torch.int32, device="cuda")
    kv = L.PagedKV(kc, vc, table, torch.arange(n + 1, dtype=torch.int32, device="cuda"), kv_len, n, max_q_len=1)
    ws = L.attn_workspace(kv, hq, n_groups=1 if prefix else 0)
    q, k, v = (torch.randn(n, h, d, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    cs = L.rope_table(256, d)
    goff, plen = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [32]))

    def step():
        r = L.kv_append_t(kv, q, k, v, cs, ws)
        return L.attn_prefix_t(kv, r, goff, plen, ws) if prefix else L.attn_paged_t(kv, r, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
    torch.cuda.synchronize()
    for i in range(4):
        graph.replay()
        got = out.clone()
        want = step()
        assert torch.equal(got, want)
        kv_len += 9 if i < 2 else 1
        q.copy_(torch.randn_like(q))
    assert L.get_error_t(ws) == 0


def test_another_stream(L):
    import torch
    c = Case([1, 60], [300, 20], 4, 2, 64, 16, seed=4)
    kv = c.kv(L)
    ws = L.attn_workspace(kv, c.hq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    L.attn_paged_t(kv, c.q, ws, out=c.out, stream=s)
    assert L.get_error_t(ws, s) == 0
    c.check(c.out)
