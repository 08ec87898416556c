"""Host-side validation of the paged-cache entry points (no GPU: nothing valid enough to
launch is passed)."""
import ctypes

import numpy as np
import pytest

FAKE = 0x10000
WS = 0x900000


@pytest.fixture(scope="module")
def L():
    from lora_serving_device_gb300 import build, lora
    build.build()
    lora.load()
    return lora


def kv(L, **kw):
    a = dict(k_cache=FAKE, v_cache=FAKE, block_table=FAKE, q_off=FAKE, kv_len=FAKE, n_pages=10, page_size=16,
             n_kv_heads=2, head_dim=64, n_seqs=3, max_pages=4, T=5, max_q_len=2)
    a.update(kw)
    return L.PagedKVStruct(**a)


def append(L, kv_kw=None, **kw):
    a = dict(q=FAKE, qs=256, k=FAKE, ks=128, v=FAKE, vs=128, hq=4, cs=FAKE, n_pos=100, rot=64, pos=None, axes=1,
             pairs=None, inter=0, qo=FAKE + 4096, qos=256, ws=WS, wsb=16)
    a.update(kw)
    pairs = None if a["pairs"] is None else (ctypes.c_int32 * len(a["pairs"]))(*a["pairs"])
    st = None if kv_kw == "null" else ctypes.byref(kv(L, **(kv_kw or {})))
    return L.lora_kv_append(st, a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["hq"], a["cs"], a["n_pos"],
                            a["rot"], a["pos"], a["axes"], pairs, a["inter"], a["qo"], a["qos"], a["ws"],
                            a["wsb"], None)


def attend(L, kv_kw=None, prefix=None, **kw):
    a = dict(q=FAKE, qs=256, hq=4, scale=0.125, window=0, sink=0, out=FAKE + 4096, os=256, ws=WS, wsb=1 << 40)
    a.update(kw)
    st = None if kv_kw == "null" else ctypes.byref(kv(L, **(kv_kw or {})))
    if prefix is None:
        return L.lora_attn_paged(st, a["q"], a["qs"], a["hq"], a["scale"], a["window"], a["sink"], a["out"],
                                 a["os"], a["ws"], a["wsb"], None)
    return L.lora_attn_prefix(st, prefix[0], prefix[1], prefix[2], a["q"], a["qs"], a["hq"], a["scale"], a["out"],
                              a["os"], a["ws"], a["wsb"], None)


INVALID, SHAPE, WORKSPACE = 1, 2, 4
CACHE = [("null", INVALID), (dict(T=-1), INVALID), (dict(n_seqs=-1), INVALID), (dict(max_q_len=-1), INVALID),
         (dict(k_cache=None), INVALID), (dict(v_cache=FAKE + 8), INVALID), (dict(block_table=None), INVALID),
         (dict(q_off=FAKE + 2), INVALID), (dict(kv_len=None), INVALID), (dict(page_size=0), SHAPE),
         (dict(page_size=24), SHAPE), (dict(page_size=512), SHAPE), (dict(head_dim=96), SHAPE),
         (dict(n_kv_heads=0), SHAPE), (dict(n_seqs=0), SHAPE), (dict(n_seqs=65537), SHAPE),
         (dict(max_pages=0), SHAPE), (dict(max_pages=1 << 28), SHAPE), (dict(T=(1 << 20) + 1), SHAPE),
         (dict(n_pages=0), SHAPE), (dict(n_pages=1 << 30), SHAPE)]


@pytest.mark.parametrize("case", range(len(CACHE)))
def test_cache_description_is_checked_by_every_call(L, case):
    kw, want = CACHE[case]
    assert append(L, kw) == want
    assert attend(L, kw) == want
    assert attend(L, kw, prefix=(FAKE, FAKE, 1)) == want


def test_append_refusals(L):
    assert append(L, q=None) == INVALID
    assert append(L, k=FAKE + 8) == INVALID
    assert append(L, v=None) == INVALID
    assert append(L, qo=None) == INVALID
    assert append(L, qo=FAKE, qos=512) == INVALID          # in place needs one stride
    assert append(L, qs=252) == SHAPE                      # not a multiple of 8
    assert append(L, qs=248) == SHAPE                      # rows overlap
    assert append(L, ks=64) == SHAPE
    assert append(L, hq=3) == SHAPE                        # not a multiple of the key heads
    assert append(L, hq=-2) == SHAPE
    assert append(L, rot=24) == SHAPE
    assert append(L, rot=80) == SHAPE
    assert append(L, cs=None) == INVALID
    assert append(L, cs=FAKE + 4) == INVALID
    assert append(L, n_pos=0) == INVALID
    assert append(L, axes=0) == SHAPE
    assert append(L, axes=5, pos=FAKE, pairs=[8, 8, 8, 4, 4]) == SHAPE
    assert append(L, axes=3, pairs=[8, 12, 12]) == INVALID            # several axes need positions
    assert append(L, axes=3, pos=FAKE) == INVALID                     # and their pairs
    assert append(L, axes=3, pos=FAKE, pairs=[8, 12, 11]) == SHAPE
    assert append(L, axes=3, pos=FAKE, pairs=[40, -4, -4]) in (INVALID, SHAPE)
    assert append(L, pairs=[31]) == SHAPE
    assert append(L, pos=FAKE + 1) == INVALID
    assert append(L, ws=None) == WORKSPACE
    assert append(L, wsb=8) == WORKSPACE
    assert append(L, dict(T=0)) == 0                                  # an empty batch launches nothing


def test_attention_refusals(L):
    for prefix in (None, (FAKE, FAKE, 2)):
        assert attend(L, prefix=prefix, q=None) == INVALID
        assert attend(L, prefix=prefix, q=FAKE + 8) == INVALID
        assert attend(L, prefix=prefix, out=None) == INVALID
        assert attend(L, prefix=prefix, out=FAKE) == INVALID          # out is q
        assert attend(L, prefix=prefix, hq=0) == SHAPE
        assert attend(L, prefix=prefix, hq=5) == SHAPE
        assert attend(L, prefix=prefix, qs=260) == SHAPE
        assert attend(L, prefix=prefix, os=64) == SHAPE
        for scale in (0.0, -1.0, float("nan"), float("inf")):
            assert attend(L, prefix=prefix, scale=scale) == INVALID
        assert attend(L, prefix=prefix, ws=None) == WORKSPACE
        assert attend(L, prefix=prefix, ws=WS + 8) == WORKSPACE
        need = L.lora_attn_workspace_bytes(ctypes.byref(kv(L)), 4, 2 if prefix else 0)
        assert need >= 16 and attend(L, prefix=prefix, wsb=need - 1) == WORKSPACE
        assert attend(L, dict(T=0), prefix=prefix) == 0
    assert attend(L, window=-1) == INVALID
    assert attend(L, sink=-1) == INVALID
    assert attend(L, prefix=(None, FAKE, 2)) == INVALID
    assert attend(L, prefix=(FAKE, FAKE + 2, 2)) == INVALID
    assert attend(L, prefix=(FAKE, FAKE, 0)) == SHAPE
    assert attend(L, prefix=(FAKE, FAKE, 4)) == SHAPE                 # more groups than sequences


def test_workspace_of_bad_arguments_is_the_error_word(L):
    assert L.lora_attn_workspace_bytes(None, 4, 0) == 16
    assert L.lora_attn_workspace_bytes(ctypes.byref(kv(L, head_dim=80)), 4, 0) == 16
    assert L.lora_attn_workspace_bytes(ctypes.byref(kv(L)), 5, 0) == 16
    assert L.lora_attn_workspace_bytes(ctypes.byref(kv(L)), 4, 9) == 16


def test_binding_refuses_wrong_tensors(L):
    torch = pytest.importorskip("torch")
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    tab, off, ln = (torch.zeros(n, dtype=torch.int32) for n in ((2, 4), (3,), (2,)))
    with pytest.raises(TypeError):
        L.PagedKV(k.float(), k, tab, off, ln, 2)
    with pytest.raises(TypeError):
        L.PagedKV(k, k, tab.long(), off, ln, 2)
    with pytest.raises(ValueError):
        L.PagedKV(k, k, tab, off[:2], ln, 2)
    with pytest.raises(ValueError):
        L.PagedKV(k, k, tab, off, ln, 2)            # not on a CUDA device


def test_rope_table_and_reference(L):
    pytest.importorskip("torch")
    from oracle import attn_ref as R
    cs = L.rope_table(50, 16, base=100.0, device="cpu").numpy()
    assert cs.shape == (50, 16)
    ang = 37 * 100.0 ** (-2.0 * 3 / 16)
    assert abs(cs[37, 3] - np.cos(ang)) < 1e-6 and abs(cs[37, 11] - np.sin(ang)) < 1e-6
    # a rotation keeps lengths, and scores depend on the distance of positions alone
    rng = np.random.default_rng(0)
    a, b = rng.normal(size=(2, 16))
    r = [R.rotate(x, cs, [p] * 8, True) for x, p in ((a, 30), (b, 21), (a, 19), (b, 10))]
    assert abs(np.linalg.norm(r[0]) - np.linalg.norm(a)) < 1e-6
    assert abs(r[0] @ r[1] - r[2] @ r[3]) < 1e-5
