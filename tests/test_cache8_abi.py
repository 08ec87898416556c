"""Host-side validation of the 8-bit cache's entry points and the batch plan, and their CPU
reference (no GPU: nothing valid enough to launch is passed)."""
import ctypes

import numpy as np
import pytest

from oracle import cache8_ref as C
from tests.test_attn_abi import CACHE, FAKE, INVALID, SHAPE, WORKSPACE, WS, L, kv  # noqa: F401


def append(L, kv_kw=None, **kw):
    a = dict(ks8=FAKE, vs8=FAKE, q=FAKE, qs=256, k=FAKE, ks=128, v=FAKE, vs=128, hq=4, cs=FAKE, n_pos=100, rot=64,
             qo=FAKE + 4096, qos=256, ws=WS, wsb=16)
    a.update(kw)
    st = None if kv_kw == "null" else ctypes.byref(kv(L, **(kv_kw or {})))
    return L.lora_kv_append_8bit(st, a["ks8"], a["vs8"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["hq"],
                                 a["cs"], a["n_pos"], a["rot"], None, 1, None, 0, a["qo"], a["qos"], a["ws"],
                                 a["wsb"], None)


def attend(L, kv_kw=None, prefix=None, **kw):
    a = dict(ks8=FAKE, vs8=FAKE, q=FAKE, qs=256, hq=4, scale=0.125, window=0, sink=0, out=FAKE + 4096, os=256, ws=WS,
             wsb=1 << 40)
    a.update(kw)
    st = None if kv_kw == "null" else ctypes.byref(kv(L, **(kv_kw or {})))
    if prefix is None:
        return L.lora_attn_paged_8bit(st, a["ks8"], a["vs8"], a["q"], a["qs"], a["hq"], a["scale"], a["window"],
                                      a["sink"], a["out"], a["os"], a["ws"], a["wsb"], None)
    return L.lora_attn_prefix_8bit(st, a["ks8"], a["vs8"], prefix[0], prefix[1], prefix[2], a["q"], a["qs"], a["hq"],
                                   a["scale"], a["out"], a["os"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("case", range(len(CACHE)))
def test_cache_description_is_checked_by_every_call(L, case):
    kw, want = CACHE[case]
    assert append(L, kw) == want
    assert attend(L, kw) == want
    assert attend(L, kw, prefix=(FAKE, FAKE, 1)) == want


def test_scales_are_checked(L):
    for bad in (None, FAKE + 8):
        assert append(L, ks8=bad) == append(L, vs8=bad) == INVALID
        for prefix in (None, (FAKE, FAKE, 2)):
            assert attend(L, prefix=prefix, ks8=bad) == attend(L, prefix=prefix, vs8=bad) == INVALID


def test_other_refusals_are_those_of_the_wide_cache(L):
    assert append(L, q=None) == append(L, k=FAKE + 8) == append(L, qo=FAKE, qos=512) == INVALID
    assert append(L, qs=252) == append(L, hq=3) == append(L, rot=24) == SHAPE
    assert append(L, ws=None) == append(L, wsb=8) == WORKSPACE
    assert append(L, dict(T=0)) == 0
    for prefix in (None, (FAKE, FAKE, 2)):
        assert attend(L, prefix=prefix, q=None) == attend(L, prefix=prefix, out=FAKE) == INVALID
        assert attend(L, prefix=prefix, hq=5) == SHAPE
        assert attend(L, prefix=prefix, scale=0.0) == INVALID
        assert attend(L, prefix=prefix, ws=WS + 8) == WORKSPACE
        need = L.lora_attn_workspace_bytes(ctypes.byref(kv(L)), 4, 2 if prefix else 0)
        assert attend(L, prefix=prefix, wsb=need - 1) == WORKSPACE
        assert attend(L, dict(T=0), prefix=prefix) == 0
    assert attend(L, window=-1) == attend(L, sink=-1) == INVALID
    assert attend(L, prefix=(FAKE, FAKE, 0)) == attend(L, prefix=(FAKE, FAKE, 4)) == SHAPE


def plan(L, **kw):
    a = dict(cached=FAKE, new=FAKE, shared=None, n=5, T=7, page=16, max_pages=4, n_pages=9, free=FAKE, cap=9,
             n_free=FAKE, table=FAKE, q_off=FAKE, kv_len=FAKE, slots=FAKE, pos=FAKE, n_out=FAKE, ws=WS, wsb=1 << 20)
    a.update(kw)
    return L.lora_batch_plan(*(a[x] for x in ("cached", "new", "shared", "n", "T", "page", "max_pages", "n_pages", "free",
                                              "cap", "n_free", "table", "q_off", "kv_len", "slots", "pos", "n_out",
                                              "ws", "wsb")), None)


def test_plan_refusals(L):
    for name in ("cached", "new", "free", "n_free", "table", "q_off", "kv_len", "n_out"):
        assert plan(L, **{name: None}) == INVALID, name
        assert plan(L, **{name: FAKE + 2}) == INVALID, name
    assert plan(L, shared=FAKE + 1) == plan(L, pos=FAKE + 2) == plan(L, slots=FAKE + 4) == INVALID
    assert plan(L, n=-1) == plan(L, T=-1) == plan(L, n_pages=-1) == INVALID
    for kw in (dict(n=0), dict(n=65537), dict(T=(1 << 20) + 1), dict(page=0), dict(page=24), dict(page=512), dict(cap=0),
               dict(max_pages=0), dict(n_pages=0), dict(max_pages=1 << 28)):
        assert plan(L, **kw) == SHAPE, kw
    # positions and the rows after them stay in 32 bits
    most = (2 ** 31 - 1024 - (1 << 20)) // 16
    assert plan(L, T=1 << 20, max_pages=most + 1) == SHAPE
    assert plan(L, T=1 << 20, max_pages=most, ws=None) == WORKSPACE
    need = L.lora_batch_plan_workspace_bytes(5)
    assert plan(L, wsb=need - 1) == plan(L, ws=WS + 8) == WORKSPACE
    assert L.lora_batch_plan_workspace_bytes(0) == L.lora_batch_plan_workspace_bytes(65537) == 16


def test_binding_refuses_wrong_tensors(L):
    torch = pytest.importorskip("torch")
    k = torch.zeros(3, 2, 16, 64, dtype=torch.uint8)
    sc = torch.zeros(3, 2, 1, dtype=torch.uint8)
    tab, off, ln = (torch.zeros(n, dtype=torch.int32) for n in ((2, 4), (3,), (2,)))
    with pytest.raises(TypeError):
        L.PagedKV8bit(k.bfloat16(), k, sc, sc, tab, off, ln, 2)
    with pytest.raises(TypeError):
        L.PagedKV(k, k, tab, off, ln, 2)
    with pytest.raises(ValueError):
        L.PagedKV8bit(k, k, sc, sc, tab, off, ln, 2)          # not on a CUDA device
    wide = object.__new__(L.PagedKV)
    narrow = object.__new__(L.PagedKV8bit)
    for call in (L.kv_append_8bit_t, L.attn_paged_8bit_t, L.attn_prefix_8bit_t):
        with pytest.raises(TypeError, match="8 bits"):
            call(wide, *[None] * 5)
    for call in (L.kv_append_t, L.attn_paged_t, L.attn_prefix_t):
        with pytest.raises(TypeError, match="16 bits"):
            call(narrow, *[None] * 5)
    out = L.BatchPlan.empty(2, 5, device="cpu")
    free, n_free = torch.zeros(9, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    ws = torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        L.batch_plan_t(tab, ln, ln, free, n_free, 16, 9, ws, out=out)
    with pytest.raises(TypeError, match="n_new"):
        L.batch_plan_t(tab, ln, ln.long(), free, n_free, 16, 9, ws, out=out)
    with pytest.raises(TypeError, match="slots"):
        L.batch_plan_t(tab, ln, ln, free, n_free, 16, 9, ws, T=6, out=out)


def test_plan_is_made_on_the_stream_of_the_call(monkeypatch):
    import contextlib
    torch = pytest.importorskip("torch")
    from lora_serving_device_gb300 import lora as L
    now, streams = [None], []

    @contextlib.contextmanager
    def on(stream):
        before, now[0] = now[0], stream
        yield
        now[0] = before

    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: streams.append(now[0]) or empty(*a, **k))
    monkeypatch.setattr(torch.cuda, "stream", on)
    one = torch.zeros(1, dtype=torch.int32)
    for stream in (None, "side"):
        streams.clear()
        with pytest.raises(ValueError, match="CUDA"):
            L.batch_plan_t(torch.zeros(1, 3, dtype=torch.int32), one, one, one, one, 16, 9, one, T=4, stream=stream)
        assert streams and set(streams) == {stream}


def test_reference_codes():
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(C.VALUES, want, equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-12, 8, 4000), [0, -0.0, 448, -448, 2.0 ** -10]])
    x = x[np.abs(x) <= 448].astype(np.float32)
    ties = (C.VALUES[:126] + C.VALUES[1:127]) / 2
    x = np.concatenate([x, ties, -ties]).astype(np.float32)
    assert np.array_equal(C.encode(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert C.scale_byte(448.0) == 127 and C.scale_byte(449.0) == 128 and C.scale_byte(0.0) == 1
    assert C.scale_byte(224.0) == 126 and C.scale_byte(3.4e38) == 247


def test_reference_append_and_plan():
    rng = np.random.default_rng(1)
    codes, scale = np.zeros((2, 1, 32, 64), np.uint8), np.zeros((2, 1, 2), np.uint8)
    x = rng.normal(size=(40, 1, 64)) * np.linspace(1, 30, 40)[:, None, None]
    places = [(1, i) for i in range(32)] + [(0, i) for i in range(8)]
    whole = codes.copy(), scale.copy()
    C.append(*whole, x, places)
    for i in range(40):   # token by token: the same scales, and values within a step of each other
        C.append(codes, scale, x[i:i + 1], places[i:i + 1])
    assert np.array_equal(scale, whole[1])
    a, b = C.dequantize(codes, scale), C.dequantize(*whole)
    assert np.all(np.abs(a - b) <= 2.0 ** -9 * np.repeat(2.0 ** (scale - 127.0), 16, -1)[..., None])
    got = b[[p for p, _ in places], :, [r for _, r in places]]
    assert np.linalg.norm(got - x) < 0.04 * np.linalg.norm(x)
    table, free = np.full((3, 4), -1), np.array([5, 6, 7, 8, -1, -1, -1])
    table[1, :3] = 1, 2, 3
    out = C.plan(table, [0, 20, 8], [9, -1, 1], [0, 1, 0], free, 4, 8, 9, 12)
    assert table.tolist() == [[3, 2, -1, -1], [1, 2, 3, -1], [-1, 8, -1, -1]]
    assert free.tolist() == [5, 6, 7, 8, 2, 3, -1] and out[4] == 3
    assert out[0].tolist() == [0, 9, 9, 10] and out[1].tolist() == [9, 0, 9]
    assert out[2].tolist() == [24 + i for i in range(8)] + [16, 64, -1, -1]
    assert out[3].tolist() == list(range(9)) + [8, -1, -1]
