"""A call of the binding that is given a stream makes its results there: memory that the
current stream has let go may still be in use on it.  Here with the library's calls
replaced, so that every helper that makes a tensor runs without a GPU."""
import contextlib

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def made(monkeypatch):
    """The binding with its C calls replaced, and the stream of each tensor made so far."""
    from lora_serving_device_gb300 import lora as L
    now, streams = [None], []

    @contextlib.contextmanager
    def on(stream):
        before, now[0] = now[0], stream
        yield
        now[0] = before

    for name in ("empty", "zeros"):
        make = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, _make=make, **k: streams.append(now[0]) or _make(*a, **k))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(L, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(L, "lora_decode_split", lambda *a: 2)
    for name in L.EXPORTS:
        if name not in ("lora_decode_split", "lora_workspace_bytes", "lora_status_string"):
            monkeypatch.setattr(L, name, lambda *a: 0, raising=False)
    return L, streams


T, D_IN, D_OUT, R, N = 6, 64, 128, 8, 3


def calls(L):
    bf = dict(dtype=torch.bfloat16)
    x, w0 = torch.ones(T, D_IN, **bf), torch.ones(D_IN, D_OUT, **bf)
    a, b = torch.ones(N, D_IN, R, **bf), torch.ones(N, R, D_OUT, **bf)
    ids, scale, ws = torch.ones(T).int(), torch.ones(N), torch.ones(64).byte()
    v, part = torch.ones(2, T, R), torch.ones(2, T, D_OUT)
    pool = L.RaggedPool([a[0], a[1]], [b[0], b[1]], device="cpu")
    base = L.Base4bit(torch.ones(D_OUT, D_IN // 2).byte(), torch.ones(1, D_OUT, **bf), torch.ones(16, **bf))
    segs = (ids, ids, ids, ids)
    return {
        "build_segments_t": (ids, N, ws),
        "bgmv_shrink_t": (x, a, ids, scale, 2, ws),
        "sgmv_shrink_t": (x, a, segs, scale, 2, ws),
        "linear_fused_t": (x, w0, a, b, ids, scale, ws),
        "base_gemm_expand_t": (x, w0, b, ids, v, ws),
        "bgmv_delta_t": (v, b, ids, ws),
        "bgmv_adapter_t": (x, a, b, ids, scale, ws),
        "base_gemm_splitk_t": (x, w0, ws),
        "bgmv_adapter_merge_t": (x, a, b, ids, scale, part, ws),
        "bgmv_adapter_ragged_t": (x, pool, ids, scale, ws),
        "linear_fused_ragged_t": (x, w0, pool, ids, scale, ws),
        "base_gemm_4bit_splitk_t": (x, base, ws),
        "linear_fused_4bit_t": (x, base, a, b, ids, scale, ws),
    }


def test_results_are_made_on_the_stream_of_the_call(made):
    L, streams = made
    every = calls(L)
    for name, args in list(every.items()) + [("quantize", (torch.ones(D_IN, D_OUT).bfloat16(), torch.ones(16)))]:
        call = L.Base4bit.quantize if name == "quantize" else getattr(L, name)
        for stream in (None, "side"):
            streams.clear()
            call(*args, stream=stream)
            assert streams and set(streams) == {stream}, name
