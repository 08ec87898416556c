"""The paged-cache helpers on the host, where a small call spends its time (an attention of one token
takes less on the GPU than its call): how many functions of the binding one runs through, and which
workspaces it refuses.  The library's calls get a null cache, so nothing is launched."""
import sys

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def L():
    from lora_serving_device_gb300 import build, lora
    build.build()
    lora.load()
    return lora


T, HQ, HKV, D = 2, 4, 2, 64


def cache(L, bits):
    """A cache's description without a GPU."""
    kv = object.__new__(L.PagedKV8bit if bits == 8 else L.PagedKV)
    kv.T, kv.n_kv_heads, kv.head_dim, kv._scale = T, HKV, D, D ** -0.5
    kv.ref, kv.scales, kv._device = None, (None, None), -1
    kv._bf16, kv._f32, kv._i32 = torch.bfloat16, torch.float32, torch.int32
    kv.new_like = torch.empty_like
    kv._current_stream, kv._current_device = int, (-1).__int__   # (not functions of Python)
    return kv


def calls(L, bits, ws, device=-1):
    kv = cache(L, bits)
    kv._device = device
    q, k = (torch.zeros(T, h, D, dtype=torch.bfloat16) for h in (HQ, HKV))
    off, lens = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    cs, pos = torch.zeros(10, D), torch.zeros(T, dtype=torch.int32)
    append, paged, prefix = ((L.kv_append_8bit_t, L.attn_paged_8bit_t, L.attn_prefix_8bit_t) if bits == 8 else
                             (L.kv_append_t, L.attn_paged_t, L.attn_prefix_t))
    return {"append": lambda: append(kv, q, k, k, cs, ws, pos=pos), "paged": lambda: paged(kv, q, ws),
            "prefix": lambda: prefix(kv, q, off, lens, ws)}


# as many as when there was no other cache: the call itself, the rows of q (and k, v), addresses, the
# result's memory, the library, the stream, the status and, here, its error
@pytest.mark.parametrize("what,most", [("append", 13), ("paged", 7), ("prefix", 7)])
def test_wide_calls_run_through_few_functions(L, what, most):
    f = calls(L, 16, torch.zeros(64, dtype=torch.uint8))[what]
    n = 0

    def count(frame, event, arg):
        nonlocal n
        n += event == "call" and frame.f_code.co_filename == L.__file__

    sys.setprofile(count)
    try:
        with pytest.raises(L.LoraError):
            f()
    finally:
        sys.setprofile(None)
    assert 2 <= n <= most


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("what", ["append", "paged", "prefix"])
def test_workspaces_elsewhere_or_with_gaps_are_refused(L, bits, what):
    """A workspace with gaps is said to have all bytes up to its last, of which it owns a part."""
    for ws, device in ((torch.zeros(1 << 21, dtype=torch.uint8)[::2], -1), (torch.zeros(1 << 20, dtype=torch.uint8), 0)):
        f = calls(L, bits, ws, device)[what]
        with pytest.raises(TypeError, match="ws"):
            f()
    with pytest.raises(L.LoraError):
        calls(L, bits, torch.zeros(1 << 20, dtype=torch.uint8))[what]()
