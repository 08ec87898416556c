"""Workspaces of the paged-cache calls that are not on the cache's device, or have gaps, reach no kernel,
whatever the cache; those that a call owns do."""
import pytest

from tests.test_gpu_attn import L  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 16])
def test_workspaces_elsewhere_are_refused(L, bits):
    import torch
    hq, hkv, d, page = 4, 2, 64, 16
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, off, lens = i32([[0, 1]]), i32([0, 1]), i32([1])
    if bits == 8:
        kv = L.PagedKV8bit(*L.PagedKV8bit.empty_cache(2, hkv, page, d), table, off, lens, 1)
        append, paged, prefix = L.kv_append_8bit_t, L.attn_paged_8bit_t, L.attn_prefix_8bit_t
    else:
        kc, vc = (torch.zeros(2, hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        kv = L.PagedKV(kc, vc, table, off, lens, 1)
        append, paged, prefix = L.kv_append_t, L.attn_paged_t, L.attn_prefix_t
    q, k = (torch.ones(1, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv))

    def calls(ws):
        return (lambda: append(kv, q, k, k, None, ws), lambda: paged(kv, q, ws),
                lambda: prefix(kv, q, i32([0, 1]), i32([0]), ws))

    size = L.attn_workspace(kv, hq, n_groups=1).numel()
    for ws in (torch.zeros(size, dtype=torch.uint8), torch.zeros(size).pin_memory(),
               torch.zeros(2 * size, dtype=torch.uint8, device="cuda")[::2]):
        for call in calls(ws):
            with pytest.raises(TypeError, match="ws"):
                call()
    ws = torch.zeros(size + 32, dtype=torch.uint8, device="cuda")[32:]
    for call in calls(ws):
        got = call()
        assert torch.equal(got, torch.ones_like(got))
    assert L.get_error_t(ws) == 0
