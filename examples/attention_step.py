"""One attention layer of a multi-adapter server, end to end on the library's operators.

Each adapter has a system prompt.  Its keys and values depend on the adapter, so they are
computed once per adapter (a prompt through the LoRA q/k/v projection, kv_append and
attn_paged) and their pages are shared by the adapter's requests.  Then all requests decode
together, one token each and step: batch_plan, which moves the lengths on and takes new pages where
a request has filled its last, the LoRA q/k/v projection, kv_append with the rotation,
attn_prefix, which reads each shared prompt once, and the LoRA output projection.  The step is
captured into a CUDA graph once; between replays only the new tokens change.

    python examples/attention_step.py [--requests 64] [--prompt 2000] [--steps 16] [--bits 8]

--bits 8 holds the cache in 8 bits.  The last step's result is compared with the same layer in
64-bit PyTorch arithmetic, with keys and values rounded as the cache stores them.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from lora_serving_device_gb300 import lora as L  # noqa: E402

PAGE = 32


class Layer:
    """q/k/v and o projections with their adapter pools, and the cache."""

    def __init__(self, d, heads, kv_heads, head_dim, adapters, rank, n_pages, gen, bits):
        def normal(*shape, scale):
            return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(torch.bfloat16)

        width = (heads + 2 * kv_heads) * head_dim
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.w_qkv, self.w_o = normal(d, width, scale=d ** -0.5), normal(heads * head_dim, d, scale=0.02)
        self.a_qkv, self.b_qkv = normal(adapters, d, rank, scale=d ** -0.5), normal(adapters, rank, width, scale=0.1)
        self.a_o, self.b_o = (normal(adapters, heads * head_dim, rank, scale=0.02),
                              normal(adapters, rank, d, scale=0.1))
        self.scale = torch.ones(adapters, device="cuda")
        self.bits = bits
        if bits == 8:
            self.cache = L.PagedKV8bit.empty_cache(n_pages, kv_heads, PAGE, head_dim)
            self.paged, self.append = L.PagedKV8bit, L.kv_append_8bit_t
            self.attend, self.attend_prefix = L.attn_paged_8bit_t, L.attn_prefix_8bit_t
        else:
            self.cache = [torch.zeros(n_pages, kv_heads, PAGE, head_dim, dtype=torch.bfloat16, device="cuda")
                          for _ in range(2)]
            self.paged, self.append = L.PagedKV, L.kv_append_t
            self.attend, self.attend_prefix = L.attn_paged_t, L.attn_prefix_t

    def project_qkv(self, x, ids, ws):
        y = L.linear_fused_t(x, self.w_qkv, self.a_qkv, self.b_qkv, ids, self.scale, ws)
        T, n, m, d = x.shape[0], self.heads, self.kv_heads, self.head_dim
        return (y[:, :n * d].view(T, n, d), y[:, n * d:(n + m) * d].view(T, m, d),
                y[:, (n + m) * d:].view(T, m, d))

    def project_out(self, o, ids, ws):
        return L.linear_fused_t(o.flatten(1), self.w_o, self.a_o, self.b_o, ids, self.scale, ws)


def workspaces(layer, T):
    d, width = layer.w_qkv.shape
    _, rank = layer.a_qkv.shape[1:]
    n = layer.a_qkv.shape[0]
    return (L.workspace(L.OP_LINEAR_FUSED, T, d, width, rank, n),
            L.workspace(L.OP_LINEAR_FUSED, T, layer.w_o.shape[0], d, rank, n))


def stored(x, bits):
    """x [tokens, heads, head_dim] as the cache holds it."""
    if bits == 16:
        return x.bfloat16().double()
    n = len(x)
    x = torch.cat([x, x.new_zeros(-n % 16, *x.shape[1:])]).view(-1, 16, *x.shape[1:])
    scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax((1, 3), keepdim=True).clamp(min=2.0 ** -100) / 448)))
    return ((x / scale).float().to(torch.float8_e4m3fn).double() * scale).flatten(0, 1)[:n]


def reference(layer, xs, ids, cos_sin):
    """The layer's output for the last token of each request, in 64 bits but for the bf16
    roundings of what the layer stores (q/k/v, the cache, the attention's result)."""
    def linear(x, w, a, b, i):
        y = x.double() @ w.double()
        return y + (x.double() @ a[i].double()) @ b[i].double() * layer.scale[i].double()

    def rotate(x, pos):
        half = cos_sin.shape[1] // 2
        c, s = cos_sin[pos, :half].double()[:, None], cos_sin[pos, half:].double()[:, None]
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    n, m, d = layer.heads, layer.kv_heads, layer.head_dim
    out = []
    for x, i in zip(xs, ids):
        qkv = linear(x, layer.w_qkv, layer.a_qkv, layer.b_qkv, i).bfloat16().double()
        pos = torch.arange(len(x), device="cuda")
        q = rotate(qkv[-1:, :n * d].view(1, n, d), pos[-1:]).bfloat16().double()
        k = stored(rotate(qkv[:, n * d:(n + m) * d].view(-1, m, d), pos), layer.bits).repeat_interleave(n // m, 1)
        v = stored(qkv[:, (n + m) * d:].view(-1, m, d), layer.bits).repeat_interleave(n // m, 1)
        w = (torch.einsum("thd,nhd->htn", q, k) * d ** -0.5).softmax(-1)
        o = torch.einsum("htn,nhd->thd", w, v).bfloat16()
        out.append(linear(o.flatten(1), layer.w_o, layer.a_o, layer.b_o, i))
    return torch.cat(out)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--adapters", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=2000, help="tokens of an adapter's system prompt")
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--d", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--bits", type=int, default=16, choices=(8, 16), help="of a value in the cache")
    a = ap.parse_args(argv)
    gen = torch.Generator("cuda").manual_seed(0)
    n, g = a.requests, a.adapters
    prompts = [a.prompt - 3 * i for i in range(g)]
    prompt_pages = [-(-p // PAGE) for p in prompts]
    own_pages = -(-(a.steps + PAGE) // PAGE) + 1
    layer = Layer(a.d, a.heads, a.kv_heads, a.head_dim, g, 16, sum(prompt_pages) + n * own_pages, gen, a.bits)
    cos_sin = L.rope_table(a.prompt + a.steps + 1, a.head_dim)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    # the system prompts, one call for all adapters: sequences of one batch
    starts = [sum(prompts[:i]) for i in range(g + 1)]
    pages = torch.arange(sum(prompt_pages), dtype=torch.int32, device="cuda").split(prompt_pages)
    table = torch.full((g, max(prompt_pages)), -1, dtype=torch.int32, device="cuda")
    for i in range(g):
        table[i, :prompt_pages[i]] = pages[i]
    kv = layer.paged(*layer.cache, table, i32(starts), i32(prompts), starts[-1], max_q_len=max(prompts))
    x = torch.randn(starts[-1], a.d, device="cuda", generator=gen).bfloat16()
    ids = torch.repeat_interleave(torch.arange(g, device="cuda"), torch.tensor(prompts, device="cuda")).int()
    ws_qkv, ws_o = workspaces(layer, starts[-1])
    ws = L.attn_workspace(kv, a.heads)
    q, k, v = layer.project_qkv(x, ids, ws_qkv)
    q = layer.append(kv, q, k, v, cos_sin, ws)
    layer.project_out(layer.attend(kv, q, ws), ids, ws_o)
    assert L.get_error_t(ws) == 0 and L.get_error_t(ws_qkv) == 0
    history = [[x[starts[i]:starts[i + 1]]] for i in range(g)]

    # the requests: adapter i's pages first, its last (partly filled) one as an own copy; all
    # other pages are free, and batch_plan takes them as they are needed
    owner = [i * g // n for i in range(n)]
    table = torch.full((n, max(prompt_pages) + own_pages), -1, dtype=torch.int32, device="cuda")
    free = list(range(sum(prompt_pages), sum(prompt_pages) + n * own_pages))
    for r in range(n):
        i = owner[r]
        full = prompts[i] // PAGE
        table[r, :full] = pages[i][:full]
        if prompts[i] % PAGE:
            own = free.pop()
            table[r, full] = own
            for c in layer.cache:
                c[own] = c[pages[i][full].item()]
    n_free, n_new = i32([len(free)]), i32([0] * n)
    free = i32(free + [-1] * (n * own_pages - len(free)))
    kv_len, n_shared = i32([prompts[i] for i in owner]), i32([prompts[i] // PAGE for i in owner])
    plan = L.BatchPlan.empty(n, n)._replace(kv_len=kv_len, n_free=n_free, slots=None, pos=None)
    kv = layer.paged(*layer.cache, table, plan.q_off, kv_len, n, max_q_len=1)
    n_pages = layer.cache[0].shape[0]
    ws_plan = L.batch_plan_workspace(n)
    group_off = i32([next((r for r in range(n) if owner[r] >= i), n) for i in range(g)] + [n])
    prefix_len = i32(prompts)
    ids = i32(owner)
    ws_qkv, ws_o = workspaces(layer, n)
    ws = L.attn_workspace(kv, a.heads, n_groups=g)
    x = torch.zeros(n, a.d, dtype=torch.bfloat16, device="cuda")

    def step():
        L.batch_plan_t(table, kv_len, n_new, free, n_free, PAGE, n_pages, ws_plan, n_shared=n_shared, T=n, out=plan)
        q, k, v = layer.project_qkv(x, ids, ws_qkv)
        q = layer.append(kv, q, k, v, cos_sin, ws)
        return layer.project_out(layer.attend_prefix(kv, q, group_off, prefix_len, ws), ids, ws_o)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                # the first run of each kernel, without new tokens
        n_new.fill_(1)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = step()
    torch.cuda.synchronize()
    tokens = torch.randn(a.steps, n, a.d, device="cuda", generator=gen).bfloat16()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for t in range(a.steps):
        x.copy_(tokens[t])
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    assert all(L.get_error_t(w) == 0 for w in (ws, ws_qkv, ws_o, ws_plan))
    ms = begin.elapsed_time(end) / a.steps
    rows = list(range(0, n, max(1, n // 8)))
    xs = [torch.cat(history[owner[r]] + [tokens[:, r]]) for r in rows]
    ref = reference(layer, xs, [owner[r] for r in rows], cos_sin)
    got = y[rows].double()
    rel = float((got - ref).norm() / ref.norm())
    print(f"{n} requests, {g} adapters with prompts of {prompts}, {a.bits} bits: {ms * 1e3:.1f} us a step, "
          f"error against 64 bits {rel:.1e}")
    assert rel < (3e-2 if a.bits == 8 else 1e-2), rel
    return rel


if __name__ == "__main__":
    main()
