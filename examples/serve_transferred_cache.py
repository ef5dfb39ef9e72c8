"""Serving the target model from a transferred cache held in 8 bits.

A prompt's cache is mapped from the pilot's (helm_kv_transfer), stored layer by
layer in an 8-bit paged cache (helm_kv8_store), and decoded from: every step
rotates the new token's query and key (helm_rope), appends the key and value,
attends (helm_kv8_attend) and accumulates the weight each cached token received
(helm_kv8_weigh).  When the context outgrows its budget, the tokens that
received the least leave it (helm_kv8_evict).  Weights and caches are random;
the model around the attention is left out.

    python examples/serve_transferred_cache.py
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import cross_model_kv_helm_amd as hk  # noqa: E402


class Layer:
    """One target layer's 8-bit pages."""

    def __init__(self, blocks, H, B, D):
        self.k_pool, self.v_pool = (torch.zeros((blocks, H, B, D), dtype=torch.uint8, device="cuda")
                                    .view(torch.float8_e4m3fn) for _ in range(2))
        self.k_scale, self.v_scale = (torch.ones((blocks, H), device="cuda") for _ in range(2))
        self.weights = torch.zeros((blocks, H, B), device="cuda")

    @property
    def cache(self):
        return self.k_pool, self.v_pool, self.k_scale, self.v_scale


def main(prompt=600, steps=24, budget=256, recent=32, L_s=6, L_t=4, H=8, Hq=40, D=128, k=2, B=16, theta=1e6, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def rand(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)

    # the prompt's cache, mapped from the pilot's
    pos = torch.arange(prompt, dtype=torch.int32, device="cuda")
    sel = torch.stack([torch.randperm(L_s, generator=gen, device="cuda")[:k] for _ in range(L_t)]).to(torch.int32)
    src = [rand(L_s, H, prompt, D) for _ in range(2)]
    W = [rand(L_t, H, k * D, D, std=(k * D) ** -0.5) for _ in range(2)]
    b = torch.zeros((L_t, H, D), device="cuda")
    out = [torch.empty((L_t, H, prompt, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    shape = hk.make_shape(src[0], W[0], sel, theta, theta)
    hk.helm_kv_transfer(src[0], src[1], pos, pos, sel, W[0], b, W[1], b, out[0], out[1], shape)

    # into 8 bits: one request, pages of B tokens
    pages, kept_pages = -(-(prompt + steps) // B), -(-(budget + steps) // B)
    order = torch.randperm(pages + kept_pages, generator=gen, device="cuda").to(torch.int32)
    table, table2 = order[None, :pages].contiguous(), order[None, pages:].contiguous()
    layers = [Layer(pages + kept_pages, H, B, D) for _ in range(L_t)]
    one, none = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, prompt], [0]))
    fill = hk.make_kv8_shape(layers[0].k_pool, table, prompt)
    for i, layer in enumerate(layers):
        hk.helm_kv8_store(out[0][i].transpose(0, 1), out[1][i].transpose(0, 1), one, none, table, *layer.cache, fill)

    # decode
    rope = hk.make_rope(D, theta)
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    step_shape = hk.make_kv8_shape(layers[0].k_pool, table, 1, n_q_heads=Hq)
    full = [[x[0].float()] for x in out]        # layer 0 in fp32, to compare with
    worst = 1.0

    def step(n, position, table, shape):
        """One token through every layer; n tokens are in the cache before it."""
        at = torch.tensor([position], dtype=torch.int32, device="cuda")
        start = torch.tensor([n], dtype=torch.int32, device="cuda")
        result = None
        for i, layer in enumerate(layers):
            qkv = rand(1, Hq + 2 * H, D)
            q, key = hk.helm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + H], at, rope)
            hk.helm_kv8_store(key, qkv[:, Hq + H:], cu, start, table, *layer.cache, shape, weights=layer.weights)
            o, lse = hk.helm_kv8_attend(q, cu, start + 1, table, *layer.cache, shape)
            hk.helm_kv8_weigh(q, lse, cu, start + 1, table, layer.k_pool, layer.k_scale, layer.weights, shape)
            if i == 0:
                result = q, key, qkv[:, Hq + H:], o
        return result

    for s in range(steps):
        q, key, value, o = step(prompt + s, prompt + s, table, step_shape)
        full[0].append(key.float().transpose(0, 1))
        full[1].append(value.float().transpose(0, 1))
        K, V = (torch.cat(x, 1).repeat_interleave(Hq // H, 0) for x in full)
        p = torch.softmax((K @ q[0].float()[..., None])[..., 0] * D ** -0.5, -1)
        want = (p[:, None] @ V)[:, 0]
        worst = min(worst, float(torch.cosine_similarity(o[0].float(), want, dim=-1).min()))

    # the context is cut to its budget, and decoding goes on
    evict = hk.make_kv8_evict_shape(layers[0].k_pool, table, table2, budget, recent)
    length = torch.tensor([prompt + steps], dtype=torch.int32, device="cuda")
    for layer in layers:
        kept, new_len = hk.helm_kv8_evict(layer.weights, length, table, table2, *layer.cache, evict)
    after = hk.make_kv8_shape(layers[0].k_pool, table2, 1, n_q_heads=Hq)
    for s in range(steps):
        _, _, _, o = step(budget + s, prompt + steps + s, table2, after)
    torch.cuda.synchronize()
    print(f"{L_t} layers, {prompt} tokens mapped, stored in 8 bits and decoded for {steps} steps: attention's cosine to "
          f"fp32 over the unrounded cache at least {worst:.5f}")
    print(f"cut to {int(new_len[0])} tokens per KV head, decoded for {steps} steps more")
    return worst, int(new_len[0]), kept, o


if __name__ == "__main__":
    main()
