"""What serving over a transferred cache computes, case by case: rotary
positions, the 8-bit paged cache's store, attention over it, the accumulated
attention weight and the eviction by it.

``run`` computes each operator in its plain form (elementary torch operations
in fp32, angles in fp64) where ``own`` is false, and through the framework's
entry points where it is true.  ``exact`` is the definition in fp64.

The 8-bit cache of one layer: k_pool, v_pool e4m3 [n_blocks, H, B, D],
k_scale, v_scale fp32 [n_blocks, H] (a code stands for code * scale), weights
fp32 [n_blocks, H, B].  A request's token t lives in slot t % B of block
block_table[r, t // B].
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GOLD = 0.6180339887498949


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 32 requests: queries and keys of a fused projection, contexts stretched fourfold
        dict(name="rope_step", op="rope", tokens=32, heads=64, kv_heads=8, dim=128, rot=128, layout="half",
             scaling="yarn", type="bf16", inverse=False),
        # a pilot's cached fp32 keys [H, T, D] un-rotated before a transfer: interleaved pairs, half of the head
        dict(name="rope_cache", op="rope", tokens=32768, heads=0, kv_heads=8, dim=128, rot=64, layout="interleaved",
             scaling="banded", type="f32", inverse=True),
        # one new token for each of 64 requests, into pages that hold some already
        dict(name="store_step", op="store", requests=64, longest=4096, new=1, kv_heads=8, dim=128, block=16,
             type="bf16"),
        # a transferred cache [H, T, D] of four prompts, taken to 8 bits
        dict(name="store_prompt", op="store", requests=4, longest=16384, new=16384, kv_heads=8, dim=128, block=32,
             type="bf16"),
        # a single request's decode step, short context: latency
        dict(name="attend_one", op="attend", requests=1, longest=511, new=1, heads=16, kv_heads=8, dim=128, block=16,
             window=0),
        # the paged workload of 32 ragged requests, one token each
        dict(name="attend_batch", op="attend", requests=32, longest=16384, new=1, heads=64, kv_heads=8, dim=128,
             block=16, window=0),
        # one request over a 131,072-token cache, five query heads to a KV head
        dict(name="attend_long", op="attend", requests=1, longest=131072, new=1, heads=40, kv_heads=8, dim=128,
             block=64, window=0),
        # two requests' next turns over their transferred prefixes
        dict(name="attend_prompt", op="attend", requests=2, longest=8192, new=2048, heads=40, kv_heads=8, dim=128,
             block=32, window=0),
        # the weight that one decode step of 32 ragged requests gives each cached token
        dict(name="weigh_batch", op="weigh", requests=32, longest=16384, new=1, heads=64, kv_heads=8, dim=128,
             block=16, window=0),
        # the same of a prompt's queries
        dict(name="weigh_prompt", op="weigh", requests=1, longest=4096, new=1023, heads=16, kv_heads=8, dim=128,
             block=32, window=0),
        # a short request cut to 256 tokens
        dict(name="evict_one", op="evict", requests=1, longest=700, budget=256, recent=32, kv_heads=8, dim=128,
             block=16),
        # 16 long ragged requests cut to 4,096 tokens each
        dict(name="evict_batch", op="evict", requests=16, longest=32768, budget=4096, recent=512, kv_heads=8, dim=128,
             block=16),
    ]


def _size(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "store", "attend", "attend", "weigh", "evict"))
    kv_heads, dim, block = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 128)), rng.choice((16, 16, 32, 48, 64))
    if op == "rope":
        dim = rng.choice((64, 96, 128))
        rot = rng.choice((dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)))
        return dict(op=op, tokens=_size(rng, 1, 16384), heads=rng.choice((0, 1, 5, 16)), kv_heads=kv_heads, dim=dim,
                    rot=rot, layout=rng.choice(("half", "interleaved")),
                    scaling=rng.choice(("plain", "linear", "ntk", "yarn", "banded")), type=rng.choice(("bf16", "f32")),
                    inverse=rng.random() < 0.3)
    if op == "store":
        longest = _size(rng, 1, 16384)
        return dict(op=op, requests=_size(rng, 1, max(1, min(64, 65536 // longest))), longest=longest,
                    new=rng.choice((1, 1, _size(rng, 1, longest))), kv_heads=kv_heads, dim=dim, block=block,
                    type=rng.choice(("bf16", "bf16", "f32")))
    if op == "evict":
        longest = _size(rng, 16, 32768)
        budget = _size(rng, 8, max(8, min(4096, longest)))
        return dict(op=op, requests=_size(rng, 1, max(1, min(32, 262144 // longest))), longest=longest, budget=budget,
                    recent=rng.randint(0, budget // 2), kv_heads=kv_heads, dim=dim, block=block)
    if rng.random() < 0.6:      # decode
        longest = _size(rng, 1, 65536)
        case = dict(op=op, requests=_size(rng, 1, max(1, min(64, 262144 // longest))), longest=longest,
                    new=rng.choice((1, 1, 1, 4)), heads=kv_heads * rng.choice((1, 2, 5, 7, 8)))
    else:
        longest = _size(rng, 32, 6000 if op == "attend" else 2500)
        case = dict(op=op, requests=rng.randint(1, 2), longest=longest,
                    new=_size(rng, 2, min(longest, 1800 if op == "attend" else 900)),
                    heads=kv_heads * rng.choice((1, 2, 5) if op == "attend" else (1, 2)))
    return dict(case, kv_heads=kv_heads, dim=dim, block=block, window=rng.choice((0, 0, 0, 1 + longest // 3)))


def _lengths(longest, requests):
    """Ragged lengths spread over 1..longest; the first is the longest."""
    return [max(1, math.ceil(longest * (1.0 - (r * GOLD) % 1.0))) for r in range(requests)]


def _lens(case):
    """(kv_len, new) per request: cached tokens, the new ones among them, and how many those are."""
    kv = _lengths(case["longest"], case["requests"])
    new = [min(a, b) for a, b in zip(_lengths(case.get("new", 1), case["requests"]), kv)]
    return kv, new


def _pairs(kv, new, window):
    """Query-key pairs that a causal mask (and a window) leaves, over one head."""
    return sum(min(p + 1, window or p + 1) for n, m in zip(kv, new) for p in range(n - m, n))


def work(case):
    op, H, D = case["op"], case["kv_heads"], case["dim"]
    if op == "rope":
        n = case["tokens"] * (case["heads"] + H)
        e = 2 if case["type"] == "bf16" else 4
        return {"bytes": 2.0 * n * D * e + 4 * case["tokens"], "flops": 3.0 * n * case["rot"]}
    kv, new = _lens(case)
    if op == "store":
        n = sum(new) * H * D * 2
        e = 2 if case["type"] == "bf16" else 4
        return {"bytes": n * (e + 1.0), "flops": 2.0 * n}
    if op == "evict":
        keep = sum(min(n, case["budget"]) for n in kv) * H
        return {"bytes": 4.0 * sum(kv) * H + keep * (4 * D + 4 + 4), "flops": 1.0 * sum(kv) * H}
    Hq, pairs = case["heads"], _pairs(kv, new, case["window"])
    seen = sum(min(n, m + case["window"] - 1) if case["window"] else n for n, m in zip(kv, new))
    if op == "weigh":
        return {"bytes": seen * H * (D + 8.0) + sum(new) * Hq * (2 * D + 4.0), "flops": 2.0 * pairs * Hq * D}
    return {"bytes": seen * H * 2.0 * D + sum(new) * Hq * (4 * D + 4.0), "flops": 4.0 * pairs * Hq * D}


# ------------------------------------------------------------------ inputs
def _tables(gen, counts, block, spare, width=None):
    """(block tables [R, width], -1 where unused, blocks in all): physical blocks in random order."""
    need = [-(-n // block) for n in counts]
    blocks = sum(need) + spare
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(counts), width or max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return table, blocks


def _pool(gen, blocks, H, B, D):
    """Codes and scales of a filled cache: one spread per head, scales that vary from block to block."""
    z = torch.randn((blocks, H, B, D), generator=gen, device="cuda")
    z.mul_(torch.exp(0.4 * torch.randn((1, H, 1, D), generator=gen, device="cuda"))).mul_(60.0).clamp_(-448.0, 448.0)
    e = torch.randint(-7, -4, (blocks, H), generator=gen, device="cuda")
    return z.to(FP8), ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(n):
    return _i32([sum(n[:r]) for r in range(len(n) + 1)])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, H, D = case["op"], case["kv_heads"], case["dim"]
    s = dict(case)
    if own:     # the shapes and plans that a serving program keeps from step to step
        import cross_model_kv_helm_amd as hk
        s["hk"] = hk
    if op == "rope":
        N, Hq, t = case["tokens"], case["heads"], TYPES[case["type"]]
        if Hq:      # slices of one fused projection's output
            x = torch.randn((N, Hq + 2 * H, D), generator=gen, device="cuda").to(t)
            s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + H]
            s["out_q"] = torch.empty((N, Hq, D), dtype=t, device="cuda")
            s["out_k"] = torch.empty((N, H, D), dtype=t, device="cuda")
        else:       # a cache's keys, head by head
            s["q"] = s["out_q"] = None
            s["k"] = torch.randn((H, N, D), generator=gen, device="cuda").to(t).transpose(0, 1)
            s["out_k"] = torch.empty((H, N, D), dtype=t, device="cuda").transpose(0, 1)
        if N > 64:  # a prompt after a prefix
            s["pos"] = (torch.arange(N, device="cuda") + int(seed) % 4096).to(torch.int32)
        else:       # one token of each request, anywhere up to a long context's end
            s["pos"] = torch.randint(0, 131072, (N,), generator=gen, device="cuda").to(torch.int32)
        s["theta"], s["factor"], s["original"] = 1e6, 4.0, 32768
        if own:
            s["rope"] = hk.make_rope(D, s["theta"], rot_dim=case["rot"],
                                     layout={"half": hk.HELM_ROPE_HALF,
                                             "interleaved": hk.HELM_ROPE_INTERLEAVED}[case["layout"]],
                                     scaling={"plain": hk.HELM_ROPE_PLAIN, "linear": hk.HELM_ROPE_LINEAR,
                                              "ntk": hk.HELM_ROPE_NTK, "yarn": hk.HELM_ROPE_YARN,
                                              "banded": hk.HELM_ROPE_BANDED}[case["scaling"]],
                                     factor=s["factor"], original_len=s["original"])
        return s
    B = case["block"]
    kv, new = _lens(case)
    s["kv_len"], s["cu"], s["n_max"] = _i32(kv), _cu(new), max(new)
    if op == "evict":
        keep = [min(n, case["budget"]) for n in kv]
        need, room = [-(-n // B) for n in kv], [-(-n // B) for n in keep]
        both, blocks = _tables(gen, [(a + b) * B for a, b in zip(need, room)], B, 8)
        s["src"] = both[:, :max(need)].clone()
        s["dst"] = torch.full((len(kv), -(-case["budget"] // B)), -1, dtype=torch.int32, device="cuda")
        for r in range(len(kv)):
            s["src"][r, need[r]:] = -1
            s["dst"][r, :room[r]] = both[r, need[r]:need[r] + room[r]]
        # accumulated weights: a heavy tail, in steps, so that some are equal
        w = torch.rand((blocks, H, B), generator=gen, device="cuda")
        s["weights"] = (w.clamp_(min=1e-6).pow_(-0.5) * 256).round_() / 256
    else:
        s["table"], blocks = _tables(gen, kv, B, 8)
    s["k_pool"], s["k_scale"] = _pool(gen, blocks, H, B, D)
    s["v_pool"], s["v_scale"] = _pool(gen, blocks, H, B, D)
    if op == "store":
        N, t = sum(new), TYPES[case["type"]]
        spread = torch.exp(0.5 * torch.randn((2, H, 1, D), generator=gen, device="cuda"))
        x = (torch.randn((2, H, N, D), generator=gen, device="cuda") * spread).to(t)
        s["k"], s["v"] = x[0].transpose(0, 1), x[1].transpose(0, 1)     # the cache's layout [H, T, D]
        s["start"] = s["kv_len"] - _i32(new)
        if own:
            s["shape"] = hk.make_kv8_shape(s["k_pool"], s["table"], N, max_kv_len=case["longest"])
    elif op == "evict":
        if own:
            s["shape"] = hk.make_kv8_evict_shape(s["k_pool"], s["src"], s["dst"], case["budget"], case["recent"],
                                                 max_kv_len=case["longest"])
    else:
        N = sum(new)
        s["q"] = (1.5 * torch.randn((N, case["heads"], D), generator=gen, device="cuda")).to(torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(D)
        if op == "weigh":
            s["lse"] = _attend(s)["lse"]
            s["weights"] = torch.rand((blocks, H, B), generator=gen, device="cuda")
        if own:
            s["shape"] = hk.make_kv8_shape(s["k_pool"], s["table"], N, n_q_heads=case["heads"],
                                           max_kv_len=case["longest"], window=case["window"])
    return s


# ------------------------------------------------------------------ the plain forms
def _frequencies(s, device):
    """(angle per position of each pair, fp64; what cos and sin are multiplied by)."""
    rot, f, theta = s["rot"], s["factor"], s["theta"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    if s["scaling"] == "ntk":
        theta = theta * f ** (rot / (rot - 2)) if rot > 2 else theta
    w = theta ** (-2.0 * i / rot)
    if s["scaling"] == "linear":
        w = w / f
    if s["scaling"] == "yarn":      # slow pairs are divided by the factor, fast ones stay, a ramp between
        at = [rot * math.log(s["original"] / (b * 2 * math.pi)) / (2 * math.log(theta)) for b in (32.0, 1.0)]
        lo, hi = max(0.0, math.floor(at[0])), min(rot - 1.0, math.ceil(at[1]))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return w / f * ramp + w * (1 - ramp), 0.1 * math.log(f) + 1.0
    if s["scaling"] == "banded":    # by wavelength: over original/1 divided, under original/4 kept, blended between
        turns = s["original"] * w / (2 * math.pi)
        keep = ((turns - 1.0) / 3.0).clamp(0, 1)
        return w / f * (1 - keep) + w * keep, 1.0
    return w, 1.0


def _turn(x, cos, sin, rot, layout):
    if x is None:
        return None
    y = x.float()
    cos, sin = cos[:, None], sin[:, None]
    if layout == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    return torch.cat((turned, y[..., rot:]), -1).to(x.dtype)


def _rope(s):
    w, m = _frequencies(s, s["pos"].device)
    angle = s["pos"].double()[:, None] * w
    cos, sin = torch.cos(angle), torch.sin(angle)
    cos, sin = (cos / m, -sin / m) if s["inverse"] else (cos * m, sin * m)
    cos, sin = cos.float(), sin.float()
    out = {n: _turn(s[n], cos, sin, s["rot"], s["layout"]) for n in ("q", "k")}
    return {n: x for n, x in out.items() if x is not None}


def _power(amax):
    """The smallest power of two 2^e, -120 <= e <= 120, with amax <= 448 * 2^e."""
    bits = amax.view(torch.int32)
    e = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    return ((e.clamp(-120, 120) + 127) << 23).view(torch.float32)


def _codes(x):
    return x.clamp(-448.0, 448.0).to(FP8).view(torch.uint8)


def _owner(cu, n):
    """Request and place within it of each packed token."""
    tok = torch.arange(n, device=cu.device)
    r = torch.searchsorted(cu[1:].contiguous(), tok.to(torch.int32), right=True)
    return r, tok - cu[r].long()


def _store_one(x, pool, scale, blk, slot, first, old):
    """One of K and V: blk, slot of each token; `first` block of each request, holding `old` tokens already."""
    B = pool.shape[2]
    amax = torch.zeros_like(scale).index_reduce_(0, blk, x.float().abs().amax(-1), "amax")
    need = _power(amax)
    held = torch.zeros(scale.shape[0], dtype=torch.bool, device=x.device)
    held[first] = old > 0
    hit = torch.zeros_like(held)
    hit[blk] = True
    grown = torch.where(held[:, None], torch.maximum(scale, need), need)
    grown = torch.where(hit[:, None], grown, scale)
    bits = pool.view(torch.uint8)
    was = bits[first]
    ratio = (scale[first] / grown[first])[..., None, None]
    again = _codes(was.view(FP8).float() * ratio)
    keep = (torch.arange(B, device=x.device) < old[:, None])[:, None, :, None]
    bits[first] = torch.where(keep, again, was)
    scale.copy_(grown)
    bits[blk, :, slot] = _codes(x.float() / scale[blk][..., None])


def _store(s):
    B = s["block"]
    r, i = _owner(s["cu"], s["k"].shape[0])
    t = s["start"].long()[r] + i
    blk, slot = s["table"].long()[r, t // B], t % B
    page = s["start"].long() // B
    first = s["table"].long()[torch.arange(page.shape[0], device=t.device), page]
    old = s["start"].long() - page * B
    for_each = (("k", "k_pool", "k_scale"), ("v", "v_pool", "v_scale"))
    [_store_one(s[x], s[p], s[c], blk, slot, first, old) for x, p, c in for_each]
    return {n: s[n] for n in ("k_pool", "v_pool", "k_scale", "v_scale")}


def _dense(pool, scale, table):
    """[R, H, tokens, D] fp32: what the codes of each request stand for."""
    blk = table.long().clamp(min=0)
    x = pool.view(torch.uint8)[blk].view(FP8).float() * scale[blk][..., None, None]
    R, M, H, B, D = x.shape
    return x.transpose(1, 2).reshape(R, H, M * B, D)


def _scores(s):
    """Masked scores [R, H, n_max, group, tokens] (-inf where masked), each packed token's request and place."""
    cu, kv, R, H, D = s["cu"], s["kv_len"].long(), s["requests"], s["kv_heads"], s["dim"]
    n = cu[1:].long() - cu[:-1].long()
    i = torch.arange(s["n_max"], device=cu.device)
    tok = (cu[:-1].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][tok].float().reshape(R, s["n_max"], H, -1, D).transpose(1, 2)
    K = _dense(s["k_pool"], s["k_scale"], s["table"])
    G, L = q.shape[3], K.shape[2]
    x = torch.matmul(q.reshape(R, H, -1, D), K.transpose(-1, -2).contiguous()) * s["scale"]
    p = (kv - n)[:, None] + i
    j = torch.arange(L, device=cu.device)
    seen = (j < kv[:, None, None]) & (j <= p[..., None]) & (i < n[:, None])[..., None]
    if s["window"]:
        seen = seen & (j > p[..., None] - s["window"])
    return x.reshape(R, H, -1, G, L).masked_fill(~seen[:, None, :, None, :], -math.inf)


def _attend(s):
    x = _scores(s)
    R, H, n, G, L = x.shape
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    V = _dense(s["v_pool"], s["v_scale"], s["table"])
    o = torch.matmul(e.reshape(R, H, n * G, L), V).reshape(R, H, n, G, -1) / total.clamp(min=1e-37)
    lse = (top + torch.log(total))[..., 0]
    r, i = _owner(s["cu"], s["q"].shape[0])
    return {"out": o[r, :, i].reshape(s["q"].shape).to(s["q"].dtype), "lse": lse[r, :, i].reshape(s["q"].shape[:2])}


def _weigh(s):
    x = _scores(s)
    R, H, n, G, L = x.shape
    cu = s["cu"]
    tok = (cu[:-1].long()[:, None] + torch.arange(n, device=cu.device)).clamp(max=s["q"].shape[0] - 1)
    lse = s["lse"][tok].reshape(R, n, H, G).transpose(1, 2)[..., None]
    p = torch.where(x == -math.inf, 0.0, torch.exp(x - lse)).sum((2, 3))
    B = s["block"]
    part = p.reshape(R, H, L // B, B).transpose(1, 2).reshape(-1, H, B)
    blk = s["table"].long().reshape(-1)
    part = torch.where((blk >= 0)[:, None, None], part, 0.0)
    s["weights"].index_add_(0, blk.clamp(min=0), part)
    return {"weights": s["weights"]}


def _chosen(s):
    """kept positions [R, H, budget], ascending, -1 beyond; how many of each request."""
    kv, budget, dev = s["kv_len"].long(), s["budget"], s["kv_len"].device
    blk = s["src"].long().clamp(min=0)
    w = s["weights"][blk].transpose(1, 2).flatten(2)        # [R, H, tokens]
    j = torch.arange(w.shape[2], device=dev)
    n = kv[:, None, None]
    w = torch.where(j >= n - s["recent"], math.inf, w)
    w = torch.where(j >= n, -math.inf, w)
    first = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    keep = kv.clamp(max=budget)
    spare = torch.arange(first.shape[2], device=dev) >= keep[:, None, None]
    first = torch.sort(first.masked_fill(spare, 1 << 30), dim=-1).values
    kept = torch.full((*w.shape[:2], budget), -1, dtype=torch.int32, device=dev)
    kept[..., :first.shape[2]] = first.masked_fill(spare, -1).to(torch.int32)
    return kept, keep


def _evict_one(pool, scale, src, dst, kept, fill):
    B, D = pool.shape[2], pool.shape[3]
    x = _dense(pool, scale, src)
    R, H, K = kept.shape
    x = torch.gather(x, 2, kept.long().clamp(min=0)[..., None].expand(-1, -1, -1, D))
    x = torch.where((kept >= 0)[..., None], x, 0.0)
    x = torch.nn.functional.pad(x, (0, 0, 0, -K % B)).reshape(R, H, -1, B, D).transpose(1, 2)
    c = _power(x.abs().amax((-1, -2)))
    blk = dst.long().clamp(min=0)
    bits = pool.view(torch.uint8)
    return fill(bits, blk, _codes(x / c[..., None, None])), fill(scale, blk, c)


def _evict(s):
    B, src, dst = s["block"], s["src"], s["dst"]
    kept, keep = _chosen(s)
    live = torch.arange(dst.shape[1], device=dst.device) * B < keep[:, None]

    def fill(pool, blk, new):
        pool[blk[live]] = new[live]

    _evict_one(s["k_pool"], s["k_scale"], src, dst, kept, fill)
    _evict_one(s["v_pool"], s["v_scale"], src, dst, kept, fill)
    w = s["weights"][src.long().clamp(min=0)].transpose(1, 2).flatten(2)
    w = torch.where(kept >= 0, torch.gather(w, 2, kept.long().clamp(min=0)), 0.0)
    w = torch.nn.functional.pad(w, (0, -kept.shape[2] % B)).reshape(*kept.shape[:2], -1, B).transpose(1, 2)
    fill(s["weights"], dst.long().clamp(min=0), w)
    return {"kept": kept, "new_len": keep.to(torch.int32), **{n: s[n] for n in _CACHE}}


_CACHE = ("k_pool", "v_pool", "k_scale", "v_scale", "weights")


# ------------------------------------------------------------------ one pass
def run(s):
    if not own:
        return {"rope": _rope, "store": _store, "attend": _attend, "weigh": _weigh, "evict": _evict}[s["op"]](s)
    hk, op = s["hk"], s["op"]
    if op == "rope":
        q, k = hk.helm_rope(s["q"], s["k"], s["pos"], s["rope"],
                            hk.HELM_ROPE_INVERSE if s["inverse"] else hk.HELM_ROPE_FORWARD,
                            out_q=s["out_q"], out_k=s["out_k"])
        return {"k": k} if q is None else {"q": q, "k": k}
    if op == "store":
        hk.helm_kv8_store(s["k"], s["v"], s["cu"], s["start"], s["table"], s["k_pool"], s["v_pool"], s["k_scale"],
                          s["v_scale"], s["shape"])
        return {n: s[n] for n in ("k_pool", "v_pool", "k_scale", "v_scale")}
    if op == "attend":
        out, lse = hk.helm_kv8_attend(s["q"], s["cu"], s["kv_len"], s["table"], s["k_pool"], s["v_pool"],
                                      s["k_scale"], s["v_scale"], s["shape"])
        return {"out": out, "lse": lse}
    if op == "weigh":
        hk.helm_kv8_weigh(s["q"], s["lse"], s["cu"], s["kv_len"], s["table"], s["k_pool"], s["k_scale"],
                          s["weights"], s["shape"])
        return {"weights": s["weights"]}
    kept, new_len = hk.helm_kv8_evict(s["weights"], s["kv_len"], s["src"], s["dst"], s["k_pool"], s["v_pool"],
                                      s["k_scale"], s["v_scale"], s["shape"])
    return {"kept": kept, "new_len": new_len, **{n: s[n] for n in _CACHE}}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_rope(s):
    rot, f, theta, L0 = s["rot"], s["factor"], s["theta"], s["original"]
    w, m = [], 1.0
    if s["scaling"] == "ntk" and rot > 2:
        theta *= math.pow(f, rot / (rot - 2))
    for i in range(rot // 2):
        x = math.pow(theta, -2.0 * i / rot)
        if s["scaling"] == "linear":
            x /= f
        elif s["scaling"] == "yarn":
            lo = max(0.0, math.floor(rot * math.log(L0 / (64 * math.pi)) / (2 * math.log(theta))))
            hi = min(rot - 1.0, math.ceil(rot * math.log(L0 / (2 * math.pi)) / (2 * math.log(theta))))
            slow = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            x, m = x * (slow / f + 1.0 - slow), 0.1 * math.log(f) + 1.0
        elif s["scaling"] == "banded":
            wave = 2 * math.pi / x
            if wave > L0:
                x /= f
            elif wave > L0 / 4.0:
                keep = (L0 / wave - 1.0) / 3.0
                x *= (1.0 - keep) / f + keep
        w.append(x)
    angle = torch.outer(s["pos"].double(), torch.tensor(w, dtype=torch.float64, device="cuda"))
    unit = torch.polar(torch.full_like(angle, m), angle)
    unit = (1.0 / unit if s["inverse"] else unit)[:, None]
    out = {}
    for n in ("q", "k"):
        if s[n] is None:
            continue
        x = s[n].double().clone()
        one, two = ((slice(0, rot // 2), slice(rot // 2, rot)) if s["layout"] == "half"
                    else (slice(0, rot, 2), slice(1, rot, 2)))
        z = torch.complex(x[..., one], x[..., two]) * unit
        x[..., one], x[..., two] = z.real, z.imag
        out[n] = x
    return out


def _exact_power(amax):
    """Per element in fp64, by trying the exponents."""
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448.0)).clamp(-120, 120)
    e = torch.where(amax <= 448.0 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    return torch.exp2(e.clamp(-120, 120))


def _exact_store(s):
    B, out = s["block"], {}
    cu, start, table = s["cu"].tolist(), s["start"].tolist(), s["table"].tolist()
    for n in ("k", "v"):
        pool, scale = s[n + "_pool"].double(), s[n + "_scale"].double()
        for r in range(len(start)):
            t0, t1 = start[r], start[r] + cu[r + 1] - cu[r]
            x = s[n][cu[r]:cu[r + 1]].double().transpose(0, 1)          # [H, new, D]
            pages = torch.tensor(table[r][t0 // B:(t1 - 1) // B + 1], device="cuda")
            lead, H, D = t0 % B, x.shape[0], x.shape[2]
            y = torch.zeros((H, len(pages) * B, D), dtype=torch.float64, device="cuda")
            y[:, lead:lead + t1 - t0] = x
            y = y.reshape(H, len(pages), B, D).transpose(0, 1)
            c = _exact_power(y.abs().amax((-1, -2)))
            was = pool[pages].clone()
            if lead:
                c[0] = torch.maximum(c[0], scale[pages[0]])
                was[0] *= (scale[pages[0]] / c[0])[:, None, None]
            at = torch.arange(len(pages) * B, device="cuda").reshape(len(pages), 1, B, 1)
            fresh = (at >= lead) & (at < lead + t1 - t0)
            if not lead or bool((c[0] == scale[pages[0]]).all()):
                rest = pool[pages]
            else:
                rest = torch.where(at < lead, was, pool[pages])
            pool[pages], scale[pages] = torch.where(fresh, y / c[..., None, None], rest), c
        out[n + "_pool"], out[n + "_scale"] = pool, scale
    return out


def _exact_rows(s, r):
    """(K, V) of request r, [H, tokens, D]; its queries [H, new * group, D]; the scores, -inf where masked."""
    B, H, D, n = s["block"], s["kv_heads"], s["dim"], int(s["kv_len"][r])
    a, b = int(s["cu"][r]), int(s["cu"][r + 1])
    pages = s["table"][r, :-(-n // B)].long()
    K, V = ((s[x + "_pool"].view(torch.uint8)[pages].view(FP8).double() * s[x + "_scale"][pages].double()[..., None, None])
            .permute(1, 0, 2, 3).reshape(H, -1, D)[:, :n] for x in ("k", "v"))
    q = s["q"][a:b].double().reshape(b - a, H, -1, D).permute(1, 0, 2, 3)
    G = q.shape[2]
    x = torch.bmm(q.reshape(H, -1, D), K.transpose(1, 2).contiguous()) / math.sqrt(D)
    behind = (torch.arange(n - (b - a), n, device="cuda").repeat_interleave(G)[:, None]
              - torch.arange(n, device="cuda"))         # how far the key lies behind the query
    ok = (behind >= 0) & (behind < (s["window"] or 1 << 40))
    return a, b, pages, V, x.masked_fill(~ok, -math.inf)


def _exact_attend(s):
    N, Hq, D = s["q"].shape
    out = torch.empty((N, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((N, Hq), dtype=torch.float64, device="cuda")
    for r in range(s["requests"]):
        a, b, _, V, x = _exact_rows(s, r)
        H, G = s["kv_heads"], Hq // s["kv_heads"]
        lse[a:b] = torch.logsumexp(x, -1).reshape(H, b - a, G).transpose(0, 1).reshape(b - a, Hq)
        o = torch.bmm(torch.softmax(x, -1), V)
        out[a:b] = o.reshape(H, b - a, G, D).transpose(0, 1).reshape(b - a, Hq, D)
    return {"out": out, "lse": lse}


def _exact_weigh(s):
    w, B, H = s["weights"].double(), s["block"], s["kv_heads"]
    for r in range(s["requests"]):
        a, b, pages, _, x = _exact_rows(s, r)
        lse = s["lse"][a:b].double().reshape(b - a, H, -1).transpose(0, 1).reshape(H, -1, 1)
        p = torch.zeros((H, len(pages) * B), dtype=torch.float64, device="cuda")
        p[:, :x.shape[2]] = torch.exp(x - lse).sum(1)
        w[pages] += p.reshape(H, -1, B).transpose(0, 1)
    return {"weights": w}


def _exact_evict(s):
    B, D, H, budget = s["block"], s["dim"], s["kv_heads"], s["budget"]
    kept = torch.full((s["requests"], H, budget), -1, dtype=torch.int32, device="cuda")
    lens = s["kv_len"].clamp(max=budget)
    out = {n: s[n].double() for n in _CACHE}
    now = {n: x.clone() for n, x in out.items()}
    for r in range(s["requests"]):
        n, m = int(s["kv_len"][r]), int(lens[r])
        src, dst = s["src"][r, :-(-n // B)].long(), s["dst"][r, :-(-m // B)].long()
        w = now["weights"][src].transpose(0, 1).reshape(H, -1)[:, :n]
        order = w.clone()
        order[:, max(0, n - s["recent"]):] = math.inf
        at = order.sort(dim=-1, descending=True, stable=True).indices[:, :m].sort(-1).values
        kept[r, :, :m] = at.to(torch.int32)
        tail = len(dst) * B - m

        def lay(x):     # [H, m, ...] into whole blocks
            x = torch.cat((x, x.new_zeros((H, tail, *x.shape[2:]))), 1)
            return x.reshape(H, len(dst), B, *x.shape[2:]).transpose(0, 1)

        out["weights"][dst] = lay(w.gather(1, at))
        for x in ("k", "v"):
            y = (now[x + "_pool"][src] * now[x + "_scale"][src][..., None, None]).transpose(0, 1).reshape(H, -1, D)
            y = lay(y.gather(1, at[..., None].expand(-1, -1, D)))
            c = _exact_power(y.abs().amax((-1, -2)))
            out[x + "_pool"][dst], out[x + "_scale"][dst] = y / c[..., None, None], c
    return {"kept": kept, "new_len": lens, **out}


def exact(case, seed):
    return {"rope": _exact_rope, "store": _exact_store, "attend": _exact_attend, "weigh": _exact_weigh,
            "evict": _exact_evict}[case["op"]](prepare(case, seed))
