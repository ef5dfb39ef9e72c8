"""Plain fp64 CPU implementations of the calls that serve over a transferred
cache, written from their formulas (include/helm_kv.h, second part), and the
inputs their tests share.  Independent of the library."""
import math

import torch

FP8 = torch.float8_e4m3fn
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step of a rounding, relative


# ------------------------------------------------------------ rotary positions
def rope_frequencies(rot, theta, scaling="plain", factor=1.0, original=0.0, fast=32.0, slow=1.0, low=1.0, high=4.0):
    out = []
    if scaling == "ntk" and rot > 2:
        theta = theta * factor ** (rot / (rot - 2))
    for i in range(rot // 2):
        w = theta ** (-2.0 * i / rot)
        if scaling == "linear":
            w /= factor
        elif scaling == "yarn":
            corner = [rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(theta)) for n in (fast, slow)]
            lo, hi = max(0, math.floor(corner[0])), min(rot - 1, math.ceil(corner[1]))
            r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = w / factor * r + w * (1 - r)
        elif scaling == "banded":
            wave = 2 * math.pi / w
            if wave > original / low:
                w /= factor
            elif wave > original / high:
                s = (original / wave - low) / (high - low)
                w = (1 - s) * w / factor + s * w
        out.append(w)
    return torch.tensor(out, dtype=torch.float64)


def rope(x, pos, freq, layout, m=1.0, mode="forward"):
    """(result, what its rounding errors are proportional to), fp64; x [N, heads, D]."""
    y, size = x.double().clone(), x.double().abs()
    P = len(freq)
    angle = pos.double()[:, None] * freq
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    m = 1.0 / m if mode == "inverse" else m
    s = s if mode == "forward" else -s
    one, two = ((slice(0, P), slice(P, 2 * P)) if layout == "half" else (slice(0, 2 * P, 2), slice(1, 2 * P, 2)))
    a, b = y[..., one].clone(), y[..., two].clone()
    y[..., one], y[..., two] = m * (a * c - b * s), m * (a * s + b * c)
    size[..., one] = size[..., two] = m * (a.abs() + b.abs())
    return y, size


# ------------------------------------------------------------ the 8-bit cache
def scale_of(amax):
    """Smallest 2^e, -120 <= e <= 120, with amax <= 448 * 2^e."""
    e = -120
    while e < 120 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def encode(x):
    return x.clamp(-448, 448).float().to(FP8)


def finite_max(x):
    x = x.double().abs().flatten()
    x = x[torch.isfinite(x)]
    return float(x.max()) if x.numel() else 0.0


def store(x, pool, scale, cu, start, table, max_len):
    """One of K and V, in place: x [N, H, D], pool [nb, H, B, D] FP8, scale [nb, H]; returns the slots written."""
    B, nb, H = pool.shape[2], pool.shape[0], pool.shape[1]
    written = []
    for r in range(len(start)):
        t0, t1 = start[r], min(start[r] + cu[r + 1] - cu[r], max_len)
        for page in range(t0 // B, -(-t1 // B) if t1 > t0 else 0):
            if page >= table.shape[1] or not 0 <= table[r, page] < nb:
                continue
            blk, a, b = int(table[r, page]), max(t0, page * B), min(t1, (page + 1) * B)
            held = a - page * B
            for h in range(H):
                new = x[cu[r] + a - t0:cu[r] + b - t0, h].double()
                c = scale_of(finite_max(new))
                if held:
                    was = float(scale[blk, h])
                    c = max(c, was)
                    if c != was:
                        pool[blk, h, :held] = encode(pool[blk, h, :held].double() * (was / c))
                pool[blk, h, held:held + b - a] = encode(new / c)
                scale[blk, h] = c
            written.append((blk, held, held + b - a))
    return written


def context(pool, scale, table_row, n):
    """[H, n, D] fp64 and which of the n tokens are in blocks of the pool."""
    nb, H, B, D = pool.shape
    x = torch.zeros((H, n, D), dtype=torch.float64)
    there = torch.zeros(n, dtype=torch.bool)
    for page in range(-(-n // B)):
        blk = int(table_row[page])
        if 0 <= blk < nb:
            m = min(B, n - page * B)
            x[:, page * B:page * B + m] = pool[blk, :, :m].double() * scale[blk].double()[:, None, None]
            there[page * B:page * B + m] = True
    return x, there


def masked_scores(q, K, there, kv, n, scale, causal, window):
    """[H, n, G, tokens] and the size of the sums behind them."""
    H, D, L = K.shape[0], K.shape[2], K.shape[1]
    qg = q.double().reshape(n, H, -1, D).transpose(0, 1)            # [H, n, G, D]
    s = torch.einsum("hngd,hld->hngl", qg, K) * scale
    size = torch.einsum("hngd,hld->hngl", qg.abs(), K.abs()) * abs(scale)
    p = (kv - n + torch.arange(n))[:, None]
    j = torch.arange(L)
    ok = there[None].expand(n, L).clone()
    if causal:
        ok &= j <= p
        if window:
            ok &= j > p - window
    return s.masked_fill(~ok[None, :, None], -math.inf), size.masked_fill(~ok[None, :, None], 0.0)


def attend(q, cu, kv_len, table, k_pool, v_pool, k_scale, v_scale, max_len, scale, causal=True, window=0):
    """(out, lse, tol_out, tol_lse) fp64.  Tolerances from the rounding count:
    scores are fp32 sums of D exact products (relative to sum |q k|), p is
    rounded to fp16 once, the sums over L tokens are fp32, out is rounded to
    bf16."""
    N, Hq, D = q.shape
    H, B = k_pool.shape[1], k_pool.shape[2]
    out, lse = torch.zeros(N, Hq, D, dtype=torch.float64), torch.full((N, Hq), -math.inf, dtype=torch.float64)
    t_out, t_lse = torch.zeros_like(out), torch.zeros_like(lse)
    u = 2.0 ** -24
    for r in range(len(kv_len)):
        n, kv = cu[r + 1] - cu[r], int(kv_len[r])
        L = max(0, min(kv, max_len, table.shape[1] * B))
        if n == 0 or L == 0:
            continue
        K, there = context(k_pool, k_scale, table[r], L)
        V, _ = context(v_pool, v_scale, table[r], L)
        s, size = masked_scores(q[cu[r]:cu[r + 1]], K, there, kv, n, scale, causal, window)
        top = s.amax(-1, keepdim=True)
        some = top[..., 0] > -math.inf
        e = torch.exp(s - top.masked_fill(top == -math.inf, 0.0))
        l = e.sum(-1)
        p = e / l.clamp(min=1e-300)[..., None]
        o = torch.einsum("hngl,hld->hngd", p, V)
        A = torch.einsum("hngl,hld->hngd", p, V.abs())
        d = (D + 8) * u * size.amax(-1) + 4 * u * s.masked_fill(s == -math.inf, 0).abs().amax(-1)     # of a score
        tol = (2.0 ** -11 * (1 + 2.0 ** -6) + 2 * d[..., None] + (L + 64) * u) * A + 2.0 ** -8 * o.abs()
        ls = top[..., 0] + torch.log(l)
        tl = d + (L + 64) * u + 4 * u * ls.abs().masked_fill(~some, 0.0)
        rows = lambda x: x.transpose(0, 1).reshape(n, Hq, *x.shape[3:])    # noqa: E731
        out[cu[r]:cu[r + 1]], t_out[cu[r]:cu[r + 1]] = rows(o), rows(tol)
        lse[cu[r]:cu[r + 1]] = rows(ls.masked_fill(~some, -math.inf))
        t_lse[cu[r]:cu[r + 1]] = rows(tl)
    return out, lse, t_out, t_lse


def weigh(q, lse, cu, kv_len, table, k_pool, k_scale, weights, max_len, scale, causal=True, window=0):
    """(weights + what the queries add, tolerance) fp64."""
    w, tol = weights.double().clone(), torch.zeros_like(weights, dtype=torch.float64)
    nb, H, B, D = k_pool.shape
    u = 2.0 ** -24
    for r in range(len(kv_len)):
        n, kv = cu[r + 1] - cu[r], int(kv_len[r])
        L = max(0, min(kv, max_len, table.shape[1] * B))
        if n == 0 or L == 0:
            continue
        K, there = context(k_pool, k_scale, table[r], L)
        s, size = masked_scores(q[cu[r]:cu[r + 1]], K, there, kv, n, scale, causal, window)
        z = lse[cu[r]:cu[r + 1]].double().reshape(n, H, -1).transpose(0, 1)[..., None]
        p = torch.where(torch.isfinite(z), torch.exp(s - z), torch.zeros_like(s))
        off = p * ((D + 8) * u * size + 8 * u * (z.abs().nan_to_num(0, 0, 0) + 1) + (p.shape[1] * p.shape[2] + 8) * u)
        add, off = p.sum((1, 2)), off.sum((1, 2))
        for t in range(L):
            if there[t]:
                w[int(table[r, t // B]), :, t % B] += add[:, t]
                tol[int(table[r, t // B]), :, t % B] += off[:, t]
    return w, tol + 2 * u * w.abs()


def evict(weights, kv_len, src, dst, k_pool, v_pool, k_scale, v_scale, budget, recent, max_len):
    """In place (CPU tensors); returns (kept, new_len)."""
    nb, H, B, D = k_pool.shape
    R = len(kv_len)
    kept = torch.full((R, H, budget), -1, dtype=torch.int32)
    new_len = torch.zeros(R, dtype=torch.int32)
    was = [x.clone() for x in (weights, k_pool, v_pool, k_scale, v_scale)]
    for r in range(R):
        n = max(0, min(int(kv_len[r]), max_len, src.shape[1] * B))
        keep = min(n, budget)
        new_len[r] = keep
        slot = [(int(src[r, t // B]), t % B) for t in range(n)]
        for h in range(H):
            if n <= budget:
                at = list(range(n))
            else:
                def rank(t):
                    w = float(was[0][slot[t][0], h, slot[t][1]]) if 0 <= slot[t][0] < nb else math.nan
                    return (1, 0.0, t) if w != w else (0, -w, t)
                at = sorted(sorted(range(n - recent), key=rank)[:budget - recent] + list(range(n - recent, n)))
            kept[r, h, :keep] = torch.tensor(at, dtype=torch.int32)
            for page in range(-(-keep // B)):
                blk = int(dst[r, page])
                if not 0 <= blk < nb:
                    continue
                for pool, scale, old, olds in ((k_pool, k_scale, was[1], was[3]), (v_pool, v_scale, was[2], was[4])):
                    x = torch.zeros(B, D, dtype=torch.float64)
                    for j, t in enumerate(at[page * B:(page + 1) * B]):
                        b, o = slot[t]
                        if 0 <= b < nb:
                            x[j] = old[b, h, o].double() * float(olds[b, h])
                    c = scale_of(finite_max(x))
                    pool[blk, h], scale[blk, h] = encode(x / c), c
                weights[blk, h] = 0.0
                for j, t in enumerate(at[page * B:(page + 1) * B]):
                    b, o = slot[t]
                    if 0 <= b < nb:
                        weights[blk, h, j] = was[0][b, h, o]
    return kept, new_len


# ------------------------------------------------------------ inputs
def cache(gen, lens, B, H, D, spare=3, width=None):
    """dict of CPU tensors: a filled cache for requests of these lengths, unused slots holding NaN codes."""
    need = [-(-n // B) for n in lens]
    nb = sum(need) + spare
    order = torch.randperm(nb, generator=gen)
    table = torch.full((len(lens), width or max(1, max(need))), -1, dtype=torch.int32)
    pools = [torch.full((nb, H, B, D), 0x7F, dtype=torch.uint8) for _ in range(2)]
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n].to(torch.int32)
        at += n
        for page in range(n):
            m = min(B, lens[r] - page * B)
            for pool in pools:
                z = torch.randn((H, m, D), generator=gen) * 60
                pool[int(table[r, page]), :, :m] = encode(z).view(torch.uint8)
    e = [torch.randint(-8, -4, (nb, H), generator=gen).double() for _ in range(2)]
    return dict(table=table, k_pool=pools[0].view(FP8), v_pool=pools[1].view(FP8), k_scale=torch.exp2(e[0]).float(),
                v_scale=torch.exp2(e[1]).float())


def cumulative(n):
    return [sum(n[:r]) for r in range(len(n) + 1)]
