"""The paged cache in plain numpy: pools filled row by row from the definition, rotation and attention in 64 bits, and the
error bounds of the kernels."""
import numpy as np

import alibi_inputs as gen


def bf16(x):
    """The values rounded to bf16, as float64, and the same as a CUDA tensor."""
    import torch
    t = gen.make_tensor(np.asarray(x, dtype=np.float32), np.shape(x), "bf16")
    return t.f32.astype(np.float64), torch.from_numpy(t.bf16.view(np.int16)).view(torch.bfloat16).cuda()


def ints(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pools(P, H, S, d, layout):
    """k_pages, v_pages [P, H, S, d] in one of the layouts that a server may have, every element NaN."""
    import torch
    def new(*shape):
        return torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    if layout == "heads":          # [P, H, S, d]
        return new(P, H, S, d), new(P, H, S, d)
    if layout == "slots":          # [P, S, H, d]
        return new(P, S, H, d).transpose(1, 2), new(P, S, H, d).transpose(1, 2)
    if layout == "together":       # [P, 2, S, H, d]
        x = new(P, 2, S, H, d)
        return x[:, 0].transpose(1, 2), x[:, 1].transpose(1, 2)
    if layout == "padded":         # rows of d + 8 elements, values from the ninth on
        return new(P, H, S, d + 8)[..., :d], new(P, H, S, d + 8)[..., 8:]
    raise ValueError(layout)


LAYOUTS = ["heads", "slots", "together", "padded"]


def paged(k, v, lens, S, seed=0, layout="heads", spare=3, M=None, unused=-1):
    """Pools that hold rows 0 .. lens[b] - 1 of k, v [B, H, N, d] (exact bf16 values) in shuffled pages, everything else NaN,
    and the table, whose entries past a sequence's pages are `unused`."""
    import torch
    B, H, N, d = k.shape
    need = [-(-n // S) for n in lens]
    P = sum(need) + spare
    order = np.random.default_rng(seed).permutation(P)
    M = max(1, *need) if M is None else M
    table = np.full((B, M), unused, dtype=np.int32)
    kp, vp = pools(P, H, S, d, layout)
    (_, kd), (_, vd) = bf16(k), bf16(v)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        for i in range(need[b]):
            m = min(S, n - i * S)
            kp[int(table[b, i]), :, :m] = kd[b, :, i * S:i * S + m]
            vp[int(table[b, i]), :, :m] = vd[b, :, i * S:i * S + m]
    torch.cuda.synchronize()
    return kp, vp, ints(table)


def rotated(x, n, R, base=10000.0, freqs=None, interleaved=False):
    """x [..., T, d] rotated by positions n [T], in 64 bits, and the bound of the kernel before the store: the angle is off
    by less than 2^-22, cosine and sine by 2^-22 more each, and products and sum by 3 2^-24: 2^-20 (|x| + |y|) covers them."""
    f = np.array([base ** (-2.0 * i / R) for i in range(R // 2)]) if freqs is None else np.asarray(freqs, dtype=np.float64)
    angle = np.asarray(n, dtype=np.float64)[:, None] * f
    c, s = np.cos(angle), np.sin(angle)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    out, err = x.copy(), np.zeros_like(x)
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    err[..., a] = err[..., b] = 2.0 ** -20 * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return out, err


def attention(q, k, v, lens, counts, m, weight=2.0 ** -16, chain=64, column=False):
    """Attention of q [B, H, T, d] over k, v [B, Hkv, N, d] (float64), query t < counts[b] of sequence b at position
    lens[b] - counts[b] + t: out, lse and the kernel's error bounds; other queries are NaN.

    Bounds. Products of bf16 numbers are exact in fp32. A tensor-core step adds 16 of them to its accumulator, each
    aligned to the largest and cut, at most 17 cuts of 2^-24 of the sum of magnitudes: d / 16 steps make the logit off by
    17 d / 16 2^-24 sum |q_e k_e| / sqrt(d). The bias, its conversion to base 2 and the sum with the logit are off
    by less than 2^-21 (m (i - j) + |x|). So dx_j. A weight is off by dx_j, 2^-19 for the exponential, for references that
    move and for the merges, and `weight`, the rounding of p for the values' products (two bf16 numbers: 2^-16); the
    normaliser by the mean of dx_j + 2^-19. The values' products are summed in chains of at most n / chain + 8 steps, each
    17 2^-24 of the magnitudes.

    column: the kernel adds the part m c of the bias, c < 128 the key's place in its tile, to the product on the tensor core, one
    more step whose cuts are relative to sum |q_e k_e| / sqrt(d) + 128 m, and takes m (i - k_0) off with one rounding, of
    numbers up to m (i - j) + 128 m: dx_j grows by 17 2^-24 (sum |q_e k_e| / sqrt(d) + 128 m) + 2^-24 128 m. (Slopes above
    4 / log2(e) are taken whole.)"""
    B, H, T, d = q.shape
    G = H // k.shape[1]
    out, lse = np.full(q.shape, np.nan), np.full(q.shape[:-1], np.nan)
    e_out, e_lse = np.zeros(q.shape), np.zeros(q.shape[:-1])
    for b in range(B):
        n, c = int(lens[b]), int(counts[b])
        i = n - c + np.arange(c)
        dist = i[:, None] - np.arange(n)[None, :]
        for h in range(H):
            if n == 0:
                out[b, h, :c], lse[b, h, :c] = 0.0, -np.inf
                continue
            K, V, Q = k[b, h // G, :n], v[b, h // G, :n], q[b, h, :c]
            bias = m[h] * np.maximum(dist, 0)
            x = np.where(dist >= 0, Q @ K.T / np.sqrt(d) - bias, -np.inf)
            M = x.max(-1, keepdims=True)
            w = np.exp(x - np.where(np.isinf(M), 0.0, M))
            l = w.sum(-1, keepdims=True)
            W = w / np.where(l == 0, 1.0, l)
            out[b, h, :c] = W @ V
            with np.errstate(divide="ignore"):
                lse[b, h, :c] = (M + np.log(l))[:, 0]
            dx = 17 * d / 16 * 2.0 ** -24 * (np.abs(Q) @ np.abs(K).T) / np.sqrt(d) + \
                2.0 ** -21 * (bias + np.where(dist >= 0, np.abs(x), 0.0)) + 2.0 ** -19
            if column:
                dx += 17 * 2.0 ** -24 * (np.abs(Q) @ np.abs(K).T) / np.sqrt(d) + (18 * 2.0 ** -24 * 128 * m[h] if m[h] < 2.78 else 0.0)
            D = (W * dx).sum(-1, keepdims=True)
            steps = 17 * 2.0 ** -24 * (n / chain + 8)
            e_out[b, h, :c] = (W * (weight + steps + dx + D)) @ np.abs(V)
            e_lse[b, h, :c] = (D + 2.0 ** -20 * (1 + np.abs(np.where(l > 0, lse[b, h, :c, None], 0.0))))[:, 0]
    return out, lse, e_out, e_lse
