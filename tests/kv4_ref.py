"""The 4-bit KV cache in plain numpy, from its definition in include/alibi.h: quantisation in
64 bits, the block layout byte by byte, attention over the held values, and error bounds."""
import numpy as np


def padded(d: int) -> int:
    return max(d, 32)


def block_bytes(d: int) -> int:
    return 36 * padded(d)


def quantise(x: np.ndarray):
    """Codes [..., D] and scales [..., D / 32] (float64) of rows x [..., d] of exact bf16 values."""
    x = np.asarray(x, dtype=np.float64)
    D = padded(x.shape[-1])
    x = np.concatenate([x, np.zeros(x.shape[:-1] + (D - x.shape[-1],))], axis=-1)
    g = x.reshape(x.shape[:-1] + (D // 32, 32))
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    hi, lo = g.max(-1), g.min(-1)
    xm = np.where(hi >= -lo, hi, lo)
    s = np.where(np.abs(xm) < 2.0 ** -100, 0.0, -xm / 8)
    safe = np.where(s == 0, 1.0, s)
    u = np.where((s == 0)[..., None], 8, np.minimum(15, np.floor(g / safe[..., None] + 8.5)))
    return u.reshape(x.shape).astype(np.int64), np.where(bad, np.nan, s)


def dequantise(u: np.ndarray, s: np.ndarray) -> np.ndarray:
    return ((u.reshape(s.shape + (32,)) - 8) * s[..., None]).reshape(u.shape)


def held(x: np.ndarray) -> np.ndarray:
    """The values the cache holds for rows x [..., d] (float64)."""
    return dequantise(*quantise(x))[..., : np.shape(x)[-1]]


def key_byte(D, r, e):
    n, c, i = e // 32, e % 32 // 8, e % 8
    return r * D // 2 + c * D // 8 + 4 * n + i // 2


def value_byte(D, r, e):
    t, p, c, z = r // 16, r % 16 // 8, r % 8 // 2, r % 2
    n, g, i = e // 32, e % 32 // 4, e % 4
    return 16 * D + 8 * D * t + 512 * (n // 2) + (4 * g + c) * min(D // 4, 16) + 8 * (n % 2) + 4 * p + 2 * z + i // 2


def scale_byte(D, r, y, n):
    return 32 * D + r * D // 8 + 2 * (y * D // 32 + n)


def bf16_bits(s: np.ndarray) -> np.ndarray:
    """bf16 bits of float64 values that bf16 holds exactly (any NaN: 0x7fc0)."""
    w = np.asarray(s, dtype=np.float32).view(np.uint32)
    assert ((w & 0xFFFF) == 0)[~np.isnan(s)].all()
    return np.where(np.isnan(s), 0x7FC0, w >> 16).astype(np.uint16)


def place(cache: np.ndarray, b, h, row, uk, sk, uv, sv):
    """Write one token's codes [D] and scales [D / 32] into cache [B, H, blocks, bytes] (uint8)."""
    D = len(uk)
    blk, r = cache[b, h, row // 32], row % 32
    e = np.arange(0, D, 2)
    blk[key_byte(D, r, e)] = uk[0::2] | (uk[1::2] << 4)
    blk[value_byte(D, r, e)] = uv[0::2] | (uv[1::2] << 4)
    for y, s in ((0, sk), (1, sv)):
        bits = bf16_bits(s)
        for n in range(D // 32):
            o = scale_byte(D, r, y, n)
            blk[o], blk[o + 1] = int(bits[n]) & 255, int(bits[n]) >> 8


def write(cache: np.ndarray, k, v, pos, count):
    """alibi_kv4_write on a numpy cache: k, v [B, H, T, d] exact bf16 values."""
    B, H, _, _ = k.shape
    uk, sk = quantise(k)
    uv, sv = quantise(v)
    for b in range(B):
        for h in range(H):
            for t in range(count[b]):
                place(cache, b, h, pos[b] + t, uk[b, h, t], sk[b, h, t], uv[b, h, t], sv[b, h, t])


def pack(k, v, C=None) -> np.ndarray:
    """A cache that holds k, v [B, H, N, d] from row 0 on; every other byte is 0xFF (scales NaN)."""
    B, H, N, d = k.shape
    D, C = padded(d), -(-N // 32) * 32 if C is None else C
    cache = np.full((B, H, C // 32, 36 * D), 0xFF, dtype=np.uint8)
    r, e = np.arange(N), np.arange(0, D, 2)
    flat = cache.reshape(B, H, -1)
    base = (r // 32 * 36 * D)[:, None]
    for x, at, y in ((k, key_byte, 0), (v, value_byte, 1)):
        u, s = quantise(x)
        flat[:, :, base + at(D, r[:, None] % 32, e[None, :])] = u[..., 0::2] | (u[..., 1::2] << 4)
        o = base + scale_byte(D, r[:, None] % 32, y, np.arange(D // 32)[None, :])
        bits = bf16_bits(s)
        flat[:, :, o], flat[:, :, o + 1] = bits & 255, bits >> 8
    return cache


def _largest(x: np.ndarray) -> np.ndarray:
    """For each element of rows x [..., d]: 2 x the largest magnitude its group holds, i.e. 16 |s|."""
    d = x.shape[-1]
    a = np.abs(np.concatenate([x, np.zeros(x.shape[:-1] + (padded(d) - d,))], -1))
    a = a.reshape(x.shape[:-1] + (padded(d) // 32, 32))
    return 2 * np.repeat(a.max(-1), 32, axis=-1)[..., :d]


def decode(q, kh, vh, lens, m):
    """Attention of q [B, H, T, d] over held keys and values [B, Hkv, N, d] (float64): out, lse and
    their error bounds for the kernel.

    Bounds. The kernel computes x_j in fp32: the codes and q are exact in its products, the group sums
    of |q_e| 16 |s| are added and scaled with at most 40 roundings of 2^-24 (below 2^-18), the bias
    m (i - j) and its conversion to base 2 with 4: dx_j = 2^-18 sum_e |q_e| 16 |s_je| / sqrt(d) +
    2^-21 (m (i - j) + |x_j|) + 2^-34 max|q| sum_e 16 |s_je| / sqrt(d), the last term for elements of q
    more than 2^32 times smaller than the row's largest, whose 16-bit form is inexact. A weight's
    relative error is then dx_j plus the same of the normaliser, plus 2^-11 for the rounding of weight
    times scale to 16 bits, plus 2^-20 for the exponentials and the sums of codes (up to 16 |s| each, fp32):
      |out - ref| <= sum_j W_j ((2^-11 + dx_j + D) |v_j| + 2^-19 16 |s_j|) + 2^-31 16 N max_j,n W_j |s_jn|,
    D = sum_j W_j dx_j, and half a bf16 ulp. The last term: 16-bit weights are relative to the largest
    product of weight and scale, of any group, which stands at 2^6 or more, and steps of 2^-24 are off
    by 2^-25 at most. lse: D + 2^-20 (1 + |lse|)."""
    B, H, T, d = q.shape
    G = H // kh.shape[1]
    out, lse = np.zeros(q.shape), np.full(q.shape[:-1], -np.inf)
    e_out, e_lse = np.zeros(q.shape), np.zeros(q.shape[:-1])
    for b in range(B):
        for h in range(H):
            for t in range(T):
                i = int(lens[b]) - T + t
                if i < 0:
                    continue
                K, V = kh[b, h // G, : i + 1], vh[b, h // G, : i + 1]
                Q = q[b, h, t]
                dist = m[h] * (i - np.arange(i + 1))
                x = K @ Q / np.sqrt(d) - dist
                M = x.max()
                w = np.exp(x - M)
                W = w / w.sum()
                out[b, h, t], lse[b, h, t] = W @ V, M + np.log(w.sum())
                tk, tv = _largest(K), _largest(V)
                dx = 2.0 ** -18 * (tk @ np.abs(Q)) / np.sqrt(d) + 2.0 ** -21 * (dist + np.abs(x)) + \
                    2.0 ** -34 * np.abs(Q).max() * tk.sum(-1) / np.sqrt(d)
                D = W @ dx
                e_out[b, h, t] = (W * (2.0 ** -11 + dx + D)) @ np.abs(V) + 2.0 ** -19 * (W @ tv) + \
                    2.0 ** -31 * (W[:, None] * tv).max() * (i + 1)
                e_lse[b, h, t] = D + 2.0 ** -20 * (1 + np.abs(lse[b, h, t]))
    return out, lse, e_out, e_lse


def decode_by_group(q, kh, vh, lens, m):
    """As `decode`, with bounds that hold group by group of 32 elements, whatever the other groups of the
    same rows hold: elements of q are inexact below 2^-32 of the largest of THEIR group of 32, and the 16-bit
    products of weight and scale are relative to the largest product of THEIR value group. So the term
    2^-34 max|q| sum_e 16 |s_je| becomes its sum over the groups, each with its own maximum, and
    2^-31 N max_j,n becomes 2^-31 N max_j of the element's own group n. Weights are fp32 numbers: one
    below 2^-126 of the row's largest may count as zero."""
    B, H, T, d = q.shape
    G, D = H // kh.shape[1], padded(d)
    out, lse = np.zeros(q.shape), np.full(q.shape[:-1], -np.inf)
    e_out, e_lse = np.zeros(q.shape), np.zeros(q.shape[:-1])
    for b in range(B):
        for h in range(H):
            for t in range(T):
                i = int(lens[b]) - T + t
                if i < 0:
                    continue
                K, V = kh[b, h // G, : i + 1], vh[b, h // G, : i + 1]
                Q = q[b, h, t]
                dist = m[h] * (i - np.arange(i + 1))
                x = K @ Q / np.sqrt(d) - dist
                M = x.max()
                w = np.exp(x - M)
                W = w / w.sum()
                out[b, h, t], lse[b, h, t] = W @ V, M + np.log(w.sum())
                tk, tv = _largest(K), _largest(V)
                q_top = np.repeat(np.abs(np.pad(Q, (0, D - d))).reshape(-1, 32).max(-1), 32)[:d]
                dx = (2.0 ** -18 * (tk @ np.abs(Q)) + 2.0 ** -34 * (tk @ q_top)) / np.sqrt(d) + \
                    2.0 ** -21 * (dist + np.abs(x))
                E = W @ dx
                e_out[b, h, t] = (W * (2.0 ** -11 + dx + E)) @ np.abs(V) + 2.0 ** -19 * (W @ tv) + \
                    2.0 ** -31 * (W[:, None] * tv).max(0) * (i + 1) + 2.0 ** -126 * tv.sum(0)
                e_lse[b, h, t] = E + 2.0 ** -20 * (1 + np.abs(lse[b, h, t]))
    return out, lse, e_out, e_lse
