"""The operators of the 4-bit key/value cache, as cases to measure.

The cache is uint8 [B, H, C / 32, 36 D] with D = max(d, 32): blocks of 32 tokens of
one head. Each 32 consecutive elements of a token's key or value row form a group with
one bf16 scale s and a 4-bit code u per element that stands for s (u - 8). The element
of largest magnitude x_m (the positive one of +x and -x) sets s = -x_m / 8, which bf16
holds exactly, and u = min(15, floor(x / s + 8.5)); a group below 2^-100 is stored as
zeros. Within a block:

    key codes     row r, element e = 32 n + 8 c + i:   byte  r D/2 + c D/8 + 4 n + i/2
    value codes   row r = 16 t + 8 p + 2 c + z, element e = 32 n + 4 g + i:
                  byte  16 D + 8 t D + 512 (n/2) + (4 g + c) min(D/4, 16) + 8 (n%2) + 4 p + 2 z + i/2
    scales        row r, key (0) or value (1) y:        byte  32 D + (r D/8) + (y D/32 + n) 2

with the even element of each pair in the low four bits of its byte.

Three kinds of cases: "store" writes new tokens into a cache and reads them back,
"read" reads rows of a cache back, "decode" attends from the newest tokens of each
sequence over its cache with the ALiBi bias.
"""
import math

import torch

own = False

BLOCK = 32  # tokens of a cache block, and elements of a group


def listed():
    return [
        # a serving step's new token of every sequence, written into a long cache
        dict(name="store_step", kind="store", B=64, Hkv=40, T=1, C=8192, d=128, ragged=True, fp32=False),
        # a decoder layer's prompt, written whole
        dict(name="store_prompt", kind="store", B=4, Hkv=32, T=2048, C=4096, d=128, ragged=False, fp32=False),
        # small heads, odd starts and odd counts: chunks that begin and end inside a block
        dict(name="store_chunk", kind="store", B=2, Hkv=6, T=1001, C=1536, d=64, ragged=True, fp32=False),
        # a long cached prefix, read back for a prefill over it
        dict(name="read_prefix", kind="read", B=1, Hkv=16, T=16384, C=16384, d=128, ragged=False, fp32=False),
        # a few odd rows in fp32, to look at what the cache holds
        dict(name="read_rows", kind="read", B=2, Hkv=6, T=333, C=1024, d=64, ragged=True, fp32=True),
        # a short conversation: launch latency
        dict(name="decode_short", kind="decode", B=1, Hkv=6, G=1, T=1, L=100, d=64, ragged=False),
        # one long sequence, one key head per query head
        dict(name="decode_one", kind="decode", B=1, Hkv=40, G=1, T=1, L=8192, d=128, ragged=False),
        # a full serving batch
        dict(name="decode_batch", kind="decode", B=64, Hkv=40, G=1, T=1, L=8192, d=128, ragged=False),
        # grouped heads and sequences of different odd lengths
        dict(name="decode_grouped", kind="decode", B=16, Hkv=8, G=4, T=1, L=4097, d=128, ragged=True),
        # a very long context, few key heads
        dict(name="decode_long", kind="decode", B=1, Hkv=4, G=4, T=1, L=131071, d=128, ragged=False),
        # four drafted tokens of every sequence checked in one pass
        dict(name="decode_draft", kind="decode", B=8, Hkv=16, G=2, T=4, L=2048, d=64, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["store", "read", "decode", "decode"])
    d = rng.choice([32, 64, 128, 128])
    B, Hkv = _log(rng, 1, 64), rng.randint(1, 40)
    if kind == "decode":
        G, T = rng.choice([1, 1, 2, 3, 4, 8]), rng.choice([1, 1, 1, 2, 5])
        most = 64 * 40 * 8192 * 128 // (B * Hkv * d * max(1, G * T // 4))
        return dict(kind=kind, B=B, Hkv=Hkv, G=G, T=T, L=_log(rng, 1, min(131072, most)), d=d, ragged=rng.random() < 0.5)
    most = 4 * 32 * 2048 * 128 // (B * Hkv * d)
    T = _log(rng, 1, max(1, min(16384, most)))
    C = -(-(T + rng.randint(0, 2048)) // BLOCK) * BLOCK
    return dict(kind=kind, B=B, Hkv=Hkv, T=T, C=C, d=d, ragged=rng.random() < 0.7, fp32=kind == "read" and rng.random() < 0.3)


# ---------------------------------------------------------------- inputs


def _lens(case):
    """Length of each sequence of a decode case."""
    L = case["L"]
    return [L - (97 * b) % (L // 2 + 1) if case["ragged"] else L for b in range(case["B"])]


def _spans(case):
    """(first row, number of rows) of each sequence of a store or read case."""
    T, room = case["T"], case["C"] - case["T"]
    if not case["ragged"]:
        return [(0, T)] * case["B"]
    return [(room - (29 * b) % (room + 1), T - b % min(3, T)) for b in range(case["B"])]


def _normal(seed, stream, *shape):
    g = torch.Generator(device="cuda").manual_seed(16 * seed + stream)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _keys_values(seed, B, H, N, d):
    """Keys with a few strong channels, as attention heads have them, and plain values."""
    k, v = _normal(seed, 1, B, H, N, d), _normal(seed, 2, B, H, N, d)
    k[..., :: max(1, d // 4)] *= 4
    return k, v


def prepare(case, seed):
    B, H, d = case["B"], case["Hkv"], case["d"]
    if case["kind"] == "decode":
        T, G, C = case["T"], case["G"], -(-case["L"] // BLOCK) * BLOCK
        k, v = _keys_values(seed, B, H, C, d)
        lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        return dict(case, q=_normal(seed, 3, B, H * G, T, d), cache=_packed(k, v), lens=lens, places=_places(d))
    pos, count = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in zip(*_spans(case)))
    state = dict(case, pos=pos, count=count, places=_places(d))
    dtype = torch.float32 if case["fp32"] else torch.bfloat16
    state["k_out"] = torch.zeros(B, H, case["T"], d, dtype=dtype, device="cuda")
    state["v_out"] = torch.zeros_like(state["k_out"])
    if case["kind"] == "store":
        state["k"], state["v"] = _keys_values(seed, B, H, case["T"], d)
        state["cache"] = torch.zeros(B, H, case["C"] // BLOCK, 36 * max(d, 32), dtype=torch.uint8, device="cuda")
    else:
        state["cache"] = _packed(*_keys_values(seed, B, H, case["C"], d))
    return state


# ------------------------------------------------------------ plain forms


def _places(d):
    """Byte offsets in a block: [32, D/2] of the key and of the value codes (element pairs),
    [2, 32, D/32, 2] of the scales' bytes."""
    D = max(d, 32)
    r = torch.arange(BLOCK, device="cuda")[:, None]
    e = torch.arange(0, D, 2, device="cuda")[None, :]
    n = e // 32
    key = r * (D // 2) + (e % 32 // 8) * (D // 8) + 4 * n + e % 8 // 2
    lane = 4 * (e % 32 // 4) + r % 8 // 2
    value = (16 * D + 8 * D * (r // 16) + 512 * (n // 2) + lane * min(D // 4, 16) + 8 * (n % 2)
             + 4 * (r % 16 // 8) + 2 * (r % 2) + e % 4 // 2)
    y = torch.arange(2, device="cuda")[:, None, None, None]
    m = torch.arange(D // 32, device="cuda")[None, None, :, None]
    scale = 32 * D + r[None, :, :, None] * (D // 8) + (y * (D // 32) + m) * 2 + torch.arange(2, device="cuda")
    return key, value, scale


def _quantised(x):
    """Code pairs [..., D/2] uint8 and the scales' bytes [..., D/32, 2] of rows x [..., d]."""
    if x.shape[-1] < 32:
        x = torch.nn.functional.pad(x, (0, 32 - x.shape[-1]))
    x = x.float().unflatten(-1, (-1, 32))
    hi, lo = x.amax(-1, keepdim=True), x.amin(-1, keepdim=True)
    s = torch.where(hi >= -lo, hi, lo) / -8
    s = torch.where(s.abs() < 2.0 ** -103, 0.0, s)
    s = torch.where(torch.isfinite(s), s, math.nan)
    u = torch.where(torch.isfinite(s) & (s != 0), (x / s + 8.5).floor().clamp(max=15), 8.0)
    u = u.to(torch.uint8).flatten(-2)
    return u[..., 0::2] | (u[..., 1::2] << 4), s.to(torch.bfloat16).view(torch.uint8)


def _values(pairs, scales):
    """fp32 values [..., D] of code pairs [..., D/2] and scale bytes [..., D/32, 2]."""
    u = torch.stack((pairs & 15, pairs >> 4), -1).flatten(-2).float() - 8
    return (u.unflatten(-1, (-1, 32)) * scales.contiguous().view(torch.bfloat16).float()).flatten(-2)


def _packed(k, v):
    """The cache that holds the rows k, v [B, H, C, d] from position 0 on."""
    B, H, C, d = k.shape
    key, value, scale = _places(d)
    cache = torch.empty(B, H, C // BLOCK, 36 * max(d, 32), dtype=torch.uint8, device="cuda")
    for x, code, y in ((k, key, 0), (v, value, 1)):
        pairs, scales = _quantised(x.unflatten(2, (-1, BLOCK)))
        cache[..., code.flatten()] = pairs.flatten(3)
        cache[..., scale[y].flatten()] = scales.flatten(3)
    return cache


def _rows(state):
    """Flat byte indices of the rows pos + t of a store or read case: of the key codes,
    the value codes, the scales of both, each [B, H, T, ...]; and which rows count, [B, 1, T, 1]."""
    cache, T = state["cache"], state["T"]
    key, value, scale = state["places"]
    t = torch.arange(T, device="cuda")
    row = (state["pos"][:, None].long() + t).clamp(max=cache.shape[2] * BLOCK - 1)[:, None, :]
    head = torch.arange(cache.shape[0] * cache.shape[1], device="cuda").view(*cache.shape[:2], 1)
    base = ((head * cache.shape[2] + row // BLOCK) * cache.shape[3])[..., None]
    r = row[:, 0] % BLOCK
    at = [base + x[r][:, None].flatten(3) for x in (key, scale[0], value, scale[1])]
    return at, (t < state["count"][:, None])[:, None, :, None]


def _plain_read(state):
    flat = state["cache"].view(-1)
    (ak, bk, av, bv), valid = _rows(state)
    for name, a, b in (("k_out", ak, bk), ("v_out", av, bv)):
        x = _values(flat[a], flat[b].unflatten(-1, (-1, 2)))[..., : state["d"]]
        state[name].copy_(torch.where(valid, x, state[name].float()))
    return state["k_out"], state["v_out"]


def _plain_store(state):
    flat = state["cache"].view(-1)
    (ak, bk, av, bv), valid = _rows(state)
    for x, a, b in ((state["k"], ak, bk), (state["v"], av, bv)):
        pairs, scales = _quantised(x)
        flat[a] = torch.where(valid, pairs, flat[a])
        flat[b] = torch.where(valid, scales.flatten(-2), flat[b])
    return _plain_read(state)


def _slopes(H):
    """ALiBi slopes: 2^(-8 (h + 1) / H), and for other head counts than powers of two every other one of the next."""
    c = 1 << (H.bit_length() - 1)
    h = torch.arange(H, device="cuda", dtype=torch.float64)
    return torch.where(h < c, torch.exp2(-8 * (h + 1) / c), torch.exp2(-4 * (2 * (h - c) + 1) / c)).float()


def _plain_decode(state):
    cache, q, T, G, d = state["cache"], state["q"], state["T"], state["G"], state["d"]
    B, H = cache.shape[:2]
    key, value, scale = state["places"]
    C = cache.shape[2] * BLOCK

    def side(code, y):
        pairs = cache[..., code.flatten()].view(B, H, C, -1)
        scales = cache[..., scale[y].flatten()].view(B, H, C, -1, 2)
        return _values(pairs, scales)[..., :d]

    rows = q.float().view(B, H, G * T, d)
    x = (rows @ side(key, 0).transpose(-1, -2)).view(B, H, G, T, C) * (1 / math.sqrt(d))
    at = state["lens"][:, None] - T + torch.arange(T, device="cuda")
    far = (at[:, :, None] - torch.arange(C, device="cuda"))[:, None, None]
    x = x - _slopes(H * G).view(1, H, G, 1, 1) * far
    x = torch.where(far >= 0, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, H, G * T, C) @ side(value, 1)).view(B, H, G, T, d)
    out = torch.where(total > 0, out / total, 0.0).view(B, H * G, T, d)
    return out.to(torch.bfloat16), (top + total.log()).view(B, H * G, T)


def run(state):
    if own:
        import alibi_positional_bias_gb300 as ab

        if state["kind"] == "decode":
            return ab.alibi_attn_decode_kv4(state["q"], state["cache"], lens=state["lens"], L=state["L"])
        if state["kind"] == "store":
            ab.alibi_kv4_write(state["k"], state["v"], state["cache"], pos=state["pos"], count=state["count"])
        return ab.alibi_kv4_read(state["cache"], state["k_out"], state["v_out"], pos=state["pos"], count=state["count"])
    return {"decode": _plain_decode, "store": _plain_store, "read": _plain_read}[state["kind"]](state)


# -------------------------------------------------- what a pass cannot do without


def work(case):
    B, H, d = case["B"], case["Hkv"], case["d"]
    if case["kind"] == "decode":
        keys, rows = H * sum(_lens(case)), case["G"] * case["T"]
        # every cached byte and query once, outputs and their log-sums once
        return {"bytes": keys * 36 * d / 32 + B * H * rows * (4 * d + 4), "flops": 4 * d * rows * keys}
    n = H * d * sum(c for _, c in _spans(case))
    values = n * (8 if case["fp32"] else 4)
    if case["kind"] == "read":
        return {"bytes": n * 36 / 32 + values, "flops": 4 * n}
    return {"bytes": 4 * n + n * 36 / 32 + values, "flops": 12 * n}


# ------------------------------------------------------------------ in 64 bits


def _held(x):
    """What the cache holds for rows x [..., d], in 64 bits."""
    n = min(32, x.shape[-1])
    g = x.double().reshape(*x.shape[:-1], -1, n)
    big = g.abs().max(-1, keepdim=True).values
    step = torch.where((g == big).any(-1, keepdim=True), -big, big) / 8
    code = torch.where(big < 2.0 ** -100, 0.0, torch.floor(g / step + 0.5).clamp(max=7))
    return (code * step).reshape(x.shape)


def exact(case, seed):
    B, H, d = case["B"], case["Hkv"], case["d"]
    if case["kind"] != "decode":
        k, v = _keys_values(seed, B, H, case["T"] if case["kind"] == "store" else case["C"], d)
        out = [torch.zeros(B, H, case["T"], d, dtype=torch.float64, device="cuda") for _ in range(2)]
        for b, (first, count) in enumerate(_spans(case)):
            if case["kind"] == "store":
                first = 0
            for x, o in zip((k, v), out):
                o[b, :, :count] = _held(x[b, :, first : first + count])
        return tuple(out)
    T, G, L = case["T"], case["G"], case["L"]
    k, v = _keys_values(seed, B, H, -(-L // BLOCK) * BLOCK, d)
    q = _normal(seed, 3, B, H * G, T, d).double()
    c = 2 ** int(math.log2(H * G))
    slope = [2.0 ** (-8 * (h + 1) / c) if h < c else 2.0 ** (-8 * (h - c + 0.5) / c) for h in range(H * G)]
    slope = torch.tensor(slope, dtype=torch.float64, device="cuda").view(H, G, 1, 1)
    out = torch.zeros(B, H * G, T, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H * G, T), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        kb, vb = _held(k[b, :, :n]), _held(v[b, :, :n])
        x = torch.einsum("hgtd,hjd->hgtj", q[b].view(H, G, T, d), kb) / math.sqrt(d)
        ago = torch.arange(n - T, n, device="cuda")[:, None] - torch.arange(n, device="cuda")[None, :]
        x = (x - slope * ago).masked_fill(ago < 0, -math.inf)
        lse[b] = x.logsumexp(-1).reshape(H * G, T)
        w = torch.exp(x - lse[b].view(H, G, T, 1)).nan_to_num(0.0)
        out[b] = torch.einsum("hgtj,hjd->hgtd", w, vb).reshape(H * G, T, d)
    return out, lse
