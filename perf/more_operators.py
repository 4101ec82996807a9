"""The operators of the paged key/value cache, as cases to measure.

Keys and values of all sequences live in pages of a common pool, bf16 [P, H_kv, S, d]
each: S tokens of every KV head to a page. Row j of sequence b is slot j % S of page
table[b, j // S], with an int32 table [B, M].

Three kinds of cases: "append" writes new tokens into the pages (and, where the case
says so, rotates keys and queries by their positions on the way), "decode" attends from
the newest tokens of each sequence over its pages, "chunk" attends from the tokens of a
prompt, or of a part of one, over the pages that hold them and what came before, both
with the ALiBi bias.

The rotation of R elements: elements i and i + R/2 turn by the angle n f_i at position n,
f_i = base^(-2 i / R).
"""
import math

import torch

own = False

BASE = 10000.0  # of the rotation's frequencies


def listed():
    return [
        # a serving step's new token of every sequence, far into its pages
        dict(name="append_step", kind="append", B=64, Hkv=40, G=1, T=1, C=8192, S=16, d=128, R=0, ragged=True),
        # a decoder layer's prompts, written whole
        dict(name="append_prompt", kind="append", B=4, Hkv=32, G=1, T=2048, C=4096, S=64, d=128, R=0, ragged=False),
        # grouped heads without bias: keys and queries rotated, odd starts and counts
        dict(name="append_rotated", kind="append", B=2, Hkv=6, G=4, T=1001, C=8192, S=32, d=64, R=64, ragged=True),
        # a short conversation: launch latency
        dict(name="decode_short", kind="decode", B=1, Hkv=6, G=1, T=1, L=100, S=16, d=64, ragged=False),
        # one long sequence, one key head per query head
        dict(name="decode_one", kind="decode", B=1, Hkv=40, G=1, T=1, L=8192, S=16, d=128, ragged=False),
        # a full serving batch
        dict(name="decode_batch", kind="decode", B=64, Hkv=40, G=1, T=1, L=8192, S=64, d=128, ragged=False),
        # grouped heads and sequences of different odd lengths
        dict(name="decode_grouped", kind="decode", B=16, Hkv=8, G=4, T=1, L=4097, S=32, d=128, ragged=True),
        # a very long context, few key heads
        dict(name="decode_long", kind="decode", B=1, Hkv=4, G=4, T=1, L=131071, S=128, d=128, ragged=False),
        # four drafted tokens of every sequence checked in one pass
        dict(name="decode_draft", kind="decode", B=8, Hkv=16, G=2, T=4, L=2048, S=16, d=64, ragged=True),
        # a few tokens of two short sequences, odd everywhere
        dict(name="chunk_short", kind="chunk", B=2, Hkv=3, G=2, T=100, L=999, S=16, d=64, ragged=True),
        # a decoder layer's prompts from their beginning, padded to one length
        dict(name="chunk_prompt", kind="chunk", B=4, Hkv=32, G=1, T=2048, L=2048, S=64, d=128, ragged=True),
        # the last part of a long prompt over the pages of the rest
        dict(name="chunk_long", kind="chunk", B=1, Hkv=8, G=4, T=2048, L=32768, S=128, d=128, ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "decode", "decode", "chunk"])
    d, S = rng.choice([32, 64, 128, 128]), rng.choice([16, 32, 64, 128])
    B, Hkv, ragged = _log(rng, 1, 64), _log(rng, 1, 40), rng.random() < 0.6
    if kind == "append":
        G, R = 1, 0
        if rng.random() < 0.5:
            G, R = rng.choice([1, 2, 4]), rng.choice([d // 2, d])
        T = _log(rng, 1, max(1, min(16384, 4 * 32 * 2048 * 128 * 2 // (B * Hkv * (2 + G) * d))))
        return dict(kind=kind, B=B, Hkv=Hkv, G=G, T=T, C=-(-(T + _log(rng, 1, 65536)) // S) * S, S=S, d=d, R=R, ragged=ragged)
    G = rng.choice([1, 1, 2, 3, 4, 8])
    if kind == "decode":
        T = rng.choice([1, 1, 1, 2, 5])
        most = 64 * 40 * 8192 * 128 // (B * Hkv * d * max(1, G * T // 4))
        return dict(kind=kind, B=B, Hkv=Hkv, G=G, T=T, L=_log(rng, 1, min(131072, most)), S=S, d=d, ragged=ragged)
    most = 32 * 2048 * 32768 * 128 // (B * Hkv * G * d)  # of T L
    T = _log(rng, 1, min(4096, math.isqrt(most)))
    return dict(kind=kind, B=B, Hkv=Hkv, G=G, T=T, L=T + _log(rng, 1, min(65536, most // T - T + 1)) - 1, S=S, d=d, ragged=ragged)


# ---------------------------------------------------------------- inputs


def _lens(case):
    """Length of each sequence of a decode or chunk case, new tokens included."""
    L = case["L"]
    return [L - (97 * b) % (L // 2 + 1) if case["ragged"] else L for b in range(case["B"])]


def _counts(case):
    """New tokens of each sequence of an append or chunk case."""
    T = case["T"]
    most = _lens(case) if case["kind"] == "chunk" else [T] * case["B"]
    return [min(n, T - (31 * b) % max(1, T // 3) if case["ragged"] else T) for b, n in enumerate(most)]


def _starts(case):
    """Position of the first new token of each sequence of an append case."""
    room = case["C"] - case["T"]
    return [room - (29 * b) % (room + 1) if case["ragged"] else 0 for b in range(case["B"])]


def _normal(seed, stream, *shape):
    g = torch.Generator(device="cuda").manual_seed(16 * seed + stream)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _keys(seed, stream, *shape):
    """Keys with a few strong channels, as attention heads have them."""
    k = _normal(seed, stream, *shape)
    k[..., :: max(1, shape[-1] // 4)] *= 4
    return k


def _shuffled(seed, n):
    g = torch.Generator(device="cuda").manual_seed(16 * seed + 9)
    return torch.randperm(n, generator=g, device="cuda", dtype=torch.int32)


def _append_table(case, seed):
    """(table, pages in the pool): pages of their own where a sequence gets new tokens; before and after those a
    prefix that all sequences share."""
    B, M, S = case["B"], case["C"] // case["S"], case["S"]
    spans = [(a // S, -(-(a + n) // S)) for a, n in zip(_starts(case), _counts(case))]
    shared = min(M, 8)
    table = torch.arange(M).remainder(shared).repeat(B, 1)
    used = shared
    for b, (first, end) in enumerate(spans):
        table[b, first:end] = torch.arange(used, used + end - first)
        used += end - first
    return _shuffled(seed, used)[table.cuda()].contiguous(), used


def prepare(case, seed):
    B, H, G, S, T, d = (case[x] for x in ("B", "Hkv", "G", "S", "T", "d"))
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["kind"] == "append":
        table, P = _append_table(case, seed)
        state = dict(case, table=table, pos=ints(_starts(case)), count=ints(_counts(case)), q=None, q_out=None)
        state["k_pages"], state["v_pages"] = _keys(seed, 1, P, H, S, d), _normal(seed, 2, P, H, S, d)
        state["k"], state["v"] = _keys(seed, 3, B, H, T, d), _normal(seed, 4, B, H, T, d)
        if case["R"]:
            state["q"] = _normal(seed, 5, B, H * G, T, d)
            state["q_out"] = torch.zeros_like(state["q"])
        return state
    M = -(-case["L"] // S)
    P = B * M
    state = dict(case, table=_shuffled(seed, P).view(B, M), lens=ints(_lens(case)), q=_normal(seed, 3, B, H * G, T, d))
    state["k_pages"], state["v_pages"] = _keys(seed, 1, P, H, S, d), _normal(seed, 2, P, H, S, d)
    if case["kind"] == "chunk":
        state["count"] = ints(_counts(case))
        state["out"] = torch.zeros_like(state["q"])
        state["lse"] = torch.zeros(B, H * G, T, device="cuda")
    return state


# ------------------------------------------------------------ plain forms


def _rotated(x, n, R):
    """x [B, H, T, d] rotated by the positions n [B, T], in 32 bits."""
    f = torch.tensor([BASE ** (-2 * i / R) for i in range(R // 2)], dtype=torch.float64, device="cuda")
    angle = n[:, None, :, None].double() * f
    c, s = angle.cos().float(), angle.sin().float()
    x = x.float()
    a, b = x[..., : R // 2], x[..., R // 2 : R]
    return torch.cat((a * c - b * s, b * c + a * s, x[..., R:]), -1)


def _plain_append(state):
    S, T = state["S"], state["T"]
    t = torch.arange(T, device="cuda")
    n = state["pos"][:, None] + t  # [B, T]
    valid = t < state["count"][:, None]
    k, v, q = state["k"], state["v"], state["q"]
    if state["R"]:
        k = _rotated(k, n, state["R"]).to(torch.bfloat16)
        q = _rotated(q, n, state["R"]).to(torch.bfloat16)
        state["q_out"].copy_(torch.where(valid[:, None, :, None], q, state["q_out"]))
    page = state["table"].gather(1, (n // S).clamp(max=state["table"].shape[1] - 1).long())[valid].long()
    slot = (n % S)[valid].long()
    for x, pages in ((k, state["k_pages"]), (v, state["v_pages"])):
        pages[page, :, slot] = x.transpose(1, 2)[valid]
    return (state["k_pages"], state["v_pages"]) + (() if q is None else (state["q_out"],))


def _slopes(H):
    """ALiBi slopes: 2^(-8 (h + 1) / H), and for other head counts than powers of two every other one of the next."""
    c = 1 << (H.bit_length() - 1)
    h = torch.arange(H, device="cuda", dtype=torch.float64)
    return torch.where(h < c, torch.exp2(-8 * (h + 1) / c), torch.exp2(-4 * (2 * (h - c) + 1) / c)).float()


def _rows(pages, table):
    """The rows [B, H, M S, d] of all sequences, in 32 bits."""
    B, M = table.shape
    return pages[table.long()].transpose(1, 2).reshape(B, pages.shape[1], M * pages.shape[2], pages.shape[3]).float()


def _plain_attention(state, count):
    q, table, G, T, d = (state[x] for x in ("q", "table", "G", "T", "d"))
    k, v = _rows(state["k_pages"], table), _rows(state["v_pages"], table)
    B, H, C = k.shape[:3]
    x = (q.float().view(B, H, G * T, d) @ k.transpose(-1, -2)).view(B, H, G, T, C).mul_(1 / math.sqrt(d))
    at = (state["lens"] - count)[:, None] + torch.arange(T, device="cuda")
    far = (at[:, :, None] - torch.arange(C, device="cuda"))[:, None]  # [B, 1, T, C]
    slope = _slopes(H * G).view(H, G, 1, 1)
    for g in range(G):  # one query head of each group at a time, to hold less at once
        x[:, :, g] -= slope[:, g] * far
        x[:, :, g].masked_fill_(far < 0, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    out = (x.view(B, H, G * T, C) @ v).view(B, H, G, T, d)
    out = torch.where(total > 0, out / total, 0.0).view(B, H * G, T, d)
    return out.to(torch.bfloat16), (top + total.log()).view(B, H * G, T)


def _plain_decode(state):
    return _plain_attention(state, state["T"])


def _plain_chunk(state):
    out, lse = _plain_attention(state, state["count"])
    valid = (torch.arange(state["T"], device="cuda") < state["count"][:, None])[:, None]
    state["out"].copy_(torch.where(valid[..., None], out, state["out"]))
    state["lse"].copy_(torch.where(valid, lse, state["lse"]))
    return state["out"], state["lse"]


def run(state):
    if own:
        import alibi_positional_bias_gb300 as ab

        pages = state["k_pages"], state["v_pages"], state["table"]
        if state["kind"] == "decode":
            return ab.alibi_attn_decode_paged(state["q"], *pages, lens=state["lens"], L=state["L"])
        if state["kind"] == "chunk":
            return ab.alibi_attn_fwd_paged(state["q"], *pages, lens=state["lens"], count=state["count"], L=state["L"],
                                           out=state["out"], lse=state["lse"])
        if state["R"]:
            ab.alibi_paged_append(state["k"], state["v"], *pages, pos=state["pos"], count=state["count"], rotate=state["R"],
                                  base=BASE, q=state["q"], q_out=state["q_out"])
            return state["k_pages"], state["v_pages"], state["q_out"]
        ab.alibi_paged_append(state["k"], state["v"], *pages, pos=state["pos"], count=state["count"])
        return state["k_pages"], state["v_pages"]
    return {"append": _plain_append, "decode": _plain_decode, "chunk": _plain_chunk}[state["kind"]](state)


# -------------------------------------------------- what a pass cannot do without


def work(case):
    H, G, d = case["Hkv"], case["G"], case["d"]
    if case["kind"] == "append":
        n, R = sum(_counts(case)), case["R"]
        heads = 2 * H + (H * G if R else 0)
        return {"bytes": 4 * d * heads * n, "flops": 3 * R * (H + H * G) * n}
    lens = _lens(case)
    counts = _counts(case) if case["kind"] == "chunk" else [case["T"]] * case["B"]
    rows = H * G * sum(counts)
    # queries i = len - count + t see keys 0 .. i
    pairs = H * G * sum(max(0, n - c + t + 1) for n, c in zip(lens, counts) for t in range(c))
    # every cached row and query once, outputs and their log-sums once
    return {"bytes": 4 * d * H * sum(lens) + rows * (4 * d + 4), "flops": 4 * d * pairs}


# ------------------------------------------------------------------ in 64 bits


def _turned(x, first, R):
    """x [H, T, d] in 64 bits, rotated by the positions first, first + 1, ..."""
    y = x.double().clone()
    n = torch.arange(first, first + x.shape[1], device="cuda", dtype=torch.float64)
    for i in range(R // 2):
        w = n / BASE ** (2 * i / R)
        y[..., i] = x[..., i].double() * torch.cos(w) - x[..., R // 2 + i].double() * torch.sin(w)
        y[..., R // 2 + i] = x[..., i].double() * torch.sin(w) + x[..., R // 2 + i].double() * torch.cos(w)
    return y


def exact(case, seed):
    B, H, G, S, T, d = (case[x] for x in ("B", "Hkv", "G", "S", "T", "d"))
    if case["kind"] == "append":
        table, P = _append_table(case, seed)
        outs = []
        for pages, new, R in ((_keys(seed, 1, P, H, S, d), _keys(seed, 3, B, H, T, d), case["R"]),
                              (_normal(seed, 2, P, H, S, d), _normal(seed, 4, B, H, T, d), 0)):
            pages = pages.double()
            for b, (first, n) in enumerate(zip(_starts(case), _counts(case))):
                j = torch.arange(first, first + n, device="cuda")
                pages[table[b].long()[j // S], :, j % S] = _turned(new[b, :, :n], first, R).transpose(0, 1)
            outs.append(pages)
        if case["R"]:
            q = _normal(seed, 5, B, H * G, T, d)
            o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
            for b, (first, n) in enumerate(zip(_starts(case), _counts(case))):
                o[b, :, :n] = _turned(q[b, :, :n], first, case["R"])
            outs.append(o)
        return tuple(outs)
    L = case["L"]
    M = -(-L // S)
    table = _shuffled(seed, B * M).view(B, M).long()
    kp, vp = _keys(seed, 1, B * M, H, S, d), _normal(seed, 2, B * M, H, S, d)
    q = _normal(seed, 3, B, H * G, T, d)
    c = 2 ** int(math.log2(H * G))
    slope = [2.0 ** (-8 * (h + 1) / c) if h < c else 2.0 ** (-8 * (h - c + 0.5) / c) for h in range(H * G)]
    chunk = case["kind"] == "chunk"
    out = torch.zeros(B, H * G, T, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H * G, T), 0.0 if chunk else -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, new) in enumerate(zip(_lens(case), _counts(case) if chunk else [T] * B)):
        i = torch.arange(n - new, n, device="cuda")[:, None]
        ago = i - torch.arange(n, device="cuda")[None, :]
        for h in range(H):
            k, v = (x[table[b], h].reshape(-1, d)[:n].double() for x in (kp, vp))
            for g in range(h * G, h * G + G):
                x = q[b, g, :new].double() @ k.T / math.sqrt(d) - slope[g] * ago
                x.masked_fill_(ago < 0, -math.inf)
                z = x.logsumexp(-1)
                lse[b, g, :new] = z
                out[b, g, :new] = torch.exp(x - z[:, None]).nan_to_num_(0.0) @ v
    return out, lse
