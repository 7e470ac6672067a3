"""Workloads of the paged 8-bit key/value cache: its attention, over all keys and over blocks that a score selects, and writing rotated
tokens into it.

A cache page holds `page` tokens of one layer, in B = page / 64 blocks of 64 tokens for each of H key/value heads:
    values [H][B]{K [dim/16][64][16] | V [4][dim][16]} | bounds [H][B][2][dim] | scales [H][B][4], and bytes up to a multiple of 128.
Values are E4M3 numbers; a scale is a biased power of two (E8M0) for all keys (byte 0) or values (byte 1) of one block and head.  K unit
[u][t] is channels 16 u .. 16 u + 15 of token t of the block; V unit [g][c] is channel c of tokens 16 j + 4 g + i, at byte 4 j + i.  Bounds are
the largest and the smallest key of the block in each channel.
Token i of sequence s is at place kv_len[s] - (q_start[s + 1] - q_start[s]) + i of the sequence.

Head counts are those of the decoder layers the benchmark runs: 32 query and 8 key/value heads (q 4096, k 1024), 40 and 8 (q 5120), 64 and
8 (q 8192), dim 128.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one conversation at a context of 512: what a token waits for between q|k|v and o
        attention_case("attention: 1 x 512 tokens, 32/8 heads", 1, 1, 512, 32, 8),
        # a serving batch in mid-flight, contexts from one page to 8K, five query heads to a key head
        attention_case("attention: 48 ragged to 8K, 40/8 heads", 48, 1, 8192, 40, 8),
        # long documents: the cache is far larger than every on-chip memory
        attention_case("attention: 16 ragged to 64K, 64/8 heads", 16, 1, 65536, 64, 8),
        # drafts of four tokens checked at once, small heads, a window
        attention_case("attention: 32 drafts of 4 to 6000, dim 64", 32, 4, 6000, 32, 8, dim=64, page=128, window=4096),
        # prompts read in chunks behind what is cached already
        attention_case("attention: 3 prompts of 4K behind 2K, 32/8", 3, 4096, 6144, 32, 8),
        # the new token of every sequence of a serving batch
        append_case("append: 48 sequences, one token", 48, 1, 4096, 32, 8),
        # short questions that go on behind what is there, pairs side by side, half of the channels rotated
        append_case("append: 13 of up to 37 behind 999, dim 64", 13, 37, 999, 20, 4, dim=64, page=128, rotary=32, interleaved=True),
        # prompts going in
        append_case("append: 3 prompts of 4K", 3, 4096, 6144, 32, 8),
        # one long conversation
        sparse_case("select: 1 x 32K, 32 blocks, 32/8", 1, 1, 32768, 32, 8, 32, 1, 2),
        # long documents, a sixteenth of each looked at
        sparse_case("select: 16 ragged to 64K, 64 blocks, 64/8", 16, 1, 65536, 64, 8, 64, 1, 4),
        # drafts of five tokens
        sparse_case("select: 24 drafts of 5 to 9001, 24 blocks", 24, 5, 9001, 40, 8, 24, 2, 2, page=256),
        # a chunk of a prompt behind what is cached already
        sparse_case("select: chunk of 512 behind 16K, 16 blocks", 1, 512, 16896, 32, 8, 16, 1, 2),
    ]


def attention_case(name, seqs, q, kv, heads, kv_heads, dim=128, page=64, window=0):
    c = {"op": "attention", "seqs": seqs, "q": q, "kv": kv, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "window": window}
    return dict(c, name=name) if name else c


def append_case(name, seqs, q, kv, heads, kv_heads, dim=128, page=64, rotary=None, interleaved=False):
    c = {"op": "append", "seqs": seqs, "q": q, "kv": kv, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
         "rotary": dim if rotary is None else rotary, "interleaved": interleaved}
    return dict(c, name=name) if name else c


def sparse_case(name, seqs, q, kv, heads, kv_heads, top, first, last, dim=128, page=64):
    c = {"op": "sparse", "seqs": seqs, "q": q, "kv": kv, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "window": 0,
         "top": top, "first": first, "last": last}
    return dict(c, name=name) if name else c


def spread(rng, low, high):
    """A whole number between two, its logarithm spread evenly."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("attention", "attention", "append", "sparse", "sparse"))
    dim, page = rng.choice((64, 128, 128)), rng.choice((64, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 4, 5, 8))
    if op == "attention":
        if rng.random() < 0.4:  # prompts
            seqs = rng.randint(1, 4)
            q = spread(rng, 9, 4096 // seqs)
            group = min(group, 4)
            kv = q + rng.choice((0, spread(rng, 1, 4096)))
        else:  # single tokens, and a few at a time where drafts are checked
            seqs = spread(rng, 1, 96)
            q = rng.choice((1, 1, 2, 5, 8))
            kv = max(q, spread(rng, 1, 400000 // seqs if seqs > 8 else 50000))
        window = rng.choice((0, 0, 0, spread(rng, 1, 4096)))
        return attention_case(None, seqs, q, kv, kv_heads * group, kv_heads, dim, page, window)
    if op == "append":
        seqs = spread(rng, 1, 128)
        q = rng.choice((1, spread(rng, 2, max(2, 8192 // seqs))))
        return append_case(None, seqs, q, q + rng.choice((0, spread(rng, 1, 4096))), kv_heads * group, kv_heads, dim, page,
                           rng.choice((0, dim // 2, dim, dim)), rng.random() < 0.3)
    top, first, last = spread(rng, 4, 128), rng.randint(0, 2), rng.randint(0, 2)
    if rng.random() < 0.3:  # a chunk of a prompt
        seqs = rng.randint(1, 2)
        top = min(top, 32)
        q = spread(rng, 9, max(9, 65536 // (top * kv_heads * seqs)))
        kv = q + spread(rng, 1, 16384)
    else:
        seqs = spread(rng, 1, 32)
        q = rng.choice((1, 1, 2, 5))
        kv = q + spread(rng, 1, 400000 // seqs if seqs > 8 else 65536)
    return sparse_case(None, seqs, q, kv, kv_heads * group, kv_heads, top, first, last, dim, page)


def lengths(case):
    """(new tokens, tokens with them) of every sequence: ragged, the same for every seed; the first sequence is the longest."""
    r = random.Random(case["seqs"] * 1000003 + case["kv"])
    q, kv = case["q"], case["kv"]
    new = [q] + [q if q <= 8 else r.randint(max(1, q // 2), q) for _ in range(case["seqs"] - 1)]
    return new, [kv] + [max(n, int(kv * math.exp(r.uniform(math.log(0.15), 0)))) for n in new[1:]]


def page_bytes(case):
    H, D, page = case["kv_heads"], case["dim"], case["page"]
    return -(-H * (page // 64) * (130 * D + 4) // 128) * 128


def visible(n, length, window):
    """Pairs of a query and a key it may look at: query i is at place length - n + i."""
    places = range(max(0, length - n), length)
    if not window:
        return (places.start + 1 + length) * len(places) // 2
    return sum(min(p + 1, window) for p in places)


def work(case):
    new, length = lengths(case)
    T, H, D, heads = sum(new), case["kv_heads"], case["dim"], case["heads"]
    if case["op"] == "attention":
        w = case["window"]
        seen = sum(min(n, w + q - 1) if w else n for q, n in zip(new, length))
        pairs = sum(visible(q, n, w) for q, n in zip(new, length))
        return {"bytes": seen * 2 * H * D + T * heads * (4 * D + 4), "flops": 4 * pairs * heads * D}
    if case["op"] == "append":  # read and written, and the written values read back
        return {"bytes": T * (H * D * (4 + 2 + 2 + 4) + heads * D * 4) + 4 * case["rotary"] * min(T, max(length)),
                "flops": T * (3 * (H + heads) * case["rotary"] + 8 * H * D)}
    blocks = [-(-n // 64) for n in length]
    taken = [min(case["top"], n) for n in blocks]  # of one row at least, of other rows they may be the same
    scored = sum(q * n for q, n in zip(new, blocks))
    looked = sum(q * n for q, n in zip(new, taken)) * 64
    return {"bytes": H * (sum(blocks) * (2 * D + 4) + sum(taken) * 128 * D) + T * (heads * (6 * D + 4) + 4 * H * case["top"]),
            "flops": 4 * scored * H * D + 4 * looked * heads * D}


# ---------------------------------------------------------------- what a program has in hand

def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def heads_like(shape, g):
    """bf16 activations of heads: normal, with a few channels several times larger than the others, as keys have them."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(shape[-2:], generator=g, device="cuda"))
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    new, length = lengths(case)
    S, T, H, D, page = case["seqs"], sum(new), case["kv_heads"], case["dim"], case["page"]
    columns = -(-max(length) // page)
    counts = [-(-n // page) for n in length]
    pages = sum(counts) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((S, columns), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(columns, device="cuda") < ints(counts)[:, None]
    table[at] = order[: sum(counts)]
    starts = [sum(new[:s]) for s in range(S + 1)]
    s = {"case": case, "table": table, "kv_len": ints(length), "q_start": ints(starts)}
    # which token of which sequence each row is: the plain form's index, a fused one goes by q_start
    s["seq"] = torch.repeat_interleave(torch.arange(S, device="cuda"), ints(new).long())
    s["row"] = torch.arange(T, device="cuda") - s["q_start"].long()[s["seq"]]
    s["place"] = (s["kv_len"] - (s["q_start"][1:] - s["q_start"][:-1])).long()[s["seq"]] + s["row"]

    # what earlier tokens left in the cache: all of a sequence's, or those before the new ones
    held = torch.zeros(pages, dtype=torch.int64, device="cuda")
    there = ints([n - q if case["op"] == "append" else n for q, n in zip(new, length)]).long()
    held[table[at].long()] = (there[:, None] - page * torch.arange(columns, device="cuda")).clamp(0, page)[at]
    s["cache"] = torch.zeros((pages, page_bytes(case)), dtype=torch.uint8, device="cuda")
    few = max(1, (1 << 26) // (H * page * D))
    size = torch.exp(0.5 * torch.randn((H, 1, D), generator=g, device="cuda"))  # larger channels, the same for all tokens
    drift = torch.randn((pages, H, 1, D), generator=g, device="cuda")  # and what the tokens of a page have in common
    for p in range(0, pages, few):
        n = min(few, pages - p)
        k, v = (torch.randn((n, H, page, D), generator=g, device="cuda") for _ in range(2))
        live = torch.arange(page, device="cuda") < held[p : p + n, None]
        s["cache"][p : p + n] = laid_out((k + drift[p : p + n]) * size, v, live[:, None, :, None], case)
    if case["op"] != "append":
        s["q"] = heads_like((T, case["heads"], D), g)
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((T, case["heads"]), device="cuda")
        if case["op"] == "sparse":
            s["selected"] = torch.empty((T, H, case["top"]), dtype=torch.int32, device="cuda")
        return s
    s["k"], s["v"] = heads_like((T, H, D), g), heads_like((T, H, D), g)
    s["q"] = heads_like((T, case["heads"], D), g)
    s["q_out"], s["k_out"], s["v_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
    s["rotation"] = None
    if case["rotary"]:  # cosine and sine of every place, in 64 bits where the angle is far
        turn = 500000.0 ** (-torch.arange(case["rotary"] // 2, dtype=torch.float64, device="cuda") * 2 / case["rotary"])
        angle = torch.arange(columns * page, dtype=torch.float64, device="cuda")[:, None] * turn
        s["rotation"] = torch.stack([torch.cos(angle), torch.sin(angle)], -1).float()
    # the blocks of 64 tokens that the new rows lie in, the sequence and number of each, and which of them is each row's
    key = s["seq"] * (columns * page // 64) + s["place"] // 64
    key, s["unit"] = torch.unique(key, return_inverse=True)
    s["unit_seq"], s["unit_block"] = key // (columns * page // 64), key % (columns * page // 64)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    H, page = case["kv_heads"], case["page"]
    if own:
        import bitmask_spmv_amd as nm

        batch = s["cache"], s["table"], s["kv_len"], s["q_start"]
        if case["op"] == "append":
            if s["rotation"] is None:  # queries stay as they are
                nm.nm_kv8_append(s["k"], s["v"], *batch, page)
            else:
                nm.nm_kv8_append(s["k"], s["v"], *batch, page, rotation=s["rotation"], interleaved=case["interleaved"], q=s["q"], q_out=s["q_out"])
            nm.nm_kv8_unpack(*batch, page, s["k_out"], s["v_out"])
            return s["k_out"], s["v_out"], s["q"] if s["rotation"] is None else s["q_out"]
        if case["op"] == "attention":
            return nm.nm_kv8_attention(s["q"], *batch, H, page, case["q"], window=case["window"], out=s["out"], lse=s["lse"])
        nm.nm_kv8_select(s["q"], *batch, H, page, case["top"], first=case["first"], last=case["last"], out=s["selected"])
        nm.nm_kv8_attention(s["q"], *batch, H, page, case["q"], selected=s["selected"], out=s["out"], lse=s["lse"])
        return s["selected"], s["out"], s["lse"]
    if case["op"] == "append":
        return plain_append(s)
    if case["op"] == "attention":
        return plain_attention(s)
    selected = plain_select(s)
    return selected, *plain_selected_attention(s, selected)


# ---------------------------------------------------------------- the plain forms

def parts(cache, case):
    """Views of the pages: K codes [N][H][B][D/16][64][16], V codes [N][H][B][4][D][16], bounds [N][H][B][2][D], scales [N][H][B][4]."""
    N, H, D, B = cache.shape[0], case["kv_heads"], case["dim"], case["page"] // 64
    a, b, c = H * B * 128 * D, H * B * 130 * D, H * B * (130 * D + 4)
    values = cache[:, :a].view(N, H, B, 2, 64 * D)
    return (values[:, :, :, 0].unflatten(-1, (D // 16, 64, 16)), values[:, :, :, 1].unflatten(-1, (4, D, 16)),
            cache[:, a:b].view(N, H, B, 2, D), cache[:, b:c].view(N, H, B, 4))


def scale_byte(top):
    """The scale byte that brings magnitudes up to `top` (fp32) to 448 and below."""
    bits = top.view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)).clamp(63, 182)


def power(byte):
    """2^(byte - 127), put together from its bits: exp2 may be off by one in the last."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def codes(x, byte):
    """fp32 values of a block whose scale byte is `byte` -> E4M3 codes."""
    return (x * power(254 - byte)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def numbers(code):
    return code.view(torch.float8_e4m3fn).float()


def k_units(x):  # [.., 64, D] -> [.., D/16, 64, 16]
    return x.unflatten(-1, (-1, 16)).transpose(-3, -2)


def v_units(x):  # [.., 64, D] -> [.., 4, D, 16]: token 16 j + 4 g + i
    n = x.dim() - 2
    return x.unflatten(-2, (4, 4, 4)).permute(*range(n), n + 1, n + 3, n, n + 2).flatten(-2)


def k_rows(u):  # and back
    return u.transpose(-3, -2).flatten(-2)


def v_rows(u):
    n = u.dim() - 3
    return u.unflatten(-1, (4, 4)).permute(*range(n), n + 2, n, n + 3, n + 1).flatten(-4, -2)


def laid_out(k, v, live, case):
    """fp32 [n][H][page][D], of which tokens are there -> bytes of whole pages."""
    n, H, page, D = k.shape
    out = torch.zeros((n, page_bytes(case)), dtype=torch.uint8, device=k.device)
    ku, vu, bounds, scales = parts(out, case)
    live = live.unflatten(2, (-1, 64))
    for i, (x, to, units) in enumerate(((k, ku, k_units), (v, vu, v_units))):
        x = x.unflatten(2, (-1, 64)) * live
        byte = scale_byte(x.abs().amax((-1, -2)))
        x = codes(x, byte[..., None, None])
        to.copy_(units(x))
        scales[..., i] = byte.to(torch.uint8)
        if i == 0:
            x = numbers(x)
            some = live.any(-2)
            bounds[..., 0, :] = torch.where(some, x.masked_fill(~live, -math.inf).amax(-2), 0.0).to(torch.float8_e4m3fn).view(torch.uint8)
            bounds[..., 1, :] = torch.where(some, x.masked_fill(~live, math.inf).amin(-2), 0.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def cached(s, table):
    """Keys and values fp32 [..., H][B * 64][D] of the pages in `table` [...], whatever is in them."""
    ku, vu, _, scales = parts(s["cache"], s["case"])
    at = table.clamp_min(0).long()
    scale = power(scales[at])[..., None, None]
    return ((numbers(k_rows(ku[at])) * scale[..., 0, :, :]).flatten(-3, -2), (numbers(v_rows(vu[at])) * scale[..., 1, :, :]).flatten(-3, -2))


def weighted(x, seen):
    """Scores [..., keys] and which of them a row sees -> weights, log-sum-exp and what the weights are divided by."""
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    x.sub_(top).exp_()
    total = x.sum(-1)
    return x, top[..., 0] + total.log(), torch.where(total == 0, 1.0, total)[..., None]


def plain_attention(s):
    case = s["case"]
    S, Q, H, D = case["seqs"], case["q"], case["kv_heads"], case["dim"]
    group = case["heads"] // H
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in cached(s, s["table"]))  # [S][H][tokens][D]
    q = torch.zeros((S, Q, H * group, D), device=k.device)
    q[s["seq"], s["row"]] = s["q"].float()
    q = q.view(S, Q, H, group, D).permute(0, 2, 1, 3, 4).reshape(S, H, Q * group, D)
    x = torch.matmul(q, k.transpose(-1, -2)).view(S, H, Q, group, -1)
    x *= 1 / math.sqrt(D)
    new = s["q_start"][1:] - s["q_start"][:-1]
    at = (s["kv_len"] - new)[:, None, None] + torch.arange(Q, device=k.device)[:, None]  # place of every query
    key = torch.arange(k.shape[2], device=k.device)
    seen = (key <= at) & ((key > at - case["window"]) if case["window"] else True)
    x, lse, total = weighted(x, seen[:, None, :, None])
    o = torch.matmul(x.view(S, H, Q * group, -1), v).view(S, H, Q, group, D) / total
    o, lse = o.permute(0, 2, 1, 3, 4).reshape(S, Q, -1, D), lse.permute(0, 2, 1, 3).reshape(S, Q, -1)
    return o[s["seq"], s["row"]].to(torch.bfloat16), lse[s["seq"], s["row"]]


def plain_select(s):
    """Blocks of 64 keys that each row and key head takes: those whose bound on the sum of the head's scores is largest, in 64 bits."""
    case = s["case"]
    S, Q, H, D, top = case["seqs"], case["q"], case["kv_heads"], case["dim"], case["top"]
    _, _, bounds, scales = parts(s["cache"], case)
    at = s["table"].clamp_min(0).long()
    b = numbers(bounds[at]).double() * power(scales[at][..., 0]).double()[..., None, None]  # [S][columns][H][B][2][D]
    b = b.permute(0, 2, 1, 3, 4, 5).reshape(S, H, -1, 2 * D)
    q = s["q"].double().unflatten(1, (H, -1))
    q = torch.cat([q.clamp_min(0).sum(2), q.clamp_max(0).sum(2)], -1)  # [T][H][2 D]
    rows = torch.zeros((S, Q, H, 2 * D), dtype=torch.float64, device=q.device)
    rows[s["seq"], s["row"]] = q
    x = torch.matmul(rows.transpose(1, 2), b.transpose(-1, -2))  # [S][H][Q][blocks]
    x = x.transpose(1, 2)[s["seq"], s["row"]]  # [T][H][blocks]
    block, mine = torch.arange(x.shape[-1], device=x.device), (s["place"] // 64)[:, None, None]
    x = torch.where((block < case["first"]) | (block > mine - case["last"]), math.inf, x)
    x = torch.where(block > mine, -math.inf, x)
    x, i = torch.sort(x, dim=-1, descending=True, stable=True)
    none = 1 << 30
    i = torch.where(torch.isneginf(x), none, i)[..., :top]
    i = torch.nn.functional.pad(i, (0, top - i.shape[-1]), value=none).sort(-1).values
    return torch.where(i == none, -1, i).to(torch.int32)


def plain_selected_attention(s, selected):
    case = s["case"]
    T, H, D, page = selected.shape[0], case["kv_heads"], case["dim"], case["page"]
    ku, vu, _, scales = parts(s["cache"], case)
    b = selected.clamp_min(0).long()  # [T][H][top]
    where = s["table"][s["seq"][:, None, None], b // (page // 64)].clamp_min(0).long(), torch.arange(H, device=b.device)[:, None], b % (page // 64)
    scale = power(scales[where])[..., None, None]
    k = (numbers(k_rows(ku[where])) * scale[..., 0, :, :]).flatten(2, 3)  # [T][H][top * 64][D]
    v = (numbers(v_rows(vu[where])) * scale[..., 1, :, :]).flatten(2, 3)
    x = torch.matmul(s["q"].float().unflatten(1, (H, -1)), k.transpose(-1, -2))
    x *= 1 / math.sqrt(D)
    key = (selected[..., None] * 64 + torch.arange(64, device=b.device)).flatten(2, 3)
    seen = (key <= s["place"][:, None, None]) & (key >= 0)
    x, lse, total = weighted(x, seen[:, :, None])
    return (torch.matmul(x, v) / total).flatten(1, 2).to(torch.bfloat16), lse.flatten(1)


def rotated(x, turn, interleaved):
    """fp64 [T][heads][D], [T][pairs][2] cosines and sines."""
    R = 2 * turn.shape[1]
    c, t = turn[:, None, :, 0], turn[:, None, :, 1]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., : R // 2], x[..., R // 2 : R])
    a, b = a * c - b * t, b * c + a * t
    y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y, x[..., R:]], -1)


def narrowed(x):
    """fp64 -> fp32 that rounds to fewer bits as x itself does: cut after 20 bits of fraction, the last of them set where something is lost."""
    bits = x.view(torch.int64)
    bits = torch.where((bits & 0xFFFFFFFF) != 0, (bits | (1 << 32)) & ~0xFFFFFFFF, bits)
    return bits.view(torch.float64).float()


def plain_append(s):
    case = s["case"]
    H, D, page = case["kv_heads"], case["dim"], case["page"]
    k, q = s["k"].double(), s["q"].double()
    if s["rotation"] is not None:
        turn = s["rotation"][s["place"]].double()
        k, q = rotated(k, turn, case["interleaved"]), rotated(q, turn, case["interleaved"])
    U, B = s["unit_seq"].shape[0], page // 64
    where = s["table"][s["unit_seq"], s["unit_block"] // B].long(), slice(None), s["unit_block"] % B
    where = where[0][:, None], torch.arange(H, device=k.device), where[2][:, None]
    token = s["place"] % 64
    fresh = torch.zeros((U, 64), dtype=torch.bool, device=k.device)
    fresh[s["unit"], token] = True
    before = torch.argmax(fresh.to(torch.uint8), -1)  # tokens of the block that were there
    old = (torch.arange(64, device=k.device) < before[:, None])[:, None, :, None]
    fresh = fresh[:, None, :, None]
    ku, vu, bounds, scales = parts(s["cache"], case)
    back = []
    for i, (x, at, units, rows) in enumerate(((k, ku, k_units, k_rows), (s["v"].double(), vu, v_units, v_rows))):
        new = torch.zeros((U, H, 64, D), device=k.device)
        new[s["unit"], :, token] = narrowed(x)
        byte, was = scale_byte(new.abs().amax((-1, -2))), scales[where][..., i].to(torch.int32)
        byte = torch.where((before > 0)[:, None], torch.maximum(byte, was), byte)
        more = power(was - byte + 127)[..., None, None]  # 1 unless the scale grows
        code = rows(at[where])
        code = torch.where(old, (numbers(code) * more).to(torch.float8_e4m3fn).view(torch.uint8), code)
        code = torch.where(fresh, codes(new, byte[..., None, None]), code)
        at[where] = units(code)
        scales[where + (i,)] = byte.to(torch.uint8)
        if i == 0:
            n = numbers(code)
            most, least = n.masked_fill(~fresh, -math.inf).amax(-2), n.masked_fill(~fresh, math.inf).amin(-2)
            b = (numbers(bounds[where]) * more).to(torch.float8_e4m3fn).float()
            had = (before > 0)[:, None, None]
            most = torch.where(had, torch.maximum(most, b[..., 0, :]), most)
            least = torch.where(had, torch.minimum(least, b[..., 1, :]), least)
            bounds[where] = torch.stack([most, least], -2).to(torch.float8_e4m3fn).view(torch.uint8)
        # what the cache now holds for these tokens
        n = numbers(rows(at[where])) * power(scales[where][..., i])[..., None, None]
        back.append(n[s["unit"], :, token].to(torch.bfloat16))
    return back[0], back[1], q.to(torch.bfloat16)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    new, length = lengths(case)
    if case["op"] == "append":
        return exact_append(s, new, length)
    H, D, w = case["kv_heads"], case["dim"], case["window"]
    group, out, lse, at = case["heads"] // H, [], [], 0
    for i, (n, length) in enumerate(zip(new, length)):
        q = s["q"][at : at + n].double()
        at += n
        place = torch.arange(length, device="cuda")
        mine = length - n + torch.arange(n, device="cuda")
        outs, sums = [], []
        for h in range(H):
            k, v = (exact_values(s, i, place, h, values) for values in (False, True))
            x = torch.einsum("nge,ke->gnk", q[:, h * group : (h + 1) * group], k) / math.sqrt(D)
            behind = mine[:, None] - place
            hidden = (behind < 0) | ((behind >= w) if w else False)
            if case["op"] == "sparse":
                hidden = hidden | ~exact_chosen(s, i, h, q[:, h * group : (h + 1) * group], mine)[:, place // 64]
            x[:, hidden] = -math.inf
            total = torch.logsumexp(x, -1)
            outs.append(torch.einsum("gnk,ke->nge", torch.exp(x - total[..., None]), v))
            sums.append(total.T)
        out.append(torch.cat(outs, 1))
        lse.append(torch.cat(sums, 1))
    out, lse = torch.cat(out), torch.cat(lse)
    return (None, out, lse) if case["op"] == "sparse" else (out, lse)


def two_to(e):
    """fp64 powers of two, from their bits: a power function may be off by one in the last."""
    return (e.long() + 1023 << 52).view(torch.float64)


def e4m3(byte):
    """The numbers that bytes stand for, from their fields."""
    byte = byte.long()
    e, m = byte >> 3 & 15, byte & 7
    x = torch.where(e == 0, m.double() * 2.0**-9, (8 + m).double() * two_to(e - 10))
    return torch.where(byte > 127, -x, x)


def exact_values(s, i, place, h, values):
    """fp64 [tokens][D] of one sequence and head, byte by byte from where the format puts them."""
    case = s["case"]
    H, D, page = case["kv_heads"], case["dim"], case["page"]
    B, c, t = page // 64, torch.arange(D, device="cuda"), place[:, None] % 64
    block = h * B + place[:, None] % page // 64
    if values:
        byte = block * 128 * D + 64 * D + (t // 4 % 4 * D + c) * 16 + t // 16 * 4 + t % 4
    else:
        byte = block * 128 * D + (c // 16 * 64 + t) * 16 + c % 16
    rows = s["table"][i].long()[place // page][:, None]
    scale = s["cache"][rows, H * B * 130 * D + block * 4 + int(values)]
    return e4m3(s["cache"][rows, byte]) * two_to(scale.long() - 127)


def exact_chosen(s, i, h, q, mine):
    """Which blocks rows at places `mine` take, by comparing each block with all others."""
    case = s["case"]
    H, D, page = case["kv_heads"], case["dim"], case["page"]
    B, c = page // 64, torch.arange(D, device="cuda")
    block = torch.arange(int(mine[-1]) // 64 + 1, device="cuda")
    at = h * B + block[:, None] % B
    rows = s["table"][i].long()[block // B][:, None]
    scale = two_to(s["cache"][rows, H * B * 130 * D + at * 4].long() - 127)
    most, least = (e4m3(s["cache"][rows, H * B * 128 * D + (at * 2 + j) * D + c]) * scale for j in (0, 1))
    x = sum(torch.maximum(q[:, g, None] * most, q[:, g, None] * least).sum(-1) if q.shape[0] == 1 else
            q[:, g].clamp_min(0) @ most.T + q[:, g].clamp_max(0) @ least.T for g in range(q.shape[1]))
    own_block = (mine // 64)[:, None]
    x = torch.where((block < case["first"]) | (block > own_block - case["last"]), math.inf, x)
    x = torch.where(block > own_block, -math.inf, x)
    chosen = torch.empty_like(x, dtype=torch.bool)
    for r in range(x.shape[0]):
        ahead = (x[r] > x[r][:, None]) | ((x[r] == x[r][:, None]) & (block < block[:, None]))
        chosen[r] = ahead.sum(-1) < case["top"]
    return chosen & (block <= own_block)


def exact_append(s, new, length):
    case = s["case"]
    H, D, page = case["kv_heads"], case["dim"], case["page"]
    k, q = s["k"].double(), s["q"].double()
    if s["rotation"] is not None:
        R, pairs = case["rotary"], torch.arange(case["rotary"] // 2, device="cuda")
        a, b = (2 * pairs, 2 * pairs + 1) if case["interleaved"] else (pairs, pairs + R // 2)
        turn = torch.complex(*s["rotation"].double().unbind(-1))[s["place"]][:, None]
        for x in (k, q):
            y = torch.complex(x[..., a], x[..., b]) * turn
            x[..., a], x[..., b] = y.real, y.imag
    outs, at = ([], []), 0
    for i, (n, length) in enumerate(zip(new, length)):
        begin = length - n
        for x, done, values in ((k, outs[0], False), (s["v"].double(), outs[1], True)):
            x = x[at : at + n]
            for b in range(begin // 64, (length - 1) // 64 + 1):  # block by block
                lo, hi = max(begin, 64 * b), min(length, 64 * b + 64)
                y = x[lo - begin : hi - begin]
                top = y.abs().amax((0, 2))
                m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1)
                byte = torch.where(top > 0, e - 1 - 8 + (m > 0.875) + 127, 0).clamp(63, 182)
                if lo > 64 * b:  # a scale that is there does not shrink
                    p, B = int(s["table"][i, lo // page]), page // 64
                    was = s["cache"][p, H * B * 130 * D :][: H * B * 4].view(H, B, 4)[:, b % B, int(values)]
                    byte = torch.maximum(byte, was.to(byte.dtype))
                unit = two_to(byte - 127)[:, None]
                y = y / unit
                step = two_to(torch.frexp(y.abs().clamp_min(2.0**-6))[1] - 4)
                done.append((torch.round(y / step) * step).clamp(-448, 448) * unit)
        at += n
    return torch.cat(outs[0]), torch.cat(outs[1]), q
