"""Workloads of the paged 4-bit key/value cache: its attention, writing tokens into it and keeping its pages.

A cache page holds `page` tokens of one layer: for each key/value head a block of
    K values [page][dim/2] | V values [page/4][dim/8][4][4] | K scales [page/64][16][dim/32][4] | V scales [page/4][dim/32][4]
bytes.  Values are E2M1 numbers, two a byte, the even channel in the low four bits; a scale is a biased power of two (E8M0) for one token
and 32 channels.  K value rows are tokens; a unit of 16 V bytes is 4 tokens of 8 channels; K scale [G][r][b][j] is token 64 G + 16 j + r.
Token i of sequence s is at place kv_len[s] - (q_start[s + 1] - q_start[s]) + i of the sequence.

Head counts are those of the decoder layers the benchmark runs: 32 query and 8 key/value heads (q 4096, k 1024), 40 and 8 (q 5120), 64 and
8 (q 8192), dim 128.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- the cases

def listed():
    a, p, f, r, c = "attention", "append", "fork", "resize", "compact"
    return [
        # one conversation at a context of 512: what a token waits for between q|k|v and o
        attention_case("attention: 1 x 512 tokens, 32/8 heads", 1, 1, 512, 32, 8),
        # a serving batch in mid-flight, contexts from one page to 8K, five query heads to a key head
        attention_case("attention: 48 ragged to 8K, 40/8 heads", 48, 1, 8192, 40, 8),
        # long documents: the cache is far larger than every on-chip memory
        attention_case("attention: 16 ragged to 64K, 64/8 heads", 16, 1, 65536, 64, 8),
        # prompts read in chunks behind what is cached already
        attention_case("attention: 3 prompts of 4K behind 2K, 32/8", 3, 4096, 6144, 32, 8),
        # the new token of every sequence of a serving batch
        {"name": "append: 48 sequences, one token", "op": p, "seqs": 48, "q": 1, "kv": 4096, "kv_heads": 8, "dim": 128, "page": 64},
        # prompts going in
        {"name": "append: 3 prompts of 4K", "op": p, "seqs": 3, "q": 4096, "kv": 6144, "kv_heads": 8, "dim": 128, "page": 64},
        # four answers sampled from one prompt, all 32 layers
        {"name": "fork: 1 prompt into 4, 32 layers", "op": f, "seqs": 8, "parents": 1, "children": 4, "kv": 500, "pages": 64, "layers": 32, "kv_heads": 8, "dim": 128, "page": 64},
        # a search over many prompts
        {"name": "fork: 32 prompts into 7 each, 8 layers", "op": f, "seqs": 256, "parents": 32, "children": 7, "kv": 4000, "pages": 2816, "layers": 8, "kv_heads": 8, "dim": 128, "page": 64},
        # the room for the next tokens of a small batch, finished ones given back
        {"name": "resize: 16 sequences, 1K pages", "op": r, "seqs": 16, "kv": 2048, "pages": 1024, "page": 64},
        # the same for a full machine
        {"name": "resize: 1024 sequences, 128K pages", "op": r, "seqs": 1024, "kv": 6000, "pages": 131072, "page": 64},
        # a small pool, half of it holes
        {"name": "compact: 256 pages, 4 layers", "op": c, "seqs": 8, "kv": 1000, "pages": 256, "layers": 4, "kv_heads": 8, "dim": 128, "page": 64},
        # a pool before it is cut to make room for other weights
        {"name": "compact: 8K pages, 2 layers", "op": c, "seqs": 96, "kv": 4000, "pages": 8192, "layers": 2, "kv_heads": 8, "dim": 128, "page": 64},
    ]


def attention_case(name, seqs, q, kv, heads, kv_heads, dim=128, page=64, window=0):
    c = {"op": "attention", "seqs": seqs, "q": q, "kv": kv, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "window": window}
    return dict(c, name=name) if name else c


def spread(rng, low, high):
    """A whole number between two, its logarithm spread evenly."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("attention", "attention", "attention", "append", "fork", "resize", "compact"))
    dim, page = rng.choice((64, 128, 128)), rng.choice((64, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8))
    if op == "attention":
        group = rng.choice((1, 2, 4, 5, 8))
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
        return {"op": op, "seqs": seqs, "q": q, "kv": q + spread(rng, 1, 4096), "kv_heads": kv_heads, "dim": dim, "page": page}
    if op == "fork":
        parents, children, kv = spread(rng, 1, 32), rng.randint(1, 8), spread(rng, 1, 4000)
        need = parents * (-(-kv // page) + children) + parents * children
        return {"op": op, "seqs": parents * (1 + children) + rng.randint(0, 5), "parents": parents, "children": children, "kv": kv,
                "pages": need + rng.randint(0, 64), "layers": rng.randint(1, 4), "kv_heads": kv_heads, "dim": dim, "page": page}
    if op == "resize":
        seqs, kv = spread(rng, 1, 1024), spread(rng, 2, 6000)
        return {"op": op, "seqs": seqs, "kv": kv, "pages": seqs * (-(-kv * 2 // page) + 1) + rng.randint(0, 999), "page": page}
    seqs, kv = spread(rng, 1, 64), spread(rng, 1, 4000)
    return {"op": op, "seqs": seqs, "kv": kv, "pages": 2 * seqs * -(-kv // page) + rng.randint(0, 99), "layers": rng.randint(1, 3),
            "kv_heads": kv_heads, "dim": dim, "page": page}


def lengths(case):
    """(new tokens, tokens with them) of every sequence: ragged, the same for every seed; the first sequence is the longest."""
    r = random.Random(case["seqs"] * 1000003 + case["kv"])
    q, kv = case["q"], case["kv"]
    new = [q] + [q if q <= 8 else r.randint(max(1, q // 2), q) for _ in range(case["seqs"] - 1)]
    return new, [kv] + [max(n, int(kv * math.exp(r.uniform(math.log(0.15), 0)))) for n in new[1:]]


def block_bytes(case):
    return case["page"] * (case["dim"] // 2 + case["dim"] // 32) * 2


def page_bytes(case):
    return case["kv_heads"] * block_bytes(case)


def visible(n, length, window):
    """Pairs of a query and a key it may look at: query i is at place length - n + i."""
    places = range(max(0, length - n), length)
    if not window:
        return (places.start + 1 + length) * len(places) // 2
    return sum(min(p + 1, window) for p in places)


def work(case):
    if case["op"] in ("attention", "append"):
        new, length = lengths(case)
        T, H, D = sum(new), case["kv_heads"], case["dim"]
        token = 2 * H * (D // 2 + D // 32)  # cached bytes of one token
    if case["op"] == "attention":
        w = case["window"]
        seen = sum(min(n, w + q - 1) if w else n for q, n in zip(new, length))
        pairs = sum(visible(q, n, w) for q, n in zip(new, length))
        return {"bytes": seen * token + T * case["heads"] * (4 * D + 4), "flops": 4 * pairs * case["heads"] * D}
    if case["op"] == "append":  # read and written, and the written values read back
        return {"bytes": 2 * T * 4 * H * D + T * token, "flops": 8 * T * H * D}
    if case["op"] == "resize":
        return {"bytes": 4 * (case["pages"] + 4 * case["seqs"] + case["seqs"] * (-(-case["kv"] // case["page"]))), "flops": case["pages"]}
    if case["op"] == "fork":
        tails = case["parents"] * case["children"] if case["kv"] % case["page"] else 0
        rows = 2 * case["parents"] * case["children"] * -(-case["kv"] // case["page"])
        return {"bytes": 2 * tails * page_bytes(case) * case["layers"] + 4 * (case["pages"] + rows), "flops": case["pages"]}
    used = sum(-(-n // case["page"]) for n in held(case))
    moved = used * (1 - used / case["pages"])  # the used pages behind the first `used` ones, where they lie evenly
    return {"bytes": 2 * moved * page_bytes(case) * case["layers"] + 4 * (2 * case["pages"] + 2 * used), "flops": case["pages"]}


def held(case):
    """Tokens that the sequences of a page-keeping case hold."""
    r = random.Random(case["seqs"] * 1000003 + case["kv"])
    if case["op"] == "fork":  # parents first, then slots with nothing in them
        return [case["kv"]] * case["parents"] + [0] * (case["seqs"] - case["parents"])
    return [case["kv"]] + [max(1, int(case["kv"] * r.uniform(0.3, 1.0))) for _ in range(case["seqs"] - 1)]


# ---------------------------------------------------------------- what a program has in hand

def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def heads_like(shape, g):
    """bf16 activations of heads: normal, with a few channels several times larger than the others, as keys have them."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(shape[-2:], generator=g, device="cuda"))
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g, r = torch.Generator("cuda").manual_seed(seed), random.Random(seed)
    if case["op"] in ("attention", "append"):
        new, length = lengths(case)
        S, T, H, D, page = case["seqs"], sum(new), case["kv_heads"], case["dim"], case["page"]
        columns = -(-max(length) // page)
        counts = [-(-n // page) for n in length]
        pages = sum(counts) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((S, columns), -1, dtype=torch.int32, device="cuda")
        at = torch.arange(columns, device="cuda") < ints(counts)[:, None]
        table[at] = order[: sum(counts)]
        cache = torch.empty((pages, page_bytes(case)), dtype=torch.uint8, device="cuda")
        scale = torch.exp(0.5 * torch.randn((H, 1, D), generator=g, device="cuda"))  # larger channels, the same for all tokens
        few = max(1, (1 << 26) // (H * page * D))
        for p in range(0, pages, few):  # what earlier tokens left in it
            n = min(few, pages - p)
            k, v = (torch.randn((n, H, page, D), generator=g, device="cuda") for _ in range(2))
            cache[p : p + n] = laid_out(*quantized((k * scale).to(torch.bfloat16)), *quantized(v.to(torch.bfloat16)))
        starts = [sum(new[:s]) for s in range(S + 1)]
        s = {"case": case, "cache": cache, "table": table, "kv_len": ints(length), "q_start": ints(starts)}
        # which token of which sequence each row is: the plain form's index, a fused one goes by q_start
        s["seq"] = torch.repeat_interleave(torch.arange(S, device="cuda"), ints(new).long())
        s["place"] = torch.arange(T, device="cuda") - s["q_start"].long()[s["seq"]]
        if case["op"] == "attention":
            s["q"] = heads_like((T, case["heads"], D), g)
            s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((T, case["heads"]), device="cuda")
        else:
            s["k"], s["v"] = heads_like((T, H, D), g), heads_like((T, H, D), g)
            s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        return s
    S, N, page = case["seqs"], case["pages"], case["page"]
    length = held(case)
    counts = [-(-n // page) for n in length]
    columns = -(-2 * max(length) // page) + 1
    ids = list(range(N))
    r.shuffle(ids)
    table, refs, at = torch.full((S, columns), -1, dtype=torch.int32), torch.zeros(N, dtype=torch.int32), 0
    for s, n in enumerate(counts):
        shared = min(n, counts[s - 1]) // 2 if case["op"] != "fork" and s % 4 == 1 else 0  # a prefix in common with the one before
        row = table[s - 1, :shared].tolist() + ids[at : at + n - shared]
        if case["op"] == "resize" and s % 8 == 3 and n == counts[s - 1] and length[s] % page:
            row[-1] = int(table[s - 1, n - 1])  # the last page too: written to, it has to be copied
        at += n - shared
        table[s, :n] = torch.tensor(row, dtype=torch.int32)
        refs.index_add_(0, table[s, :n].long(), torch.ones(n, dtype=torch.int32))
    s = {"case": case}
    # tables, lengths and counts as the scheduler sends them: one buffer
    first = torch.cat([table.reshape(-1), torch.tensor(length, dtype=torch.int32), refs]).cuda()
    s["first"], s["now"] = first, first.clone()
    a, b = table.numel(), table.numel() + S
    s["table"], s["kv_len"], s["refs"] = s["now"][:a].view(S, columns), s["now"][a:b], s["now"][b:]
    s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] != "resize":
        s["cache"] = torch.randint(-(2**31), 2**31 - 1, (case["layers"], N, page_bytes(case) // 4), generator=g, device="cuda", dtype=torch.int32).view(torch.uint8)
    if case["op"] == "fork":
        P, C = case["parents"], case["children"]
        s["parent"], s["child"] = ints([i // C for i in range(P * C)]), ints([P + i for i in range(P * C)])
        s["moves"] = torch.empty((P * C, 2), dtype=torch.int32, device="cuda")
    elif case["op"] == "resize":  # most take a few tokens more, some have ended, some take their draft back
        s["new_len"] = ints([0 if i % 16 == 5 else n // 2 if i % 16 == 9 else n + (i * 7) % (page + 9) for i, n in enumerate(length)])
        s["moves"] = torch.empty((S, 2), dtype=torch.int32, device="cuda")
    else:
        s["moves"] = torch.empty((N // 2 + 1, 2), dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        import bitmask_spmv_amd as nm

        if case["op"] == "attention":
            return nm.nm_kv4_attention(s["q"], s["cache"], s["table"], s["kv_len"], s["q_start"], case["kv_heads"], case["page"], case["q"],
                                       window=case["window"], out=s["out"], lse=s["lse"])
        if case["op"] == "append":
            nm.nm_kv4_append(s["k"], s["v"], s["cache"], s["table"], s["kv_len"], s["q_start"], case["page"])
            return nm.nm_kv4_unpack(s["cache"], s["table"], s["kv_len"], s["q_start"], case["page"], s["k_out"], s["v_out"])
        if case["op"] == "fork":
            # the children's old pages go back first, so another pass gives the same
            nm.nm_kv_fork(s["parent"], s["child"], s["table"], s["kv_len"], s["refs"], case["page"], s["moves"], s["count"])
            nm.nm_kv_copy_pages(s["cache"], s["moves"])
            return s["table"], s["kv_len"], s["refs"], s["moves"], s["count"], s["cache"]
        s["now"].copy_(s["first"])
        if case["op"] == "resize":
            nm.nm_kv_resize(s["new_len"], s["table"], s["kv_len"], s["refs"], case["page"], s["moves"], s["count"])
            return s["table"], s["kv_len"], s["refs"], s["moves"], s["count"]
        nm.nm_kv_compact(s["table"], s["kv_len"], s["refs"], case["page"], s["moves"], s["count"])
        nm.nm_kv_copy_pages(s["cache"], s["moves"])
        return s["table"], s["kv_len"], s["refs"], s["moves"], s["count"], s["cache"]
    if case["op"] == "attention":
        return plain_attention(s)
    if case["op"] == "append":
        return plain_append(s)
    if case["op"] == "fork":
        plain_fork(s)
        plain_copy(s)
        return s["table"], s["kv_len"], s["refs"], s["moves"], s["count"], s["cache"]
    s["now"].copy_(s["first"])
    if case["op"] == "resize":
        plain_resize(s)
        return s["table"], s["kv_len"], s["refs"], s["moves"], s["count"]
    plain_compact(s)
    plain_copy(s)
    return s["table"], s["kv_len"], s["refs"], s["moves"], s["count"], s["cache"]


# ---------------------------------------------------------------- the plain forms

def quantized(x):
    """bf16 [..., D] -> (E2M1 codes uint8 [..., D], scale bytes uint8 [..., D/32])."""
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    top = blocks.abs().amax(-1).view(torch.int16).to(torch.int32)  # exponent and fraction of the largest magnitude
    byte = ((top >> 7) - 2 + ((top & 127) > 96).to(torch.int32)).clamp(16, 252)
    a = blocks.float() * torch.exp2((127 - byte).float())[..., None]
    m = a.abs()  # to nearest, a tie to the even code
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)).to(torch.uint8)
    code |= torch.signbit(a).to(torch.uint8) << 3
    return code.reshape(x.shape), byte.to(torch.uint8)


def laid_out(k, ks, v, vs):
    """Codes [n][H][page][D] and scales [n][H][page][D/32] of whole pages -> bytes [n][page_bytes]."""
    n, H, page, D = k.shape
    k = k[..., ::2] | k[..., 1::2] << 4
    v = (v[..., ::2] | v[..., 1::2] << 4).reshape(n, H, page // 4, 4, D // 8, 4).transpose(3, 4)
    ks = ks.reshape(n, H, page // 64, 4, 16, D // 32).permute(0, 1, 2, 4, 5, 3)
    vs = vs.reshape(n, H, page // 4, 4, D // 32).transpose(3, 4)
    return torch.cat([t.reshape(n, H, -1) for t in (k, v, ks, vs)], -1).reshape(n, -1)


def dequantized(code, byte):
    """Codes [..., D] and scale bytes [..., D/32] -> fp32 [..., D]."""
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=code.device)
    x = torch.index_select(value, 0, code.reshape(-1).to(torch.int32)).view(*byte.shape, 32)
    return (x * torch.exp2(byte.float() - 127)[..., None]).view(code.shape)


def pairs(x):
    """The two codes of every byte, the low one first."""
    return torch.stack([x & 15, x >> 4], -1).flatten(-2)


def cached(s):
    """Keys and values fp32 [S][H][columns * page][D] of every sequence's pages, whatever is in them."""
    case = s["case"]
    H, D, page = case["kv_heads"], case["dim"], case["page"]
    S, columns = s["table"].shape
    x = s["cache"][s["table"].clamp_min(0).long()].view(S, columns, H, -1).transpose(1, 2)
    k, v, ks, vs = x.split([page * D // 2, page * D // 2, page * D // 32, page * D // 32], -1)
    v = v.reshape(S, H, columns, page // 4, D // 8, 4, 4).transpose(4, 5)
    ks = ks.reshape(S, H, columns, page // 64, 16, D // 32, 4).permute(0, 1, 2, 3, 6, 4, 5)
    vs = vs.reshape(S, H, columns, page // 4, D // 32, 4).transpose(4, 5)
    n = columns * page
    k = dequantized(pairs(k.reshape(S, H, n, D // 2)), ks.reshape(S, H, n, D // 32))
    return k, dequantized(pairs(v.reshape(S, H, n, D // 2)), vs.reshape(S, H, n, D // 32))


def plain_attention(s):
    case = s["case"]
    S, Q, H, D = case["seqs"], case["q"], case["kv_heads"], case["dim"]
    group = case["heads"] // H
    k, v = cached(s)
    q = torch.zeros((S, Q, H * group, D), device=k.device)
    q[s["seq"], s["place"]] = s["q"].float()
    q = q.view(S, Q, H, group, D).permute(0, 2, 1, 3, 4).reshape(S, H, Q * group, D)
    x = torch.matmul(q, k.transpose(-1, -2)).view(S, H, Q, group, -1)
    x *= 1 / math.sqrt(D)
    new = s["q_start"][1:] - s["q_start"][:-1]
    at = (s["kv_len"] - new)[:, None, None] + torch.arange(Q, device=k.device)[:, None]  # place of every query
    key = torch.arange(k.shape[2], device=k.device)
    seen = (key <= at) & ((key > at - case["window"]) if case["window"] else True)
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    x.sub_(top).exp_()
    total = x.sum(-1)
    o = torch.matmul(x.view(S, H, Q * group, -1), v).view(S, H, Q, group, D) / torch.where(total == 0, 1.0, total)[..., None]
    lse = top[..., 0] + total.log()
    o, lse = o.permute(0, 2, 1, 3, 4).reshape(S, Q, -1, D), lse.permute(0, 2, 1, 3).reshape(S, Q, -1)
    return o[s["seq"], s["place"]].to(torch.bfloat16), lse[s["seq"], s["place"]]


def plain_append(s):
    case = s["case"]
    H, D, page = case["kv_heads"], case["dim"], case["page"]
    new = s["q_start"][1:] - s["q_start"][:-1]
    at = (s["kv_len"] - new).long()[s["seq"]] + s["place"]
    where, t = s["table"][s["seq"], at // page].long()[:, None], (at % page)[:, None]
    h = torch.arange(H, device=t.device)
    x = s["cache"].view(s["cache"].shape[0], H, -1)
    k, v, ks, vs = x.split([page * D // 2, page * D // 2, page * D // 32, page * D // 32], -1)
    k = k.unflatten(-1, (page, D // 2))
    v = v.unflatten(-1, (page // 4, D // 8, 4, 4))
    ks = ks.unflatten(-1, (page // 64, 16, D // 32, 4))
    vs = vs.unflatten(-1, (page // 4, D // 32, 4))
    (kc, kb), (vc, vb) = quantized(s["k"]), quantized(s["v"])
    k[where, h, t] = kc[..., ::2] | kc[..., 1::2] << 4
    v[where, h, t // 4, :, t % 4] = (vc[..., ::2] | vc[..., 1::2] << 4).view(-1, H, D // 8, 4)
    ks[where, h, t // 64, t % 16, :, t % 64 // 16] = kb
    vs[where, h, t // 4, :, t % 4] = vb
    # what the cache now holds for these tokens
    kn = dequantized(pairs(k[where, h, t]), ks[where, h, t // 64, t % 16, :, t % 64 // 16])
    vn = dequantized(pairs(v[where, h, t // 4, :, t % 4].flatten(-2)), vs[where, h, t // 4, :, t % 4])
    return kn.to(torch.bfloat16), vn.to(torch.bfloat16)


def released(rows, keep, have, refs):
    """Gives back the pages of table rows between `keep` and `have`; the rows without them."""
    column = torch.arange(rows.shape[1], device=rows.device)
    gone = (column >= keep[:, None]) & (column < have[:, None])
    refs.index_add_(0, rows.clamp_min(0).flatten().long(), -gone.flatten().to(torch.int32))
    return torch.where(gone, -1, rows)


def free_pages(refs):
    """Free pages, lowest first, and how many there are."""
    at = torch.arange(refs.shape[0], dtype=torch.int32, device=refs.device)
    free = refs <= 0
    return torch.where(free, at, refs.shape[0]).sort().values, free.sum()


def plain_fork(s):
    page, table, kv_len, refs = s["case"]["page"], s["table"], s["kv_len"], s["refs"]
    parent, child = s["parent"].long(), s["child"].long()
    table[child] = released(table[child], torch.zeros_like(child), (kv_len[child] + page - 1) // page, refs)
    length = kv_len[parent]
    full, part = length // page, (length % page > 0).to(torch.int32)
    ids, count = free_pages(refs)
    rank = part.cumsum(0)
    ok = (part == 0) | (rank <= count)
    part = (part > 0) & ok
    fresh = ids[(rank - 1).clamp_min(0)].clamp_max(refs.shape[0] - 1)
    column = torch.arange(table.shape[1], device=table.device)
    rows = table[parent]
    share = (column < full[:, None]) & ok[:, None]
    refs.index_add_(0, rows.clamp_min(0).flatten().long(), share.flatten().to(torch.int32))
    refs.index_add_(0, fresh.long(), part.to(torch.int32))
    tail = rows.gather(1, full.long().clamp_max(table.shape[1] - 1)[:, None])[:, 0]
    table[child] = torch.where(share, rows, torch.where((column == full[:, None]) & part[:, None], fresh[:, None], -1))
    kv_len[child] = torch.where(ok, length, 0)
    s["moves"].copy_(torch.where(part[:, None], torch.stack([tail, fresh], 1), -1))
    s["count"].copy_((rank[-1:] - count).clamp_min(0))


def plain_resize(s):
    page, table, kv_len, refs, new = s["case"]["page"], s["table"], s["kv_len"], s["refs"], s["new_len"]
    have, want = (kv_len + page - 1) // page, (new + page - 1) // page
    table.copy_(released(table, want, have, refs))
    last = table.gather(1, (have - 1).clamp_min(0).long()[:, None])[:, 0]
    copied = (new > kv_len) & (kv_len % page > 0) & (refs[last.clamp_min(0).long()] > 1)
    ids, count = free_pages(refs)
    first = torch.where(copied, have - 1, have)  # the first column that gets a new page
    need = (want - first).clamp_min(0)
    rank = need.cumsum(0)
    ok = (need == 0) | (rank <= count)
    column = torch.arange(table.shape[1], device=table.device)
    fill = (column >= first[:, None]) & (column < want[:, None]) & ok[:, None]
    fresh = ids[((rank - need)[:, None] + column - first[:, None]).clamp(0, refs.shape[0] - 1)].clamp_max(refs.shape[0] - 1)
    copied &= ok
    refs.index_add_(0, fresh.flatten().long(), fill.flatten().to(torch.int32))
    refs.index_add_(0, last.clamp_min(0).long(), -copied.to(torch.int32))
    table.copy_(torch.where(fill, fresh, table))
    to = table.gather(1, (have - 1).clamp_min(0).long()[:, None])[:, 0]
    s["moves"].copy_(torch.where(copied[:, None], torch.stack([last, to], 1), -1))
    kv_len.copy_(torch.where(ok, new, kv_len))
    s["count"].copy_((rank[-1:] - count).clamp_min(0))


def plain_compact(s):
    page, table, refs, moves = s["case"]["page"], s["table"], s["refs"], s["moves"]
    N, most = refs.shape[0], moves.shape[0]
    at = torch.arange(N, dtype=torch.int32, device=refs.device)
    used = refs > 0
    count = used.sum()
    hole, mover = ~used & (at < count), used & (at >= count)
    to = torch.where(hole, at, N).sort().values[:most]
    of = torch.where(mover, at, N).sort().values[:most]
    moves.copy_(torch.where((of < N)[:, None], torch.stack([of, to], 1), -1))
    new = torch.cat([at, at[:1]])  # where every page goes; one place more for the moves that are none
    new[of.long()] = to
    new = new[:N]
    column = torch.arange(table.shape[1], device=table.device)
    have = column < ((s["kv_len"] + page - 1) // page)[:, None]
    table.copy_(torch.where(have, new[table.clamp_min(0).long()], table))
    left = torch.cat([refs, refs[:1]])
    left[to.long()] = torch.cat([refs, refs[:1]])[of.long()]
    left[of.long()] = 0
    refs.copy_(left[:N])
    s["count"].copy_(count[None])  # this operator says here how many pages are used


def plain_copy(s):
    moves = s["moves"][s["moves"][:, 0] >= 0].long()
    s["cache"][:, moves[:, 1]] = s["cache"][:, moves[:, 0]]


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    if case["op"] not in ("attention", "append"):
        return None  # whole numbers only
    s = prepare(case, seed)
    new, length = lengths(case)
    if case["op"] == "append":
        return exact_rounded(s["k"]), exact_rounded(s["v"])
    H, D, page, w = case["kv_heads"], case["dim"], case["page"], case["window"]
    group, out, lse, at = case["heads"] // H, [], [], 0
    for i, (n, length) in enumerate(zip(new, length)):
        q = s["q"][at : at + n].double() / math.sqrt(D)
        at += n
        place = torch.arange(length, device="cuda")
        rows = s["table"][i].long()[place // page]
        outs, sums = [], []
        for h in range(H):
            k, v = (exact_values(s["cache"], rows, place % page, h, case, values) for values in (False, True))
            x = torch.einsum("nge,ke->gnk", q[:, h * group : (h + 1) * group], k)
            behind = (length - n + torch.arange(n, device="cuda"))[:, None] - place
            x[:, (behind < 0) | ((behind >= w) if w else False)] = -math.inf
            total = torch.logsumexp(x, -1)
            outs.append(torch.einsum("gnk,ke->nge", torch.exp(x - total[..., None]), v))
            sums.append(total.T)
        out.append(torch.cat(outs, 1))
        lse.append(torch.cat(sums, 1))
    return torch.cat(out), torch.cat(lse)


def exact_values(cache, rows, t, h, case, values):
    """fp64 [tokens][D] of one head, byte by byte from where the format puts them."""
    D, page = case["dim"], case["page"]
    c = torch.arange(D, device="cuda")
    t, base = t[:, None], h * block_bytes(case)
    if values:
        byte = page * D // 2 + ((t // 4 * (D // 8) + c // 8) * 4 + t % 4) * 4 + c % 8 // 2
        scale = page * D + page * D // 32 + (t // 4 * (D // 32) + c // 32) * 4 + t % 4
    else:
        byte = t * (D // 2) + c // 2
        scale = page * D + ((t // 64 * 16 + t % 16) * (D // 32) + c // 32) * 4 + t % 64 // 16
    x, e = cache[rows[:, None], base + byte].int(), cache[rows[:, None], base + scale].double()
    x = x >> (4 * (c % 2)) & 15
    two = x >> 1 & 3  # exponent field
    m = torch.where(two == 0, 0.5 * (x & 1), (2 + (x & 1)) * 2.0 ** (two - 2))
    return torch.where(x > 7, -m, m).double() * 2.0 ** (e - 127)


def exact_rounded(x):
    """bf16 [T][H][D] as the cache holds it: the nearest E2M1 multiple of each block's power of two."""
    b = x.double().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1)
    byte = torch.where(top > 0, e - 1 - 2 + (m > 0.875) + 127, 0).clamp(16, 252)
    y = b * 2.0 ** (127 - byte).double()
    step = 2.0 ** (torch.frexp(y.abs().clamp_min(1.0))[1] - 2).double()
    return ((torch.round(y / step) * step).clamp(-6, 6) * 2.0 ** (byte - 127).double()).flatten(-2)
