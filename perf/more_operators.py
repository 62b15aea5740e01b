"""Cases, plain forms and work of the operators around a cache held in 4 bits, its pages and the residual stream.

* ``qk_norm_rope_fp4``  RMS norm and rotation of every query and key head, keys and values written to a cache of NVFP4
                        rows, followed by ``kv_gather_fp4``, which reads a chunk's context and its own rows back as the
                        contiguous rows that ``attn_prompt`` takes;
* ``attn_decode_fp4``   one new token per request over that cache, with a prefix that all requests share;
* ``kv_fork``, ``kv_free_pages``, ``kv_compact``  pages of a cache: requests that continue as several, the pages that no
                        request holds, live pages moved to the front of the pool;
* ``block_norm``        the norm behind a block, its gate, its residual scale, the residual and the norm before the next
                        block in one pass.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, where ``own`` is true, by the
calls of ``block_scaled_fp4_group_amd``.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # A few users behind a short instruction: latency is all there is.
        {"name": "decode 8 + 777 x 32/8 x 128", "op": "decode", "requests": 8, "prefix": 777, "longest": 301, "hq": 32,
         "hkv": 8, "dq": 128, "dv": 128, "page": 16, "lens": 7},
        # The 64-token decode batch behind a long system prompt.
        {"name": "decode 64 + 8192 x 64/8 x 128", "op": "decode", "requests": 64, "prefix": 8192, "longest": 2048,
         "hq": 64, "hkv": 8, "dq": 128, "dv": 128, "page": 64, "lens": 8},
        # What a cache of 4 bits is for: many requests with long contexts of their own; wide keys.
        {"name": "decode 48 of 16384 x 64/4 x 192", "op": "decode", "requests": 48, "prefix": 0, "longest": 16384,
         "hq": 64, "hkv": 4, "dq": 192, "dv": 128, "page": 64, "lens": 9},
        # One user with a very long conversation.
        {"name": "decode 1 of 131072 x 32/8 x 128", "op": "decode", "requests": 1, "prefix": 0, "longest": 131072,
         "hq": 32, "hkv": 8, "dq": 128, "dv": 128, "page": 64, "lens": 10},
        # A short question on a conversation: a few tokens written, a few hundred read back.
        {"name": "write 64 + 300 x 32/8 x 128", "op": "write", "requests": 2, "tokens": 64, "context": 300, "hq": 32,
         "hkv": 8, "dq": 128, "dv": 128, "rot": 128, "interleaved": False, "norm": True, "page": 16, "keep_k": False,
         "lens": 1},
        # A batch of prompts of an odd number of tokens, wide key heads of which a third is rotated, adjacent pairs.
        {"name": "write 8191 + 1500 x 64/4 x 192", "op": "write", "requests": 5, "tokens": 8191, "context": 1500,
         "hq": 64, "hkv": 4, "dq": 192, "dv": 128, "rot": 64, "interleaved": True, "norm": True, "page": 64,
         "keep_k": True, "lens": 2},
        # Between the halves of a layer in a decode step: residual and norm.
        {"name": "norm 64 x 4096", "op": "norm", "tokens": 64, "hidden": 4096, "post": False, "gate": "none",
         "scale": 1.0, "residual": True},
        # The same in a prompt batch, with a norm behind the block, a gate for each channel and a residual scale.
        {"name": "norm 8191 x 4096 post gate", "op": "norm", "tokens": 8191, "hidden": 4096, "post": True,
         "gate": "channel", "scale": 0.5, "residual": True},
        # A gate of each token's own, no residual; rows that are no multiple of a wave's.
        {"name": "norm 500 x 1224 token gate", "op": "norm", "tokens": 500, "hidden": 1224, "post": False,
         "gate": "token", "scale": 1.0, "residual": False},
        # Eight conversations that go on in four ways each.
        {"name": "fork 8 to 32 of 2048", "op": "fork", "requests": 64, "parents": 8, "children": 32, "longest": 2048,
         "hkv": 8, "dq": 128, "dv": 128, "page": 64, "fp4": False, "lens": 11},
        # A large pool of small pages after many requests have ended.
        {"name": "free 1500 of 4096", "op": "free", "requests": 1500, "longest": 4096, "page": 16, "ended": 0.3,
         "lens": 12},
        # The pool's live pages moved to its front, so that the rest can be given back.
        {"name": "compact 64 of 4096", "op": "compact", "requests": 64, "longest": 4096, "hkv": 8, "dq": 128, "dv": 128,
         "page": 64, "ended": 0.5, "fp4": True, "lens": 13},
    ]


def draw(rng):
    """One more case of the same ranges; sizes spread over their logarithm."""
    def log(lo, hi):
        return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))

    op = rng.choice(["decode", "decode", "decode", "write", "write", "norm", "norm", "fork", "free", "compact"])
    dq, dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = min(hkv * rng.choice([1, 2, 4, 5, 8, 16]), 64)
    hq -= hq % hkv
    page = rng.choice([16, 32, 64, 128])
    lens = rng.randrange(1, 1 << 30)
    if op == "decode":
        requests = log(1, 96)
        prefix = rng.choice([0, log(1, 4000)])
        longest = log(1, max(300, min(131072, 3000000 // (hkv * (requests + 1)))))
        return {"op": op, "requests": requests, "prefix": prefix, "longest": longest, "hq": hq, "hkv": hkv, "dq": dq,
                "dv": dv, "page": page, "lens": lens}
    if op == "write":
        tokens = log(1, 6000)
        return {"op": op, "requests": min(tokens, log(1, 12)), "tokens": tokens, "context": rng.choice([0, log(1, 1500)]),
                "hq": hq, "hkv": hkv, "dq": dq, "dv": dv, "rot": rng.choice([dq, dq // 64 * 32, 32, 0]),
                "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.8, "page": page,
                "keep_k": rng.random() < 0.5, "lens": lens}
    if op == "norm":
        hidden = 8 * log(8, 1024)
        return {"op": op, "tokens": log(1, min(8191, 6000 * 4096 // hidden)), "hidden": hidden,
                "post": rng.random() < 0.5, "gate": rng.choice(["none", "channel", "token"]),
                "scale": rng.choice([1.0, 0.5, 0.22]), "residual": rng.random() < 0.8}
    if op == "fork":
        parents = log(1, 16)
        children = log(1, 64)
        return {"op": op, "requests": parents + children + rng.randrange(4), "parents": parents, "children": children,
                "longest": log(1, 2048), "hkv": hkv, "dq": dq, "dv": dv, "page": page, "fp4": rng.random() < 0.5,
                "lens": lens}
    if op == "free":
        return {"op": op, "requests": log(1, 1500), "longest": log(1, 4096), "page": page, "ended": rng.uniform(0, 1),
                "lens": lens}
    return {"op": op, "requests": log(1, 24), "longest": log(1, 2048), "hkv": hkv, "dq": dq, "dv": dv, "page": page,
            "ended": rng.uniform(0.1, 0.9), "fp4": rng.random() < 0.5, "lens": lens}


# ------------------------------------------------------------------ lengths
def lengths(case):
    """What the host knows of a batch: the lengths of its requests."""
    r = random.Random(case["lens"])
    n = case["requests"]
    if case["op"] == "write":
        cuts = sorted(r.sample(range(1, case["tokens"]), n - 1)) if n > 1 else []
        new = [b - a for a, b in zip([0] + cuts, cuts + [case["tokens"]])]
        return [r.randint(0, case["context"]) if case["context"] else 0 for _ in range(n)], new
    if case["op"] == "decode":
        s = [case["longest"]] + [r.randint(0 if case["prefix"] else 1, case["longest"]) for _ in range(n - 1)]
        r.shuffle(s)
        return s
    s = [r.randint(1, case["longest"]) for _ in range(n)]
    if case["op"] == "fork":
        # the parents come first, the children hold nothing yet
        return [x if b < case["parents"] or b >= case["parents"] + case["children"] else 0 for b, x in enumerate(s)]
    return s


def ended(case):
    """Which requests of a pool have ended."""
    r = random.Random(case["lens"] + 1)
    return [r.random() < case["ended"] for _ in range(case["requests"])]


def offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def pages(tokens, page):
    return (tokens + page - 1) // page


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=DEV)

    return {"decode": prepare_decode, "write": prepare_write, "norm": prepare_norm, "fork": prepare_fork,
            "free": prepare_free, "compact": prepare_compact}[case["op"]](case, g, normal, ints)


def fp4_rows(g, n, page, heads, dim, blocks_first):
    """Codes and scales of a cache's keys or values: any codes, scales spread as those of values around 1."""
    codes = torch.randint(0, 256, (n, heads, page, dim // 2), generator=g, device=DEV, dtype=torch.uint8)
    shape = (n, heads, dim // 16, page) if blocks_first else (n, heads, page, dim // 16)
    return codes, torch.randint(0x24, 0x34, shape, generator=g, device=DEV, dtype=torch.uint8)


def paged(g, ints, lens, page, blocks, spare):
    """A table whose requests hold pages in any order, and the pages that are left."""
    counts = ints([pages(n, page) for n in lens])
    held = sum(pages(n, page) for n in lens)
    pool = torch.randperm(held + spare, generator=g, device=DEV).to(torch.int32)
    block = torch.arange(blocks, device=DEV)[None, :]
    at = counts.to(torch.int64).cumsum(0)[:, None] - counts[:, None] + block
    table = torch.where(block < counts[:, None], pool[at.clamp(max=held + spare - 1)], -1).to(torch.int32)
    return table.contiguous(), pool[held:].contiguous()


def heads_of(normal, rows, heads, d):
    """Queries: heads look about sharply or widely, so scores spread over 0.5 to 3 standard deviations."""
    x = normal(rows, heads, d).float()
    return (x * torch.linspace(0.5, 3.0, heads, device=DEV)[None, :, None]).to(torch.bfloat16)


def prepare_decode(case, g, normal, ints):
    lens, page, b = lengths(case), case["page"], case["requests"]
    shared = pages(case["prefix"], page)
    table, left = paged(g, ints, lens, page, max(1, pages(case["longest"], page)), shared + 4)
    n = sum(pages(x, page) for x in lens) + shared + 4
    k, ks = fp4_rows(g, n, page, case["hkv"], case["dq"], False)
    v, vs = fp4_rows(g, n, page, case["hkv"], case["dv"], True)
    s = {"case": case, "q": heads_of(normal, b, case["hq"], case["dq"]), "k": k, "ks": ks, "v": v, "vs": vs,
         "table": table, "lens": ints(lens), "prefix_table": left[:shared].contiguous(), "host_lens": lens}
    return with_cache(s)


def with_cache(s, k_global=1.0, v_global=1.0):
    """The handle that a program keeps of its cache (the framework's own where it is there)."""
    s["k_global"], s["v_global"] = k_global, v_global
    if own:
        import block_scaled_fp4_group_amd as moe
        s["cache"] = moe.Fp4Cache(s["k"], s["ks"], s["v"], s["vs"], k_global, v_global)
    return s


def prepare_write(case, g, normal, ints):
    t, hq, hkv, dq, dv, page = (case[n] for n in ("tokens", "hq", "hkv", "dq", "dv", "page"))
    before, new = lengths(case)
    total = [a + b for a, b in zip(before, new)]
    table, _ = paged(g, ints, total, page, max(1, pages(max(total), page)), 4)
    n = sum(pages(x, page) for x in total) + 4
    # a few more rows than tokens: a padded batch, whose last rows have no slot
    pad = t // 97
    rows = normal(t + pad, hq * dq + hkv * dq + hkv * dv)
    longest = 16384
    angle = torch.arange(longest, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / max(case["rot"], 1))
    cu, nt = ints(offsets(new)).to(torch.int64), torch.arange(t, device=DEV)
    b = torch.searchsorted(cu, nt, right=True) - 1
    pos = ints(before).to(torch.int64)[b] + nt - cu[b]
    slots = table.to(torch.int64)[b, pos // page] * page + pos % page
    k, ks = fp4_rows(g, n, page, hkv, dq, False)
    v, vs = fp4_rows(g, n, page, hkv, dv, True)
    s = {"case": case, "q": rows[:, :hq * dq].unflatten(1, (hq, dq)),
         "k_in": rows[:, hq * dq:(hq + hkv) * dq].unflatten(1, (hkv, dq)),
         "v_in": rows[:, (hq + hkv) * dq:].unflatten(1, (hkv, dv)),
         "positions": torch.cat([pos, pos.new_zeros(pad)]).to(torch.int32),
         "slots": torch.cat([slots, slots.new_full((pad,), -1)]).to(torch.int32),
         "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32) if case["rot"] else None,
         "qw": 1 + 0.2 * torch.randn(dq, generator=g, device=DEV) if case["norm"] else None,
         "kw": 1 + 0.2 * torch.randn(dq, generator=g, device=DEV) if case["norm"] else None,
         "k": k, "ks": ks, "v": v, "vs": vs, "table": table, "cu_k": ints(offsets(total)), "total": sum(total)}
    return with_cache(s, 1.0, 0.25)


def prepare_norm(case, g, normal, ints):
    t, h = case["tokens"], case["hidden"]
    gate = None
    if case["gate"] == "channel":
        gate = 0.5 + 0.3 * torch.randn(h, generator=g, device=DEV)
    elif case["gate"] == "token":
        gate = normal(t, h).sigmoid()
    return {"case": case, "x": (normal(t, h).float() * 3).to(torch.bfloat16),
            "residual": (normal(t, h).float() * 5).to(torch.bfloat16) if case["residual"] else None,
            "post": 1 + 0.2 * torch.randn(h, generator=g, device=DEV) if case["post"] else None, "gate": gate,
            "weight": 1 + 0.2 * torch.randn(h, generator=g, device=DEV)}


def buffers_of(case, g, normal, n):
    """A pool of n pages: keys and values in bf16, or their codes and scales in 4 bits."""
    page, hkv, dq, dv = case["page"], case["hkv"], case["dq"], case["dv"]
    if case["fp4"]:
        return [*fp4_rows(g, n, page, hkv, dq, False), *fp4_rows(g, n, page, hkv, dv, True)]
    return [normal(n, page, hkv, dq), normal(n, page, hkv, dv)]


def prepare_fork(case, g, normal, ints):
    lens, page, b, p, c = lengths(case), case["page"], case["requests"], case["parents"], case["children"]
    table, left = paged(g, ints, lens, page, pages(case["longest"], page) + 1, c + 8)
    n = sum(pages(x, page) for x in lens) + c + 8
    return {"case": case, "table": table, "lens": ints(lens), "free": left,
            "parents": torch.randint(0, p, (c,), generator=g, device=DEV).to(torch.int32),
            "children": (p + torch.randperm(c, generator=g, device=DEV)).to(torch.int32),
            "buffers": buffers_of(case, g, normal, n)}


def pool_after(case, g, ints):
    """A pool whose requests have grown together, some of which have ended since: (table, lengths, pages)."""
    lens, page = lengths(case), case["page"]
    table, _ = paged(g, ints, lens, page, pages(case["longest"], page), 16)
    n = sum(pages(x, page) for x in lens) + 16
    return table, ints([0 if gone else x for x, gone in zip(lens, ended(case))]), n


def prepare_free(case, g, normal, ints):
    table, lens, n = pool_after(case, g, ints)
    return {"case": case, "table": table, "lens": lens, "pages": n}


def prepare_compact(case, g, normal, ints):
    table, lens, n = pool_after(case, g, ints)
    return {"case": case, "table": table, "lens": lens, "pages": n, "buffers": buffers_of(case, g, normal, n)}


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"decode": own_decode, "write": own_write, "norm": own_norm, "fork": own_fork, "free": own_free,
                "compact": own_compact}[op](state)
    return {"decode": plain_decode, "write": plain_write, "norm": plain_norm, "fork": plain_fork, "free": plain_free,
            "compact": plain_compact}[op](state)


def own_decode(s):
    import block_scaled_fp4_group_amd as moe
    c = s["case"]
    out, lse = moe.attn_decode_fp4(s["q"], s["cache"], s["table"], s["lens"], c["longest"],
                                   prefix_table=s["prefix_table"], prefix_len=c["prefix"], want_lse=True)
    return {"out": out, "lse": lse}


def own_write(s):
    import block_scaled_fp4_group_amd as moe
    c = s["case"]
    q, k = moe.qk_norm_rope_fp4(s["q"], s["k_in"], s["v_in"], s["positions"], s["cos_sin"], s["cache"], s["slots"],
                                q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, interleaved=c["interleaved"],
                                want_k=c["keep_k"])
    keys, values = moe.kv_gather_fp4(s["cache"], s["table"], s["cu_k"], s["total"])
    return {"q": q, "k": k, "keys": keys, "values": values}


def own_norm(s):
    import block_scaled_fp4_group_amd as moe
    h, y = moe.block_norm(s["x"], s["weight"], residual=s["residual"], post_weight=s["post"], gate=s["gate"],
                          scale=s["case"]["scale"], eps=1e-6)
    return {"h": h, "y": y}


def own_fork(s):
    import block_scaled_fp4_group_amd as moe
    counts = moe.kv_fork(s["table"], s["lens"], s["parents"], s["children"], s["free"], s["case"]["page"], s["buffers"])
    return {"table": s["table"], "lens": s["lens"], "counts": counts, "buffers": s["buffers"]}


def own_free(s):
    import block_scaled_fp4_group_amd as moe
    free, counts = moe.kv_free_pages(s["table"], s["lens"], s["case"]["page"], s["pages"])
    return {"free": free, "counts": counts}


def own_compact(s):
    import block_scaled_fp4_group_amd as moe
    table, counts = moe.kv_compact(s["table"], s["lens"], s["case"]["page"], s["buffers"])
    return {"table": table, "counts": counts, "buffers": s["buffers"]}


# ------------------------------------------------------------------ plain forms
def nibbles(codes):
    """Codes [..., n] -> their values [..., 2 n]: the low nibble first, 8 and up negative."""
    values = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
    c = codes.to(torch.int64)
    return torch.stack([values[c & 15], values[c >> 4]], -1).flatten(-2)


def e4m3(scales):
    return scales.view(torch.float8_e4m3fn).float()


def rows_k(codes, scales, scale):
    """Rows [..., dim / 2] and [..., dim / 16] -> values [..., dim]."""
    return (nibbles(codes).unflatten(-1, (-1, 16)) * e4m3(scales)[..., None]).flatten(-2) * scale


def cache_rows(s, at_page, at_row):
    """Keys and values [rows, heads, dim] at places (page, row in it) of the cache."""
    k = rows_k(s["k"][at_page, :, at_row], s["ks"][at_page, :, at_row], s["k_global"])
    v = rows_k(s["v"][at_page, :, at_row], s["vs"][at_page, :, :, at_row], s["v_global"])
    return k, v


def plain_decode(s):
    c = s["case"]
    hq, hkv, dq, dv, page, b = (c[n] for n in ("hq", "hkv", "dq", "dv", "page", "requests"))
    shared, longest, group = c["prefix"], c["longest"], c["hq"] // c["hkv"]
    q = s["q"].float().unflatten(1, (hkv, group))
    p = torch.arange(shared, device=DEV)
    front_k, front_v = cache_rows(s, s["prefix_table"].to(torch.int64)[p // page], p % page)
    # the shared part: every request's heads against the same rows, at once
    front = torch.matmul(q.permute(1, 0, 2, 3).reshape(hkv, b * group, dq), front_k.permute(1, 2, 0).contiguous())
    front = front.unflatten(1, (b, group)).permute(1, 0, 2, 3) * dq ** -0.5
    out = torch.zeros(b, hkv, group, dv, device=DEV)
    lse = torch.zeros(b, hkv, group, device=DEV)
    w_front = torch.zeros(b, hkv, group, shared, device=DEV)
    for i, n in enumerate(s["host_lens"]):                      # each request's own part
        j = torch.arange(n, device=DEV)
        k, v = cache_rows(s, s["table"][i].to(torch.int64)[j // page], j % page)
        scores = torch.cat([front[i], torch.matmul(q[i], k.permute(1, 2, 0).contiguous()) * dq ** -0.5], -1)
        if scores.shape[-1] == 0:
            lse[i] = -math.inf
            continue
        top = scores.amax(-1, keepdim=True)
        weights = (scores - top).exp()
        total = weights.sum(-1, keepdim=True)
        weights = weights / total
        w_front[i] = weights[..., :shared]
        out[i] = torch.matmul(weights[..., shared:], v.permute(1, 0, 2).contiguous())
        lse[i] = (top + total.log()).squeeze(-1)
    part = torch.matmul(w_front.permute(1, 0, 2, 3).reshape(hkv, b * group, shared), front_v.permute(1, 0, 2).contiguous())
    out = out + part.unflatten(1, (b, group)).permute(1, 0, 2, 3)
    return {"out": out.reshape(b, hq, dv).to(torch.bfloat16), "lse": lse.reshape(b, hq)}


def quantized(x, scale):
    """NVFP4 codes of x [..., dim] float64, 16 values to a scale -> (codes [..., dim / 2], scales [..., dim / 16])."""
    x = x.unflatten(-1, (-1, 16))
    want = (x.abs().amax(-1) / (6.0 * scale)).clamp(max=448.0)
    # to E4M3: a step of 2^(exponent - 3), 2^-9 below 2^-6; round() takes ties to even
    step = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -6))) - 3)
    sv = torch.round(want / step) * step
    s8 = sv.to(torch.float32).to(torch.float8_e4m3fn)
    unit = (s8.to(torch.float64) * scale)[..., None]
    a = x.abs()
    code = torch.zeros_like(a, dtype=torch.int32)
    for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (a >= mid * unit) if i % 2 else (a > mid * unit)   # a tie goes to the even code
    code = torch.where(unit > 0, code + 8 * torch.signbit(x).to(torch.int32), 0).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), s8.view(torch.uint8)


def plain_write(s):
    c = s["case"]
    page, rot = c["page"], c["rot"]
    half = rot // 2
    if rot:
        table = s["cos_sin"][s["positions"].to(torch.int64)][:, None, :]

    def head(x, w, dtype):
        x = x.to(dtype)
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.to(dtype)
        if not rot:
            return x
        cos, sin = table[..., :half].to(dtype), table[..., half:].to(dtype)
        r, rest = x[..., :rot], x[..., rot:]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, rest], -1)

    q, k = head(s["q"], s["qw"], torch.float32), head(s["k_in"], s["kw"], torch.float64)
    t = c["tokens"]
    at = s["slots"][:t].to(torch.int64)
    at_page, at_row = at // page, at % page
    s["k"][at_page, :, at_row], s["ks"][at_page, :, at_row] = quantized(k[:t], s["k_global"])
    s["v"][at_page, :, at_row], s["vs"][at_page, :, :, at_row] = quantized(s["v_in"][:t].double(), s["v_global"])
    j = torch.arange(s["total"], device=DEV)
    cu = s["cu_k"].to(torch.int64)
    b = torch.searchsorted(cu, j, right=True) - 1
    keys, values = cache_rows(s, s["table"].to(torch.int64)[b, (j - cu[b]) // page], (j - cu[b]) % page)
    return {"q": q.to(torch.bfloat16), "k": k.to(torch.bfloat16) if c["keep_k"] else None,
            "keys": keys.to(torch.bfloat16), "values": values.to(torch.bfloat16)}


def plain_norm(s):
    def norm(x, w):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w

    b = s["x"].float()
    if s["post"] is not None:
        b = norm(b, s["post"])
    if s["gate"] is not None:
        b = b * s["gate"].float()
    h = b * s["case"]["scale"]
    if s["residual"] is not None:
        h = s["residual"].float() + h
    return {"h": h.to(torch.bfloat16), "y": norm(h, s["weight"]).to(torch.bfloat16)}


def plain_fork(s):
    page, table, lens, free = s["case"]["page"], s["table"], s["lens"], s["free"]
    parents, children = s["parents"].to(torch.int64), s["children"].to(torch.int64)
    n = lens[parents].to(torch.int64)
    whole = n // page
    part = n % page != 0
    rank = part.to(torch.int64).cumsum(0) - 1
    new = free[rank.clamp(min=0)]
    block = torch.arange(table.shape[1], device=DEV)[None, :]
    rows = torch.where(block < whole[:, None], table[parents], table[children])
    rows = torch.where((block == whole[:, None]) & part[:, None], new[:, None], rows)
    old = table[parents, torch.where(part, whole, 0)].to(torch.int64)
    for x in s["buffers"]:                                      # (without a part of a page: a page onto itself)
        x[torch.where(part, new.to(torch.int64), old)] = x[old]
    table[children] = rows
    lens[children] = lens[parents]
    total = part.sum()
    return {"table": table, "lens": lens, "counts": torch.stack([total, total]).to(torch.int32), "buffers": s["buffers"]}


def live_pages(s):
    """Which pages of the pool the requests hold, and which entries of the table say so."""
    table, page = s["table"], s["case"]["page"]
    held = (s["lens"] + page - 1) // page
    there = torch.arange(table.shape[1], device=DEV)[None, :] < held[:, None]
    live = torch.zeros(s["pages"] + 1, dtype=torch.bool, device=DEV)
    live[torch.where(there, table, s["pages"]).to(torch.int64)] = True
    return live[:-1], there


def plain_free(s):
    live, _ = live_pages(s)
    at = torch.where(live, s["pages"], (~live).to(torch.int64).cumsum(0) - 1)
    free = torch.full((s["pages"] + 1,), -1, dtype=torch.int32, device=DEV)
    free[at] = torch.arange(s["pages"], dtype=torch.int32, device=DEV)
    free[-1] = -1
    n = live.sum()
    return {"free": free[:-1], "counts": torch.stack([s["pages"] - n, n]).to(torch.int32)}


def plain_compact(s):
    live, there = live_pages(s)
    n, p = live.sum(), torch.arange(s["pages"], device=DEV)
    hole, far = ~live & (p < n), live & (p >= n)
    # the i-th live page behind the first n goes to the i-th hole among them
    hole_rank, far_rank = hole.to(torch.int64).cumsum(0) - 1, far.to(torch.int64).cumsum(0) - 1
    spot = torch.full((s["pages"] + 1,), -1, dtype=torch.int64, device=DEV)
    spot[torch.where(hole, hole_rank, s["pages"])] = p
    to = torch.where(far, spot[far_rank.clamp(min=0)], p)
    back = torch.arange(s["pages"] + 1, device=DEV)              # where each page's content comes from
    back[torch.where(far, to, s["pages"])] = p
    back = back[:-1]
    for x in s["buffers"]:
        x.copy_(x[back])
    table = torch.where(there, to[s["table"].to(torch.int64).clamp(min=0)], -1).to(torch.int32)
    return {"table": table, "counts": torch.stack([n, far.sum()]).to(torch.int32), "buffers": s["buffers"]}


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "norm":
        t, h = case["tokens"], case["hidden"]
        rows = 1 + case["residual"] + (case["gate"] == "token")
        vectors = 1 + case["post"] + (case["gate"] == "channel")
        return {"bytes": 2 * t * h * (rows + 2) + 4 * h * vectors, "flops": t * h * (6 + 4 * case["post"])}
    if op == "free":
        lens, page = lengths(case), case["page"]
        n = sum(pages(x, page) for x in lens) + 16
        live = sum(pages(x, page) for x, gone in zip(lens, ended(case)) if not gone)
        return {"bytes": 4 * (len(lens) + live + n + 2), "flops": 0}
    hkv, dq, dv, page = (case[n] for n in ("hkv", "dq", "dv", "page"))
    row = hkv * (dq + dv) * 9 // 16                              # codes and scales
    if op in ("fork", "compact"):
        whole = page * (row if case["fp4"] else 2 * hkv * (dq + dv))
        lens = lengths(case)
        if op == "fork":
            # about as many children as not continue from a page that is not full, and copy it
            c = case["children"]
            blocks = sum(pages(x, page) for x in lens[:case["parents"]]) // case["parents"]
            return {"bytes": 2 * c * whole + 4 * c * (2 * blocks + 5), "flops": 0}
        n = sum(pages(x, page) for x in lens) + 16
        live = sum(pages(x, page) for x, gone in zip(lens, ended(case)) if not gone)
        moved = live * (n - live) // n                           # live pages lie anywhere in the pool
        return {"bytes": 2 * moved * whole + 4 * (len(lens) + 2 * live), "flops": 0}
    hq = case["hq"]
    if op == "write":
        before, new = lengths(case)
        t, total = sum(new), sum(before) + sum(new)
        q, k, v = 2 * t * hq * dq, 2 * t * hkv * dq, 2 * t * hkv * dv
        moved = 2 * q + k + v + (k if case["keep_k"] else 0) + t * (8 + 4 * case["rot"]) + t * row
        context = total * row + 2 * total * hkv * (dq + dv) + 4 * sum(pages(a + b, page) for a, b in zip(before, new))
        return {"bytes": moved + context, "flops": t * (hq + hkv) * (4 * dq + 3 * case["rot"])}
    lens, b = lengths(case), case["requests"]
    rows = case["prefix"] + sum(lens)
    tables = 4 * (pages(case["prefix"], page) + sum(pages(n, page) for n in lens) + b)
    return {"bytes": rows * row + 2 * b * hq * (dq + dv) + 4 * b * hq + tables,
            "flops": 2 * (b * case["prefix"] + sum(lens)) * hq * (dq + dv)}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definition in 64 bits."""
    if case["op"] in ("fork", "free", "compact"):
        return None
    s = prepare(case, seed)
    if case["op"] == "norm":
        return exact_norm(case, s)
    if case["op"] == "write":
        return exact_write(case, s)
    return exact_decode(case, s)


def exact_rows(codes, scales, scale):
    """From the bits: sign, two bits of exponent, one of mantissa; the scale's four and three."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int64)
    e, m = (c >> 1) & 3, (c & 1).double()
    x = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1)) * torch.where(c >= 8, -1.0, 1.0)
    b = scales.to(torch.int64)
    e, m = b >> 3, (b & 7).double()
    unit = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    return x * unit.repeat_interleave(16, -1) * scale


def exact_decode(case, s):
    hq, hkv, dq, dv, page = (case[n] for n in ("hq", "hkv", "dq", "dv", "page"))
    out = torch.zeros(case["requests"], hq, dv, dtype=torch.float64, device=DEV)
    lse = torch.full((case["requests"], hq), -math.inf, dtype=torch.float64, device=DEV)
    p = s["prefix_table"].long()
    front = s["k"][p], s["ks"][p], s["v"][p], s["vs"][p]
    for b, n in enumerate(s["host_lens"]):
        t = s["table"][b, :pages(n, page)].long()
        parts = [(x, m) for x, m in ((front, case["prefix"]), ((s["k"][t], s["ks"][t], s["v"][t], s["vs"][t]), n)) if m]
        for g in range(hkv):
            # a head's whole pages as rows, then as many as there are keys
            k = [exact_rows(x[0][:, g].flatten(0, 1)[:m], x[1][:, g].flatten(0, 1)[:m], 1.0) for x, m in parts]
            v = [exact_rows(x[2][:, g].flatten(0, 1)[:m], x[3][:, g].transpose(1, 2).flatten(0, 1)[:m], 1.0) for x, m in parts]
            if not k:
                continue
            hs = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
            z = s["q"][b, hs].double() @ torch.cat(k).t() / math.sqrt(dq)
            lse[b, hs] = torch.logsumexp(z, 1)
            out[b, hs] = torch.exp(z - lse[b, hs][:, None]) @ torch.cat(v)
    return {"out": out, "lse": lse}


def exact_norm(case, s):
    x = s["x"].double()
    if s["post"] is not None:
        x = s["post"].double() * x / ((x * x).sum(1, keepdim=True) / case["hidden"] + 1e-6).sqrt()
    if s["gate"] is not None:
        x = x * s["gate"].double()
    x = x * float(torch.tensor(case["scale"], dtype=torch.float32))
    if s["residual"] is not None:
        x = x + s["residual"].double()
    return {"h": x, "y": s["weight"].double() * x / ((x * x).sum(1, keepdim=True) / case["hidden"] + 1e-6).sqrt()}


def exact_write(case, s):
    """Each rotated pair as a complex number times the table's cos + i sin; each block's scale and codes as the nearest
    of all there are, the even one of two equally near."""
    rot, page = case["rot"], case["page"]
    if rot:
        turn = s["cos_sin"].double()[s["positions"].long()]
        turn = torch.complex(turn[:, :rot // 2], turn[:, rot // 2:])[:, None]

    def head(x, w):
        x = x.double()
        if w is not None:
            x = w.double() * x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt()
        y = x.clone()
        if rot and case["interleaved"]:
            z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * turn
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        elif rot:
            z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        return y

    def nearest(x, grid):
        """Index of the nearest of the ascending grid to x >= 0."""
        mid = (grid[1:] + grid[:-1]) / 2
        down, up = torch.searchsorted(mid, x), torch.searchsorted(mid, x, right=True)
        return torch.where(up % 2 == 0, up, down)

    units = torch.arange(127, device=DEV)
    e, m = units >> 3, (units & 7).double()
    units = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    steps = torch.tensor(E2M1, dtype=torch.float64, device=DEV)

    def values(x, scale):
        x = x.unflatten(-1, (-1, 16))
        unit = units[nearest(x.abs().amax(-1) / 6 / scale, units)][..., None] * scale
        y = torch.zeros_like(x)
        for i in range(1, 8):
            mid = (steps[i] + steps[i - 1]) / 2 * unit
            y = torch.where((x.abs() > mid) | ((x.abs() == mid) & (i % 2 == 0)), steps[i] * unit, y)
        return (y * torch.where(x < 0, -1.0, 1.0)).flatten(-2)

    q, k = head(s["q"], s["qw"]), head(s["k_in"], s["kw"])
    n = s["k"].shape[0]
    at = s["slots"][:case["tokens"]].long()
    old_k = exact_rows(s["k"], s["ks"], s["k_global"]).transpose(1, 2).reshape(n * page, case["hkv"], -1)
    old_v = exact_rows(s["v"], s["vs"].transpose(2, 3), s["v_global"]).transpose(1, 2).reshape(n * page, case["hkv"], -1)
    old_k[at] = values(k[:case["tokens"]], s["k_global"])
    old_v[at] = values(s["v_in"][:case["tokens"]].double(), s["v_global"])
    cu = s["cu_k"].tolist()
    rows = []
    for b in range(case["requests"]):
        j = torch.arange(cu[b + 1] - cu[b], device=DEV)
        rows.append(s["table"][b].long()[j // page] * page + j % page)
    rows = torch.cat(rows)
    return {"q": q, "k": k if case["keep_k"] else None, "keys": old_k[rows], "values": old_v[rows]}
