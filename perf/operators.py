"""Cases, plain forms and work of the attention operators that sit beside the routed-expert layer.

Four operators make up the attention half of a decoder layer whose other half is ``MoELayer``:

* ``kv_slots``      block tables and cache slots of the new tokens, built on the GPU from the request lengths;
* ``qk_norm_rope``  RMS norm of every query and key head, the position rotation and the cache write in one pass;
* ``attn_prompt``   causal attention over whole prompts, grouped heads, packed sequences;
* ``attn_decode``   one new token per request over a paged cache, with a prefix that all requests share.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, where ``own`` is true, by the
calls of ``block_scaled_fp4_group_amd``.
"""
import math
import random

import torch

own = False

DEV = "cuda"
# What the widest plain form holds at once: the scores of one 16384-token prompt with 32 heads.
MOST_SCORES = 32 * 16384 * 16384
MOST_PROMPT_FLOPS = 32 * (16384 * 16385 // 2) * 2 * (128 + 128)


def listed():
    return [
        # One decode step of a full serving batch: every request appends one token; latency is all there is.
        {"name": "slots 64 decode", "op": "slots", "requests": 64, "page": 64, "cached": 8192, "new": 1, "table": 160,
         "lens": 1},
        # A large mixed step: prompts that enter and requests that decode, small pages, a pool handed out in order.
        {"name": "slots 1500 mixed", "op": "slots", "requests": 1500, "page": 16, "cached": 4096, "new": 700,
         "table": 400, "lens": 2},
        # The decode batch of the layer's 64-token workload.
        {"name": "rope 64 x 32/8 x 128", "op": "rope", "tokens": 64, "hq": 32, "hkv": 8, "dq": 128, "dv": 128,
         "rot": 128, "interleaved": False, "norm": True, "page": 64, "keep_k": False},
        # A prompt batch of an odd length, wide key heads of which a third is rotated, adjacent pairs.
        {"name": "rope 8191 x 64/4 x 192", "op": "rope", "tokens": 8191, "hq": 64, "hkv": 4, "dq": 192, "dv": 128,
         "rot": 64, "interleaved": True, "norm": True, "page": 16, "keep_k": True},
        # The smallest prompt in earnest: a short question, small heads; latency counts.
        {"name": "prompt 129 x 16/2 x 64", "op": "prompt", "requests": 1, "longest": 129, "context": 0, "hq": 16,
         "hkv": 2, "dq": 64, "dv": 64, "lens": 3},
        # Prompts of very different lengths packed into one batch.
        {"name": "prompt 32 ragged x 32/8 x 128", "op": "prompt", "requests": 32, "longest": 2048, "context": 0,
         "hq": 32, "hkv": 8, "dq": 128, "dv": 128, "lens": 4},
        # Prompts whose first part was answered before: more keys than queries; 192-wide keys, 128-wide values.
        {"name": "prompt 3 + context x 64/4 x 192", "op": "prompt", "requests": 3, "longest": 3500, "context": 1500,
         "hq": 64, "hkv": 4, "dq": 192, "dv": 128, "lens": 5},
        # One long document.
        {"name": "prompt 16384 x 32/4 x 128", "op": "prompt", "requests": 1, "longest": 16384, "context": 0, "hq": 32,
         "hkv": 4, "dq": 128, "dv": 128, "lens": 6},
        # A few users behind a short instruction.
        {"name": "decode 8 + 777 x 32/8 x 128", "op": "decode", "requests": 8, "prefix": 777, "longest": 301,
         "hq": 32, "hkv": 8, "dq": 128, "dv": 128, "page": 16, "lens": 7},
        # The 64-token decode batch behind a long system prompt.
        {"name": "decode 64 + 8192 x 64/8 x 128", "op": "decode", "requests": 64, "prefix": 8192, "longest": 2048,
         "hq": 64, "hkv": 8, "dq": 128, "dv": 128, "page": 64, "lens": 8},
        # Many questions about one long document: nearly all keys are shared; wide keys.
        {"name": "decode 96 + 32768 x 64/4 x 192", "op": "decode", "requests": 96, "prefix": 32768, "longest": 500,
         "hq": 64, "hkv": 4, "dq": 192, "dv": 128, "page": 64, "lens": 9},
        # One user with a very long conversation and nothing shared.
        {"name": "decode 1 of 131072 x 32/8 x 128", "op": "decode", "requests": 1, "prefix": 0, "longest": 131072,
         "hq": 32, "hkv": 8, "dq": 128, "dv": 128, "page": 64, "lens": 10},
    ]


def draw(rng):
    """One more case of the same ranges; sizes spread over their logarithm."""
    def log(lo, hi):
        return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))

    op = rng.choice(["slots", "rope", "prompt", "prompt", "decode", "decode"])
    dq, dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8, 16])
    lens = rng.randrange(1, 1 << 30)
    if op == "slots":
        page = rng.choice([16, 32, 64, 128])
        cached, new = log(1, 8192), log(1, 700)
        return {"op": op, "requests": log(1, 1500), "page": page, "cached": cached, "new": new,
                "table": (cached + new + page - 1) // page + 1, "lens": lens}
    if op == "rope":
        hq = min(hq, 64)
        return {"op": op, "tokens": log(1, 7000), "hq": hq - hq % hkv, "hkv": hkv, "dq": dq, "dv": dv,
                "rot": rng.choice([dq, dq // 2, 32]), "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.8,
                "page": rng.choice([16, 64]), "keep_k": rng.random() < 0.5}
    if op == "prompt":
        hq = min(hq, 64)
        hq -= hq % hkv
        longest = log(1, 16384 if hq <= 32 and dq <= 128 else 6000)
        context = rng.choice([0, 0, log(1, 2000)])
        most = MOST_SCORES // (hq * longest * (longest + context))
        return {"op": op, "requests": log(1, max(1, min(48, most, 40000 // longest + 1))), "longest": longest,
                "context": context, "hq": hq, "hkv": hkv, "dq": dq, "dv": dv, "lens": lens}
    hq = min(hq, 64)
    hq -= hq % hkv
    requests = log(1, 96)
    prefix = rng.choice([0, log(1, 32768)])
    longest = log(1, max(300, (131072 - 2 * prefix) // requests))
    return {"op": op, "requests": requests, "prefix": prefix, "longest": longest, "hq": hq, "hkv": hkv, "dq": dq,
            "dv": dv, "page": rng.choice([16, 32, 64, 128]), "lens": lens}


# ------------------------------------------------------------------ lengths
def lengths(case):
    """What the host knows of a batch: the lengths of its requests, the longest first drawn and then shuffled."""
    r = random.Random(case["lens"])
    n = case["requests"]
    if case["op"] == "slots":
        cached = [r.randint(0, case["cached"]) for _ in range(n)]
        if case["new"] == 1:
            return cached, [1] * n
        # half of the requests decode one token, the others bring a prompt; some bring nothing
        return cached, [r.choice([1, 1, 0, r.randint(1, case["new"])]) for _ in range(n)]
    if case["op"] == "prompt":
        q = [case["longest"]] + [max(1, int(case["longest"] ** r.uniform(0.4, 1.0))) for _ in range(n - 1)]
        r.shuffle(q)
        c = [r.randint(0, case["context"]) if case["context"] else 0 for _ in range(n)]
        return q, [a + b for a, b in zip(q, c)]
    s = [case["longest"]] + [r.randint(0 if case["prefix"] else 1, case["longest"]) for _ in range(n - 1)]
    r.shuffle(s)
    return s


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

    return {"slots": prepare_slots, "rope": prepare_rope, "prompt": prepare_prompt, "decode": prepare_decode}[
        case["op"]](case, g, normal, ints)


def prepare_slots(case, g, normal, ints):
    cached, new = lengths(case)
    page = case["page"]
    held = [pages(c, page) for c in cached]
    need = sum(pages(c + n, page) - h for c, n, h in zip(cached, new, held))
    # the pool: pages in any order; the requests hold some, the free list the others (with a few to spare)
    pool = torch.randperm(sum(held) + need + 32, generator=g, device=DEV).to(torch.int32)
    ends = ints(held).to(torch.int64).cumsum(0)
    block = torch.arange(case["table"], device=DEV)[None, :]
    at = ends[:, None] - ints(held)[:, None] + block
    table = torch.where(block < ints(held)[:, None], pool[at.clamp(max=pool.numel() - 1)], -1).to(torch.int32)
    return {"case": case, "cached": ints(cached), "new": ints(new), "table": table.contiguous(),
            "free": pool[sum(held):].contiguous(), "most": max(1, sum(new))}


def prepare_rope(case, g, normal, ints):
    t, hq, hkv, dq, dv, page = (case[n] for n in ("tokens", "hq", "hkv", "dq", "dv", "page"))
    # the projection's output: one row per token, the query, key and value heads side by side
    rows = normal(t, hq * dq + hkv * dq + hkv * dv)
    longest = 16384
    angle = torch.arange(longest, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
    slots_there = (pages(t, page) + 8) * page
    slots = torch.randperm(slots_there, generator=g, device=DEV)[:t].to(torch.int32)
    if t > 97:
        slots[::97] = -1  # tokens of a padded batch have no slot
    # a row behind each cache takes what the plain form writes for tokens without a slot
    k_rows, v_rows = normal(slots_there + 1, hkv, dq), normal(slots_there + 1, hkv, dv)
    return {"case": case, "q": rows[:, :hq * dq].unflatten(1, (hq, dq)),
            "k": rows[:, hq * dq:(hq + hkv) * dq].unflatten(1, (hkv, dq)),
            "v": rows[:, (hq + hkv) * dq:].unflatten(1, (hkv, dv)),
            "positions": torch.randint(0, longest, (t,), generator=g, device=DEV, dtype=torch.int32), "slots": slots,
            "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32),
            "qw": 1 + 0.2 * torch.randn(dq, generator=g, device=DEV) if case["norm"] else None,
            "kw": 1 + 0.2 * torch.randn(dq, generator=g, device=DEV) if case["norm"] else None,
            "k_rows": k_rows, "v_rows": v_rows, "k_cache": k_rows[:-1].unflatten(0, (-1, page)),
            "v_cache": v_rows[:-1].unflatten(0, (-1, page))}


def heads_of(normal, rows, heads, d):
    """Queries: heads look about sharply or widely, so scores spread over 0.5 to 3 standard deviations."""
    x = normal(rows, heads, d).float()
    return (x * torch.linspace(0.5, 3.0, heads, device=DEV)[None, :, None]).to(torch.bfloat16)


def prepare_prompt(case, g, normal, ints):
    lq, lk = lengths(case)
    return {"case": case, "q": heads_of(normal, sum(lq), case["hq"], case["dq"]),
            "k": normal(sum(lk), case["hkv"], case["dq"]), "v": normal(sum(lk), case["hkv"], case["dv"]),
            "cu_q": ints(offsets(lq)), "cu_k": ints(offsets(lk)), "max_q": max(lq), "max_k": max(lk)}


def prepare_decode(case, g, normal, ints):
    lens, page, b = lengths(case), case["page"], case["requests"]
    blocks = max(1, pages(case["longest"], page))
    shared = pages(case["prefix"], page)
    held = sum(pages(n, page) for n in lens)
    pool = torch.randperm(held + shared + 4, generator=g, device=DEV).to(torch.int32)
    counts = ints([pages(n, page) for n in lens])
    block = torch.arange(blocks, device=DEV)[None, :]
    at = counts.to(torch.int64).cumsum(0)[:, None] - counts[:, None] + block
    table = torch.where(block < counts[:, None], pool[at.clamp(max=held + shared + 3)], -1).to(torch.int32)
    n = pool.numel()
    return {"case": case, "q": heads_of(normal, b, case["hq"], case["dq"]),
            "k_cache": normal(n, page, case["hkv"], case["dq"]), "v_cache": normal(n, page, case["hkv"], case["dv"]),
            "table": table.contiguous(), "lens": ints(lens), "prefix_table": pool[held:held + shared].contiguous(),
            "host_lens": lens}


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"slots": own_slots, "rope": own_rope, "prompt": own_prompt, "decode": own_decode}[op](state)
    return {"slots": plain_slots, "rope": plain_rope, "prompt": plain_prompt, "decode": plain_decode}[op](state)


def own_slots(s):
    import block_scaled_fp4_group_amd as moe
    table = s["table"]
    slots, positions, cu, counts = moe.kv_slots(s["cached"], s["new"], s["free"], table, s["case"]["page"], s["most"])
    return {"table": table, "slots": slots, "positions": positions, "cu": cu, "counts": counts}


def own_rope(s):
    import block_scaled_fp4_group_amd as moe
    c = s["case"]
    q, k = moe.qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
                            interleaved=c["interleaved"], v=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"],
                            slots=s["slots"], want_k=c["keep_k"])
    return {"q": q, "k": k, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def own_prompt(s):
    import block_scaled_fp4_group_amd as moe
    out, lse = moe.attn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], want_lse=True)
    return {"out": out, "lse": lse}


def own_decode(s):
    import block_scaled_fp4_group_amd as moe
    c = s["case"]
    out, lse = moe.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], c["longest"],
                               prefix_table=s["prefix_table"], prefix_len=c["prefix"], want_lse=True)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ plain forms
def plain_slots(s):
    page, table, cached, free = s["case"]["page"], s["table"], s["cached"], s["free"]
    n, c = s["new"].to(torch.int64), cached.to(torch.int64)
    cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
    held = (c + page - 1) // page
    need = (c + n + page - 1) // page - held
    first = need.cumsum(0) - need
    block = torch.arange(table.shape[1], device=DEV)[None, :]
    at = first[:, None] + block - held[:, None]
    fresh = (block >= held[:, None]) & (block < (held + need)[:, None])
    table = torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table)
    t = torch.arange(s["most"], device=DEV)
    real = t < cu[-1]
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=c.numel() - 1)
    pos = c[b] + t - cu[b]
    slot = table[b, (pos // page).clamp(max=table.shape[1] - 1)].to(torch.int64) * page + pos % page
    total = need.sum()
    return {"table": table, "slots": torch.where(real, slot, -1).to(torch.int32),
            "positions": torch.where(real, pos, 0).to(torch.int32), "cu": cu.to(torch.int32),
            "counts": torch.stack([total, total, torch.zeros_like(total)]).to(torch.int32)}


def plain_rope(s):
    c = s["case"]
    half = c["rot"] // 2
    table = s["cos_sin"][s["positions"].to(torch.int64)][:, None, :]
    cos, sin = table[..., :half], table[..., half:]

    def head(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, rest], -1).to(torch.bfloat16)

    q, k = head(s["q"], s["qw"]), head(s["k"], s["kw"])
    at = s["slots"].to(torch.int64)
    at = torch.where(at < 0, s["k_rows"].shape[0] - 1, at)
    s["k_rows"][at] = k
    s["v_rows"][at] = s["v"]
    return {"q": q, "k": k if c["keep_k"] else None, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def softmax_values(scores, allowed, v):
    """Weights of the allowed places and their sum of v: (out, log of the sum of exponentials); a row without any: 0, -inf."""
    scores.masked_fill_(~allowed, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    out = torch.matmul(weights, v) / torch.where(total == 0, 1.0, total)
    return out, (top + total.log()).squeeze(-1)


def plain_prompt(s):
    c = s["case"]
    hq, hkv, dq, dv = c["hq"], c["hkv"], c["dq"], c["dv"]
    cu_q, cu_k = s["cu_q"].to(torch.int64), s["cu_k"].to(torch.int64)
    b, group, mq, mk = cu_q.numel() - 1, hq // hkv, s["max_q"], s["max_k"]
    i, j = torch.arange(mq, device=DEV), torch.arange(mk, device=DEV)
    lq, lk = cu_q.diff()[:, None], cu_k.diff()[:, None]
    q = s["q"].float()[(cu_q[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)]
    rows_k = (cu_k[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    k, v = s["k"].float()[rows_k], s["v"].float()[rows_k]
    q = q.unflatten(2, (hkv, group)).permute(0, 2, 3, 1, 4).reshape(b, hkv, group * mq, dq)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(dq ** -0.5).unflatten(2, (group, mq))
    allowed = (j[None, None, :] <= (i[None, :] + lk - lq)[:, :, None]) & (j[None, :] < lk)[:, None, :]
    out, lse = softmax_values(scores, allowed[:, None, None], v.permute(0, 2, 1, 3)[:, :, None])
    t = torch.arange(s["q"].shape[0], device=DEV)
    at = torch.searchsorted(cu_q, t, right=True) - 1
    out = out.permute(0, 3, 1, 2, 4)[at, t - cu_q[at]]
    lse = lse.permute(0, 3, 1, 2)[at, t - cu_q[at]]
    return {"out": out.reshape(-1, hq, dv).to(torch.bfloat16), "lse": lse.reshape(-1, hq)}


def plain_decode(s):
    c = s["case"]
    hq, hkv, dq, dv, page, b = (c[n] for n in ("hq", "hkv", "dq", "dv", "page", "requests"))
    shared, longest, group = c["prefix"], c["longest"], c["hq"] // c["hkv"]
    j = torch.arange(longest, device=DEV)
    pages_of = s["table"].to(torch.int64)[:, j // page].clamp(min=0)
    own_rows = pages_of * page + j % page
    p = torch.arange(shared, device=DEV)
    shared_rows = s["prefix_table"].to(torch.int64)[p // page] * page + p % page
    k_rows, v_rows = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    q = s["q"].float().unflatten(1, (hkv, group))
    # the shared part: every request's heads against the same rows, at once
    front = torch.matmul(q.permute(1, 0, 2, 3).reshape(hkv, b * group, dq), k_rows[shared_rows].float().permute(1, 2, 0))
    front = front.unflatten(1, (b, group)).permute(1, 0, 2, 3)
    # each request's own part
    back = torch.matmul(q, k_rows[own_rows].float().permute(0, 2, 3, 1))
    scores = torch.cat([front, back], -1).mul_(dq ** -0.5)
    there = torch.cat([p.new_ones(b, shared, dtype=torch.bool), j[None, :] < s["lens"][:, None]], 1)[:, None, None]
    scores.masked_fill_(~there, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    w_front = weights[..., :shared].permute(1, 0, 2, 3).reshape(hkv, b * group, shared)
    out = torch.matmul(w_front, v_rows[shared_rows].float().permute(1, 0, 2)).unflatten(1, (b, group)).permute(1, 0, 2, 3)
    out = out + torch.matmul(weights[..., shared:], v_rows[own_rows].float().permute(0, 2, 1, 3))
    out = out / torch.where(total == 0, 1.0, total)
    return {"out": out.reshape(b, hq, dv).to(torch.bfloat16), "lse": (top + total.log()).reshape(b, hq)}


# ------------------------------------------------------------------ work
def work(case):
    if case["op"] == "slots":
        cached, new = lengths(case)
        page = case["page"]
        fresh = sum(pages(c + n, page) - pages(c, page) for c, n in zip(cached, new))
        # lengths in, offsets out; a slot and a position for each token; each new page read from the pool and written
        # to the table, the last page held read where it has room
        held = sum(1 for c, n in zip(cached, new) if n and c % page)
        return {"bytes": 4 * (3 * len(new) + 1 + 2 * sum(new) + 2 * fresh + held + 3), "flops": 0}
    if case["op"] == "rope":
        t, hq, hkv, dq, dv = (case[n] for n in ("tokens", "hq", "hkv", "dq", "dv"))
        q, k, v = t * hq * dq * 2, t * hkv * dq * 2, t * hkv * dv * 2
        weights = 8 * dq if case["norm"] else 0
        return {"bytes": 2 * (q + k + v) + (k if case["keep_k"] else 0) + t * (8 + 4 * case["rot"]) + weights,
                "flops": t * (hq + hkv) * (4 * dq + 3 * case["rot"])}
    hq, hkv, dq, dv = (case[n] for n in ("hq", "hkv", "dq", "dv"))
    if case["op"] == "prompt":
        lq, lk = lengths(case)
        # row i of a prompt sees its lk - lq + i + 1 keys
        pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(lq, lk))
        moved = 2 * (sum(lq) * hq * (dq + dv) + sum(lk) * hkv * (dq + dv)) + 4 * sum(lq) * hq + 8 * (len(lq) + 1)
        return {"bytes": moved, "flops": 2 * pairs * hq * (dq + dv)}
    lens, b = lengths(case), case["requests"]
    rows = case["prefix"] + sum(lens)
    tables = 4 * (pages(case["prefix"], case["page"]) + sum(pages(n, case["page"]) for n in lens) + b)
    return {"bytes": 2 * rows * hkv * (dq + dv) + 2 * b * hq * (dq + dv) + 4 * b * hq + tables,
            "flops": 2 * (b * case["prefix"] + sum(lens)) * hq * (dq + dv)}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definition in 64 bits, request by request and head by head."""
    if case["op"] == "slots":
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return exact_rope(case, s)
    hq, hkv, dq, dv = (case[n] for n in ("hq", "hkv", "dq", "dv"))
    rows = s["q"].shape[0]
    out = torch.zeros(rows, hq, dv, dtype=torch.float64, device=DEV)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device=DEV)

    def attend(q, k, v, behind):
        """q [n, d], k [m, d], v [m, e]; query i sees the keys up to i + behind."""
        z = q.double() @ k.double().t() / math.sqrt(dq)
        if behind is not None:
            z = z + torch.full_like(z, -math.inf).triu(behind + 1)
        norm = torch.logsumexp(z, 1)
        return torch.exp(z - norm[:, None]) @ v.double(), norm

    if case["op"] == "prompt":
        lq, lk = lengths(case)
        at_q, at_k = offsets(lq), offsets(lk)
        for b in range(len(lq)):
            kk, vv = s["k"][at_k[b]:at_k[b + 1]], s["v"][at_k[b]:at_k[b + 1]]
            for lo in range(0, lq[b], 4096):
                hi = min(lq[b], lo + 4096)
                seen = lk[b] - lq[b] + hi
                a = slice(at_q[b] + lo, at_q[b] + hi)
                for h in range(hq):
                    g = h // (hq // hkv)
                    out[a, h], lse[a, h] = attend(s["q"][a, h], kk[:seen, g], vv[:seen, g], lk[b] - lq[b] + lo)
        return {"out": out, "lse": lse}
    page = case["page"]

    def rows_of(table, n):
        order = torch.arange(n, device=DEV)
        at = table.to(torch.int64)[order // page] * page + order % page
        return s["k_cache"].flatten(0, 1)[at], s["v_cache"].flatten(0, 1)[at]

    front_k, front_v = rows_of(s["prefix_table"], case["prefix"])
    for b, n in enumerate(s["host_lens"]):
        k, v = rows_of(s["table"][b], n)
        k, v = torch.cat([front_k, k]).double(), torch.cat([front_v, v]).double()
        for g in range(hkv):
            if k.shape[0]:
                hs = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
                out[b, hs], lse[b, hs] = attend(s["q"][b, hs], k[:, g], v[:, g], None)
    return {"out": out, "lse": lse}


def exact_rope(case, s):
    """Each rotated pair as a complex number times the table's cos + i sin."""
    rot = case["rot"]
    turn = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(turn[:, :rot // 2], turn[:, rot // 2:])[:, None]

    def head(x, w):
        x = x.double()
        if w is not None:
            x = w.double() * x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt()
        y = x.clone()
        if case["interleaved"]:
            z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * turn
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        return y

    q, k = head(s["q"], s["qw"]), head(s["k"], s["kw"])
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    has = s["slots"] >= 0
    at = s["slots"][has].long()
    kc.view(-1, case["hkv"], case["dq"])[at] = k[has]
    vc.view(-1, case["hkv"], case["dv"])[at] = s["v"].double()[has]
    return {"q": q, "k": k if case["keep_k"] else None, "k_cache": kc, "v_cache": vc}
