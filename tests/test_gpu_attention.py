"""GPU parity of the attention operators against the float64 oracle.

Whole numbers (tables, slots, positions) are compared exactly.

Tolerance of an attention output o = sum_j p_j v_j, from the arithmetic, with
u = 2^-24 (float) and r = 2^-8 (half an ulp of bf16, relative):
  * the result is rounded once to bf16:                       r |o|
  * each weight is rounded to bf16 for the matrix cores:      r sum p |v|
  * a score is a float sum of D exact products, then scaled:  d = 2 D u max_j sum_i |q_i k_ji| scale
    and formed against the rounded maximum in base 2:         t = 4 u (|s|max + 1) log2(e)
    both change a weight by e^(...), numerator and denominator alike:  2 (d + t) sum p |v|
  * 2^x is good to a few ulp and sums of n weights to n u (n / 32 in any one partial sum, taken as n):
    2 (8 u + n u) sum p |v|
Tolerance of lse: d + t + (8 + n) u + 2 u |lse|.
"""
import numpy as np
import pytest

import synth
from gpu_util import bf16_to_f64, dev_bf16, dev_f32, dev_i32, host, host_bf16_bits, say
from oracle import attention as oa

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_group_amd as moe  # noqa: E402

U, R = 2.0 ** -24, 2.0 ** -8
HEADS = [(64, 64), (128, 128), (192, 128)]


def bf16(seed, shape, std=1.0):
    bits = synth.random_bf16(seed, shape, std)
    return bits, bf16_to_f64(bits)


# ------------------------------------------------------------------- slots
def slots_case(seed, B, page, cached_max, new_max, blocks, free, position_base=0, max_new=None, zeros=True):
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, cached_max + 1, B)
    new = rng.integers(0 if zeros else 1, new_max + 1, B)
    pool = rng.permutation(4 * B * blocks + free).astype(np.int32)
    table = np.full((B, blocks + 3), -7, np.int32)                  # 3 columns that are not the table's
    at = 0
    for b in range(B):
        n = min(-(-int(cached[b]) // page), blocks)
        table[b, :n] = pool[at:at + n]
        at += n
    free_pages = pool[at:at + free]
    max_new = int(new.sum()) + 5 if max_new is None else max_new
    want = oa.kv_slots(cached, new, free_pages, table[:, :blocks], page, max_new, position_base)
    dt = dev_i32(table)
    got = moe.kv_slots(dev_i32(cached), dev_i32(new), dev_i32(free_pages), dt[:, :blocks], page, max_new, position_base)
    torch.cuda.synchronize()
    assert np.array_equal(host(dt)[:, blocks:], table[:, blocks:]), "columns beside the table changed"
    for name, g, w in zip(("table", "slots", "positions", "cu_new", "counts"), (dt[:, :blocks], *got), want):
        assert np.array_equal(host(g), w), f"{name} differs"
    return want


@pytest.mark.parametrize("B,page,cached,new,blocks", [
    (1, 16, 0, 1, 4), (1, 1, 3, 40, 64), (3, 16, 50, 33, 8), (64, 64, 8192, 1, 129), (255, 32, 100, 9, 6),
    (256, 16, 17, 17, 4), (257, 128, 1000, 300, 12), (1500, 16, 300, 90, 32), (4096, 4, 30, 5, 16), (2, 1024, 5000, 3000, 9)])
def test_kv_slots(B, page, cached, new, blocks):
    say(f"kv_slots B={B} page={page}")
    want = slots_case(B + page, B, page, cached, new, blocks, 2 * B * blocks)
    assert want[4][2] == 0 or cached + new > blocks * page


def test_kv_slots_runs_out():
    say("kv_slots: short free list, full table, short outputs")
    assert slots_case(1, 40, 16, 60, 50, 8, 30)[4][2] > 0          # the free list ends inside the batch
    assert slots_case(2, 40, 16, 60, 50, 8, 0)[4][0] == 0          # nothing free
    assert slots_case(3, 20, 8, 100, 60, 10, 500)[4][2] > 0        # tables too narrow (cached lengths beyond them too)
    slots_case(4, 33, 16, 60, 50, 8, 200, position_base=12345, max_new=100)
    slots_case(5, 5, 16, 60, 50, 8, 200, max_new=0)


def test_kv_slots_negative_and_empty():
    say("kv_slots: negative lengths, no requests")
    t = dev_i32(np.full((2, 4), -1))
    s, p, cu, n = moe.kv_slots(dev_i32(np.array([-5, 3])), dev_i32(np.array([2, -1])), dev_i32(np.array([11, 12])), t, 4, 4)
    assert host(t).tolist() == [[11, -1, -1, -1], [-1] * 4]
    assert host(s).tolist() == [44, 45, -1, -1] and host(p).tolist() == [0, 1, 0, 0]
    assert host(cu).tolist() == [0, 2, 2] and host(n).tolist() == [1, 1, 0]
    e = dev_i32(np.zeros(0))
    s, p, cu, n = moe.kv_slots(e, e, e, torch.empty((0, 4), dtype=torch.int32, device="cuda"), 4, 3)
    assert host(s).tolist() == [-1] * 3 and host(cu).tolist() == [0] and host(n).tolist() == [0, 0, 0]


# -------------------------------------------------------------------- rope
@pytest.mark.parametrize("T,Hq,Hkv,D,Dv,rot,inter,norm,page,keep", [
    (1, 1, 1, 64, 64, 64, False, True, 16, True), (5, 8, 2, 128, 128, 128, False, True, 16, False),
    (33, 5, 5, 192, 128, 64, True, True, 1, True), (300, 4, 1, 128, 128, 32, True, False, 64, True),
    (70, 16, 4, 64, 64, 16, False, True, 32, False), (9, 3, 3, 192, 128, 192, False, False, 16, True),
    (17, 2, 1, 128, 40, 0, False, True, 16, True), (129, 12, 4, 192, 128, 96, False, True, 128, True)])
def test_qk_norm_rope(T, Hq, Hkv, D, Dv, rot, inter, norm, page, keep):
    say(f"qk_norm_rope T={T} D={D} rot={rot} interleaved={inter} norm={norm}")
    rng = np.random.default_rng(T + D + rot)
    width = Hq * D + Hkv * D + Hkv * Dv
    bits, x = bf16(T, (T, width + 8), 2.0)                          # 8 more columns: rows are not dense
    rows = dev_bf16(bits)
    cut = lambda a, i, h, d: a[:, i:i + h * d].reshape(T, h, d) if isinstance(a, np.ndarray) else a[:, i:i + h * d].unflatten(1, (h, d))  # noqa: E731
    at = (0, Hq * D, Hq * D + Hkv * D)
    qw, kw = (rng.uniform(0.5, 1.5, D).astype(np.float32) if norm else None for _ in range(2))
    P = 50
    ang = rng.uniform(0, 6.3, (P, rot // 2))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32) if rot else None
    pos = rng.integers(-3, P + 3, T)                                # values outside are clamped
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T]
    slots[::7] = -1
    if T > 3:
        slots[3] = pages * page                                     # outside the cache: skipped
    kb, _ = bf16(77, (pages, page, Hkv, D))
    vb, _ = bf16(78, (pages, page, Hkv, Dv))
    kc, vc = dev_bf16(kb), dev_bf16(vb)
    q_want = oa.norm_rope(cut(x, at[0], Hq, D), qw, 1e-6, cs, pos, inter)
    k_want = oa.norm_rope(cut(x, at[1], Hkv, D), kw, 1e-6, cs, pos, inter)
    f = lambda a: None if a is None else dev_f32(a)  # noqa: E731
    q, k = moe.qk_norm_rope(cut(rows, at[0], Hq, D), cut(rows, at[1], Hkv, D), dev_i32(pos), f(cs), f(qw), f(kw), 1e-6,
                            inter, cut(rows, at[2], Hkv, Dv), kc, vc, dev_i32(slots), want_k=keep)
    torch.cuda.synchronize()

    def near(got, want, what):
        # one rounding to bf16; float before it: the norm's sum of D squares, three products and a sum
        big = np.abs(want).max(axis=-1, keepdims=True)
        assert np.all(np.abs(got - want) <= R * np.abs(want) + (D + 16) * U * big), what

    near(bf16_to_f64(host_bf16_bits(q)), q_want, "q")
    if keep:
        near(bf16_to_f64(host_bf16_bits(k)), k_want, "k")
    else:
        assert k is None
    kg, vg = host_bf16_bits(kc).reshape(-1, Hkv, D), host_bf16_bits(vc).reshape(-1, Hkv, Dv)
    used = [(t, s) for t, s in enumerate(slots) if 0 <= s < pages * page]
    for t, s in used:
        near(bf16_to_f64(kg[s]), k_want[t], "cached k")
        assert np.array_equal(vg[s], cut(bits, at[2], Hkv, Dv)[t]), "cached v"
    rest = np.setdiff1d(np.arange(pages * page), [s for _, s in used])
    assert np.array_equal(kg[rest], kb.reshape(-1, Hkv, D)[rest]) and np.array_equal(vg[rest], vb.reshape(-1, Hkv, Dv)[rest])
    # in place, without a cache: the same bits
    q2, k2 = cut(rows, at[0], Hq, D), cut(rows, at[1], Hkv, D)
    moe.qk_norm_rope(q2, k2, dev_i32(pos), f(cs), f(qw), f(kw), 1e-6, inter, q_out=q2, k_out=k2)
    torch.cuda.synchronize()
    assert torch.equal(q2, q) and (k is None or torch.equal(k2, k))
    assert np.array_equal(host_bf16_bits(rows)[:, at[2]:], bits[:, at[2]:]), "values or padding changed"


def test_qk_norm_rope_zero_and_infinite_heads():
    say("qk_norm_rope: a head of zeros, one with an infinity")
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    x[1, 1, 5] = float("inf")
    w = torch.ones(64, device="cuda")
    q, k = moe.qk_norm_rope(x, x, None, None, w, w)
    torch.cuda.synchronize()
    assert (q[0] == 0).all() and (q[1, 0] == 0).all()
    assert torch.isnan(q[1, 1, 5])                                  # inf / inf, as in the formula
    assert (q[1, 1, :5] == 0).all()


# ------------------------------------------------------------------ prompts
def bounds(q, k, v, allowed_n, scale, ref, lse, n):
    """Tolerances of one row: (out [Dv], lse); see the file's head."""
    big = np.abs(k) @ np.abs(q) * scale
    smax = np.abs(k @ q).max() * scale
    d = 2 * len(q) * U * big.max()
    t = 4 * U * (smax + 1) * 1.4427
    pv, _ = oa.attend(q, k, np.abs(v), scale)
    return R * np.abs(ref) + (R + 2 * (d + t) + 2 * (8 + n) * U) * pv, d + t + (8 + n) * U + 2 * U * abs(lse)


def check_prompt(q, k, v, cu_q, cu_k, scale, out, lse, what):
    want, wlse = oa.attn_prompt(q, k, v, cu_q, cu_k, scale)
    Hq, G = q.shape[1], q.shape[1] // k.shape[1]
    worst = 0.0
    for b in range(len(cu_q) - 1):
        lq, lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(lq):
            row, n = cu_q[b] + i, min(lk, i + lk - lq + 1)
            for h in range(Hq):
                if n <= 0:
                    assert np.all(out[row, h] == 0) and lse[row, h] == -np.inf, f"{what}: row {row} sees nothing"
                    continue
                at = slice(cu_k[b], cu_k[b] + n)
                bo, bl = bounds(q[row, h], k[at, h // G], v[at, h // G], n, scale, want[row, h], wlse[row, h], n)
                e = np.abs(out[row, h] - want[row, h])
                assert np.all(e <= bo), f"{what}: row {row} head {h}: {e.max()} over {bo.min()}"
                assert abs(lse[row, h] - wlse[row, h]) <= bl, f"{what}: lse of row {row} head {h}"
                worst = max(worst, float((e / bo).max()))
    say(f"  {what}: worst error / bound {worst:.2f}")


def offs(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def run_prompt(seed, lq, lk, Hq, Hkv, D, Dv, std=1.0, scale=None, **kw):
    cu_q, cu_k = offs(lq), offs(lk)
    qb, q = bf16(seed, (cu_q[-1], Hq, D), std)
    kb, k = bf16(seed + 1, (cu_k[-1], Hkv, D))
    vb, v = bf16(seed + 2, (cu_k[-1], Hkv, Dv))
    out, lse = moe.attn_prompt(dev_bf16(qb), dev_bf16(kb), dev_bf16(vb), dev_i32(cu_q), dev_i32(cu_k), scale,
                               want_lse=True, **kw)
    torch.cuda.synchronize()
    return q, k, v, cu_q, cu_k, bf16_to_f64(host_bf16_bits(out)), host(lse).astype(np.float64)


@pytest.mark.parametrize("D,Dv", HEADS)
@pytest.mark.parametrize("lq,lk,Hq,Hkv", [
    ([1], [1], 1, 1), ([2, 1, 0, 65], [2, 1, 0, 65], 4, 2), ([64], [64], 3, 3), ([31, 32, 33], [31, 32, 33], 2, 1),
    ([129], [129], 4, 1), ([257, 3], [257, 3], 2, 2), ([1, 7], [300, 70], 5, 1), ([40, 100], [200, 163], 2, 1),
    ([70, 5], [3, 0], 2, 1), ([130], [129], 1, 1), ([0, 0, 6], [4, 0, 6], 2, 2), ([300], [301], 16, 1)])
def test_attn_prompt(D, Dv, lq, lk, Hq, Hkv):
    what = f"attn_prompt {D}/{Dv} lq={lq} lk={lk} heads {Hq}/{Hkv}"
    say(what)
    r = run_prompt(len(lq) * 31 + lq[0] + D, lq, lk, Hq, Hkv, D, Dv)
    check_prompt(*r[:5], D ** -0.5, *r[5:], what)


@pytest.mark.parametrize("lens", [[600], [513, 255, 256, 257]])
def test_attn_prompt_longer(lens):
    """Several key tiles in front of the diagonal, sharp and flat heads."""
    for std, scale in ((4.0, None), (0.05, 0.5)):
        r = run_prompt(900, lens, lens, 2, 1, 128, 128, std, scale)
        check_prompt(*r[:5], 128 ** -0.5 if scale is None else scale, *r[5:], f"attn_prompt {lens} std {std}")


def test_attn_prompt_many_sequences():
    """More sequences than one round of the search looks at: 64, 65, 4097 and 5000."""
    rng = np.random.default_rng(8)
    for n, most in ((64, 9), (65, 9), (4097, 1), (5000, 2)):
        say(f"attn_prompt {n} sequences")
        lens = rng.integers(0, most + 1, n)
        r = run_prompt(n, lens, lens, 1, 1, 64, 64)
        check_prompt(*r[:5], 0.125, *r[5:], f"{n} sequences")


def test_attn_prompt_strides():
    """Heads cut from a fused projection, outputs into a wider buffer; heads before tokens; one key row for all."""
    T, Hq, Hkv, D = 100, 4, 2, 128
    bits, x = bf16(5, (T, (Hq + 2 * Hkv) * D + 16))
    rows = dev_bf16(bits)
    f = lambda a, i, h: a[:, i * D:(i + h) * D].reshape(T, h, D) if isinstance(a, np.ndarray) else a[:, i * D:(i + h) * D].unflatten(1, (h, D))  # noqa: E731
    wide = torch.full((T, Hq * D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = np.array([0, 37, T])
    out, lse = moe.attn_prompt(f(rows, 0, Hq), f(rows, Hq, Hkv), f(rows, Hq + Hkv, Hkv), dev_i32(cu), out=f(wide, 0, Hq),
                               want_lse=True)
    torch.cuda.synchronize()
    q, k, v = f(x, 0, Hq), f(x, Hq, Hkv), f(x, Hq + Hkv, Hkv)
    check_prompt(q, k, v, cu, cu, D ** -0.5, bf16_to_f64(host_bf16_bits(out)), host(lse).astype(np.float64), "fused rows")
    assert (wide[:, Hq * D:] == 7).all()
    # [heads, tokens, dim] in memory
    qt, kt, vt = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (f(rows, 0, Hq), f(rows, Hq, Hkv), f(rows, Hq + Hkv, Hkv)))
    out2, _ = moe.attn_prompt(qt, kt, vt, dev_i32(cu), out=torch.empty((Hq, T, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1))
    torch.cuda.synchronize()
    assert torch.equal(out2, out)
    # a broadcast key: every weight equal
    one = dev_bf16(synth.random_bf16(6, (1, Hkv, D))).expand(T, Hkv, D)
    out3, _ = moe.attn_prompt(f(rows, 0, Hq), one, f(rows, Hq + Hkv, Hkv), dev_i32(np.array([0, T])))
    torch.cuda.synchronize()
    mean = np.cumsum(np.repeat(v, Hq // Hkv, 1), 0) / np.arange(1, T + 1)[:, None, None]
    amean = np.cumsum(np.abs(np.repeat(v, Hq // Hkv, 1)), 0) / np.arange(1, T + 1)[:, None, None]
    assert np.all(np.abs(bf16_to_f64(host_bf16_bits(out3)) - mean) <= R * np.abs(mean) + (R + 1e-4) * amean)


def test_attn_prompt_rows_outside_the_offsets():
    say("attn_prompt: rows before, between and after the sequences")
    q = dev_bf16(synth.random_bf16(1, (50, 2, 64)))
    out = torch.full((50, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((50, 2), 5.0, device="cuda")
    moe.attn_prompt(q, q, q, dev_i32(np.array([10, 20, 40])), out=out, lse=lse)
    torch.cuda.synchronize()
    assert (out[:10] == 3).all() and (out[40:] == 3).all() and (lse[:10] == 5).all() and (lse[40:] == 5).all()
    assert (lse[10:40] != 5).all()
    moe.attn_prompt(q, q, q, dev_i32(np.array([-5, 30, 90])), out=out)   # entries are clamped to the rows
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("D,Dv", HEADS)
@pytest.mark.parametrize("where", [0, 40, 70, 199])
def test_attn_prompt_masked_places_do_not_leak(D, Dv, where):
    """Infinities and NaN in keys and values reach the rows that see them and no other, in this sequence and the next."""
    say(f"attn_prompt {D}/{Dv}: not finite at {where}")
    cu = np.array([0, 200, 260])
    qb, kb, vb = (synth.random_bf16(40 + i, (260, 2, d)) for i, d in enumerate((D, D, Dv)))
    clean = [dev_bf16(a) for a in (qb, kb, vb)]
    ref, rlse = moe.attn_prompt(*clean, dev_i32(cu), want_lse=True)
    for which, value in ((1, float("nan")), (1, float("inf")), (2, float("nan")), (2, float("inf")), (2, -float("inf"))):
        t = [a.clone() for a in clean]
        t[which][where, 1, 3] = value
        t[which][259, 0] = value                                    # the packed batch's last row too
        out, lse = moe.attn_prompt(*t, dev_i32(cu), want_lse=True)
        torch.cuda.synchronize()
        same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
        assert same(out[:where, 1], ref[:where, 1]) and torch.equal(lse[:where], rlse[:where]), (which, value)
        assert same(out[:200, 0], ref[:200, 0]) and same(out[200:259], ref[200:259]), (which, value)
        if which == 2:
            hit = out[where:200, 1, 3].float()
            assert (torch.isnan(hit) if value != value else hit == value).all(), (which, value)
            others = [i for i in range(Dv) if i != 3]
            assert torch.isfinite(out[where:200, 1][:, others].float()).all()
            # the other columns: the ordinary result (the sum's order may differ there by nothing: same bits)
            assert same(out[where:200, 1][:, others].contiguous(), ref[where:200, 1][:, others].contiguous())
            assert torch.equal(lse[:259], rlse[:259])
        else:
            s = torch.isnan(out[where:200, 1].float()).any(-1)
            if value != value:
                assert s.all()


def test_attn_prompt_lowest_scores():
    """Scores that overflow to -inf for some keys get no weight; a row with nothing else gives 0."""
    say("attn_prompt: scores of -inf")
    T, D = 90, 64
    q = torch.full((T, 1, D), 3e38, dtype=torch.bfloat16, device="cuda")
    k = torch.full((T, 1, D), -3e38, dtype=torch.bfloat16, device="cuda")
    v = dev_bf16(synth.random_bf16(2, (T, 1, D)))
    out, lse = moe.attn_prompt(q, k, v, dev_i32(np.array([0, T])), want_lse=True)
    torch.cuda.synchronize()
    assert (out == 0).all() and (lse == -float("inf")).all()
    k[70] = 0                                                       # one key with a score of 0
    out, lse = moe.attn_prompt(q, k, v, dev_i32(np.array([0, T])), want_lse=True)
    torch.cuda.synchronize()
    assert (out[:70] == 0).all() and torch.equal(out[70:], v[70].expand(T - 70, 1, D)) and (lse[70:] == 0).all()


def test_attn_prompt_same_bits_other_stream_and_graph():
    say("attn_prompt: repeated, on another stream, in a graph")
    cu = dev_i32(np.array([0, 300, 333]))
    q, k, v = (dev_bf16(synth.random_bf16(60 + i, (333, h, 128))) for i, h in enumerate((8, 2, 2)))
    ref, rl = moe.attn_prompt(q, k, v, cu, want_lse=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = moe.attn_prompt(q, k, v, cu, want_lse=True, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.attn_prompt(q, k, v, cu, out=out, lse=lse)
    for i in range(3):
        out.zero_()
        q.mul_(1.5 if i else 1.0)
        g.replay()
        eager, el = moe.attn_prompt(q, k, v, cu, want_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(lse, el), i


# ------------------------------------------------------------------- decode
def paged(seed, lens, prefix, page, Hkv, D, Dv, spare=3, blocks=None):
    """A cache whose unused rows are all NaN, in shuffled pages."""
    rng = np.random.default_rng(seed)
    blocks = max([1] + [-(-n // page) for n in lens]) if blocks is None else blocks
    need = sum(-(-n // page) for n in lens) + -(-prefix // page)
    pages = need + spare
    order = rng.permutation(pages)
    kb = np.full((pages, page, Hkv, D), 0x7FC0, np.uint16)
    vb = np.full((pages, page, Hkv, Dv), 0x7FC0, np.uint16)
    at = 0

    def fill(n):
        nonlocal at
        mine = order[at:at + -(-n // page)]
        at += len(mine)
        for j in range(n):
            kb[mine[j // page], j % page] = synth.random_bf16(seed * 7919 + at * 1000 + j, (Hkv, D))
            vb[mine[j // page], j % page] = synth.random_bf16(seed * 104729 + at * 1000 + j, (Hkv, Dv))
        return mine

    ptab = fill(prefix)
    table = np.full((len(lens), blocks + 2), -9, np.int64)          # entries past a length: not a page
    for b, n in enumerate(lens):
        mine = fill(n)
        table[b, :len(mine)] = mine
    return kb, vb, table, ptab, blocks


def check_decode(q, kb, vb, table, lens, ptab, prefix, scale, out, lse, what):
    k, v = bf16_to_f64(kb), bf16_to_f64(vb)
    page, Hkv = k.shape[1], k.shape[2]
    G = q.shape[1] // Hkv
    want, wlse = oa.attn_decode(q, k, v, table, lens, ptab, prefix, scale)
    worst = 0.0
    for b, n in enumerate(lens):
        at = [(ptab[j // page], j % page) for j in range(prefix)] + [(table[b][j // page], j % page) for j in range(n)]
        for h in range(q.shape[1]):
            if not at:
                assert np.all(out[b, h] == 0) and lse[b, h] == -np.inf, f"{what}: request {b} has no key"
                continue
            pg, off = np.array(at).T
            kk, vv = k[pg, off, h // G], v[pg, off, h // G]
            bo, bl = bounds(q[b, h], kk, vv, len(at), scale, want[b, h], wlse[b, h], len(at))
            e = np.abs(out[b, h] - want[b, h])
            assert np.all(e <= bo), f"{what}: request {b} head {h}: {e.max()} over {bo.min()}"
            assert abs(lse[b, h] - wlse[b, h]) <= bl, f"{what}: lse of request {b} head {h}"
            worst = max(worst, float((e / bo).max()))
    say(f"  {what}: worst error / bound {worst:.2f}")


def run_decode(seed, lens, prefix, page, Hq, Hkv, D, Dv, max_len=None, std=1.0):
    kb, vb, table, ptab, blocks = paged(seed, lens, prefix, page, Hkv, D, Dv)
    qb, q = bf16(seed + 5, (len(lens), Hq, D), std)
    dt = dev_i32(table)
    args = (dev_bf16(qb), dev_bf16(kb), dev_bf16(vb), dt[:, :blocks], dev_i32(np.array(lens)),
            max(lens) if max_len is None else max_len)
    out, lse = moe.attn_decode(*args, prefix_table=dev_i32(ptab), prefix_len=prefix, want_lse=True)
    torch.cuda.synchronize()
    return args, dev_i32(ptab), (q, kb, vb, table, lens, ptab, prefix, D ** -0.5, bf16_to_f64(host_bf16_bits(out)),
                                 host(lse).astype(np.float64)), out, lse


@pytest.mark.parametrize("D,Dv", HEADS)
@pytest.mark.parametrize("lens,prefix,page,Hq,Hkv", [
    ([1], 0, 16, 1, 1), ([0], 0, 16, 2, 1), ([5, 0, 33], 0, 16, 4, 2), ([0, 0], 7, 4, 8, 2), ([3, 64, 31, 32], 1, 1, 4, 1),
    ([130, 2, 0], 65, 64, 5, 1), ([300], 300, 32, 8, 8), ([17] * 9, 40, 16, 16, 2), ([70, 9], 130, 128, 40, 1),
    ([700, 1, 513], 260, 16, 2, 1), ([2] * 40, 33, 1024, 2, 2)])
def test_attn_decode(D, Dv, lens, prefix, page, Hq, Hkv):
    what = f"attn_decode {D}/{Dv} lens={lens[:4]} prefix={prefix} page={page} heads {Hq}/{Hkv}"
    say(what)
    *_, ref, _, _ = run_decode(len(lens) * 13 + prefix + D, lens, prefix, page, Hq, Hkv, D, Dv)
    check_decode(*ref, what)


def test_attn_decode_long_and_sharp():
    for lens, prefix in (([3000], 0), ([40, 0, 900], 2500), ([5] * 70, 1100)):
        *_, ref, _, _ = run_decode(3, lens, prefix, 32, 8, 2, 128, 128, std=4.0)
        check_decode(*ref, f"attn_decode {lens[:3]} behind {prefix}")


def test_attn_decode_bounds_on_the_host_side():
    """max_len over the lengths plans more parts than there are; lengths over max_len count as max_len."""
    lens = [100, 0, 37]
    _, _, ref, out, _ = run_decode(9, lens, 20, 16, 4, 2, 128, 128, max_len=112)
    check_decode(*ref, "attn_decode max_len over the lengths")
    args, pt, ref, _, _ = run_decode(9, lens, 20, 16, 4, 2, 128, 128)
    short, _ = moe.attn_decode(*args[:5], 37, prefix_table=pt, prefix_len=20)
    cut, _ = moe.attn_decode(*args[:4], dev_i32(np.array([37, 0, 37])), 37, prefix_table=pt, prefix_len=20)
    torch.cuda.synchronize()
    assert torch.equal(short, cut)


def test_attn_decode_shared_prefix_equals_private_copies():
    """The prefix in every request's own pages gives the result of the shared one (within the rounding of the weights)."""
    prefix, page = 96, 32
    kb, vb, table, ptab, blocks = paged(21, [10, 50, 1], prefix, page, 2, 128, 128)
    q = dev_bf16(synth.random_bf16(22, (3, 8, 128)))
    k, v, lens = dev_bf16(kb), dev_bf16(vb), np.array([10, 50, 1])
    a, la = moe.attn_decode(q, k, v, dev_i32(table), dev_i32(lens), 50, dev_i32(ptab), prefix, want_lse=True)
    both = np.concatenate([np.repeat(ptab[None], 3, 0), table], 1)
    b, lb = moe.attn_decode(q, k, v, dev_i32(both), dev_i32(lens + prefix), 50 + prefix, want_lse=True)
    torch.cuda.synchronize()
    np.testing.assert_allclose(host(la), host(lb), rtol=0, atol=2e-6)
    assert (a.float() - b.float()).abs().max() <= 4 * R * v[~torch.isnan(v)].float().abs().max()


def test_attn_decode_entries_outside_the_cache():
    """Table entries that are no page never address memory outside the cache (results of those requests: unspecified)."""
    say("attn_decode: bad table entries")
    kb, vb, table, ptab, blocks = paged(30, [40, 40], 0, 16, 1, 64, 64)
    t = table[:, :blocks].copy()
    t[0, 1] = 1 << 30
    t[0, 2] = -(1 << 30)
    q = dev_bf16(synth.random_bf16(31, (2, 2, 64)))
    args = (dev_bf16(kb), dev_bf16(vb))
    good, _ = moe.attn_decode(q, *args, dev_i32(table[:, :blocks]), dev_i32(np.array([40, 40])), 40)
    bad, _ = moe.attn_decode(q, *args, dev_i32(t), dev_i32(np.array([40, 40])), 40)
    torch.cuda.synchronize()
    assert torch.equal(good[1], bad[1])


def test_attn_decode_infinite_values():
    say("attn_decode: infinities in seen values")
    kb, vb, table, ptab, blocks = paged(33, [40, 70], 35, 16, 1, 128, 128)
    q = dev_bf16(synth.random_bf16(34, (2, 4, 128)))
    v = dev_bf16(vb)
    k = dev_bf16(kb)
    args = (dev_i32(table), dev_i32(np.array([40, 70])), 70, dev_i32(ptab), 35)
    ref, _ = moe.attn_decode(q, k, v, *args)
    v[table[1][4], 5, 0, 9] = float("inf")                          # request 1's last key (69)
    v[ptab[2], 2, 0, 11] = -float("inf")                            # the prefix's last key (34)
    out, _ = moe.attn_decode(q, k, v, *args)
    torch.cuda.synchronize()
    assert (out[1, :, 9] == float("inf")).all() and (out[:, :, 11] == -float("inf")).all()
    rest = [i for i in range(128) if i not in (9, 11)]
    assert torch.equal(out[..., rest], ref[..., rest]) and torch.equal(out[0, :, 9], ref[0, :, 9])


def test_attn_decode_far_rows():
    """Rows whose bytes lie past 2^32 (and 2^31 elements) in the cache."""
    page, Hkv, D = 64, 8, 128
    pages = (1 << 32) // (page * Hkv * D * 2) + 40
    say(f"attn_decode: {pages * page * Hkv * D * 2 / 2**30:.1f} GiB of keys")
    k = torch.empty((pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty((pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    far = [pages - 1, pages - 7, pages - 20, 3]
    kb, vb = synth.random_bf16(50, (4, page, Hkv, D)), synth.random_bf16(51, (4, page, Hkv, D))
    for i, p in enumerate(far):
        k[p], v[p] = dev_bf16(kb[i]), dev_bf16(vb[i])
    q = dev_bf16(synth.random_bf16(52, (1, 16, D)))
    a, _ = moe.attn_decode(q, k, v, dev_i32(np.array([far[1:]])), dev_i32(np.array([150])), 150, dev_i32(np.array(far[:1])), 50)
    b, _ = moe.attn_decode(q, dev_bf16(kb), dev_bf16(vb), dev_i32(np.array([[1, 2, 3]])), dev_i32(np.array([150])), 150,
                           dev_i32(np.array([0])), 50)
    # and the write: the last slot of the cache
    row = dev_bf16(synth.random_bf16(53, (1, Hkv, D)))
    moe.qk_norm_rope(q, row, None, None, v=row, k_cache=k, v_cache=v, slots=dev_i32(np.array([pages * page - 1])))
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    assert torch.equal(k[-1, -1], row[0]) and torch.equal(v[-1, -1], row[0])


def test_attn_decode_same_bits_other_stream_and_graph():
    say("attn_decode: repeated, on another stream, in a graph")
    args, pt, _, ref, rl = run_decode(70, [400, 20, 0, 129], 600, 16, 8, 2, 128, 128)
    ws = torch.empty(max(16, moe.attn_decode_workspace_bytes(4, 600, 400, 8, 2, 128, 128)), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = moe.attn_decode(*args, prefix_table=pt, prefix_len=600, want_lse=True, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.attn_decode(*args, prefix_table=pt, prefix_len=600, workspace=ws, out=out, lse=lse)
    for i in range(3):
        args[4].sub_(i * 7)                                          # the lengths are read on the device
        g.replay()
        eager, el = moe.attn_decode(*args, prefix_table=pt, prefix_len=600, want_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(lse, el), i


# ----------------------------------------------- variants chosen by size, and other streams
@pytest.mark.parametrize("D,inter,heads", [(64, False, 216), (128, True, 108), (192, False, 72)])
def test_qk_norm_rope_large_equals_small(D, inter, heads):
    """Outputs over 128 MiB take the stores that bypass the cache: the bits of the same tokens in small calls."""
    Hkv, T, page = 4, 5200, 16
    Hq = heads - 2 * Hkv
    say(f"qk_norm_rope {T} x {Hq}/{Hkv} x {D}")
    assert T * heads * D * 2 > 128 << 20
    g = torch.Generator(device="cuda").manual_seed(D)
    rows = torch.randn((T, heads, D), generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    pos = torch.randint(0, 300, (T,), generator=g, device="cuda", dtype=torch.int32)
    cs, w = torch.randn((300, D), generator=g, device="cuda"), torch.rand(D, generator=g, device="cuda")
    pages = T // page + 4
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    caches = [torch.zeros((pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    ql, kl = moe.qk_norm_rope(q, k, pos, cs, w, w, 1e-6, inter, v, *caches[:2], slots, want_k=True)
    for i in range(0, T, 1300):
        s = slice(i, i + 1300)
        qs, ks = moe.qk_norm_rope(q[s], k[s], pos[s], cs, w, w, 1e-6, inter, v[s], *caches[2:], slots[s], want_k=True)
        torch.cuda.synchronize()
        assert torch.equal(qs, ql[s]) and torch.equal(ks, kl[s]), i
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    assert torch.equal(caches[1].view(-1, Hkv, D)[slots.long()], v)


@pytest.mark.parametrize("lens,prefix,Hq,Hkv", [([5, 40], 70, 70, 1), ([33], 0, 130, 1), ([1, 0, 65], 64, 132, 2)])
def test_attn_decode_many_heads_per_key_head(lens, prefix, Hq, Hkv):
    """More than 64 query heads of a key head: several row blocks of the own keys."""
    what = f"attn_decode lens={lens} prefix={prefix} heads {Hq}/{Hkv}"
    say(what)
    *_, ref, _, _ = run_decode(Hq + prefix, lens, prefix, 16, Hq, Hkv, 128, 128)
    check_decode(*ref, what)


@pytest.mark.parametrize("D,Dv", HEADS)
@pytest.mark.parametrize("B", [2, 3, 20])
def test_attn_decode_places_past_the_end(D, Dv, B):
    """Few and many rows (32, 48 and 320 to a key head): the last page's unused rows hold infinities that nothing sees;
    an infinity in the last key's value is seen by exactly the rows that read it."""
    say(f"attn_decode {D}/{Dv}: infinities behind the last key, {B} requests")
    lens, prefix = [40 + b for b in range(B)], 75
    kb, vb, table, ptab, blocks = paged(80 + B, lens, prefix, 16, 1, D, Dv)
    q = dev_bf16(synth.random_bf16(81, (B, 16, D)))
    v, k = dev_bf16(vb), dev_bf16(kb)
    args = (dev_i32(table), dev_i32(np.array(lens)), max(lens), dev_i32(ptab), prefix)
    ref, rl = moe.attn_decode(q, k, v, *args, want_lse=True)
    dirt = torch.isnan(v)
    assert dirt.any() and torch.isfinite(ref.float()).all()
    for value in (float("inf"), -float("inf")):
        k2, v2 = k.clone(), v.clone()
        k2[torch.isnan(k)], v2[dirt] = value, value
        out, lse = moe.attn_decode(q, k2, v2, *args, want_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(lse, rl), value
    v[ptab[74 // 16], 74 % 16, 0, 7] = float("inf")
    last = lens[-1] - 1
    v[table[B - 1][last // 16], last % 16, 0, 21] = -float("inf")
    out, lse = moe.attn_decode(q, k, v, *args, want_lse=True)
    torch.cuda.synchronize()
    assert (out[:, :, 7] == float("inf")).all() and (out[-1, :, 21] == -float("inf")).all()
    rest = [i for i in range(Dv) if i not in (7, 21)]
    assert torch.equal(out[..., rest], ref[..., rest]) and torch.equal(out[:-1, :, 21], ref[:-1, :, 21])
    assert torch.equal(lse, rl)


def test_slots_and_rope_other_stream_and_graph():
    """The tables of a step that are built and used on another stream, and in a graph: the bits of the eager calls."""
    say("kv_slots + qk_norm_rope: another stream, a graph")
    B, page, Hq, Hkv, D = 5, 16, 4, 2, 64
    rng = np.random.default_rng(4)
    new, cached = dev_i32(rng.integers(0, 20, B)), dev_i32(rng.integers(0, 20, B))
    free, cs = dev_i32(rng.permutation(40)), torch.randn((64, D), device="cuda")
    rows = dev_bf16(synth.random_bf16(9, (100, Hq + 2 * Hkv, D)))

    def step(table, kc, vc, out, **kw):
        s, p, cu, n = moe.kv_slots(cached, new, free, table, page, 100, 0, *out, **kw)
        return moe.qk_norm_rope(rows[:, :Hq], rows[:, Hq:Hq + Hkv], p, cs, v=rows[:, Hq + Hkv:], k_cache=kc, v_cache=vc,
                                slots=s, want_k=True, **kw)

    def fresh():
        caches = [torch.zeros((40, page, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        outs = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (100, 100, B + 1, 3)]
        return torch.full((B, 4), -1, dtype=torch.int32, device="cuda"), *caches, outs

    a, b, c = fresh(), fresh(), fresh()
    qa, ka = step(*a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    qb, kb = step(*b, stream=s)
    s.synchronize()
    assert torch.equal(qa, qb) and torch.equal(ka, kb) and all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qc, kc = step(*c)
    for i in range(3):
        for t in c[:3]:
            t.fill_(-1 if t.dtype == torch.int32 else 0)
        d = fresh()
        new.copy_(dev_i32(rng.integers(0, 20, B)))
        g.replay()
        qd, kd = step(*d)
        torch.cuda.synchronize()
        assert torch.equal(qc, qd) and torch.equal(kc, kd), i
        assert all(torch.equal(x, y) for x, y in zip(c[:3], d[:3])) and all(torch.equal(x, y) for x, y in zip(c[3], d[3])), i


# ----------------------------------------------- many keys: parts that are joined
def makes_parts(lens, prefix, Hq, Hkv, D, Dv):
    return moe.attn_decode_workspace_bytes(len(lens), prefix, max(lens), Hq, Hkv, D, Dv) > 0


@pytest.mark.parametrize("D,Dv", HEADS)
@pytest.mark.parametrize("lens,prefix,page,Hq,Hkv", [
    ([5, 0, 33], 2901, 16, 4, 2), ([0, 0], 2985, 4, 8, 2), ([17] * 9, 3000, 16, 16, 2), ([70, 9], 2930, 128, 40, 1),
    ([2] * 40, 2857, 64, 2, 2), ([130, 2, 0], 2945, 64, 5, 1), ([700, 1, 513], 2900, 16, 2, 1), ([3500, 0, 33, 1], 0, 32, 8, 2),
    ([2900, 3100, 2999], 0, 1024, 4, 4), ([64] * 12, 2816, 64, 12, 2), ([31] * 12, 2823, 32, 12, 2)])
def test_attn_decode_parts(D, Dv, lens, prefix, page, Hq, Hkv):
    """Parts and runs that end inside a tile, a page or a request; few rows and many, small pages and large."""
    what = f"attn_decode {D}/{Dv} lens={lens[:4]} prefix={prefix} page={page} heads {Hq}/{Hkv}"
    say(what)
    assert makes_parts(lens, prefix, Hq, Hkv, D, Dv)
    *_, ref, _, _ = run_decode(len(lens) * 17 + prefix + D, lens, prefix, page, Hq, Hkv, D, Dv)
    check_decode(*ref, what)


@pytest.mark.parametrize("B,page", [(2, 16), (3, 64), (20, 16), (20, 64)])
def test_attn_decode_parts_past_the_end(B, page):
    """As test_attn_decode_places_past_the_end, where parts are joined."""
    say(f"attn_decode parts: infinities behind the last key, {B} requests, pages of {page}")
    D, lens, prefix = 128, [40 + b for b in range(B)], 3075
    assert makes_parts(lens, prefix, 16, 1, D, D)
    kb, vb, table, ptab, blocks = paged(90 + B, lens, prefix, page, 1, D, D)
    q = dev_bf16(synth.random_bf16(81, (B, 16, D)))
    v, k = dev_bf16(vb), dev_bf16(kb)
    args = (dev_i32(table), dev_i32(np.array(lens)), max(lens), dev_i32(ptab), prefix)
    ref, rl = moe.attn_decode(q, k, v, *args, want_lse=True)
    k2, v2 = k.clone(), v.clone()
    k2[torch.isnan(k)], v2[torch.isnan(v)] = float("inf"), float("inf")
    out, lse = moe.attn_decode(q, k2, v2, *args, want_lse=True)
    torch.cuda.synchronize()
    assert torch.isfinite(ref.float()).all() and torch.equal(out, ref) and torch.equal(lse, rl)
    v[ptab[(prefix - 1) // page], (prefix - 1) % page, 0, 7] = float("inf")
    last = lens[-1] - 1
    v[table[B - 1][last // page], last % page, 0, 21] = -float("inf")
    out, lse = moe.attn_decode(q, k, v, *args, want_lse=True)
    torch.cuda.synchronize()
    assert (out[:, :, 7] == float("inf")).all() and (out[-1, :, 21] == -float("inf")).all()
    rest = [i for i in range(D) if i not in (7, 21)]
    assert torch.equal(out[..., rest], ref[..., rest]) and torch.equal(out[:-1, :, 21], ref[:-1, :, 21])
    assert torch.equal(lse, rl)


def test_attn_decode_parts_bounds_and_bad_entries():
    """max_len over and under the lengths, and table entries outside the cache, where parts are joined."""
    lens = [3100, 0, 2037]
    _, _, ref, _, _ = run_decode(9, lens, 20, 16, 4, 2, 128, 128, max_len=194 * 16)
    check_decode(*ref, "attn_decode max_len over the lengths, parts")
    args, pt, _, out, _ = run_decode(9, lens, 20, 16, 4, 2, 128, 128)
    assert makes_parts([2837] * 3, 20, 4, 2, 128, 128)
    short, _ = moe.attn_decode(*args[:5], 2837, prefix_table=pt, prefix_len=20)
    cut, _ = moe.attn_decode(*args[:4], dev_i32(np.array([2837, 0, 2037])), 2837, prefix_table=pt, prefix_len=20)
    t = args[3].clone()
    t[0, 5], t[0, 150] = 1 << 30, -(1 << 30)
    bad, _ = moe.attn_decode(*args[:3], t, *args[4:], prefix_table=pt, prefix_len=20)
    torch.cuda.synchronize()
    assert torch.equal(short, cut) and torch.equal(bad[2], out[2])


def test_attn_decode_parts_far_rows():
    """As test_attn_decode_far_rows with every page many times, so that parts are joined."""
    page, Hkv, D, times = 64, 8, 128, 30
    pages = (1 << 32) // (page * Hkv * D * 2) + 40
    say("attn_decode parts: rows past 2^32 bytes")
    k = torch.empty((pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty((pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    far = [pages - 1, pages - 7, pages - 20, 3]
    kb, vb = synth.random_bf16(50, (4, page, Hkv, D)), synth.random_bf16(51, (4, page, Hkv, D))
    for i, p in enumerate(far):
        k[p], v[p] = dev_bf16(kb[i]), dev_bf16(vb[i])
    for B in (1, 40):                                                # few rows and many to a key head
        q = dev_bf16(synth.random_bf16(52, (B, 16, D)))
        n = 3 * page * times - 42
        rows = lambda t: dev_i32(np.array([t * times] * B))  # noqa: E731
        lens = dev_i32(np.array([n] * B))
        assert moe.attn_decode_workspace_bytes(B, 4 * page * times - 14, n, 16, Hkv, D, D) > 0
        a, _ = moe.attn_decode(q, k, v, rows(far[1:]), lens, n, dev_i32(np.array(far * times)), 4 * page * times - 14)
        b, _ = moe.attn_decode(q, dev_bf16(kb), dev_bf16(vb), rows([1, 2, 3]), lens, n,
                               dev_i32(np.array([0, 1, 2, 3] * times)), 4 * page * times - 14)
        torch.cuda.synchronize()
        assert torch.equal(a, b), B


def test_attn_decode_alone_equals_parts():
    """A request's answer where one workgroup gives it and where parts are joined: the rounding of the weights apart."""
    say("attn_decode: one workgroup against parts")
    lens, prefix = [300, 7, 120], 200
    args, pt, _, small, sl = run_decode(33, lens, prefix, 16, 8, 2, 128, 128)
    assert not makes_parts(lens, prefix, 8, 2, 128, 128)
    # the same requests among others that need parts
    wide = torch.zeros((3, 200), dtype=torch.int32, device="cuda")
    wide[:, :args[3].shape[1]] = args[3]
    assert moe.attn_decode_workspace_bytes(3, prefix, 3200, 8, 2, 128, 128) > 0
    parts, pl = moe.attn_decode(*args[:3], wide, args[4], 3200, prefix_table=pt, prefix_len=prefix, want_lse=True)
    torch.cuda.synchronize()
    np.testing.assert_allclose(host(sl), host(pl), rtol=0, atol=2e-6)
    big = args[2][~torch.isnan(args[2])].float().abs().max()
    assert (small.float() - parts.float()).abs().max() <= 4 * R * big


# ----------------------------------------------- prompts of few rows and many keys: keys split, parts joined
@pytest.mark.parametrize("D,Dv", HEADS)
@pytest.mark.parametrize("lq,lk,Hq,Hkv", [
    ([1], [1500], 1, 1), ([16], [2100], 4, 2), ([3, 0, 40], [2000, 700, 1345], 4, 1), ([33, 2], [65, 3900], 5, 1),
    ([200], [1999], 2, 2), ([1, 1, 1, 1], [700, 3000, 0, 1], 8, 2), ([64], [4097], 3, 1), ([50, 9], [40, 2500], 2, 1)])
def test_attn_prompt_split_keys(D, Dv, lq, lk, Hq, Hkv):
    """Runs of keys that end before the diagonal, in it, or see nothing; rows without keys."""
    what = f"attn_prompt {D}/{Dv} lq={lq} lk={lk} heads {Hq}/{Hkv}, split"
    say(what)
    # (3701 keys of four sequences are too few on average to split for the smallest heads)
    assert moe.attn_prompt_workspace_bytes(len(lq), sum(lq), sum(lk), Hq, Hkv, D, Dv) > 0 or (D == 64 and len(lq) == 4)
    r = run_prompt(len(lq) * 37 + lq[0] + D, lq, lk, Hq, Hkv, D, Dv)
    check_prompt(*r[:5], D ** -0.5, *r[5:], what)


def test_attn_prompt_split_masked_places_and_other_rows():
    """Infinities and NaN in values and keys reach the rows that see them alone; rows outside the sequences stay."""
    say("attn_prompt split: not finite values, rows outside")
    cu_q, cu_k = np.array([3, 40, 60]), np.array([0, 1800, 3100])
    qb, kb, vb = synth.random_bf16(70, (70, 4, 128)), synth.random_bf16(71, (3100, 2, 128)), synth.random_bf16(72, (3100, 2, 128))
    q, k, v = dev_bf16(qb), dev_bf16(kb), dev_bf16(vb)
    args = (dev_i32(cu_q), dev_i32(cu_k))
    assert moe.attn_prompt_workspace_bytes(2, 70, 3100, 4, 2, 128, 128) > 0

    def call(q, k, v):
        out = torch.full((70, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((70, 4), 5.0, device="cuda")
        moe.attn_prompt(q, k, v, *args, out=out, lse=lse)
        torch.cuda.synchronize()
        return out, lse

    ref, rl = call(q, k, v)
    assert (ref[:3] == 3).all() and (ref[60:] == 3).all() and (rl[:3] == 5).all() and (rl[60:] == 5).all()
    assert torch.isfinite(ref.float()).all() and torch.isfinite(rl).all()
    where = 1780                                                     # rows 20 .. 36 of the first sequence see it
    for which, value in ((1, float("nan")), (2, float("nan")), (2, float("inf")), (2, -float("inf"))):
        t = [q, k.clone(), v.clone()]
        t[which][where, 1, 5] = value
        out, lse = call(*t)
        row = 3 + where - (1800 - 37)
        same = lambda a, b: torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))  # noqa: E731
        assert same(out[:row], ref[:row]) and same(out[40:], ref[40:]) and same(out[:, :2], ref[:, :2]), (which, value)
        if which == 2:
            hit = out[row:40, 2:, 5].float()
            assert (torch.isnan(hit) if value != value else hit == value).all()
            rest = [i for i in range(128) if i != 5]
            assert same(out[..., rest], ref[..., rest]) and torch.equal(lse, rl)
        else:
            assert torch.isnan(out[row:40, 2:].float()).all()


def test_attn_prompt_split_stream_graph_and_workspace():
    say("attn_prompt split: repeated, on another stream, in a graph, with a workspace that is given")
    cu_q, cu_k = dev_i32(np.array([0, 20, 33])), dev_i32(np.array([0, 2500, 4000]))
    q, k, v = (dev_bf16(synth.random_bf16(60 + i, (n, h, 128))) for i, (n, h) in enumerate(((33, 8), (4000, 2), (4000, 2))))
    ref, rl = moe.attn_prompt(q, k, v, cu_q, cu_k, want_lse=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = moe.attn_prompt(q, k, v, cu_q, cu_k, want_lse=True, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    ws = torch.full((moe.attn_prompt_workspace_bytes(2, 33, 4000, 8, 2, 128, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.attn_prompt(q, k, v, cu_q, cu_k, out=out, lse=lse, workspace=ws)
    for i in range(3):
        out.zero_()
        ws.fill_(0xFF)
        q.mul_(1.5 if i else 1.0)
        g.replay()
        eager, el = moe.attn_prompt(q, k, v, cu_q, cu_k, want_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(lse, el), i


# ----------------------------------------------- the Python side
def test_calls_refuse_and_keep_no_references():
    """Wrong tensors are named; refused and finished calls leave every argument's reference count as it was."""
    import gc
    import sys
    say("attention calls: refusals from Python, reference counts")
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    q, k, v, cu = z(8, 4, 128), z(8, 2, 128), z(8, 2, 128), dev_i32(np.array([0, 8]))
    kc, vc, tb, ln = z(4, 16, 2, 128), z(4, 16, 2, 128), dev_i32(np.zeros((8, 2))), dev_i32(np.full(8, 5))
    f = torch.zeros(128, device="cuda")
    cases = [
        (ValueError, "q must be a 3-d", lambda: moe.attn_prompt(q.float(), k, v, cu)),
        (ValueError, "k must be a 3-d", lambda: moe.attn_prompt(q, k[..., ::2], v, cu)),
        (ValueError, "k: shape", lambda: moe.attn_prompt(q, k[..., :64], v, cu)),
        (ValueError, "v: shape", lambda: moe.attn_prompt(q, k, v[:4], cu)),
        (ValueError, "cu_q must be a 1-d", lambda: moe.attn_prompt(q, k, v, cu.long())),
        (ValueError, "entry for each sequence", lambda: moe.attn_prompt(q, k, v, cu, dev_i32(np.zeros(3)))),
        (ValueError, "out: shape", lambda: moe.attn_prompt(q, k, v, cu, out=k)),
        (ValueError, "lse must be", lambda: moe.attn_prompt(q, k, v, cu, lse=z(8, 2, d=torch.float32))),
        (ValueError, "workspace must be", lambda: moe.attn_prompt(q, k, v, cu, workspace=torch.zeros(8))),
        (TypeError, None, lambda: moe.attn_prompt(q, k, v, cu, scale="x")),
        (moe.MoeError, "scale", lambda: moe.attn_prompt(q, k, v, cu, scale=-1.0)),
        (ValueError, "k_cache must be", lambda: moe.attn_decode(q, kc[0], vc, tb, ln, 5)),
        (ValueError, "do not fit", lambda: moe.attn_decode(q, kc, vc[:2], tb, ln, 5)),
        (ValueError, "block_table needs", lambda: moe.attn_decode(q, kc, vc, tb[:3], ln, 5)),
        (ValueError, "lens needs", lambda: moe.attn_decode(q, kc, vc, tb, ln[:3], 5)),
        (moe.MoeError, "max_len", lambda: moe.attn_decode(q, kc, vc, tb, ln, 50)),
        (TypeError, None, lambda: moe.attn_decode(q, kc, vc, tb, ln, None)),
        (ValueError, "positions must be", lambda: moe.qk_norm_rope(q, k, None, z(4, 64, d=torch.float32))),
        (ValueError, "positions needs", lambda: moe.qk_norm_rope(q, k, cu, z(4, 64, d=torch.float32))),
        (ValueError, "need 128", lambda: moe.qk_norm_rope(q, k, None, None, f[:64])),
        (ValueError, "slots needs", lambda: moe.qk_norm_rope(q, k, None, None, v=v, k_cache=kc, v_cache=vc, slots=cu)),
        (moe.MoeError, "nowhere", lambda: moe.qk_norm_rope(q, k, None, None, want_k=False)),
        (ValueError, "entry for each request", lambda: moe.kv_slots(ln, cu, cu, tb, 16, 4)),
        (ValueError, "slots needs 4", lambda: moe.kv_slots(ln, ln, cu, tb, 16, 4, slots=cu)),
        (ValueError, "32-bit", lambda: moe.kv_slots(ln, ln, cu, tb, 1 << 40, 4)),
        (moe.MoeError, "page_size", lambda: moe.kv_slots(ln, ln, cu, tb, 24, 4)),
    ]
    fine = [lambda: moe.attn_prompt(q, k, v, cu, want_lse=True), lambda: moe.attn_prompt(q, k, v, cu, cu, 0.1, out=q.clone()),
            lambda: moe.attn_decode(q, kc, vc, tb, ln, 5, tb[0], 7, want_lse=True),
            lambda: moe.qk_norm_rope(q, k, None, None, f, f, v=v, k_cache=kc, v_cache=vc, slots=ln),
            lambda: moe.kv_slots(ln, ln, cu, tb.clone(), 16, 4), lambda: moe.kv_slots(ln, ln, cu, tb.clone(), 16, 4, counts=ln)]
    watched = [q, k, v, cu, kc, vc, tb, ln, f, None]
    count = lambda: [sys.getrefcount(x) for x in watched[:-1]]  # noqa: E731
    before = None
    for turn in range(3):
        for kind, match, call in cases:
            with pytest.raises(kind, match=match):
                call()
        for call in fine:
            call()
        gc.collect()
        assert before is None or count() == before, turn
        before = count()
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    for _ in range(50):
        for call in fine:
            call()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == held
    assert [tuple(t.shape) for t in fine[4]()] == [(4,), (4,), (9,), (3,)]


# ----------------------------------------------- memory of two streams
def stream_calls():
    """Each call on inputs of its own, with outputs (and a workspace where there is one) made by the call."""
    z = lambda i, *s: dev_bf16(synth.random_bf16(900 + i, s))  # noqa: E731
    q, k, v, cs = z(0, 64, 8, 128), z(1, 64, 2, 128), z(2, 64, 2, 128), torch.randn((64, 128), device="cuda")
    kc, vc = z(3, 300, 16, 2, 128), z(4, 300, 16, 2, 128)
    kl, vl = z(5, 4000, 2, 128), z(6, 4000, 2, 128)
    i = lambda a: dev_i32(np.asarray(a))  # noqa: E731
    ints = [i(np.full(40, 9)), i(np.full(40, 30)), i(np.arange(200)), i(np.zeros((40, 4)))]
    pos, cu_q, cu_k, tb, ln, pt = i(np.arange(64)), i([0, 64]), i([0, 4000]), i(np.arange(128).reshape(64, 2)), i(np.full(64, 20)), i(np.arange(250))
    assert moe.attn_prompt_workspace_bytes(1, 64, 4000, 8, 2, 128, 128) > 0 and makes_parts([20] * 64, 4000, 8, 2, 128, 128)
    return {
        "kv_slots": lambda **kw: moe.kv_slots(*ints, 16, 1300, **kw),
        "qk_norm_rope": lambda **kw: moe.qk_norm_rope(q, k, pos, cs, **kw),
        "attn_prompt": lambda **kw: moe.attn_prompt(q, kl, vl, cu_q, cu_k, want_lse=True, **kw),
        "attn_decode": lambda **kw: moe.attn_decode(q, kc, vc, tb, ln, 20, pt, 4000, want_lse=True, **kw)}


SIZES = [1 << b for b in range(9, 24)]                              # of freed blocks: each call finds one that fits


@pytest.mark.parametrize("name", ["kv_slots", "qk_norm_rope", "attn_prompt", "attn_decode"])
def test_outputs_do_not_lie_in_memory_that_queued_work_writes(name):
    """Blocks freed while work on them is queued belong to the current stream's order; a call on another stream runs
    before that work does."""
    say(f"{name}: freed blocks of the current stream, still written")
    call = stream_calls()[name]
    want = [t.clone() for t in call() if t is not None]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in SIZES for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(30_000_000)
    for t in junk:
        t.fill_(0xFF)
    del junk, t
    got = call(stream=s)
    assert torch.cuda.current_stream() != s
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("name", ["kv_slots", "qk_norm_rope", "attn_prompt", "attn_decode"])
def test_outputs_of_another_stream_outlive_their_readers(name):
    """An output read on the current stream and freed there: the next call on its own stream gets other memory until
    the reader is done."""
    say(f"{name}: outputs read on the current stream after they are freed")
    call = stream_calls()[name]
    want = [t.clone() for t in call() if t is not None]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(30_000_000)
    read = [t.clone() for t in got]
    del got
    with torch.cuda.stream(s):
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in SIZES for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(read, want))
    del junk


# ----------------------------------------------- slots of requests that ran out of pages before
@pytest.mark.parametrize("B,page,blocks", [(1, 16, 4), (70, 16, 8), (300, 4, 30), (1500, 32, 12), (4096, 8, 16)])
def test_kv_slots_behind_a_short_free_list(B, page, blocks):
    """Steps one after another where the free list ends inside the first: tokens that go into a page entered as -1 have
    no slot, and are counted in every step."""
    say(f"kv_slots after the pages ran out: B={B} page={page}")
    rng = np.random.default_rng(B)
    table = np.full((B, blocks), -1, np.int64)
    dt = dev_i32(table)
    cached, lost = np.zeros(B, np.int64), []
    for step in range(4):
        new = rng.integers(0, 2 * page if step == 0 else 3, B)
        if B == 1:
            new[:] = 10 if step == 0 else 1
        free = rng.permutation(8 * B)[:(B // 2 if step == 0 else 3)] if B > 1 else np.zeros(0, np.int64)
        most = int(new.sum()) + 1
        want = oa.kv_slots(cached, new, free, table, page, most)
        got = moe.kv_slots(dev_i32(cached), dev_i32(new), dev_i32(free), dt, page, most)
        torch.cuda.synchronize()
        for name, g, w in zip(("table", "slots", "positions", "cu_new", "counts"), (dt, *got), want):
            assert np.array_equal(host(g), w), (step, name)
        assert host(got[3])[2] == (host(got[0])[:new.sum()] < 0).sum()
        table, cached = want[0], cached + new
        lost.append(int(want[4][2]))
    assert all(lost)


# ----------------------------------------------- more workgroups than the chip holds
@pytest.mark.parametrize("B,Hq,Hkv,prefix,longest,D", [(520, 128, 16, 100, 700, 64), (300, 128, 8, 40, 900, 128)])
def test_attn_decode_many_rows_behind_a_short_prefix(B, Hq, Hkv, prefix, longest, D):
    """The prefix's row blocks take most of the chip or all of it; the own keys' workgroups come behind them."""
    say(f"attn_decode {B} requests x {Hq}/{Hkv} x {D} behind {prefix}")
    lens = [int(n) for n in np.random.default_rng(B).integers(0, 40, B)]
    lens[3], lens[B - 2] = longest, 0
    assert makes_parts(lens, prefix, Hq, Hkv, D, D)
    _, _, case, *_ = run_decode(B, lens, prefix, 16, Hq, Hkv, D, D)
    check_decode(*case, f"attn_decode {B} x {Hq}/{Hkv}")
