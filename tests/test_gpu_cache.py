"""GPU parity of the 4-bit cache's calls, the page calls and the residual stream's norms against the float64 oracle.

Whole numbers -- tables, lengths, counts, codes and scales of values and of keys without norm and rotation, copied
bytes -- are compared exactly, and so is what codes stand for.

Tolerance of an attention output over a 4-bit cache, o = sum_j p_j v_j, from the arithmetic, with u = 2^-24 (float),
r = 2^-8 and f = 2^-11 (half a step of bf16 and f16, relative):
  * the result is rounded once to bf16:                        r |o|
  * each weight is rounded to f16, below 2^-21 of the reference maximum to a multiple of 2^-31 of it:
                                                               f sum p |v| + n 2^-32 max |v|
  * codes times scales are exact in f16; a query's values are, down to 2^-28 of its row's largest, and off by 2^-39
    of it below; a score is a float sum of D exact products, then scaled:
        d = 2 D u max_j sum_i |q_i k_ji| scale + 2^-39 max |q| max_j sum_i |k_ji| scale
    and formed against the rounded maximum in base 2:          t = 4 u (|s|max + 1) log2(e)
    both change a weight by e^(...), numerator and denominator alike:  2 (d + t) sum p |v|
  * 2^x is good to a few ulp and sums of n weights to n u:     2 (8 u + n u) sum p |v|
Tolerance of lse: d + t + (8 + n) u + 2 u |lse|.
"""
import numpy as np
import pytest

import synth
from gpu_util import bf16_to_f64, dev_bf16, dev_f32, dev_i32, dev_u8, host, host_bf16_bits, say
from oracle import attention as oa
from oracle import cache as oc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_group_amd as moe  # noqa: E402

U, R, F = 2.0 ** -24, 2.0 ** -8, 2.0 ** -11
HEADS = [(64, 64), (128, 128), (192, 128)]


def bf16(seed, shape, std=1.0):
    bits = synth.random_bf16(seed, shape, std)
    return bits, bf16_to_f64(bits)


# ------------------------------------------------------------------- decode
class Paged:
    """A 4-bit cache in shuffled pages; rows that no request reaches hold codes of 0xFF and scales that are NaN."""

    def __init__(self, seed, lens, prefix, page, Hkv, D, Dv, spare=3, kg=1.0, vg=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.prefix, self.page = list(lens), prefix, page
        self.blocks = max([1] + [-(-n // page) for n in lens])
        pages = sum(-(-n // page) for n in lens) + -(-prefix // page) + spare
        order = rng.permutation(pages)
        self.k = np.full((pages, Hkv, page, D // 2), 0xFF, np.uint8)
        self.ks = np.full((pages, Hkv, page, D // 16), 0x7F, np.uint8)
        self.v = np.full((pages, Hkv, page, Dv // 2), 0xFF, np.uint8)
        self.vs = np.full((pages, Hkv, Dv // 16, page), 0xFF, np.uint8)
        self.kg, self.vg = kg, vg
        at = 0

        def fill(n):
            nonlocal at
            mine = order[at:at + -(-n // page)]
            at += len(mine)
            kc, ks = oc.nvfp4_rows(rng.standard_normal((n, Hkv, D)) * kg, kg)
            vc, vs = oc.nvfp4_rows(rng.standard_normal((n, Hkv, Dv)) * vg, vg)
            for j in range(n):
                p, r = mine[j // page], j % page
                self.k[p, :, r], self.ks[p, :, r], self.v[p, :, r], self.vs[p, :, :, r] = kc[j], ks[j], vc[j], vs[j]
            return mine

        self.ptab = fill(prefix).astype(np.int64)
        self.table = np.full((len(lens), self.blocks + 2), -9, np.int64)
        for b, n in enumerate(lens):
            mine = fill(n)
            self.table[b, :len(mine)] = mine

    def cache(self):
        return moe.Fp4Cache(dev_u8(self.k), dev_u8(self.ks), dev_u8(self.v), dev_u8(self.vs), self.kg, self.vg)

    def values(self):
        return oc.cache_values(self.k, self.ks, self.v, self.vs, self.kg, self.vg)


def bounds(q, k, v, scale, ref, lse):
    n = len(k)
    big = np.abs(k) @ np.abs(q) * scale
    d = 2 * len(q) * U * big.max() + 2.0 ** -39 * np.abs(q).max() * np.abs(k).sum(-1).max() * scale
    t = 4 * U * (np.abs(k @ q).max() * scale + 1) * 1.4427
    pv, _ = oa.attend(q, k, np.abs(v), scale)
    return (R * np.abs(ref) + (F + 2 * (d + t) + 2 * (8 + n) * U) * pv + n * 2.0 ** -32 * np.abs(v).max(),
            d + t + (8 + n) * U + 2 * U * abs(lse))


def check_decode(c, q, scale, out, lse, what, lens=None):
    k, v = c.values()
    G = q.shape[1] // k.shape[2]
    worst = 0.0
    for b, n in enumerate(c.lens if lens is None else lens):
        at = [(c.ptab[j // c.page], j % c.page) for j in range(c.prefix)] + [(c.table[b][j // c.page], j % c.page) for j in range(n)]
        for h in range(q.shape[1]):
            if not at:
                assert np.all(out[b, h] == 0) and lse[b, h] == -np.inf, f"{what}: request {b} has no key"
                continue
            pg, off = np.array(at).T
            kk, vv = k[pg, off, h // G], v[pg, off, h // G]
            want, wl = oa.attend(q[b, h], kk, vv, scale)
            bo, bl = bounds(q[b, h], kk, vv, scale, want, wl)
            e = np.abs(out[b, h] - want)
            assert np.all(e <= bo), f"{what}: request {b} head {h}: {e.max()} over {bo.min()}"
            assert abs(lse[b, h] - wl) <= bl, f"{what}: lse of request {b} head {h}: {lse[b, h]} for {wl}"
            worst = max(worst, float((e / bo).max()))
    say(f"  {what}: worst error / bound {worst:.2f}")


def run_decode(seed, lens, prefix, page, Hq, Hkv, D, Dv, max_len=None, std=1.0, **kw):
    c = Paged(seed, lens, prefix, page, Hkv, D, Dv, **kw)
    qb, q = bf16(seed + 5, (len(lens), Hq, D), std)
    args = (dev_bf16(qb), c.cache(), dev_i32(c.table)[:, :c.blocks], dev_i32(np.array(lens)),
            max(lens) if max_len is None else max_len)
    pre = dict(prefix_table=dev_i32(c.ptab), prefix_len=prefix)
    out, lse = moe.attn_decode_fp4(*args, **pre, want_lse=True)
    torch.cuda.synchronize()
    return c, q, args, pre, out, lse


def check_run(run, what, **kw):
    c, q, args, pre, out, lse = run
    check_decode(c, q, q.shape[2] ** -0.5, bf16_to_f64(host_bf16_bits(out)), host(lse).astype(np.float64), what, **kw)


@pytest.mark.parametrize("D,Dv", HEADS)
@pytest.mark.parametrize("lens,prefix,page,Hq,Hkv", [
    ([1], 0, 16, 1, 1), ([0], 0, 16, 2, 1), ([5, 0, 33], 0, 16, 4, 2), ([0, 0], 7, 16, 8, 2), ([3, 64, 31, 32], 1, 16, 4, 1),
    ([130, 2, 0], 65, 64, 5, 1), ([300], 300, 32, 8, 8), ([17] * 9, 40, 16, 16, 2), ([63, 65, 15, 16], 0, 128, 16, 1),
    ([2] * 40, 33, 1024, 2, 2), ([3, 0, 70, 130, 1] * 26 + [64] * 3, 70, 16, 8, 4)])               # more workgroups than CUs
def test_decode(D, Dv, lens, prefix, page, Hq, Hkv):
    what = f"attn_decode_fp4 {D}/{Dv} lens={lens[:4]} prefix={prefix} page={page} heads {Hq}/{Hkv}"
    say(what)
    check_run(run_decode(len(lens) * 13 + prefix + D, lens, prefix, page, Hq, Hkv, D, Dv), what)


@pytest.mark.parametrize("D,Dv", HEADS)
@pytest.mark.parametrize("lens,prefix,page,Hq,Hkv", [
    ([3000], 0, 16, 4, 1), ([3000, 0, 1, 65], 0, 64, 8, 2), ([70, 9, 2500], 130, 128, 40, 1),          # heads over 16
    ([700, 1, 5130], 260, 16, 2, 1), ([900, 30], 2600, 32, 8, 1),                                   # a narrow prefix
    ([40, 0, 900] * 5, 2500, 32, 8, 2), ([5] * 70, 1100, 16, 2, 1), ([0] * 9, 3000, 64, 16, 1)])    # many rows
def test_decode_in_parts(D, Dv, lens, prefix, page, Hq, Hkv):
    what = f"attn_decode_fp4 {D}/{Dv} lens={lens[:4]} prefix={prefix} page={page} heads {Hq}/{Hkv}"
    say(what)
    check_run(run_decode(len(lens) * 17 + prefix + D, lens, prefix, page, Hq, Hkv, D, Dv), what)


@pytest.mark.parametrize("D,Dv", HEADS)
@pytest.mark.parametrize("lens,prefix,page,Hq,Hkv", [
    ([70, 0, 1] * 5 + [64, 500], 30900, 64, 64, 4), ([9] * 20, 26300, 16, 64, 8), ([0] * 95 + [33], 22000, 1024, 16, 2),
    ([33] * 30, 28000, 32, 40, 1)])                                                                   # heads over 16
def test_decode_behind_a_long_prefix(D, Dv, lens, prefix, page, Hq, Hkv):
    """Workgroups of 128 rows (partial last blocks, pages inside a tile and over it); all requests in 64 bits on the device."""
    what = f"attn_decode_fp4 {D}/{Dv} {len(lens)} requests prefix={prefix} page={page} heads {Hq}/{Hkv}"
    say(what)
    c, q, _, _, out, lse = run_decode(len(lens) + D, lens, prefix, page, Hq, Hkv, D, Dv)
    k, v = (torch.from_numpy(x).cuda() for x in c.values())
    qd, G, scale = torch.from_numpy(q).cuda(), Hq // Hkv, D ** -0.5
    at = lambda pages, n: (torch.as_tensor(np.asarray(pages)[np.arange(n) // page], device="cuda"),
                           torch.as_tensor(np.arange(n) % page, device="cuda"))
    pk, pv = k[at(c.ptab, prefix)].transpose(0, 1), v[at(c.ptab, prefix)].transpose(0, 1)     # [Hkv, n, D]
    worst = 0.0
    for b, n in enumerate(lens):
        kk = torch.cat((pk, k[at(c.table[b], n)].transpose(0, 1)), 1) if n else pk
        vv = torch.cat((pv, v[at(c.table[b], n)].transpose(0, 1)), 1) if n else pv
        N, qq = prefix + n, qd[b].view(Hkv, G, D)
        s = qq @ kk.transpose(1, 2).contiguous() * scale
        wl = s.logsumexp(-1, keepdim=True)
        p = (s - wl).exp()
        ref, mass = p @ vv, p @ vv.abs()
        d = 2 * D * U * (qq.abs() @ kk.abs().transpose(1, 2).contiguous()).amax(-1, keepdim=True) * scale
        d = d + 2.0 ** -39 * qq.abs().amax(-1, keepdim=True) * kk.abs().sum(-1).amax(-1)[:, None, None] * scale
        t = 4 * U * (s.abs().amax(-1, keepdim=True) + 1) * 1.4427
        bo = R * ref.abs() + (F + 2 * (d + t) + 2 * (8 + N) * U) * mass + N * 2.0 ** -32 * vv.abs().amax((1, 2))[:, None, None]
        e = (out[b].double().view(Hkv, G, Dv) - ref).abs()
        assert (e <= bo).all(), f"{what}: request {b}: {(e / bo).max()}"
        el = (lse[b].double().view(Hkv, G, 1) - wl).abs()
        assert (el <= d + t + (8 + N) * U + 2 * U * wl.abs()).all(), f"{what}: lse of request {b}"
        worst = max(worst, float((e / bo).max()))
    say(f"  {what}: worst error / bound {worst:.2f}")


def test_decode_sharp_flat_and_scaled():
    for std, kg, vg in ((4.0, 1.0, 1.0), (0.01, 0.125, 64.0), (300.0, 2.0 ** -7, 2.0 ** -20)):
        for lens, prefix in (([200, 3], 77), ([4000], 0), ([40] * 30, 1000)):
            r = run_decode(3, lens, prefix, 32, 8, 2, 128, 128, std=std, kg=kg, vg=vg)
            check_run(r, f"attn_decode_fp4 {lens[:2]} behind {prefix}, queries {std}, globals {kg} {vg}")


def test_decode_bounds_on_the_host_side():
    """max_len over the lengths; lengths over max_len count as max_len."""
    for lens in ([100, 0, 37], [100, 0, 3000]):
        r = run_decode(9, lens, 20, 16, 4, 2, 128, 128, max_len=-(-max(lens) // 16) * 16)
        check_run(r, "attn_decode_fp4 max_len over the lengths")
        args, pre = r[2], r[3]
        short, _ = moe.attn_decode_fp4(*args[:4], 37, **pre)
        cut, _ = moe.attn_decode_fp4(*args[:3], dev_i32(np.minimum(lens, 37)), 37, **pre)
        torch.cuda.synchronize()
        assert torch.equal(short, cut)


@pytest.mark.parametrize("D,Dv", HEADS)
@pytest.mark.parametrize("lens,prefix", [([33, 200, 0], 50), ([33, 6000, 0], 50), ([33, 200, 0] * 6, 1500)])
def test_decode_agrees_with_the_gathered_cache(D, Dv, lens, prefix):
    """The bf16 decode over the values that the codes stand for: twice the tolerance (its own weights round to 2^-8)."""
    say(f"attn_decode_fp4 against attn_decode {D}/{Dv} {lens[:3]}")
    c, q, args, pre, out, lse = run_decode(5, lens, prefix, 16, 8, 2, D, Dv)
    k, v = c.values()
    ok = ~np.isnan(k).any(axis=(2, 3))
    to = lambda a: dev_f32(np.where(ok[:, :, None, None], a, 0).astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    ref, rl = moe.attn_decode(args[0], to(k), to(v), *args[2:], **pre, want_lse=True)
    torch.cuda.synchronize()
    assert (lse - rl).abs().nan_to_num(0).max() < 1e-4
    vmax = float(np.abs(np.where(ok[:, :, None, None], v, 0)).max())
    assert (out.float() - ref.float()).abs().max() <= 4 * R * vmax


@pytest.mark.parametrize("D,Dv", HEADS)
@pytest.mark.parametrize("lens,prefix", [([33, 200, 0], 50), ([33, 6000, 0], 0), ([33, 0, 200] * 6, 1500)])
def test_decode_lse_agrees_with_the_gathered_cache(D, Dv, lens, prefix):
    """-inf for the same rows, a number for every other, as near as test_decode_agrees_with_the_gathered_cache asks."""
    say(f"attn_decode_fp4 against attn_decode {D}/{Dv} {lens[:3]}: lse")
    c, q, args, pre, out, lse = run_decode(6, lens, prefix, 16, 8, 2, D, Dv)
    k, v = c.values()
    to = lambda a: dev_f32(np.nan_to_num(a, nan=0.0).astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    ref, rl = moe.attn_decode(args[0], to(k), to(v), *args[2:], **pre, want_lse=True)
    torch.cuda.synchronize()
    none = torch.tensor([n + prefix == 0 for n in lens], device="cuda")[:, None].expand(lse.shape)
    assert torch.equal(lse == -np.inf, none) and torch.equal(rl == -np.inf, none)
    assert torch.isfinite(lse[~none]).all() and torch.isfinite(rl[~none]).all() and torch.isfinite(out.float()).all()
    assert (lse[~none] - rl[~none]).abs().max() < 1e-4


def test_decode_bad_entries_stay_inside():
    """Table entries that are no page never address memory outside the cache (results of those requests: unspecified)."""
    say("attn_decode_fp4: bad table entries")
    for lens in ([40, 40], [40, 5000]):
        c, q, args, pre, out, lse = run_decode(30, lens, 20, 16, 2, 1, 64, 64)
        t = args[2].clone()
        t[0, 1], t[0, 2] = 1 << 30, -(1 << 30)
        bad, _ = moe.attn_decode_fp4(args[0], args[1], t, *args[3:], **pre)
        torch.cuda.synchronize()
        assert torch.equal(bad[1], out[1])


@pytest.mark.parametrize("D,Dv", HEADS)
@pytest.mark.parametrize("lens", [[20, 300], [20, 6000], [20, 300] * 12])
def test_decode_not_finite(D, Dv, lens):
    """A scale that is NaN reaches the rows that see it and no other; queries that are not finite their own row."""
    say(f"attn_decode_fp4 {D}/{Dv}: NaN scales and queries")
    c, q, args, pre, out, lse = run_decode(8, lens, 70, 16, 8, 2, D, Dv)
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    cache = args[1]
    page, row = int(c.table[0][1]), 3                                 # key 19 of request 0, the last
    cache.v_scale[page, 1, 2, row] = 0x7F
    got, gl = moe.attn_decode_fp4(*args, **pre, want_lse=True)
    torch.cuda.synchronize()
    assert same(got[1:], out[1:]) and same(got[0, :4], out[0, :4]) and torch.equal(gl, lse)
    assert torch.isnan(got[0, 4:, 32:48].float()).all() and same(got[0, 4:, :32].contiguous(), out[0, 4:, :32].contiguous())
    cache.k_scale[page, 0, row, 0] = 0xFF
    got, gl = moe.attn_decode_fp4(*args, **pre, want_lse=True)
    torch.cuda.synchronize()
    assert same(got[1:], out[1:]) and torch.isnan(got[0, :4].float()).all() and torch.isnan(gl[0, :4]).all()
    x = args[0].clone()
    x[1, 3, 5], x[1, 0, 7] = float("nan"), float("inf")
    got, gl = moe.attn_decode_fp4(x, *args[1:], **pre, want_lse=True)
    torch.cuda.synchronize()
    assert torch.isnan(got[1, 3].float()).all() and same(got[1, 1:3], out[1, 1:3]) and same(got[1, 4:], out[1, 4:])


def test_decode_queries_of_any_size():
    """Rows of huge, tiny and zero queries side by side: each keeps its own scale."""
    say("attn_decode_fp4: queries from 2^-120 to 2^100")
    c, q, args, pre, out, lse = run_decode(12, [90, 0, 31], 40, 16, 4, 1, 128, 128)
    x = args[0].clone()
    x[:, 0] *= 2.0 ** -120
    x[:, 1] = 0
    x[:, 2] *= 2.0 ** 60
    got, gl = moe.attn_decode_fp4(x, args[1], *args[2:], **pre, want_lse=True)
    one, ol = moe.attn_decode_fp4(torch.zeros_like(x), *args[1:], **pre, want_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(got[:, 0], one[:, 0]) and torch.equal(got[:, 1], one[:, 1]) and torch.equal(gl[:, :2], ol[:, :2])
    assert torch.equal(got[:, 3], out[:, 3])
    k, v = c.values()
    at = [(c.ptab[j // 16], j % 16) for j in range(40)] + [(c.table[0][j // 16], j % 16) for j in range(90)]
    pg, off = np.array(at).T
    best = int(np.argmax(k[pg, off, 0] @ q[0, 2]))                    # its score wins by far: its value alone
    assert np.array_equal(bf16_to_f64(host_bf16_bits(got))[0, 2], v[pg[best], off[best], 0])


FORMS = [([90, 0, 31], 40, 4, 1), ([5000, 3, 70], 0, 8, 2), ([90, 30], 2600, 8, 1), ([40, 0, 90] * 5, 2500, 8, 2)]   # alone, own keys in parts, prefix in parts, of 128 rows


@pytest.mark.parametrize("D,Dv", HEADS)
@pytest.mark.parametrize("lens,prefix,Hq,Hkv", FORMS)
@pytest.mark.parametrize("kg", [1.0, 2.0 ** -20, 2.0 ** -32])
def test_decode_tiny_queries_and_globals(D, Dv, lens, prefix, Hq, Hkv, kg):
    """Scores next to zero weigh all keys alike, and keys that are not there count as none, however small the queries (the
    smallest numbers of bf16 among them) and the keys' global scale are."""
    say(f"attn_decode_fp4 {D}/{Dv} lens={lens[:3]} prefix={prefix}: tiny queries, keys of 2^{int(np.log2(kg))}")
    c, q, args, pre, _, _ = run_decode(21, lens, prefix, 16, Hq, Hkv, D, Dv, kg=kg)
    x = torch.from_numpy(q).float()
    for h, e in enumerate((-101, -119, -126, -132)):
        x[:, h::4] *= 2.0 ** e
    x = x.to(torch.bfloat16)
    out, lse = moe.attn_decode_fp4(x.cuda(), *args[1:], **pre, want_lse=True)
    torch.cuda.synchronize()
    check_decode(c, x.double().numpy(), D ** -0.5, bf16_to_f64(host_bf16_bits(out)), host(lse).astype(np.float64), "tiny queries")


def test_decode_keys_of_zeros_and_huge_queries():
    """Scores that are zero stay zero where the factor they are multiplied by is past float's range."""
    say("attn_decode_fp4: keys of zeros, queries of 2^120, scales at both ends of float's range")
    for lens, prefix, Hq, Hkv in FORMS:
        c, q, args, pre, _, _ = run_decode(22, lens, prefix, 16, Hq, Hkv, 128, 128, kg=2.0 ** 32)
        for t in (c.k, c.ks):
            t[:] = 0
        x = args[0] * 2.0 ** 120
        assert torch.isfinite(x.float()).all()
        out, lse = moe.attn_decode_fp4(x, c.cache(), *args[2:], **pre, want_lse=True)
        torch.cuda.synchronize()
        check_decode(c, bf16_to_f64(host_bf16_bits(x)), 128 ** -0.5, bf16_to_f64(host_bf16_bits(out)),
                     host(lse).astype(np.float64), "keys of zeros")
        # scale and global past float's range, the queries' size in it again: the bits of the same product at size one
        c, q, args, pre, _, _ = run_decode(23, lens, prefix, 16, Hq, Hkv, 128, 128)
        run = lambda q, cache, scale: moe.attn_decode_fp4(q, cache, *args[2:], **pre, scale=scale, want_lse=True)  # noqa: E731
        want = run(args[0], args[1], 2.0 ** 29), run(args[0] * 0, args[1], 1.0)
        c.kg = 2.0 ** 32
        got = [run(args[0] * 2.0 ** -100, c.cache(), 2.0 ** 97)]
        c.kg = 2.0 ** -32
        got.append(run(args[0] * 2.0 ** 100, c.cache(), 2.0 ** -130))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


@pytest.mark.parametrize("lens,prefix,Hq,Hkv,every", [
    ([1000], 0, 2, 1, 8), ([300] * 260, 0, 1, 1, 4),                                                  # alone: 8 and 4 waves
    ([32798], 0, 8, 8, 4), ([9, 0, 70], 32790, 64, 8, 4), ([40, 0, 90] * 5, 2500, 8, 2, 1)])          # parts: own keys, prefix, 128 rows
@pytest.mark.parametrize("bits", [24, 25, 26])
@pytest.mark.parametrize("sign", [1, -1])
def test_decode_maxima_that_rise_by_8_far_from_zero(lens, prefix, Hq, Hkv, every, bits, sign):
    """Scores of +-1.25 x 2^24 .. 2^26 (base 2), where maxima are rounded to multiples of 2 to 8, the largest in some tiles 8
    over those in others: of a wave's successive tiles the second's has weights 2^8 the first's.

    Scores are integers that float holds and the scale times log2(e) is 1 in float, so the weights are powers of two, exactly:
    what is left is the result's rounding and that of the sums.  lse: the scale, ln 2, and the maximum with the weights' sum
    are each rounded once, and the scale is 2^-24 off ln 2: 6 U of it."""
    say(f"attn_decode_fp4 lens={lens[:2]} prefix={prefix}: maxima of {sign} x 1.25 x 2^{bits} that rise by 8")
    c = Paged(24, lens, prefix, 16, Hkv, 128, 128)
    c.k[:], c.ks[:] = 0, 0

    def key(pages, n):
        low = high = 0
        for t in range(-(-n // 64)):
            rows = [(pages[j // 16], j % 16) for j in range(64 * t, min(64 * t + 64, n))]
            if sign < 0:                                              # the others far below
                for p, r in rows:
                    c.k[p, :, r, 0], c.ks[p, :, r, 0] = 7, 0x78       # 6 x 256
            p, r = rows[0]
            c.k[p, :, r, 0], c.ks[p, :, r, 0] = 6, 0x78               # 4 x 256
            if t // every % 2:
                c.k[p, :, r, 8], c.ks[p, :, r, 1] = 2, 0x38           # 1
                high += 1
            else:
                low += 1
        return low, high

    counts = [key(c.ptab, prefix)] + [key(c.table[b], n) for b, n in enumerate(lens)]
    q = np.zeros((len(lens), Hq, 128))
    q[:, :, 0], q[:, :, 16] = sign * 1.25 * 2.0 ** (bits - 10), 8.0
    out, lse = moe.attn_decode_fp4(torch.from_numpy(q).to(torch.bfloat16).cuda(), c.cache(), dev_i32(c.table)[:, :c.blocks],
                                   dev_i32(np.array(lens)), max(lens), prefix_table=dev_i32(c.ptab), prefix_len=prefix,
                                   scale=float(np.float32(np.log(2.0))), want_lse=True)
    torch.cuda.synchronize()
    out, lse = bf16_to_f64(host_bf16_bits(out)), host(lse).astype(np.float64)
    values = c.values()[1]

    def sums(pages, n):
        s = np.zeros((2, Hkv, 128))
        for t in range(-(-n // 64)):
            s[t // every % 2] += values[pages[64 * t // 16], 0]       # a tile's first key is a page's first row
        return s

    front, G = sums(c.ptab, prefix), Hq // Hkv
    for b, n in enumerate(lens):
        s = front + sums(c.table[b], n)
        low, high = counts[0][0] + counts[b + 1][0], counts[0][1] + counts[b + 1][1]
        if low + high == 0:
            assert np.all(out[b] == 0) and np.all(lse[b] == -np.inf)
            continue
        w = 2.0 ** -8 if high else 1.0
        top, mass = sign * 1.25 * 2.0 ** bits + (8 if high else 0), w * low + high
        want = ((w * s[0] + s[1]) / mass).repeat(G, 0)
        # sums of low + high weights and products, the division
        assert np.all(np.abs(out[b] - want) <= R * np.abs(want) + 2 * (low + high + 8) * U * np.abs(values[np.isfinite(values)]).max()), b
        wl = top * np.log(2.0) + np.log(mass)
        assert np.all(np.abs(lse[b] - wl) <= 6 * U * abs(wl) + (low + high + 8) * U), (b, lse[b], wl)


def test_decode_other_stream_graph_and_workspace():
    say("attn_decode_fp4: repeated, on another stream, in graphs that share a workspace")
    for lens, prefix in (([100, 3], 40), ([5000, 3], 0), ([100, 3] * 20, 900)):
        c, q, args, pre, ref, rl = run_decode(14, lens, prefix, 32, 8, 2, 128, 128)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        out, lse = moe.attn_decode_fp4(*args, **pre, want_lse=True, stream=s)
        s.synchronize()
        assert torch.equal(out, ref) and torch.equal(lse, rl)
        need = moe.attn_decode_fp4_workspace_bytes(len(lens), prefix, max(lens), 8, 2, 128, 128)
        ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        outs, graphs = [torch.zeros_like(out) for _ in range(2)], []
        for o in outs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                moe.attn_decode_fp4(*args, **pre, out=o, workspace=ws)
            graphs.append(g)
        for i in range(3):
            args[0].mul_(1.5 if i else 1.0)
            for o, g in zip(outs, graphs):
                o.zero_()
                g.replay()
            eager, _ = moe.attn_decode_fp4(*args, **pre)
            torch.cuda.synchronize()
            assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager), i


def test_decode_strides():
    """Queries cut from a projection's rows, heads before tokens; output into a wider buffer, rows beside it kept."""
    say("attn_decode_fp4: strides")
    for lens in ([50, 7, 0], [50, 7, 4000]):
        c, q, args, pre, ref, _ = run_decode(15, lens, 30, 16, 6, 2, 128, 128)
        wide = torch.full((3, 6 * 128 + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        rows = torch.zeros((3, 6 * 128 + 40), dtype=torch.bfloat16, device="cuda")
        rows[:, :768] = args[0].flatten(1)
        moe.attn_decode_fp4(rows[:, :768].unflatten(1, (6, 128)), *args[1:], **pre, out=wide[:, :768].unflatten(1, (6, 128)))
        t = args[0].transpose(0, 1).contiguous().transpose(0, 1)
        out2, _ = moe.attn_decode_fp4(t, *args[1:], **pre)
        torch.cuda.synchronize()
        assert torch.equal(wide[:, :768], ref.flatten(1)) and (wide[:, 768:] == 7).all() and torch.equal(out2, ref)


def test_decode_far_pages():
    """Rows whose byte offsets pass 2^32 in every one of the cache's tensors."""
    say("attn_decode_fp4: a cache of 5 GiB of codes")
    D, page, H = 128, 1024, 8
    pages = (5 << 30) // (page * H * D // 2)
    cache = moe.Fp4Cache.zeros(pages, page, H, D, D)
    lens, near = [70, 1500], [3, 4, 5]
    far = [pages - 2, pages - 1, pages - 7]
    for p in near:
        for x in (cache.k, cache.v):
            x[p].random_(0, 256)
        for x in (cache.k_scale, cache.v_scale):
            x[p].random_(0x28, 0x40)
    for a, b in zip(near, far):
        for x in cache.buffers:
            x[b] = x[a]
    q = dev_bf16(synth.random_bf16(1, (2, 16, D)))
    r = []
    for t in (near, far):
        table = torch.tensor([[t[0], -1], [t[1], t[2]]], dtype=torch.int32, device="cuda")
        r.append(moe.attn_decode_fp4(q, cache, table, dev_i32(np.array(lens)), 1500, want_lse=True))
        r[-1] += moe.kv_gather_fp4(cache, table, dev_i32(np.array([0, 70, 1570])), 1570)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*r)) and r[0][2].abs().max() > 0


# ------------------------------------------------------- write and read back
@pytest.mark.parametrize("T,Hq,Hkv,D,Dv,rot,inter,norm,page,keep", [
    (1, 1, 1, 64, 64, 64, False, True, 16, True), (5, 8, 2, 128, 128, 128, False, True, 16, False),
    (33, 5, 5, 192, 128, 64, True, True, 32, True), (300, 4, 1, 128, 128, 32, True, False, 64, True),
    (70, 16, 4, 64, 64, 32, False, True, 32, False), (9, 3, 3, 192, 128, 192, False, False, 16, True),
    (17, 2, 1, 128, 48, 0, False, True, 16, True), (129, 12, 4, 192, 128, 96, False, True, 128, True)])
def test_write(T, Hq, Hkv, D, Dv, rot, inter, norm, page, keep):
    say(f"qk_norm_rope_fp4 T={T} D={D} rot={rot} interleaved={inter} norm={norm}")
    rng = np.random.default_rng(T + D + rot)
    width = Hq * D + Hkv * D + Hkv * Dv
    bits, x = bf16(T, (T, width + 8), 2.0)                          # 8 more columns: rows are not dense
    x[:, Hq * D:Hq * D + 16] = 0
    bits[:, Hq * D:Hq * D + 16] = 0                                 # a block of zeros
    rows = dev_bf16(bits)
    cut = lambda a, i, h, d: a[:, i:i + h * d].reshape(T, h, d) if isinstance(a, np.ndarray) else a[:, i:i + h * d].unflatten(1, (h, d))  # noqa: E731
    at = (0, Hq * D, Hq * D + Hkv * D)
    qw, kw = (rng.uniform(0.5, 1.5, D).astype(np.float32) if norm else None for _ in range(2))
    P = 50
    ang = rng.uniform(0, 6.3, (P, rot // 2))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32) if rot else None
    pos = rng.integers(-3, P + 3, T)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T]
    slots[::7] = -1
    if T > 3:
        slots[3] = pages * page                                     # outside the cache: skipped
    start = [rng.integers(0, 256, s).astype(np.uint8) for s in (
        (pages, Hkv, page, D // 2), (pages, Hkv, page, D // 16), (pages, Hkv, page, Dv // 2), (pages, Hkv, Dv // 16, page))]
    cache = moe.Fp4Cache(*[dev_u8(a) for a in start], k_global=0.5, v_global=2.0)
    q_want = oa.norm_rope(cut(x, at[0], Hq, D), qw, 1e-6, cs, pos, inter)
    k_want = oa.norm_rope(cut(x, at[1], Hkv, D), kw, 1e-6, cs, pos, inter)
    f = lambda a: None if a is None else dev_f32(a)  # noqa: E731
    q, k = moe.qk_norm_rope_fp4(cut(rows, at[0], Hq, D), cut(rows, at[1], Hkv, D), cut(rows, at[2], Hkv, Dv), dev_i32(pos), f(cs),
                                cache, dev_i32(slots), f(qw), f(kw), 1e-6, inter, want_k=keep)
    torch.cuda.synchronize()

    def near(got, want, what):
        # one rounding to bf16; float before it: the norm's sum of D squares, three products and a sum
        big = np.abs(want).max(axis=-1, keepdims=True)
        assert np.all(np.abs(got - want) <= R * np.abs(want) + (D + 16) * U * big), what

    near(bf16_to_f64(host_bf16_bits(q)), q_want, "q")
    assert k is None if not keep else True
    if keep:
        near(bf16_to_f64(host_bf16_bits(k)), k_want, "k")
    # the cache: every byte
    kc, ks = oc.nvfp4_rows(k_want, 0.5)
    vc, vs = oc.nvfp4_rows(cut(x, at[2], Hkv, Dv), 2.0)
    want = [a.copy() for a in start]
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            p, r = s // page, s % page
            want[0][p, :, r], want[1][p, :, r], want[2][p, :, r], want[3][p, :, :, r] = kc[t], ks[t], vc[t], vs[t]
    for name, g, w in zip(("k", "k_scale", "v", "v_scale"), cache.buffers, want):
        assert np.array_equal(host(g), w), name


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter", [(33, 5, 5, 192, 64, True), (70, 16, 4, 64, 32, False), (129, 6, 2, 128, 128, False),
                                                  (6000, 64, 4, 192, 64, True), (6000, 64, 4, 192, 96, False)])   # the last two past 128 MB
def test_write_in_place(T, Hq, Hkv, D, rot, inter):
    """q_out and k_out the rows of the projection that q and k come from: the same bits, v and the columns beside them kept."""
    say(f"qk_norm_rope_fp4 in place, T={T} heads {Hq}/{Hkv} x {D}")
    torch.manual_seed(T + D)
    rows = torch.randn((T, (Hq + 2 * Hkv) * D + 8), device="cuda").to(torch.bfloat16)
    w = torch.rand((2, D), device="cuda") + 0.5
    cs = torch.rand((T, rot), device="cuda") * 2 - 1
    pages = -(-T // 16)
    slots = torch.randperm(pages * 16, device="cuda")[:T].int()

    def call(rows, **kw):
        q, k, v = (rows[:, i * D:(i + h) * D].unflatten(1, (h, D)) for i, h in ((0, Hq), (Hq, Hkv), (Hq + Hkv, Hkv)))
        cache = moe.Fp4Cache.zeros(pages, 16, Hkv, D, D)
        kw = dict(q_out=q, k_out=k) if kw else {}
        return [*moe.qk_norm_rope_fp4(q, k, v, torch.arange(T, device="cuda").int(), cs, cache, slots, w[0], w[1], 1e-6, inter, **kw),
                *cache.buffers]

    want = call(rows)
    own = rows.clone()
    got = call(own, in_place=True)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(own[:, (Hq + Hkv) * D:], rows[:, (Hq + Hkv) * D:])
    assert not torch.equal(own[:, :D], rows[:, :D])


def test_write_special_values():
    """Without norm and rotation the rows are quantize_nvfp4's, byte for byte, infinities, NaN and ties among them."""
    say("qk_norm_rope_fp4: any bf16 values, against quantize_nvfp4")
    rng = np.random.default_rng(4)
    T, H, D = 512, 2, 128
    bits = rng.integers(0, 1 << 16, (T, H, D)).astype(np.uint16)    # every exponent, NaN and infinities too
    bits[:256] = synth.random_bf16(3, (256, H, D), 4.0)
    bits[0, 0, :16], bits[1, 1, 3], bits[2, 1, 5] = 0x8000, 0x7F80, 0x7FC0
    x = dev_bf16(bits)
    for g in (1.0, 2.0 ** -6):
        cache = moe.Fp4Cache.zeros(T // 16, 16, H, D, D, g, g)
        moe.qk_norm_rope_fp4(x, x, x, None, None, cache, dev_i32(np.arange(T)), want_k=False)
        c, s = moe.quantize_nvfp4(x.reshape(T * H, D), g)
        torch.cuda.synchronize()
        want_c = host(c).reshape(T // 16, 16, H, D // 2).swapaxes(1, 2)
        want_s = host(s).reshape(T // 16, 16, H, D // 16).swapaxes(1, 2)
        assert np.array_equal(host(cache.v), want_c) and np.array_equal(host(cache.k), want_c)
        assert np.array_equal(host(cache.k_scale), want_s) and np.array_equal(host(cache.v_scale), want_s.swapaxes(2, 3))


@pytest.mark.parametrize("D,Dv,page,prefix", [(64, 64, 16, 0), (128, 128, 64, 40), (192, 128, 32, 33), (16, 48, 16, 5)])
def test_gather(D, Dv, page, prefix):
    say(f"kv_gather, kv_gather_fp4 {D}/{Dv} page={page} prefix={prefix}")
    lens = [70, 0, 1, 16, 33]
    c = Paged(6, lens, prefix, page, 3, D, Dv, kg=0.25, vg=4.0)
    counts = [n + prefix for n in lens]
    counts[0] = min(counts[0], 50)                                  # the first keys only
    cu = np.cumsum([3] + counts)                                    # three rows before, two behind the sequences
    total = cu[-1] + 2
    ok, ov = (torch.full((total, 3, d), 7.0, dtype=torch.bfloat16, device="cuda") for d in (D, Dv))
    t = dev_i32(c.table)
    moe.kv_gather_fp4(c.cache(), t, dev_i32(cu), total, dev_i32(c.ptab), prefix, k_out=ok, v_out=ov)
    k, v = c.values()
    torch.cuda.synchronize()
    for got, rows, d in ((ok, k, D), (ov, v, Dv)):
        want = oc.gather(rows, c.table, cu, total, c.ptab, prefix, np.full((total, 3, d), 7.0))
        assert np.array_equal(bf16_to_f64(host_bf16_bits(got)), want)
    # a bf16 cache, heads-first outputs
    kb, vb = synth.random_bf16(1, k.shape), synth.random_bf16(2, v.shape)
    ok2, ov2 = (torch.zeros((3, total, d), dtype=torch.bfloat16, device="cuda").transpose(0, 1) for d in (D, Dv))
    moe.kv_gather(dev_bf16(kb), dev_bf16(vb), t, dev_i32(cu), total, dev_i32(c.ptab), prefix, k_out=ok2, v_out=ov2)
    torch.cuda.synchronize()
    for got, rows, d in ((ok2, kb, D), (ov2, vb, Dv)):
        want = oc.gather(rows, c.table, cu, total, c.ptab, prefix, np.zeros((total, 3, d), np.uint16))
        assert np.array_equal(host_bf16_bits(got.contiguous()), want)


def test_gather_pages_that_are_not_there():
    say("kv_gather: entries of -1, past the table, outside the cache; offsets that descend stay inside")
    c = Paged(6, [40, 40], 0, 16, 1, 64, 64)
    t = c.table[:, :3].copy()
    t[0, 1], t[1, 2] = -1, 1 << 20
    cu = np.array([0, 60, 100])                                     # keys 48 .. 59 are past the table's three columns
    k, v = moe.kv_gather_fp4(c.cache(), dev_i32(t), dev_i32(cu), 100)
    torch.cuda.synchronize()
    for got, rows in zip((k, v), c.values()):
        want = oc.gather(rows, t, cu, 100, [], 0, np.zeros((100, 1, 64)))
        assert np.array_equal(bf16_to_f64(host_bf16_bits(got))[:40], want[:40])
        assert np.all(want[48:60] == 0) and np.all(host(got.float())[48:60] == 0) and np.all(host(got.float())[92:] == 0)
    moe.kv_gather_fp4(c.cache(), dev_i32(t), dev_i32(np.array([-5, 300, 20])), 100)
    torch.cuda.synchronize()


def test_write_gather_other_stream_and_graph():
    say("qk_norm_rope_fp4 and kv_gather_fp4: on another stream, in a graph")
    T, H, D = 100, 2, 128
    x = dev_bf16(synth.random_bf16(3, (T, H, D), 2.0))
    cache = moe.Fp4Cache.zeros(8, 16, H, D, D)
    slots, cu, table = dev_i32(np.arange(T)), dev_i32(np.array([0, T])), dev_i32(np.arange(8)[None])
    w = torch.ones(D, device="cuda")

    def step(**kw):
        q, k = moe.qk_norm_rope_fp4(x, x, x, None, None, cache, slots, w, w, **kw)
        return (q, k) + moe.kv_gather_fp4(cache, table, cu, T, **kw)

    ref = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    q, k, kk, vv = (torch.zeros_like(a) for a in ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.qk_norm_rope_fp4(x, x, x, None, None, cache, slots, w, w, q_out=q, k_out=k)
        moe.kv_gather_fp4(cache, table, cu, T, k_out=kk, v_out=vv)
    for i in range(3):
        x.mul_(1.25 if i else 1.0)
        g.replay()
        got = [a.clone() for a in (q, k, kk, vv)]
        for b in cache.buffers:
            b.zero_()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


# -------------------------------------------------------------------- pages
def pool(seed, rows, blocks, page, pages, shapes, lens=None, beyond=0):
    """A table over a pool of pages with random content; rows may share pages, some entries are no page (``beyond`` pages
    follow that no row may hold), entries past a length are any number."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(-2, blocks * page + 3, rows) if lens is None else np.array(lens)
    table = rng.integers(0, pages, (rows, blocks + 2))
    table[rng.random(table.shape) < 0.05] = -1
    table[rng.random(table.shape) < 0.02] = pages + beyond + 5
    bufs = [rng.integers(0, 256, (pages,) + s).astype(np.uint8) for s in shapes]
    return table.astype(np.int32), lens.astype(np.int32), bufs


SHAPES = [(16,), (3, 16, 64), (4096 + 48,), (2, 8, 32)]


@pytest.mark.parametrize("rows,blocks,page,forks,free", [
    (2, 1, 1, 1, 3), (5, 4, 16, 3, 9), (40, 9, 32, 20, 12), (700, 3, 64, 350, 400), (3, 2, 1024, 0, 0), (300, 5, 16, 150, 0)])
@pytest.mark.parametrize("shapes", [SHAPES[:1], SHAPES])
def test_fork(rows, blocks, page, forks, free, shapes):
    say(f"kv_fork {forks} of {rows} rows, page {page}, {free} free, {len(shapes)} buffers")
    rng = np.random.default_rng(rows + forks)
    used, pages = 50, 50 + free + 4
    table, lens, bufs = pool(rows, rows, blocks, page, used, shapes, beyond=pages - used)
    order = rng.permutation(rows)
    children, parents = order[:forks].copy(), rng.choice(order[forks:], forks) if forks else order[:0]
    bufs = [np.concatenate([b, rng.integers(0, 256, (pages - used,) + b.shape[1:]).astype(np.uint8)]) for b in bufs]
    if forks > 2:
        parents[1], children[2] = -1, rows                           # not rows of the table: nothing
    fp = used + rng.permutation(pages - used)[:free]
    want = oc.fork(table[:, :blocks], lens, parents, children, fp, page, bufs)
    dt, dl, db = dev_i32(table), dev_i32(lens), [dev_u8(b) for b in bufs]
    counts = moe.kv_fork(dt[:, :blocks], dl, dev_i32(parents), dev_i32(children), dev_i32(fp), page, db)
    torch.cuda.synchronize()
    assert np.array_equal(host(dt)[:, :blocks], want[0]) and np.array_equal(host(dt)[:, blocks:], table[:, blocks:])
    assert np.array_equal(host(dl), want[1]) and np.array_equal(host(counts), want[3])
    for g, w in zip(db, want[2]):
        assert np.array_equal(host(g), w)


@pytest.mark.parametrize("forks,free", [(1, 1), (6, 6), (700, 690), (5000, 60)])
def test_fork_of_large_pages(forks, free):
    """Pages that several workgroups copy, in the last part not a whole step; by fewer each for many forks, by one for 5000."""
    say(f"kv_fork {forks} of large pages, {free} free")
    rng = np.random.default_rng(forks)
    shape = (1 << 20) + (1 << 14) + 48 if forks <= 6 else 100016 if forks < 1000 else 40000
    rows, used = 2 * forks, 12
    table, lens, (buf,) = pool(forks, rows, 3, 16, used, [(shape,)], beyond=free)
    buf = np.concatenate([buf, np.zeros((free, shape), np.uint8)])
    parents, children = rng.integers(0, forks, forks), forks + rng.permutation(forks)
    fp = used + rng.permutation(free)
    want = oc.fork(table[:, :3], lens, parents, children, fp, 16, [buf])
    dt, dl, db = dev_i32(table), dev_i32(lens), dev_u8(buf)
    counts = moe.kv_fork(dt[:, :3], dl, dev_i32(parents), dev_i32(children), dev_i32(fp), 16, [db])
    torch.cuda.synchronize()
    assert np.array_equal(host(dt)[:, :3], want[0]) and np.array_equal(host(dl), want[1]) and np.array_equal(host(counts), want[3])
    assert np.array_equal(host(db), want[2][0])


def test_fork_from_a_list_with_an_end():
    """The whole list of kv_free_pages, -1 behind its pages, and an entry past the pool: no page left there."""
    table, lens, bufs = pool(8, 12, 3, 16, 20, SHAPES, lens=[20, 33] + [0] * 10)
    par, chi = np.array([0, 1, 0, 1, 0, 1]), np.arange(2, 8)
    free, counts = moe.kv_free_pages(dev_i32(table)[:, :3], dev_i32(lens), 16, 20)
    for fp in (host(free)[host(counts)[0] - 4:], np.concatenate([host(free)[:2], [20, 2 ** 31 - 1, -7], host(free)[2:]]), np.full(9, -1)):
        say(f"kv_fork, free pages {fp.tolist()}")
        want = oc.fork(table[:, :3], lens, par, chi, fp, 16, bufs)
        dt, dl, db = dev_i32(table), dev_i32(lens), [dev_u8(b) for b in bufs]
        got = moe.kv_fork(dt[:, :3], dl, dev_i32(par), dev_i32(chi), dev_i32(fp), 16, db)
        torch.cuda.synchronize()
        assert np.array_equal(host(dt)[:, :3], want[0]) and np.array_equal(host(dl), want[1])
        assert np.array_equal(host(got), want[3])
        for g, w in zip(db, want[2]):
            assert np.array_equal(host(g), w)


@pytest.mark.parametrize("rows,blocks,page,pages", [
    (1, 1, 16, 1), (3, 4, 16, 31), (3, 4, 16, 32), (40, 9, 32, 33), (300, 20, 64, 5000), (20, 30, 1, 100000), (0, 3, 16, 70),
    (64, 2000, 16, 1 << 20), (900, 3, 16, 3000), (200, 33, 16, 9000), (90, 64, 16, 16385), (4000, 5, 16, 30000), (700, 1, 16, 500)])
def test_free_pages(rows, blocks, page, pages):
    say(f"kv_free_pages {rows} rows of {blocks}, {pages} pages")
    table, lens, _ = pool(rows + pages, rows, blocks, page, pages, [])
    want, counts = oc.free_pages(table[:, :blocks], lens, page, pages)
    out = torch.full((pages + 3,), 77, dtype=torch.int32, device="cuda")
    f, c = moe.kv_free_pages(dev_i32(table)[:, :blocks], dev_i32(lens), page, pages, free_pages=out)
    torch.cuda.synchronize()
    assert np.array_equal(host(f)[:pages], want) and (f[pages:] == 77).all() and np.array_equal(host(c), counts)
    f2, c2 = moe.kv_free_pages(dev_i32(table)[:, :blocks], dev_i32(np.zeros_like(lens)), page, pages)
    torch.cuda.synchronize()
    assert torch.equal(f2, torch.arange(pages, dtype=torch.int32, device="cuda")) and host(c2).tolist() == [pages, 0]


@pytest.mark.parametrize("rows,blocks,page,pages", [(1, 1, 16, 1), (3, 4, 16, 31), (4, 9, 32, 40), (40, 20, 64, 2000), (0, 3, 16, 70),
                                                    (30, 30, 1, 100000), (900, 3, 16, 3000), (500, 33, 16, 2000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(rows, blocks, page, pages, in_place):
    say(f"kv_compact {rows} rows of {blocks}, {pages} pages")
    table, lens, bufs = pool(rows + pages, rows, blocks, page, pages, SHAPES if pages <= 2000 else SHAPES[:1])
    want, wb, wc = oc.compact(table[:, :blocks], lens, page, bufs)
    dt, db = dev_i32(table), [dev_u8(b) for b in bufs]
    out, counts = moe.kv_compact(dt[:, :blocks], dev_i32(lens), page, db, out_table=dt[:, :blocks] if in_place else None)
    torch.cuda.synchronize()
    assert np.array_equal(host(out), want) and np.array_equal(host(counts), wc)
    for g, w in zip(db, wb):
        assert np.array_equal(host(g), w)
    assert np.array_equal(host(dt)[:, blocks:], table[:, blocks:]) and (in_place or np.array_equal(host(dt), table))


@pytest.mark.parametrize("rows,blocks", [((1 << 25) + 70, 1), ((1 << 26) + 70, 2), ((1 << 20) + 300, 40)])
def test_pages_of_tables_of_many_rows(rows, blocks):
    """Row numbers that, taken 256 at a time by every wave, pass 2^31; more rows than one turn of all workgroups."""
    say(f"kv_free_pages, kv_compact: {rows} rows of {blocks}")
    page, pages = 16, 3000
    rng = np.random.default_rng(blocks)
    at = np.unique(np.concatenate([rng.integers(0, rows, 800), [0, 255, rows // 2, rows - 71, rows - 70, rows - 1]]))
    lens, table = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.full((rows, blocks), -1, dtype=torch.int32, device="cuda")
    n, entries = rng.integers(1, page * blocks + 1, len(at)), rng.integers(0, pages, (len(at), blocks))
    lens[torch.from_numpy(at).cuda()], table[torch.from_numpy(at).cuda()] = dev_i32(n), dev_i32(entries)
    want, counts = oc.free_pages(entries, n, page, pages)
    f, c = moe.kv_free_pages(table, lens, page, pages)
    buf = np.arange(pages * 16).astype(np.uint8).reshape(pages, 16) ^ rng.integers(0, 256, (pages, 1)).astype(np.uint8)
    wt, (wb,), wc = oc.compact(entries, n, page, [buf])
    db = dev_u8(buf)
    out, cc = moe.kv_compact(table, lens, page, [db])
    torch.cuda.synchronize()
    assert np.array_equal(host(f), want) and np.array_equal(host(c), counts)
    assert np.array_equal(host(out[torch.from_numpy(at).cuda()]), wt) and int((out >= 0).sum()) == int((wt >= 0).sum())
    assert np.array_equal(host(db), wb) and np.array_equal(host(cc), wc)


def test_pages_other_stream_and_graph():
    say("kv_fork, kv_free_pages, kv_compact: on another stream, in a graph")
    table, lens, bufs = pool(5, 30, 6, 16, 200, SHAPES, lens=[50] * 20 + [0] * 10)
    args = lambda: (dev_i32(table), dev_i32(lens), [dev_u8(b) for b in bufs])  # noqa: E731
    par, chi, fp = dev_i32(np.arange(10)), dev_i32(20 + np.arange(10)), dev_i32(150 + np.arange(12))

    def step(t, n, b, **kw):
        moe.kv_fork(t, n, par, chi, fp, 16, b, **kw)
        free, fc = moe.kv_free_pages(t, n, 16, 200, **kw)
        out, cc = moe.kv_compact(t, n, 16, b, **kw)
        return [t, n, free, fc, out, cc, *b]

    ref = step(*args())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a = args()
    torch.cuda.synchronize()
    got = step(*a, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, got))
    a = args()
    keep = [x.clone() for x in (a[0], a[1], *a[2])]
    ws = torch.empty(moe.kv_compact_workspace_bytes(200), dtype=torch.uint8, device="cuda")
    free, fc, out, cc = (torch.zeros_like(ref[i]) for i in (2, 3, 4, 5))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.kv_fork(a[0], a[1], par, chi, fp, 16, a[2], counts=torch.zeros(2, dtype=torch.int32, device="cuda"))
        moe.kv_free_pages(a[0], a[1], 16, 200, free_pages=free, counts=fc)
        moe.kv_compact(a[0], a[1], 16, a[2], out_table=out, counts=cc, workspace=ws)
    for i in range(3):
        for x, y in zip((a[0], a[1], *a[2]), keep):
            x.copy_(y)
        ws.fill_(0xEE)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(ref, [a[0], a[1], free, fc, out, cc, *a[2]])), i


# --------------------------------------------------------------------- norms
def near_norm(got, want, terms, what):
    """One rounding to bf16 and float terms before it, relative to the row's largest summand."""
    e = np.abs(got - want)
    assert np.all(e <= R * np.abs(want) + terms), f"{what}: {np.max(e / (R * np.abs(want) + terms))}"


@pytest.mark.parametrize("T,hidden", [(1, 8), (3, 64), (5, 504), (2, 512), (7, 520), (64, 1224), (33, 2048), (4, 4096), (2, 6000),
                                      (3, 8192), (2, 8200), (2, 20000), (1, 32768)])
@pytest.mark.parametrize("post,gate,scale,residual", [(False, None, 1.0, True), (True, "channel", 0.5, True),
                                                      (False, "value", -1.5, False), (True, None, 1.0, False), (True, "value", 0.1, True)])
def test_block_norm(T, hidden, post, gate, scale, residual):
    say(f"block_norm {T} x {hidden} post={post} gate={gate} scale={scale} residual={residual}")
    rng = np.random.default_rng(hidden + T)
    wide = hidden + 24
    xb, x = bf16(1, (T, wide), 3.0)
    rb, r = bf16(2, (T, wide), 5.0)
    gb, gv = bf16(3, (T, wide))
    pw, w, gc = rng.uniform(-1.5, 1.5, (3, hidden)).astype(np.float32)
    cut = lambda b: dev_bf16(b)[:, :hidden]  # noqa: E731
    g = {None: None, "channel": dev_f32(gc), "value": cut(gb)}[gate]
    gr = {None: None, "channel": gc.astype(np.float64), "value": gv[:, :hidden]}[gate]
    dx, dr = cut(xb), cut(rb) if residual else None
    kw = dict(post_weight=dev_f32(pw) if post else None, gate=g, scale=scale, eps=1e-5)
    h, y = moe.block_norm(dx, dev_f32(w), residual=dr, **kw)
    torch.cuda.synchronize()
    s32, e32 = float(np.float32(scale)), float(np.float32(1e-5))
    wh, wy = oc.block_norm(x[:, :hidden], w.astype(np.float64), r[:, :hidden] if residual else None,
                           pw.astype(np.float64) if post else None, gr, s32, e32)
    # float: a norm's sum of n squares, its root and division, three products; the residual's sum; twice for y
    part = np.abs(wh) + (2 * np.abs(r[:, :hidden]) if residual else 0)
    sum_terms = (hidden / 8 + 16) * U
    near_norm(bf16_to_f64(host_bf16_bits(h)), wh, sum_terms * part, "h")
    rms = np.sqrt((wh ** 2).mean(-1, keepdims=True) + e32)
    near_norm(bf16_to_f64(host_bf16_bits(y)), wy, 2 * sum_terms * (part / rms * np.abs(w) + np.abs(wy) * part.max(-1, keepdims=True) / rms),
              "y")
    # parts of the result, in place, rows beside: the same bits
    h2, y2 = moe.block_norm(dx, dev_f32(w), residual=dr, want_h=False, **kw)
    h3, y3 = moe.block_norm(dx, None, residual=dr, **kw)
    assert h2 is None and y3 is None and torch.equal(y2, y) and torch.equal(h3, h)
    store = dev_bf16(xb)
    moe.block_norm(store[:, :hidden], dev_f32(w), residual=dr, h=store[:, :hidden], y=None, **kw)
    torch.cuda.synchronize()
    assert torch.equal(store[:, :hidden], h) and np.array_equal(host_bf16_bits(store)[:, hidden:], xb[:, hidden:])


def test_block_norm_one_row_for_all_zeros_and_infinities():
    say("block_norm: broadcast rows, zeros, infinities")
    w = torch.ones(64, device="cuda")
    x = torch.zeros((5, 64), dtype=torch.bfloat16, device="cuda")
    x[1] = 1
    x[2, 3] = float("inf")
    x[3, 3] = float("nan")
    h, y = moe.block_norm(x, w, residual=dev_bf16(synth.random_bf16(1, (1, 64))).expand(5, 64) * 0)
    torch.cuda.synchronize()
    assert (y[0] == 0).all() and (y[1] == 1).all() and torch.isnan(y[2, 3]) and (y[2, :3] == 0).all() and torch.isnan(y[3]).all()
    r = dev_bf16(synth.random_bf16(1, (1, 64)))
    h, _ = moe.block_norm(x[:2], w, residual=r.expand(2, 64))
    torch.cuda.synchronize()
    assert torch.equal(h[0], r[0]) and torch.equal(h[1], (r.float() + 1).to(torch.bfloat16)[0])
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    h, y = moe.block_norm(e, w)
    assert h.shape == (0, 64) and y.shape == (0, 64)


def test_block_norm_more_rows_than_a_launch_takes():
    say("block_norm: 2^26 rows and some")
    T, hidden = (1 << 26) + 5, 8
    x = torch.empty((T, hidden), dtype=torch.bfloat16, device="cuda").normal_()
    r, g = x[:1].expand(T, hidden), x.flip(1)
    w = dev_f32(np.linspace(0.5, 1.5, hidden).astype(np.float32))
    h, y = moe.block_norm(x, w, residual=r, gate=g)
    for a, b in ((0, 300), ((1 << 21) - 150, (1 << 21) + 150), (33 * (1 << 20), 33 * (1 << 20) + 300), (T - 300, T)):
        hs, ys = moe.block_norm(x[a:b], w, residual=r[a:b], gate=g[a:b])
        assert torch.equal(h[a:b], hs) and torch.equal(y[a:b], ys), a


def test_block_norm_other_stream_and_graph():
    say("block_norm: on another stream, in a graph")
    x, r = (dev_bf16(synth.random_bf16(i, (100, 1024))) for i in (1, 2))
    w = torch.rand(1024, device="cuda")
    ref = moe.block_norm(x, w, residual=r, post_weight=w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.block_norm(x, w, residual=r, post_weight=w, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    h, y = (torch.zeros_like(x) for _ in range(2))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.block_norm(x, w, residual=r, post_weight=w, h=h, y=y)
    for i in range(3):
        x.mul_(1.5 if i else 1.0)
        h.zero_()
        g.replay()
        want = moe.block_norm(x, w, residual=r, post_weight=w)
        torch.cuda.synchronize()
        assert torch.equal(h, want[0]) and torch.equal(y, want[1]), i


def test_two_calls_at_once():
    """Two streams at the same time, each call with its own workspace and outputs, give the bits of one after the other."""
    say("attn_decode_fp4, kv_free_pages, kv_compact, block_norm: two at once")
    runs = [run_decode(15 + i, lens, prefix, 16, 8, 2, 128, 128) for i, (lens, prefix) in
            enumerate((([6000, 3], 40), ([100, 900] * 20, 900)))]
    tables = [pool(31 + i, 2000, 9, 16, 17000, SHAPES[:1]) for i in range(2)]
    x = [bf16(40 + i, (300, 4096))[0] for i in range(2)]
    w = dev_f32(np.linspace(0.5, 1.5, 4096).astype(np.float32))
    inputs = [(r[2], r[3], dev_i32(t[0])[:, :9], dev_i32(t[1]), dev_u8(t[2][0]), dev_bf16(b)) for r, t, b in zip(runs, tables, x)]

    def calls(at, **kw):
        args, pre, table, lens, buf, rows = at
        moved = buf.clone()
        return [*moe.attn_decode_fp4(*args, **pre, want_lse=True, **kw), *moe.kv_free_pages(table, lens, 16, 17000, **kw),
                *moe.kv_compact(table, lens, 16, [moved], **kw), moved, *moe.block_norm(rows, w, residual=rows, **kw)]

    want = [calls(at) for at in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for at, s in zip(inputs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(calls(at, stream=s))
        torch.cuda.synchronize()
        for g, h in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, h))


def test_two_writes_forks_and_read_backs_at_once():
    """Two streams at the same time, each with a cache and a table of its own."""
    say("qk_norm_rope_fp4, kv_fork, kv_gather_fp4, kv_gather: two at once")
    T, H, D, page, rows = 700, 4, 128, 16, 40
    cs = dev_f32(synth.random_bf16(3, (T, 64)).astype(np.float32) / 65536)
    at = []
    for i in range(2):
        x = dev_bf16(bf16(50 + i, (T, 3 * H, D))[0])
        table, lens, _ = pool(60 + i, rows, 4, page, 100, [], lens=[37, 20] * (rows // 2))
        order = np.random.default_rng(i).permutation(rows)
        par, chi = dev_i32(np.repeat(order[:8], 2)), dev_i32(order[8:24])
        cache = moe.Fp4Cache.zeros(130, page, H, D, D)
        wide = dev_bf16(bf16(70 + i, (130, page, H, D))[0])
        slots = dev_i32(np.random.default_rng(9 + i).permutation(130 * page)[:T])
        at.append((x, dev_i32(table)[:, :4], dev_i32(lens), par, chi, cache, wide, slots))
    positions, free = dev_i32(np.arange(T)), dev_i32(100 + np.arange(30))
    cu = dev_i32(np.arange(rows + 1) * 20)

    def calls(a, **kw):
        x, table, lens, par, chi, cache, wide, slots = a
        for t in cache.buffers:
            t.zero_()
        table, lens, wide = table.clone(), lens.clone(), wide.clone()
        q, k = moe.qk_norm_rope_fp4(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], positions, cs, cache, slots, **kw)
        counts = moe.kv_fork(table, lens, par, chi, free, page, [*cache.buffers, wide], **kw)
        return [q, k, counts, table, lens, *moe.kv_gather_fp4(cache, table, cu, 20 * rows, **kw),
                *moe.kv_gather(wide, wide, table, cu, 20 * rows, **kw), *(t.clone() for t in cache.buffers)]

    want = [calls(a) for a in at]
    torch.cuda.synchronize()
    assert all((w[0] != 0).any() and (w[5] != 0).any() and (w[7] != 0).any() and host(w[2]).tolist() == [16, 16] for w in want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for a, s in zip(at, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(calls(a, stream=s))
        torch.cuda.synchronize()
        for g, h in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(g, h))
