"""The attention layer on a cache held in 4 bits, requests that grow, fork, end and move, and the norms of the residual
stream, on the GPU.

Step-wise against the float64 oracle from the GPU's own inputs to each step, and the paths against one another: equal bits
where the same keys are read by the same call, else within the rounding of the attention's weights.
"""
import numpy as np
import pytest

import synth
from gpu_util import bf16_to_f64, dev_bf16, dev_f32, dev_u8, host, host_bf16_bits, say
from oracle import attention as oa
from oracle import cache as oc
import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_group_amd as moe  # noqa: E402

H, HQ, HKV = 512, 8, 2
R = 2.0 ** -8


def make_layer(D=128, Dv=128, requests=4, context=96, max_tokens=96, page=16, cache="nvfp4", pages=None, **norms):
    n = (HQ + HKV) * D + HKV * Dv
    wq = synth.random_mx_small(1, 1, n, H, 119, 122)
    wo = synth.random_mx_small(2, 1, H, HQ * Dv, 119, 122)
    rng = np.random.default_rng(3)
    qn, kn = rng.uniform(0.5, 1.5, (2, D)).astype(np.float32)
    ang = np.arange(512)[:, None] * 1000.0 ** (-np.arange(0, D, 2) / D)
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    w = moe.AttentionWeights(moe.Weights(dev_u8(wq[0]), dev_u8(wq[1])), moe.Weights(dev_u8(wo[0]), dev_u8(wo[1])),
                             dev_f32(qn), dev_f32(kn), **norms)
    pages = (requests + 1) * -(-context // page) if pages is None else pages
    layer = moe.AttentionLayer(w, HQ, HKV, D, Dv, dev_f32(cs), pages, page, requests, context, max_tokens, cache=cache,
                               v_global=2.0 ** -4)
    return layer, oracle.dequant_mx(wo[0][0], wo[1][0])


def tokens(seed, n):
    return dev_bf16(synth.random_bf16(seed, (n, H)))


def weights_bound(layer, wo, y):
    """Two attentions over the same keys whose weights are rounded differently, through the output projection."""
    if layer.fp4 is None:
        vmax = float(layer.v_cache.float().abs().max())
    else:
        vmax = float(np.abs(oc.cache_values(*[host(b) for b in layer.buffers], 1.0, layer.fp4.v_global)[1]).max())
    return 4 * R * vmax * np.abs(wo).sum(-1).max() + 2 * R * float(y.float().abs().max())


@pytest.mark.parametrize("D,Dv", [(64, 64), (128, 128), (192, 128)])
def test_decode_steps_against_the_oracle(D, Dv):
    say(f"4-bit attention layer {D}/{Dv}: prefix, then decode steps")
    layer, wo = make_layer(D, Dv)
    layer.prompt(tokens(1, 37), [37], prefix=True)
    for i in range(3):
        x = tokens(10 + i, 4)
        y = layer.decode(x, residual=x)
    torch.cuda.synchronize()
    # the last step: queries and cache as the layer has them
    k, v = oc.cache_values(*[host(b) for b in layer.buffers], 1.0, layer.fp4.v_global)
    table = host(layer.table)
    q = bf16_to_f64(host_bf16_bits(layer.q[:4]))
    want, _ = oa.attn_decode(q, k, v, table, [3] * 4, table[-1], 37, D ** -0.5)
    got = bf16_to_f64(host_bf16_bits(layer.a[:4]))
    vmax = np.abs(v).max()
    assert np.all(np.abs(got - want) <= R * np.abs(want) + (2.0 ** -11 + 1e-5) * vmax)
    # the cache: the keys as k_out has them within half a code (the last token's), the values' own rounding
    kc = k[table[:4, 0], 2]
    ko = bf16_to_f64(host_bf16_bits(layer.k[:4]))
    block = np.abs(ko.reshape(4, HKV, -1, 16)).max(-1).repeat(16, -1).reshape(ko.shape)
    assert np.all(np.abs(kc - ko) <= block / 6 * (1 + 2.0 ** -4) + R * np.abs(ko) + 2.0 ** -9)
    out = got.reshape(4, -1) @ wo.T + bf16_to_f64(host_bf16_bits(x))
    assert np.abs(bf16_to_f64(host_bf16_bits(y)) - out).max() <= 4 * R * np.abs(out).max()


@pytest.mark.parametrize("cache", ["bf16", "nvfp4"])
@pytest.mark.parametrize("prefix", [0, 21])
def test_extend_agrees_with_decode(cache, prefix):
    """Tokens that come together, in pieces and one by one: the same keys, so the same rows but for the weights' rounding."""
    say(f"extend {cache} prefix {prefix}")
    (a, wo), (b, _), (c, _) = (make_layer(cache=cache) for _ in range(3))
    px = tokens(1, 21)
    if prefix:
        for l in (a, b, c):
            l.prompt(px, [prefix], prefix=True)
    lens = [19, 0, 33]
    x = tokens(2, 52)
    y = a.extend(x, [0, 2], [19, 33], residual=x).clone()
    first = np.concatenate([[0], np.cumsum(lens)])
    rows = [np.arange(first[r], first[r] + lens[r]) for r in range(3)]
    cuts = {0: 7, 2: 16}
    xs = torch.cat([x[rows[r][:cuts[r]]] for r in (0, 2)])
    got = {r: [] for r in (0, 2)}
    y1 = b.extend(xs, [0, 2], [7, 16], residual=xs)
    got[0].append(y1[:7].clone()), got[2].append(y1[7:].clone())
    x2 = x[rows[2][16:]].contiguous()
    got[2].append(b.extend(x2, [2], [17], residual=x2).clone())
    x0 = x[rows[0][7:]].contiguous()
    got[0].append(b.extend(x0, [0], [12], residual=x0).clone())
    bound = weights_bound(a, wo, y)
    for r in (0, 2):
        assert (torch.cat(got[r]).float() - y[rows[r]].float()).abs().max() <= bound, r
    assert a.host_lens == b.host_lens == [19, 0, 33, 0, prefix]
    for t in range(19):                                               # one by one: request 0 alone
        xt = x[t:t + 1].contiguous()
        yt = c.decode(xt, residual=xt)
        assert (yt.float() - y[t:t + 1].float()).abs().max() <= bound, t


@pytest.mark.parametrize("cache", ["bf16", "nvfp4"])
def test_fork(cache):
    """A fork answers as its parent would, and neither sees the other's later tokens."""
    say(f"fork {cache}")
    (a, _), (b, _), (c, _) = (make_layer(cache=cache, requests=3) for _ in range(3))
    x = tokens(1, 21)
    for l in (a, b, c):
        l.extend(x, [0], [21])
    a.fork(0, [2, 1])
    same = tokens(2, 1)
    y = a.decode(same.expand(3, H).contiguous()).clone()
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
    later = [tokens(20 + i, 3) for i in range(14)]                    # over the copied page's end
    ys = [a.decode(t).clone() for t in later]
    for l, r in ((b, 0), (c, 2)):                                     # the same tokens without a fork
        z = l.decode(same)
        assert torch.equal(z[0], y[r])
        for t, w in zip(later, ys):
            assert torch.equal(l.decode(t[r:r + 1].contiguous())[0], w[r])
    used = set(host(a.table)[:3, :3].ravel().tolist())
    assert a._in_use() == len(used) and a.host_lens == [36, 36, 36, 0]


@pytest.mark.parametrize("cache", ["bf16", "nvfp4"])
def test_release_and_reuse(cache):
    """Pages of requests that ended go to others, and nothing that is held changes; the pool is never larger than needed."""
    say(f"release {cache}")
    (a, _), (b, _) = make_layer(cache=cache, pages=8), make_layer(cache=cache)
    px = tokens(1, 20)
    for l in (a, b):
        l.prompt(px, [20], prefix=True)                               # 2 pages
    rng = np.random.default_rng(1)
    for i in range(12):
        n, r = int(rng.integers(1, 33)), int(rng.integers(0, 3))
        x = tokens(30 + i, n)
        if a.host_lens[r]:
            for l in (a, b):
                l.release([r])
        ya, yb = a.extend(x, [r], [n]).clone(), b.extend(x, [r], [n])
        assert torch.equal(ya, yb), i
        d = tokens(60 + i, 3)
        if all(l % 16 for l in a.host_lens[:3]):
            assert torch.equal(a.decode(d), b.decode(d)), i
        held = host(a.table)
        mine = [set(held[j, :-(-m // 16)].tolist()) for j, m in enumerate(a.host_lens)]
        assert sum(map(len, mine)) == len(set().union(*mine)) == a._in_use()
        left = set(host(a.free)[a.taken:].tolist())
        assert not left & set().union(*mine) and len(left) + a._in_use() == 8
    for l in (a, b):
        l.release([0, 1, 2])
    assert a._in_use() == 2 and a.free.numel() == 6


@pytest.mark.parametrize("cache", ["bf16", "nvfp4"])
def test_compact(cache):
    say(f"compact {cache}")
    (a, _), (b, _) = make_layer(cache=cache), make_layer(cache=cache)
    x = tokens(1, 90)
    for l in (a, b):
        l.prompt(tokens(5, 20), [20], prefix=True)
        l.extend(x, [0, 1, 2, 3], [40, 17, 30, 3])
        l.fork(1, []) if l is a else None
        l.release([0, 2])
    n = a.compact()
    assert n == a._in_use() == 2 + 2 + 1 and a.free.tolist() == list(range(5, a.pool.numel()))
    t = host(a.table)
    assert set(t[1, :2].tolist()) | set(t[3, :1].tolist()) | set(t[-1, :2].tolist()) == set(range(5))
    for i in range(3):
        d = tokens(50 + i, 4)
        assert torch.equal(a.decode(d), b.decode(d)), i


def test_norms_of_the_residual_stream():
    """in_norm, post_norm, gate, residual_scale and next_norm in the layer equal block_norm around a layer without."""
    say("attention layer with the residual stream's norms")
    rng = np.random.default_rng(5)
    inn, post, gate, nxt = (dev_f32(rng.uniform(0.5, 1.5, H).astype(np.float32)) for _ in range(4))
    a, _ = make_layer(in_norm=inn, post_norm=post, gate=gate, residual_scale=0.5, next_norm=nxt)
    b, _ = make_layer()
    c, _ = make_layer(in_norm=inn)
    for step, x in ((lambda l, x, **kw: l.prompt(x, [20, 9], **kw), tokens(1, 29)),
                    (lambda l, x, **kw: l.extend(x, [1], [5], **kw), tokens(2, 5)),
                    (lambda l, x, **kw: l.decode(x, **kw), tokens(3, 4))):
        h, z = step(a, x, residual=x)
        xn = moe.block_norm(x, inn, want_h=False)[1]
        o = step(b, xn)
        wh, wz = moe.block_norm(o, nxt, x, post, gate, 0.5)
        assert torch.equal(h, wh) and torch.equal(z, wz)
        assert torch.equal(step(c, x), o)
        y = torch.full_like(h, float("nan"))
    h2, _ = a.decode(x, residual=x, y=y)
    assert h2 is y and torch.isfinite(y.float()).all()


def test_layer_refuses():
    layer, _ = make_layer(requests=2, context=32, pages=3)
    with pytest.raises(ValueError, match="max_context"):
        layer.extend(tokens(1, 33), [1], [33])
    layer.extend(tokens(1, 30), [1], [30])
    with pytest.raises(ValueError, match="max_context"):
        layer.extend(tokens(1, 3), [1], [3])
    with pytest.raises(ValueError, match="pages needed"):
        layer.extend(tokens(1, 20), [0], [20])
    assert layer.host_lens == [0, 30, 0]


@pytest.mark.parametrize("cache", ["bf16", "nvfp4"])
@pytest.mark.parametrize("seed,pages", [(1, 18), (2, 30)])
def test_any_order_of_calls(cache, seed, pages):
    """Requests that grow, are answered, fork, end and move in any order, in a pool that may be too small: a row once
    written keeps its bits for every request that holds it, pages are shared only by forks, a refused call changes nothing."""
    say(f"layer {cache}, calls in any order {seed}")
    a, _ = make_layer(64, 64, requests=6, context=80, cache=cache, pages=pages)
    a.prompt(tokens(9, 20), [20], prefix=True)
    rng = np.random.default_rng(seed)
    rows = [None] * 6                                                  # what each request's rows were when they were written

    def read():
        cu = np.concatenate([[0], np.cumsum(a.host_lens[:6])])
        at = torch.tensor(cu, dtype=torch.int32).cuda()
        k, v = (moe.kv_gather(a.k_cache, a.v_cache, a.table[:6], at, int(cu[-1])) if a.fp4 is None else
                moe.kv_gather_fp4(a.fp4, a.table[:6], at, int(cu[-1])))
        kv = np.concatenate([host_bf16_bits(k.flatten(1)), host_bf16_bits(v.flatten(1))], 1)
        return [kv[cu[r]:cu[r + 1]] for r in range(6)]

    done = dict.fromkeys(("extend", "decode", "fork", "release", "compact", "refused"), 0)
    prefix = host(a.table)[-1, :2].tolist()
    for i in range(60):
        op = rng.choice(["extend", "extend", "decode", "decode", "fork", "release", "compact"])
        some = sorted(rng.choice(6, int(rng.integers(1, 4)), replace=False).tolist())
        before, lens = host(a.table).copy(), list(a.host_lens)
        try:
            if op == "extend":
                new = rng.integers(1, 25, len(some)).tolist()
                y = a.extend(tokens(100 + i, sum(new)), some, new)
                assert torch.isfinite(y).all()
            elif op == "decode":
                y = a.decode(tokens(200 + i, some[-1] + 1))
                assert torch.isfinite(y).all()
            elif op == "fork":
                free = [r for r in range(6) if not a.host_lens[r] and r != some[0]]
                a.fork(some[0], free[:2])
                for r in free[:2]:
                    rows[r] = rows[some[0]]
            elif op == "release":
                a.release(some)
                for r in some:
                    rows[r] = None
            else:
                assert a.compact() == a._in_use()
                prefix = host(a.table)[-1, :2].tolist()
            done[op] += 1
        except ValueError:
            done["refused"] += 1
            assert np.array_equal(host(a.table), before) and a.host_lens == lens, (i, op)
        assert host(a.lens).tolist() == a.host_lens, (i, op)
        for r, kv in enumerate(read()):
            old = rows[r]
            assert old is None or np.array_equal(kv[:len(old)], old), (i, op, r)
            rows[r] = kv if len(kv) else None
        table = host(a.table)
        mine = [table[r, :-(-n // 16)].tolist() for r, n in enumerate(a.host_lens)]
        assert mine[-1] == prefix and all(len(set(m)) == len(m) for m in mine)
        used = set().union(*mine)
        left = host(a.free)[a.taken:].tolist()
        # (a request that a call replaced may have left pages that only release() or compact() finds)
        assert not used & set(left) and len(used) == a._in_use() and len(set(left)) == len(left)
        last = [m[-1] for r, m in enumerate(mine[:-1]) if a.host_lens[r] % 16]
        assert len(set(last)) == len(last), "two requests write to one page"
    say(f"  {done}")
    assert all(n for what, n in done.items() if what != "refused" or pages < 30)      # (30 pages hold nearly all)
