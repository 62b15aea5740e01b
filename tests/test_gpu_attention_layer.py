"""The attention layer and a decoder layer made of it and the MoE layer, on the GPU.

Step-wise against the float64 oracle (each stage from the GPU's own input to it), and the paths against one another:
a sequence read as one prompt, read as a prefix with its rest decoded token by token, and decoded from the first token.
"""
import os
import sys

import numpy as np
import pytest

import oracle
import synth
from gpu_util import bf16_to_f64, dev_bf16, dev_f32, dev_u8, host, host_bf16_bits, say
from oracle import attention as oa

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_group_amd as moe  # noqa: E402

H, HQ, HKV = 512, 8, 2
R = 2.0 ** -8


def make_layer(D=128, Dv=128, requests=4, context=96, max_tokens=96, page=16):
    n = (HQ + HKV) * D + HKV * Dv
    wq = synth.random_mx_small(1, 1, n, H, 119, 122)
    wo = synth.random_mx_small(2, 1, H, HQ * Dv, 119, 122)
    rng = np.random.default_rng(3)
    qn, kn = rng.uniform(0.5, 1.5, (2, D)).astype(np.float32)
    ang = np.arange(512)[:, None] * 1000.0 ** (-np.arange(0, D, 2) / D)
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    w = moe.AttentionWeights(moe.Weights(dev_u8(wq[0]), dev_u8(wq[1])), moe.Weights(dev_u8(wo[0]), dev_u8(wo[1])),
                             dev_f32(qn), dev_f32(kn))
    pages = (requests + 1) * -(-context // page)
    layer = moe.AttentionLayer(w, HQ, HKV, D, Dv, dev_f32(cs), pages, page, requests, context, max_tokens)
    return layer, (oracle.dequant_mx(wq[0][0], wq[1][0]), oracle.dequant_mx(wo[0][0], wo[1][0]), qn, kn, cs)


def near(got, want, what, slack):
    """One rounding to bf16 and ``slack`` of the largest value of the row (float sums, weights rounded to bf16)."""
    big = np.abs(want).max(axis=-1, keepdims=True)
    e = np.abs(got - want)
    say(f"  {what}: worst error / bound {np.max(e / (R * np.abs(want) + slack * big)):.2f}")
    assert np.all(e <= R * np.abs(want) + slack * big), what


@pytest.mark.parametrize("D,Dv", [(64, 64), (128, 128), (192, 128)])
def test_prompt_steps_against_the_oracle(D, Dv):
    say(f"attention layer prompt {D}/{Dv}")
    layer, (wq, wo, qn, kn, cs) = make_layer(D, Dv)
    lens = [33, 1, 62]
    xb = synth.random_bf16(5, (96, H))
    x = dev_bf16(xb)
    y = layer.prompt(x, lens, residual=x)
    torch.cuda.synchronize()
    f = lambda t: bf16_to_f64(host_bf16_bits(t))  # noqa: E731
    xv, qkv = bf16_to_f64(xb), f(layer.qkv)
    near(qkv, xv @ wq.T, "projection", 2e-3)
    nq, nk = HQ * D, HKV * D
    pos = np.concatenate([np.arange(n) for n in lens])
    q = oa.norm_rope(qkv[:, :nq].reshape(96, HQ, D), qn, 1e-6, cs, pos, False)
    k = oa.norm_rope(qkv[:, nq:nq + nk].reshape(96, HKV, D), kn, 1e-6, cs, pos, False)
    near(f(layer.q), q, "q", 1e-5)
    near(f(layer.k), k, "k", 1e-5)
    cu = np.concatenate([[0], np.cumsum(lens)])
    v = qkv[:, nq + nk:].reshape(96, HKV, Dv)
    a, _ = oa.attn_prompt(f(layer.q), f(layer.k), v, cu, cu, D ** -0.5)
    av, _ = oa.attn_prompt(f(layer.q), f(layer.k), np.abs(v), cu, cu, D ** -0.5)
    assert np.all(np.abs(f(layer.a) - a) <= R * np.abs(a) + (R + 1e-3) * av)
    o = f(layer.a).reshape(96, -1) @ wo.T
    near(f(layer.o), o, "output projection", 2e-3)
    near(f(y), xv + f(layer.o), "residual", 1e-6)
    # the cache holds the keys and values, in the pages that the table names
    table, kc, vc = host(layer.table), f(layer.k_cache), f(layer.v_cache)
    for b, n in enumerate(lens):
        at = [(table[b, j // 16], j % 16) for j in range(n)]
        assert np.array_equal(np.stack([kc[p] for p in at]), f(layer.k)[cu[b]:cu[b + 1]])
        assert np.array_equal(np.stack([vc[p] for p in at]), v[cu[b]:cu[b + 1]])
    assert layer.taken == 3 + 1 + 4 and host(layer.lens).tolist() == [33, 1, 62, 0, 0]


@pytest.mark.parametrize("D,Dv", [(128, 128), (192, 128)])
def test_prompt_prefix_and_decode_agree(D, Dv):
    """Token t of a sequence gives the same output however the tokens before it were read: the attention differs by the
    rounding of its weights, r sum p |v| <= r max |v| per value; through the output projection by that times sum |w|."""
    say(f"attention layer: prompt, prefix + decode, decode only {D}/{Dv}")
    n, cut = 60, 37
    xb = synth.random_bf16(8, (n, H))
    x = dev_bf16(xb)
    whole, (_, wo, *_) = make_layer(D, Dv)
    y = whole.prompt(x, [n]).clone()
    vmax = float(whole.v_cache.float().abs().max())
    behind, _ = make_layer(D, Dv)
    yp = behind.prompt(x[:cut], [cut], prefix=True).clone()
    alone, _ = make_layer(D, Dv)
    torch.cuda.synchronize()
    bound = 4 * R * vmax * np.abs(wo).sum(-1).max()
    assert torch.equal(yp, y[:cut])                                  # rows do not depend on the rows after them
    for t in range(n):
        ya = alone.decode(x[t:t + 1])[0]
        assert (ya.float() - y[t].float()).abs().max() <= bound, ("decode only", t)
        if t >= cut:
            # the request decodes the rest; a second one repeats it and gets the same bits
            yb = behind.decode(x[t:t + 1].repeat(2, 1))
            assert (yb[0].float() - y[t].float()).abs().max() <= bound, ("behind the prefix", t)
            assert torch.equal(yb[0], yb[1])
    assert behind.prefix_len == cut and behind.host_lens[:2] == [n - cut, n - cut]


def test_layer_refusals():
    layer, _ = make_layer(requests=2, context=32)
    x = dev_bf16(synth.random_bf16(1, (64, H)))
    with pytest.raises(ValueError, match="bring"):
        layer.prompt(x[:10], [4, 5])
    with pytest.raises(ValueError, match="max_context"):
        layer.prompt(x[:33], [33])
    with pytest.raises(ValueError, match="first tokens"):
        layer.prompt(x[:3], [1, 1, 1])
    with pytest.raises(ValueError, match="at most 2"):
        layer.decode(x[:3])
    layer.prompt(x[:20], [20], prefix=True)
    with pytest.raises(ValueError, match="prefix"):
        layer.prompt(x[:2], [2])
    with pytest.raises(ValueError, match="first tokens"):
        layer.prompt(x[:2], [2], prefix=True)
    layer.free = layer.free[:2]                                       # the prefix has both
    with pytest.raises(ValueError, match="pages"):
        layer.decode(x[:1])
    assert layer.host_lens == [0, 0, 20]


def test_decoder_layer_example():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decoder_layer
    y = decoder_layer.main()
    assert y.shape == (8, 512) and torch.isfinite(y.float()).all()


def test_prefix_after_requests_is_refused():
    """The requests' keys in the cache are rotated to positions from 0 on; a prefix would come to lie on the same ones."""
    for start in ("prompt", "decode"):
        layer, _ = make_layer(requests=2, context=32)
        x = dev_bf16(synth.random_bf16(1, (20, H)))
        layer.prompt(x[:3], [0, 3]) if start == "prompt" else layer.decode(x[:1])
        held = list(layer.host_lens)
        with pytest.raises(ValueError, match="before the first tokens"):
            layer.prompt(x, [20], prefix=True)
        assert layer.host_lens == held and layer.prefix_len == 0


def test_positions_past_the_table_are_refused():
    """Past the last row every position would be turned by the same angle.  Prefix and own tokens count together."""
    layer, _ = make_layer(requests=2, context=32)
    x = dev_bf16(synth.random_bf16(1, (40, H)))
    layer.cos_sin = layer.cos_sin[:22].contiguous()
    with pytest.raises(ValueError, match="22 rows"):
        layer.prompt(x[:24], [1, 23])
    layer.prompt(x[:20], [20], prefix=True)
    layer.decode(x[:2])
    layer.decode(x[:1])                                               # position 21, the last
    with pytest.raises(ValueError, match="22 rows"):
        layer.decode(x[:1])
    with pytest.raises(ValueError, match="22 rows"):
        layer.decode(x[:2])
    assert layer.host_lens == [2, 1, 20]


def test_negative_lengths_are_refused():
    """Even where the sum fits: the host's lengths would differ from the GPU's, which counts a negative one as 0."""
    layer, _ = make_layer(requests=2, context=32)
    x = dev_bf16(synth.random_bf16(1, (4, H)))
    for lens in ([5, -1], [-1, 5]):
        with pytest.raises(ValueError, match="bring"):
            layer.prompt(x, lens)
    with pytest.raises(ValueError):
        layer.prompt(x[:0], [])
    assert layer.host_lens == [0, 0, 0] and layer.taken == 0


def test_results_go_to_y():
    """With and without a residual: the result is written to y and returned."""
    xb = dev_bf16(synth.random_bf16(1, (9, H)))
    a, b = make_layer(requests=2, context=32)[0], make_layer(requests=2, context=32)[0]
    for step in (lambda l, **kw: l.prompt(xb, [4, 5], **kw), lambda l, **kw: l.decode(xb[:2], **kw),
                 lambda l, **kw: l.decode(xb[:2], residual=xb[:2], **kw)):
        want = step(a).clone()
        y = torch.full_like(want, float("nan"))
        assert step(b, y=y) is y and torch.equal(y, want)


@pytest.mark.parametrize("D,Dv", [(64, 64), (128, 128), (192, 128)])
def test_prompt_then_decode_agrees_with_prompt(D, Dv):
    """Requests that are read as prompts and then answered: token t of each gives the output that it has in a whole
    prompt, within the rounding of the attention's weights (as where a prefix and decode steps are compared)."""
    say(f"attention layer: prompt, then decode {D}/{Dv}")
    lens, cuts = [33, 18, 38], [30, 16, 37]                            # 16: the next token begins a page
    first = np.concatenate([[0], np.cumsum(lens)])
    x = dev_bf16(synth.random_bf16(11, (sum(lens), H)))
    whole, (_, wo, *_) = make_layer(D, Dv)
    y = whole.prompt(x, lens, residual=x).clone()
    vmax = float(whole.v_cache.float().abs().max())
    bound = 4 * R * vmax * np.abs(wo).sum(-1).max() + 2 * R * float(y.abs().max())   # (and the residual sum's own rounding)
    layer, _ = make_layer(D, Dv)
    xs = torch.cat([x[a:a + c] for a, c in zip(first, cuts)])
    yp = layer.prompt(xs, cuts, residual=xs).clone()
    at = 0
    for a, c in zip(first, cuts):
        assert torch.equal(yp[at:at + c], y[a:a + c])                  # rows do not depend on the rows after them
        at += c
    for i, n in enumerate((3, 2, 1)):                                  # all requests, then the first ones
        rows = torch.tensor([f + c + i for f, c in zip(first, cuts[:n])], device="cuda")
        xd = x[rows].contiguous()
        yd = layer.decode(xd, residual=xd)
        assert (yd.float() - y[rows].float()).abs().max() <= bound, i
    assert layer.host_lens == lens + [0, 0]
