"""What the attention layer refuses on the host before anything of a step is done (no GPU needed)."""
import pytest
import torch

moe = pytest.importorskip("block_scaled_fp4_group_amd")

H, HQ, HKV, D = 512, 4, 2, 64


def weights(n, k):
    return moe.Weights(torch.zeros((1, n, k // 2), dtype=torch.uint8), torch.zeros((1, n, k // 32), dtype=torch.uint8))


@pytest.fixture
def layer(monkeypatch):
    """A layer in host memory; a launch would be an error."""
    def no_launch(*a, **kw):
        raise AssertionError("launched")
    for name in ("grouped_gemm", "kv_slots", "qk_norm_rope", "attn_prompt", "attn_decode", "combine"):
        monkeypatch.setattr(moe.attention, name, no_launch)

    w = moe.AttentionWeights(weights((HQ + 2 * HKV) * D, H), weights(H, HQ * D))
    return moe.AttentionLayer(w, HQ, HKV, D, D, torch.zeros((64, D)), 8, 16, 2, 32, 32, device="cpu")


def rows(t, h=H, dtype=torch.bfloat16):
    return torch.zeros((t, h), dtype=dtype)


@pytest.mark.parametrize("bad", [
    dict(x=rows(2, H - 8)), dict(x=rows(2, dtype=torch.float32)), dict(x=rows(4)[::2]), dict(x=torch.zeros(2, dtype=torch.bfloat16)),
    dict(residual=rows(1)), dict(residual=rows(3)), dict(residual=rows(2, dtype=torch.float32)), dict(residual=rows(2, 2 * H)[:, ::2]),
    dict(y=rows(1)), dict(y=rows(2, H + 8)[:, :H]), dict(y=rows(2, dtype=torch.float16))])
def test_rows_that_do_not_fit_are_refused(layer, bad):
    """The kernels read and write T x hidden values from each address."""
    kw = dict(x=rows(2), residual=None, y=None)
    kw.update(bad)
    with pytest.raises(ValueError, match=f"{next(iter(bad))} must be a contiguous bfloat16"):
        layer.decode(**kw)
    with pytest.raises(ValueError, match=f"{next(iter(bad))} must be a contiguous bfloat16"):
        layer.prompt(kw["x"], [1, 1], kw["residual"], False, kw["y"])
    assert layer.host_lens == [0, 0, 0] and layer.taken == 0


@pytest.mark.parametrize("name", ["x", "residual", "y"])
def test_rows_off_a_16_byte_boundary_are_refused(layer, name):
    """Refused by a kernel's check, they would leave the cache a token ahead."""
    off = torch.zeros(2 * H + 1, dtype=torch.bfloat16)[1:].view(2, H)
    assert off.is_contiguous()
    with pytest.raises(ValueError, match="16-byte aligned"):
        layer.decode(**{"x": rows(2), name: off})
    assert layer.host_lens == [0, 0, 0]


def test_rows_that_fit_reach_the_step(layer):
    with pytest.raises(AssertionError, match="launched"):
        layer.decode(rows(2), residual=rows(2), y=rows(2))


@pytest.mark.parametrize("qkv,out", [((HQ * D, H), (H, HQ * D)), (((HQ + 2 * HKV) * D, 2 * H), (H, HQ * D)),
                                     (((HQ + 2 * HKV) * D, H), (H, 2 * HQ * D)), (((HQ + 2 * HKV) * D, H), (2 * H, HQ * D))])
def test_projections_that_do_not_fit_the_heads_are_refused(qkv, out):
    """A projection reads rows as wide as its weights, from buffers made for the heads."""
    with pytest.raises(ValueError, match="these heads need"):
        moe.AttentionLayer(moe.AttentionWeights(weights(*qkv), weights(*out)), HQ, HKV, D, D, torch.zeros((64, D)), 8, 16, 2, 32,
                           32, device="cpu")


@pytest.mark.parametrize("bad,match", [
    (dict(cache="fp8"), "bf16"), (dict(cache="nvfp4", page_size=8), "16 tokens"),
    (dict(cache="nvfp4", cos_sin=torch.zeros((64, 48))), "multiple of 32")])
def test_caches_that_are_not_built_are_refused(bad, match):
    kw = dict(cos_sin=torch.zeros((64, D)), num_pages=8, page_size=16, max_requests=2, max_context=32, max_tokens=32, device="cpu")
    kw.update(bad)
    with pytest.raises(ValueError, match=match):
        moe.AttentionLayer(moe.AttentionWeights(weights((HQ + 2 * HKV) * D, H), weights(H, HQ * D)), HQ, HKV, D, D, **kw)


@pytest.mark.parametrize("name", ["in_norm", "post_norm", "gate", "next_norm"])
@pytest.mark.parametrize("t", [torch.zeros(H + 8), torch.zeros(H, dtype=torch.bfloat16), torch.zeros((1, H))])
def test_norms_that_do_not_fit_are_refused(name, t):
    w = moe.AttentionWeights(weights((HQ + 2 * HKV) * D, H), weights(H, HQ * D), **{name: t})
    with pytest.raises(ValueError, match=f"{name} must be a float32"):
        moe.AttentionLayer(w, HQ, HKV, D, D, torch.zeros((64, D)), 8, 16, 2, 32, 32, device="cpu")


@pytest.fixture
def counting(monkeypatch, layer):
    """A layer whose launches are only counted."""
    calls = []
    for name in ("grouped_gemm", "kv_slots", "qk_norm_rope", "attn_prompt", "attn_decode", "combine", "kv_fork", "kv_free_pages",
                 "kv_compact", "kv_gather"):
        def call(*a, name=name, **kw):
            calls.append(name)
            return kw.get("out") if name == "grouped_gemm" else (torch.zeros(1), torch.zeros(1))
        monkeypatch.setattr(moe.attention, name, call)
    layer.calls = calls
    return layer


@pytest.mark.parametrize("requests,lens", [([], []), ([0], []), ([1, 0], [1, 1]), ([0, 0], [1, 1]), ([-1], [2]), ([2], [2])])
def test_extend_refuses_requests_that_are_not(counting, requests, lens):
    with pytest.raises(ValueError, match="ascend"):
        counting.extend(rows(2), requests, lens)
    assert not counting.calls and counting.taken == 0


def test_fork_and_release_refuse(counting):
    layer = counting
    layer.extend(rows(20), [0], [20])
    for parent, children in ((0, [0]), (0, [1, 1]), (0, [2]), (-1, [1]), (2, [1])):
        with pytest.raises(ValueError, match="different requests"):
            layer.fork(parent, children)
    layer.extend(rows(1), [1], [1])
    with pytest.raises(ValueError, match="release"):
        layer.fork(0, [1])
    for r in ([2], [-1], [0, 5]):
        with pytest.raises(ValueError, match="requests are"):
            layer.release(r)
    assert layer.host_lens == [20, 1, 0]


def test_pages_are_counted_once(counting):
    """The host's count of pages in use: shared ones once, a request's own copies by themselves, none behind release()."""
    layer = counting                                                  # 8 pages of 16
    layer.extend(rows(20), [0], [20])                                 # 2 pages
    layer.fork(0, [1])                                                # shares one, copies one
    assert layer._in_use() == 3 and layer.taken == 3 and layer.host_lens == [20, 20, 0]
    layer.extend(rows(10), [1], [10])                                 # ends in the copy, and one more... 30 tokens: 2 pages
    assert layer._in_use() == 3
    layer.extend(rows(2), [1], [2])
    layer.release([0])
    assert layer._in_use() == 2 and layer.taken == 0 and layer.free.numel() == 6 and layer.host_lens == [0, 32, 0]
    layer.fork(1, [0])                                                # no page that is not full: nothing copied
    assert layer._in_use() == 2 and layer.taken == 0
    layer.release([1])
    assert layer._in_use() == 2                                       # request 0 holds them still
    assert layer.compact() == 2 and layer.free.tolist() == [2, 3, 4, 5, 6, 7]
    layer.release([0, 1])
    assert layer._in_use() == 0 and layer.free.numel() == 8


def test_fork_without_a_page_left_is_refused(counting):
    layer = counting
    layer.extend(rows(20), [0], [20])
    layer.free = layer.free[:2]
    with pytest.raises(ValueError, match="1 pages needed, 0 free"):
        layer.fork(0, [1])
    assert layer.host_lens == [20, 0, 0] and layer.calls[-1] != "kv_fork"


def test_a_refused_page_call_leaves_the_layer_as_it_was(counting, monkeypatch):
    """release() and compact() of pools that the page calls do not take: requests keep their tokens and pages."""
    layer = counting

    def refuse(*a, **kw):
        raise RuntimeError("pages, at most")
    layer.extend(rows(20), [0], [20])
    layer.fork(0, [1])
    layer.lens[:2] = 20
    for name in ("kv_free_pages", "kv_compact"):
        monkeypatch.setattr(moe.attention, name, refuse)
    for call in (lambda: layer.release([0]), lambda: layer.release([0, 1]), layer.compact):
        free, held = layer.free, [list(h) for h in layer.held]
        with pytest.raises(RuntimeError, match="at most"):
            call()
        assert layer.lens.tolist() == [20, 20, 0] and layer.host_lens == [20, 20, 0]
        assert layer.held == held and layer.free is free and layer.taken == 3
