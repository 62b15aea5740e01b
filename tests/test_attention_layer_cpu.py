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
