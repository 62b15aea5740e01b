"""The routed layer's calls on another stream: their outputs do not lie in memory that work queued on the current stream
still writes, and outlive readers there."""
import numpy as np
import pytest

import synth
from gpu_util import dev_bf16, dev_f32, dev_i32, dev_u8, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_group_amd as moe  # noqa: E402

SIZES = [1 << b for b in range(9, 22)]                              # of freed blocks: each call finds one that fits


def routed_calls():
    x = dev_bf16(synth.random_bf16(1, (64, 512)))
    packed, scale = synth.random_mx_small(2, 4, 512, 512, 119, 122)
    w = moe.Weights(dev_u8(packed), dev_u8(scale))
    logits = dev_f32(synth.random_logits(3, 64, 16))
    rng = np.random.default_rng(4)
    ids = dev_i32(rng.integers(0, 16, (64, 4)))
    off, slot_rows, topw = dev_i32(np.array([0, 10, 10, 40, 64])), dev_i32(rng.permutation(64)), torch.rand((16, 4), device="cuda")
    counter = torch.zeros(1, dtype=torch.int32, device="cuda")
    flat = lambda w: [t for t in (w.packed, w.scale, w.global_scale) if t is not None]  # noqa: E731
    return {
        "route": lambda **k: moe.route(logits, None, 16, 4, 2, 4, 1.0, **k),
        "permute": lambda **k: moe.permute(ids, 16, **k),
        "route_permute": lambda **k: moe.route_permute(logits, None, 16, 4, 2, 4, 1.0, counter, **k),
        "grouped_gemm": lambda **k: [moe.grouped_gemm(x, w, None, off, 64, **k)],
        "combine": lambda **k: [moe.combine(x, slot_rows, topw, **k)],
        "transcode": lambda **k: moe.transcode_mx_to_nv(w.scale, w.packed, **k),
        "tile_weights": lambda **k: flat(moe.tile_weights(w, **k)),
        "compact_weights": lambda **k: flat(moe.compact_weights(w, **k)[0]),
        "quantize_nvfp4": lambda **k: moe.quantize_nvfp4(x, **k),
        "quantize_mxfp8": lambda **k: moe.quantize_mxfp8(x, **k)}


@pytest.mark.parametrize("name", ["route", "permute", "route_permute", "grouped_gemm", "combine", "transcode", "tile_weights",
                                  "compact_weights", "quantize_nvfp4", "quantize_mxfp8"])
def test_outputs_of_another_stream(name):
    say(f"{name}: on another stream beside work that is queued on the current one")
    call = routed_calls()[name]
    want = [t.clone() for t in call()]
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
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(30_000_000)
    read = [t.clone() for t in got]
    del got
    with torch.cuda.stream(s):
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in SIZES for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(read, want))
    del junk
