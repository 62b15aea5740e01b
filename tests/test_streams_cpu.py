"""Where the routed layer's calls make their tensors, with stand-ins for the library and torch's streams (no GPU)."""
import inspect

import pytest
import torch

moe = pytest.importorskip("block_scaled_fp4_group_amd")

U8, I32, F32, BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16


class Stream:
    device, device_index = torch.device("cuda", 0), 0

    def __init__(self, name, handle):
        self.name, self.cuda_stream = name, handle


class Library:
    """Every entry point: refuses nothing, writes nothing."""
    def __getattr__(self, name):
        return lambda *a: World.launch(name, a)


class World:
    log, streams, device, devices = [], [], 0, []

    @staticmethod
    def launch(name, args):
        if not name.endswith("_bytes"):
            World.devices.append(World.device)
            World.log.append(("launched", World.streams[-1].name, args[-1].value))
            return 0
        return 64


class Under:
    """Stands in for torch.cuda.stream()."""
    def __init__(self, stream):
        self.stream = stream

    def __enter__(self):
        World.streams.append(self.stream)

    def __exit__(self, *a):
        World.streams.pop()


class OnDevice:
    """Stands in for torch.cuda.device()."""
    def __init__(self, index):
        self.index = index

    def __enter__(self):
        self.before, World.device = World.device, self.index

    def __exit__(self, *a):
        World.device = self.before


@pytest.fixture
def world(monkeypatch):
    World.log, World.streams, World.device, World.devices = [], [Stream("current", 0x10)], 0, []
    empty, like = torch.empty, torch.empty_like
    for name, f in (("empty", empty), ("empty_like", like)):
        def made(*a, f=f, **kw):
            World.log.append(("made on", World.streams[-1].name))
            return f(*a, **kw)
        monkeypatch.setattr(torch, name, made)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: World.streams[-1])
    monkeypatch.setattr(torch.cuda, "stream", Under)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: World.log.append(("known to", s.name)))
    monkeypatch.setattr(moe, "lib", Library())
    monkeypatch.setattr(moe, "_dev", lambda t, name: None)
    monkeypatch.setattr(torch.cuda, "device", OnDevice)
    monkeypatch.setattr(moe, "_get_device", lambda: World.device)
    yield World
    assert [s.name for s in World.streams] == ["current"] and World.device == 0


def routed_calls():
    """name -> (call, its own tensors are returned)."""
    z = torch.zeros
    w = moe.Weights(z((2, 64, 32), dtype=U8), z((2, 64, 2), dtype=U8))
    x, off, ids, topw = z((4, 64), dtype=BF16), z(3, dtype=I32), z((4, 2), dtype=I32), z((4, 2))
    made = [z((4, 2), dtype=I32), z((4, 2)), off, z(8, dtype=I32), z(8, dtype=I32)]
    return {
        "route": lambda **k: moe.route(topw, None, 2, 1, 1, 2, 1.0, **k),
        "route_gemv": lambda **k: moe.route_gemv(x, z((2, 64)), None, 2, 1, 1, 2, 1.0, z(64, dtype=U8), **k),
        "permute": lambda **k: moe.permute(ids, 2, **k),
        "route_permute": lambda **k: moe.route_permute(topw, None, 2, 1, 1, 2, 1.0, z(1, dtype=I32), **k),
        "route_permute_noalloc": lambda **k: moe.route_permute_noalloc(topw, None, 2, 1, 1, 2, 1.0, *made, **k),
        "grouped_gemm": lambda **k: moe.grouped_gemm(x, w, None, off, 4, **k),
        "combine": lambda **k: moe.combine(x, ids, topw, **k),
        "transcode_mx_to_nv": lambda **k: moe.transcode_mx_to_nv(w.scale, w.packed, **k),
        "tile_weights": lambda **k: moe.tile_weights(w, **k),
        "compact_mx": lambda **k: moe.compact_mx(w.scale, w.packed, **k),
        "compact_weights": lambda **k: moe.compact_weights(w, **k),
        "quantize_nvfp4": lambda **k: moe.quantize_nvfp4(x, **k),
        "quantize_mxfp8": lambda **k: moe.quantize_mxfp8(x, **k),
        "quantize_nvfp4_planes": lambda **k: moe.quantize_nvfp4_planes(x, **k),
        "reap_saliency_accumulate": lambda **k: moe.reap_saliency_accumulate(
            topw, off, ids, topw, z(2, dtype=torch.float64), z(2, dtype=torch.int64), 8, **k)}


def test_every_call_with_a_stream_is_looked_at():
    have = {n for n, f in vars(moe).items() if inspect.isfunction(f) and "stream" in inspect.signature(f).parameters
            and not n.startswith("_")}
    assert have == set(routed_calls())


@pytest.mark.parametrize("name", sorted(routed_calls()))
def test_outputs_are_made_on_the_callers_stream(world, name):
    """Memory from the current stream's pool may still be written by what is queued there; the caller's stream does not
    wait for that."""
    routed_calls()[name](stream=Stream("s", 0x20))
    made = [x for x in world.log if x[0] == "made on"]
    assert all(x == ("made on", "s") for x in made)
    assert [x for x in world.log if x[0] == "launched"] == [("launched", "s", 0x20)]
    known = [x for x in world.log if x[0] == "known to"]
    assert all(x == ("known to", "current") for x in known) and (not made or known)


@pytest.mark.parametrize("name", sorted(routed_calls()))
def test_without_a_stream_everything_is_on_the_current_one(world, name):
    routed_calls()[name]()
    assert [x for x in world.log if x[0] == "launched"] == [("launched", "current", 0x10)]
    assert {x for x in world.log if x[0] != "launched"} <= {("made on", "current")}


def test_an_error_leaves_the_current_stream(world):
    with pytest.raises(ValueError):
        moe.compact_weights(moe.Weights(*routed_weights(), tiled=True), stream=Stream("s", 0x20))


def routed_weights():
    return torch.zeros((2, 64, 32), dtype=U8), torch.zeros((2, 64, 2), dtype=U8)


@pytest.mark.parametrize("name", sorted(routed_calls()))
@pytest.mark.parametrize("device", [0, 1])
def test_calls_run_on_the_device_of_their_arguments(world, monkeypatch, name, device):
    """The default stream has one handle on all devices: the current device decides where a launch goes."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: device)
    routed_calls()[name]()
    assert world.devices == [device]
    if device == 1:
        with pytest.raises(ValueError, match="stream of cuda:0, the arguments are on cuda:1"):
            routed_calls()[name](stream=Stream("s", 0x20))
