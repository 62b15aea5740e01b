"""Where the attention calls make their tensors and run, with stand-ins for torch's tensors and streams (no GPU: calls
without rows launch nothing, refused ones neither)."""
import pytest
import torch

moe = pytest.importorskip("block_scaled_fp4_group_amd")

BF16, I32 = torch.bfloat16, torch.int32


class Tensor:
    """Contiguous, at an address that nothing follows."""
    log = []

    def __init__(self, shape, dtype=BF16, device=0):
        self.shape, self.dtype, self.device = tuple(shape), dtype, device

    def get_device(self):
        return self.device

    def stride(self):
        st, n = [], 1
        for d in reversed(self.shape):
            st.insert(0, n)
            n *= d
        return tuple(st)

    def data_ptr(self):
        return 0x10000

    def is_contiguous(self):
        return True

    def new_empty(self, shape, dtype=None):
        self.log.append(("made on", Streams.now[-1]))
        self.log.append(("device", Devices.now[-1]))
        return Tensor(shape, dtype or self.dtype, self.device)

    def unsafe_split_with_sizes(self, sizes):
        return [Tensor((n,), self.dtype, self.device) for n in sizes]

    def record_stream(self, s):
        self.log.append(("known to", s.name))


class Stream:
    cuda_stream = 0x5000

    def __init__(self, name, device_index=0):
        self.name, self.device_index = name, device_index


class Streams:
    """The stack of current streams; stands in for torch.cuda.stream()."""
    now = ["current"]

    def __init__(self, stream):
        self.stream = stream

    def __enter__(self):
        Streams.now.append(self.stream.name)

    def __exit__(self, *a):
        Streams.now.pop()


class Devices:
    """The stack of current devices; stands in for torch.cuda.device()."""
    now = [0]

    def __init__(self, index):
        self.index = index

    def __enter__(self):
        Devices.now.append(self.index)

    def __exit__(self, *a):
        Devices.now.pop()


@pytest.fixture
def calls():
    """The package's calls on the stand-ins."""
    Tensor.log.clear()
    moe._calls.setup(Tensor, BF16, I32, torch.float32, torch.uint8, lambda index: 0, moe._check, moe._bad,
                     lambda index: Stream("current"), Streams, lambda: Devices.now[-1], Devices)
    yield moe._calls
    moe._setup_calls()
    assert Streams.now == ["current"] and Devices.now == [0]


def empty_calls(calls, device=0, **kw):
    """Each call, without rows to work on (kv_slots is refused after its outputs are made)."""
    x, i = Tensor((0, 2, 128), BF16, device), Tensor((0,), I32, device)
    c, t = Tensor((4, 16, 2, 128), BF16, device), Tensor((0, 4), I32, device)
    return {
        "qk_norm_rope": lambda: calls.qk_norm_rope(x, x, None, None, **kw),
        "attn_prompt": lambda: calls.attn_prompt(x, x, x, Tensor((1,), I32, device), want_lse=True, **kw),
        "attn_decode": lambda: calls.attn_decode(x, c, c, t, i, 4, want_lse=True, **kw),
        "kv_slots": lambda: pytest.raises(moe.MoeError, calls.kv_slots, i, i, i, t, 24, 4, **kw),
    }


@pytest.mark.parametrize("name", ["qk_norm_rope", "attn_prompt", "attn_decode", "kv_slots"])
def test_outputs_are_made_on_the_callers_stream(calls, name):
    """Memory from the current stream's pool may still be written by what is queued there; the caller's stream does not
    wait for that."""
    empty_calls(calls, stream=Stream("s"))[name]()
    made = [x for x in Tensor.log if x[0] == "made on"]
    assert made and all(where == "s" for _, where in made)
    assert [x for x in Tensor.log if x[0] == "known to"] == [("known to", "current")] * len(made)


@pytest.mark.parametrize("name", ["qk_norm_rope", "attn_prompt", "attn_decode", "kv_slots"])
def test_without_a_stream_everything_is_on_the_current_one(calls, name):
    empty_calls(calls)[name]()
    assert {x for x in Tensor.log if x[0] != "device"} == {("made on", "current")}


def test_a_refused_call_leaves_the_current_stream(calls):
    for make in ("qk_norm_rope", "attn_prompt"):
        with pytest.raises(ValueError):
            getattr(calls, make)(Tensor((3, 2, 128)), Tensor((2, 2, 64)), None, None, stream=Stream("s"))
        assert Streams.now == ["current"]


@pytest.mark.parametrize("name", ["qk_norm_rope", "attn_prompt", "attn_decode", "kv_slots"])
@pytest.mark.parametrize("device", [0, 1])
def test_calls_run_on_the_device_of_their_arguments(calls, name, device):
    """The default stream has one handle on all devices: the current device decides where a launch goes."""
    empty_calls(calls, device)[name]()
    assert {x for x in Tensor.log if x[0] == "device"} == {("device", device)}


def test_a_stream_of_another_device_is_refused(calls):
    for name in ("qk_norm_rope", "attn_prompt", "attn_decode"):
        with pytest.raises(ValueError, match="stream of cuda:0, the arguments are on cuda:1"):
            empty_calls(calls, 1, stream=Stream("s", 0))[name]()
    assert not Tensor.log
