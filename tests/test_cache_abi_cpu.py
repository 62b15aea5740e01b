"""The calls around the cache and the residual stream's norms refuse bad arguments on the host, before any launch, and make
their tensors where they run (no GPU needed)."""
import ctypes
import inspect

import pytest
import torch

moe = pytest.importorskip("block_scaled_fp4_group_amd")

from test_attention_streams_cpu import BF16, Devices, I32, Stream, Streams, Tensor as Plain  # noqa: E402

P = ctypes.c_void_p(0x10000)          # an aligned address that the checks never follow
FAR = ctypes.c_void_p(0x90000000)
ODD = ctypes.c_void_p(0x10008)
INVALID, UNSUPPORTED, WORKSPACE, OK = moe.MOE_ERR_INVALID, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE, moe.MOE_OK


def refuses(status, expect):
    assert status == expect, (status, moe.lib.moe_last_error())
    assert bool(moe.lib.moe_last_error()) == (expect != OK)


def heads(h, d, data=0x10000, ts=None, hs=None):
    return moe.Heads(data, h * d if ts is None else ts, d if hs is None else hs)


def cache4(k=0x10000, ks=0x10000, v=0x10000, vs=0x10000, pages=8, page=16, kg=1.0, vg=0.25):
    return moe.KvCacheFp4(k, ks, v, vs, pages, page, kg, vg)


BAD_CACHES = [dict(k=None), dict(ks=None), dict(v=None), dict(vs=None), dict(k=0x10008), dict(vs=0x10004), dict(page=8), dict(page=24),
              dict(page=2048), dict(pages=0), dict(pages=1 << 28), dict(kg=0.0), dict(kg=3.0), dict(vg=-1.0), dict(vg=float("inf")),
              dict(vg=float("nan")), dict(kg=2.0 ** 33), dict(vg=2.0 ** -33)]


def rope(T=4, q=None, k=None, v=None, qo=None, ko=None, cache=None, slots=P, pos=P, cs=P, qw=P, **kw):
    f = dict(q_heads=4, kv_heads=2, head_dim=128, v_dim=128, rot_dim=64, interleaved=0, max_position=100, eps=1e-6)
    f.update(kw)
    D = f["head_dim"]
    return moe.lib.moe_qk_norm_rope_fp4(heads(4, D) if q is None else q, heads(2, D) if k is None else k,
                                        heads(2, 128) if v is None else v, T, moe.RopeParams(*f.values()), pos, cs, qw, None,
                                        heads(4, D) if qo is None else qo, ko, cache4() if cache is None else cache, slots, None)


def test_qk_norm_rope_fp4_refuses():
    for kw in (dict(T=-1), dict(q_heads=0), dict(eps=-1.0), dict(rot_dim=-32), dict(rot_dim=160), dict(pos=None), dict(cs=None),
               dict(max_position=0), dict(qw=ODD), dict(q=heads(4, 128, None)), dict(k=heads(2, 128, hs=-128)),
               dict(qo=heads(4, 128, ts=504)), dict(ko=heads(2, 128, ts=120)), dict(slots=None), dict(v_dim=24), dict(v_dim=0),
               dict(v=heads(2, 128, 0x10002)), dict(T=1 << 30), *(dict(cache=cache4(**c)) for c in BAD_CACHES)):
        refuses(rope(**kw), INVALID)
    for kw in (dict(head_dim=96), dict(rot_dim=16), dict(rot_dim=48)):
        refuses(rope(**kw), UNSUPPORTED)
    refuses(rope(T=0), OK)


def decode(B=4, c=None, table=P, stride=16, blocks=16, lens=P, most=100, ptab=P, pblocks=4, prefix=40, q=None, out=None,
           lse=None, ws=P, nbytes=1 << 40, hq=8, hkv=2, D=128, Dv=128, scale=0.1):
    p = moe.AttnParams(hq, hkv, D, Dv, scale)
    return moe.lib.moe_attn_decode_fp4(heads(hq, D) if q is None else q, cache4() if c is None else c, table, stride, blocks, lens,
                                       B, most, ptab, pblocks, prefix, p, heads(hq, Dv) if out is None else out, lse, ws, nbytes,
                                       None)


def test_attn_decode_fp4_refuses():
    for kw in (dict(B=-1), dict(most=-1), dict(prefix=-1), dict(blocks=-1), dict(most=257), dict(stride=15), dict(table=None),
               dict(lens=None), dict(prefix=65), dict(ptab=None), dict(hq=9), dict(scale=0.0), dict(q=heads(8, 128, None)),
               dict(out=heads(8, 128, hs=64)), dict(lse=ctypes.c_void_p(0x10001)), *(dict(c=cache4(**c)) for c in BAD_CACHES)):
        refuses(decode(**kw), INVALID)
    refuses(decode(D=192, Dv=192), UNSUPPORTED)
    f = moe.attn_decode_fp4_workspace_bytes
    assert f(4, 40, 100, 8, 2, 128, 128) == 0 and f(0, 40, 100, 8, 2, 128, 128) == 0 and f(4, -1, 100, 8, 2, 128, 128) == 0
    need = f(4, 40, 16000, 8, 2, 128, 128)
    assert need > 0
    for kw in (dict(ws=None), dict(nbytes=need - 1), dict(ws=ODD)):
        refuses(decode(most=16000, blocks=1000, stride=1000, **kw), WORKSPACE)
    refuses(decode(B=0), OK)


def test_attn_decode_fp4_workspace_stays_bounded():
    """Parts are for the workgroups that the chip holds, whatever the sizes, and one for each request and run."""
    for B, prefix, most, hq, hkv in ((1, 0, 1 << 20, 64, 1), (4096, 100, 2048, 64, 8), (2000, 1 << 20, 1 << 16, 8, 8), (70, 40000, 0, 64, 4)):
        rows = B * hq
        assert 0 < moe.attn_decode_fp4_workspace_bytes(B, prefix, most, hq, hkv, 128, 128) <= (1100 * 128 * 2 + 4 * rows) * 520 + 4 * B + 4


def gather(fp4=True, c=None, H=2, D=64, Dv=64, table=P, stride=4, blocks=4, ptab=P, pblocks=2, prefix=20, cu=P, seqs=2, total=50,
           ko=None, vo=None):
    f = moe.lib.moe_kv_gather_fp4 if fp4 else moe.lib.moe_kv_gather
    c = (cache4() if fp4 else moe.KvCache(0x10000, 0x10000, 8, 16)) if c is None else c
    return f(c, H, D, Dv, table, stride, blocks, ptab, pblocks, prefix, cu, seqs, total,
             heads(max(H, 1), D) if ko is None else ko, heads(max(H, 1), Dv) if vo is None else vo, None)


@pytest.mark.parametrize("fp4", [True, False])
def test_kv_gather_refuses(fp4):
    bad = (cache4(page=8), cache4(vg=3.0)) if fp4 else (moe.KvCache(None, 0x10000, 8, 16), moe.KvCache(0x10000, 0x10000, 8, 24))
    for kw in (dict(H=0), dict(D=24), dict(Dv=0), dict(D=2048), dict(table=None), dict(stride=3), dict(blocks=-1), dict(ptab=None),
               dict(prefix=33), dict(prefix=-1), dict(pblocks=-1, prefix=0), dict(cu=None), dict(seqs=-1), dict(total=-1),
               dict(total=1 << 31), dict(total=(1 << 31) - 64, H=64, ko=heads(64, 64), vo=heads(64, 64)),
               dict(ko=heads(2, 64, ts=64)), dict(vo=heads(2, 64, 0x10004)), *(dict(c=c) for c in bad)):
        refuses(gather(fp4, **kw), INVALID)
    refuses(gather(fp4, seqs=0), OK)
    refuses(gather(fp4, total=0), OK)


def buffers(*pairs, count=None):
    b = moe.PageBuffers()
    for i, (p, n) in enumerate(pairs):
        b.data[i], b.page_bytes[i] = p, n
    b.count = len(pairs) if count is None else count
    return b


GOOD = buffers((0x10000, 256), (0x20000, 64))
BAD_BUFFERS = [buffers((None, 256)), buffers((0x10008, 256)), buffers((0x10000, 8)), buffers((0x10000, 0)), buffers((0x10000, -16)),
               buffers((0x10000, 1 << 41)), buffers(count=9), buffers(count=-1)]
BAD_TABLES = [dict(rows=-1), dict(blocks=-1), dict(stride=3), dict(table=None), dict(lens=None), dict(page=0), dict(page=24), dict(page=2048),
              dict(pages=0), dict(pages=1 << 28), dict(blocks=1 << 28, stride=1 << 28)]


def fork(table=P, stride=4, rows=3, blocks=4, lens=P, par=P, chi=P, n=2, pool=P, free=5, page=16, buf=GOOD, pages=100, counts=P):
    return moe.lib.moe_kv_fork(table, stride, rows, blocks, lens, par, chi, n, pool, free, page, buf, pages, counts, None)


def test_kv_fork_refuses():
    for kw in (*BAD_TABLES, *(dict(buf=b) for b in BAD_BUFFERS), dict(n=-1), dict(free=-1), dict(par=None), dict(chi=None),
               dict(pool=None), dict(counts=None)):
        refuses(fork(**kw), INVALID)
    refuses(fork(n=65537), UNSUPPORTED)


def free_pages(table=P, stride=4, rows=3, blocks=4, lens=P, page=16, pages=100, out=P, counts=P, ws=None, nbytes=0):
    return moe.lib.moe_kv_free_pages(table, stride, rows, blocks, lens, page, pages, out, counts, ws, nbytes, None)


def test_kv_free_pages_refuses():
    for kw in (*BAD_TABLES, dict(out=None), dict(counts=None)):
        refuses(free_pages(**kw), INVALID)
    refuses(free_pages(pages=(1 << 20) + 1), UNSUPPORTED)
    need = moe.kv_free_pages_workspace_bytes(3, 4, 70000)
    assert need >= 70000 and moe.kv_free_pages_workspace_bytes(3, 4, 100) == 0 and moe.kv_free_pages_workspace_bytes(300, 400, 100) >= 100
    for kw in (dict(), dict(ws=P, nbytes=need - 1), dict(ws=ODD, nbytes=need)):
        refuses(free_pages(pages=70000, **kw), WORKSPACE)


def compact(table=P, stride=4, rows=3, blocks=4, lens=P, page=16, buf=GOOD, pages=100, out=FAR, ostride=4, counts=P, ws=P, nbytes=1 << 30):
    return moe.lib.moe_kv_compact(table, stride, rows, blocks, lens, page, buf, pages, out, ostride, counts, ws, nbytes, None)


def test_kv_compact_refuses():
    near = ctypes.c_void_p(0x10000 + 40)                              # 10 entries in: rows of both overlap
    for kw in (*BAD_TABLES, *(dict(buf=b) for b in BAD_BUFFERS), dict(out=None), dict(ostride=3), dict(counts=None), dict(out=near),
               dict(out=P, ostride=5)):
        refuses(compact(**kw), INVALID)
    refuses(compact(pages=(1 << 20) + 1), UNSUPPORTED)
    need = moe.kv_compact_workspace_bytes(100)
    assert need > 0 and moe.kv_compact_workspace_bytes(0) == 0 and moe.kv_compact_workspace_bytes(1 << 21) == 0
    for kw in (dict(ws=None), dict(nbytes=need - 1), dict(ws=ODD)):
        refuses(compact(**kw), WORKSPACE)


def norm(T=4, hidden=64, x=0x10000, xs=64, r=None, post=None, g=None, gc=None, scale=1.0, w=P, eps=1e-6, h=(0x20000, 64), y=(0x30000, 64)):
    rows = lambda a: None if a is None else moe.Rows(*a)  # noqa: E731
    return moe.lib.moe_block_norm(moe.Rows(x, xs), T, hidden, rows(r), post, rows(g), gc, scale, w, eps, rows(h), rows(y), None)


def test_block_norm_refuses():
    for kw in (dict(T=-1), dict(T=1 << 31), dict(hidden=0), dict(hidden=60), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(eps=-1.0), dict(eps=float("nan")), dict(h=None, y=None), dict(w=None), dict(w=ODD), dict(post=ODD), dict(gc=ODD),
               dict(g=(0x40000, 64), gc=P), dict(x=None), dict(x=0x10002), dict(xs=60), dict(xs=-64), dict(r=(None, 64)),
               dict(r=(0x40000, 4)), dict(g=(0x40008, 64)), dict(h=(0x20000, 56)), dict(y=(0x30000, 0)), dict(y=(None, 64))):
        refuses(norm(**kw), INVALID)
    refuses(norm(hidden=32776, xs=32776), UNSUPPORTED)
    refuses(norm(T=0), OK)


def test_sizes_past_a_launch_are_refused():
    """A launch's threads are counted in 32 bits: by name, not by the launch."""
    for kw in (dict(q_heads=64, kv_heads=8, head_dim=192, T=1 << 23), dict(q_heads=4, kv_heads=2, head_dim=64, T=1 << 28)):
        D, hq, hkv = kw["head_dim"], kw["q_heads"], kw["kv_heads"]
        refuses(rope(q=heads(hq, D), k=heads(hkv, D), v=heads(hkv, 128), qo=heads(hq, D), **kw), INVALID)
        assert b"too many heads" in moe.lib.moe_last_error()
    for kw in (dict(B=1 << 20, hq=64, hkv=64, most=100), dict(B=1 << 20, hq=64, hkv=1, most=1 << 13, blocks=512, stride=512)):
        refuses(decode(**{**dict(prefix=0), **kw}), INVALID)
        assert b"too many rows" in moe.lib.moe_last_error()
    for fp4 in (True, False):
        refuses(gather(fp4, total=1 << 25, H=16, ko=heads(16, 64), vo=heads(16, 64)), INVALID)
        assert b"too many rows" in moe.lib.moe_last_error()


# --------------------------------------------------------------- Python's side
def test_wrappers_refuse_before_the_library():
    x, i = torch.zeros((2, 2, 128), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    c = moe.Fp4Cache.zeros(2, 16, 2, 128, 128, device="cpu")
    for call in (lambda: moe.qk_norm_rope_fp4(x, x, x, None, None, c, i), lambda: moe.attn_decode_fp4(x, c, i[None], i, 1),
                 lambda: moe.kv_gather(x[None], x[None], i[None], i, 3), lambda: moe.kv_gather_fp4(c, i[None], i, 3),
                 lambda: moe.kv_fork(i[None], i, i, i, i, 16, c.buffers), lambda: moe.kv_free_pages(i[None], i, 16, 4),
                 lambda: moe.kv_compact(i[None], i, 16, c.buffers), lambda: moe.block_norm(x[0], None)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    assert list(inspect.signature(moe.attn_decode_fp4).parameters)[:3] == ["q", "cache", "block_table"]
    assert inspect.signature(moe.block_norm).parameters["scale"].default == 1.0


def test_cache_shapes():
    c = moe.Fp4Cache.zeros(5, 32, 3, 192, 128, device="cpu")
    assert [tuple(b.shape) for b in c.buffers] == [(5, 3, 32, 96), (5, 3, 32, 12), (5, 3, 32, 64), (5, 3, 8, 32)]


class Tensor(Plain):
    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def element_size(self):
        return {BF16: 2, I32: 4, torch.float32: 4, torch.uint8: 1}[self.dtype]

    def dim(self):
        return len(self.shape)

    def new_empty(self, shape, dtype=None):
        self.log.append(("made on", Streams.now[-1]))
        self.log.append(("device", Devices.now[-1]))
        return Tensor(shape, dtype or self.dtype, self.device)


@pytest.fixture
def calls():
    Tensor.log.clear()
    moe._calls.setup(Tensor, BF16, I32, torch.float32, torch.uint8, lambda index: 0, moe._check, moe._bad,
                     lambda index: Stream("current"), Streams, lambda: Devices.now[-1], Devices)
    yield moe._calls
    moe._setup_calls()
    assert Streams.now == ["current"] and Devices.now == [0]


def fp4_cache(device, H=2, D=128, page=16):
    u8 = lambda *s: Tensor(s, torch.uint8, device)  # noqa: E731
    return moe.Fp4Cache(u8(4, H, page, D // 2), u8(4, H, page, D // 16), u8(4, H, page, D // 2), u8(4, H, D // 16, page))


def empty_calls(calls, device=0, **kw):
    """Each call, without rows to work on (the page calls are refused after their outputs are made)."""
    i = lambda *s: Tensor(s, I32, device)  # noqa: E731
    x, c, b = Tensor((0, 2, 128), BF16, device), fp4_cache(device), [Tensor((4, 3, 8), BF16, device)]
    refused = lambda f, *a: pytest.raises(moe.MoeError, f, *a, **kw)  # noqa: E731
    return {
        "qk_norm_rope_fp4": lambda: calls.qk_norm_rope_fp4(x, x, x, None, None, c, i(0), **kw),
        "attn_decode_fp4": lambda: calls.attn_decode_fp4(x, c, i(0, 4), i(0), 4, want_lse=True, **kw),
        "kv_gather_fp4": lambda: calls.kv_gather_fp4(c, i(0, 4), i(1), 0, **kw),
        "kv_gather": lambda: calls.kv_gather(Tensor((4, 16, 2, 128), BF16, device), Tensor((4, 16, 2, 64), BF16, device), i(0, 4), i(1), 0, **kw),
        "kv_fork": lambda: refused(calls.kv_fork, i(2, 4), i(2), i(1), i(1), i(3), 24, b),
        "kv_free_pages": lambda: refused(calls.kv_free_pages, i(2, 4), i(2), 24, 4),
        "kv_compact": lambda: refused(calls.kv_compact, i(2, 4), i(2), 24, b),
        "block_norm": lambda: calls.block_norm(Tensor((0, 64), BF16, device), Tensor((64,), torch.float32, device), **kw),
    }


NAMES = ["qk_norm_rope_fp4", "attn_decode_fp4", "kv_gather_fp4", "kv_gather", "kv_fork", "kv_free_pages", "kv_compact", "block_norm"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_made_on_the_callers_stream(calls, name):
    empty_calls(calls, stream=Stream("s"))[name]()
    made = [x for x in Tensor.log if x[0] == "made on"]
    known = [x for x in Tensor.log if x[0] == "known to"]
    assert made and all(where == "s" for _, where in made)
    # (a workspace is made too, and nobody else's)
    assert known == [("known to", "current")] * (len(made) - (name == "kv_compact"))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("device", [0, 1])
def test_calls_run_on_the_device_of_their_arguments(calls, name, device):
    empty_calls(calls, device)[name]()
    assert {x for x in Tensor.log if x[0] == "device"} == {("device", device)}
    assert {x for x in Tensor.log if x[0] != "device"} == {("made on", "current")}


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(calls, name):
    with pytest.raises(ValueError, match="stream of cuda:0, the arguments are on cuda:1"):
        empty_calls(calls, 1, stream=Stream("s", 0))[name]()
    assert not Tensor.log


@pytest.mark.parametrize("bad", ["k", "k_scale", "v", "v_scale"])
def test_caches_that_do_not_fit_are_refused(calls, bad):
    x, i = Tensor((3, 2, 128)), lambda *s: Tensor(s, I32)
    for shape in ((4, 2, 16, 65), (4, 2, 32, 64), (5, 2, 16, 64), (4, 2, 16)):
        c = fp4_cache(0)
        setattr(c, bad, Tensor(shape, torch.uint8))
        with pytest.raises(ValueError):
            calls.attn_decode_fp4(x, c, i(3, 4), i(3), 4)
    for make in (lambda: fp4_cache(1), lambda: fp4_cache(0, H=3), lambda: fp4_cache(0, D=64), lambda: None):
        with pytest.raises((ValueError, AttributeError)):
            calls.qk_norm_rope_fp4(x, x, x, None, None, make(), i(3))
    assert not [e for e in Tensor.log if e[0] == "made on"]


def test_page_calls_refuse_tables_and_buffers(calls):
    i, b = lambda *s: Tensor(s, I32), lambda *s: Tensor(s, torch.uint8)
    good = [b(4, 16), b(4, 32)]
    for bufs in ([], [b(4, 16), b(5, 16)], [b(0, 16)], [Tensor((4, 16), torch.uint8, 1)], [1], [b(4, 16)] * 9):
        with pytest.raises((ValueError, TypeError)):
            calls.kv_compact(i(2, 3), i(2), 16, bufs)
    for args in ((i(1, 3), i(2), i(1), i(1)), (i(2, 3), i(2), i(1), i(2)), (b(2, 3), i(2), i(1), i(1)), (i(2, 3), b(2), i(1), i(1))):
        with pytest.raises(ValueError):
            calls.kv_fork(*args, i(3), 16, good)
    for kw in (dict(free_pages=i(3)), dict(counts=i(1)), dict(free_pages=b(4)), dict(counts=Tensor((2,), I32, 1))):
        with pytest.raises(ValueError):
            calls.kv_free_pages(i(2, 3), i(2), 16, 4, **kw)
    for kw in (dict(out_table=i(1, 3)), dict(out_table=i(2, 2)), dict(out_table=b(2, 3))):
        with pytest.raises(ValueError):
            calls.kv_compact(i(2, 3), i(2), 16, good, **kw)
    with pytest.raises(ValueError, match="positive"):
        calls.kv_free_pages(i(2, 3), i(2), 16, 0)


def test_block_norm_refuses_rows_that_do_not_fit(calls):
    x, w = Tensor((3, 64)), Tensor((64,), torch.float32)
    for kw in (dict(residual=Tensor((2, 64))), dict(residual=Tensor((3, 64), torch.float32)), dict(post_weight=Tensor((32,), torch.float32)),
               dict(gate=Tensor((3, 32))), dict(gate=Tensor((3,), torch.float32)), dict(gate=Tensor((64,))), dict(h=Tensor((3, 72))),
               dict(y=Tensor((4, 64))), dict(gate=3)):
        with pytest.raises(ValueError):
            calls.block_norm(x, w, **kw)
    with pytest.raises(ValueError, match="y needs weight"):
        calls.block_norm(x, None, y=Tensor((3, 64)))
    with pytest.raises(ValueError):
        calls.block_norm(Tensor((3, 2, 64)), w)
