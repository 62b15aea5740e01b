"""The attention entry points refuse bad arguments on the host, before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

moe = pytest.importorskip("block_scaled_fp4_group_amd")

P = ctypes.c_void_p(0x10000)          # an aligned address that the checks never follow
ODD = ctypes.c_void_p(0x10008)
INVALID, UNSUPPORTED, WORKSPACE, OK = moe.MOE_ERR_INVALID, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE, moe.MOE_OK


def refuses(status, expect):
    assert status == expect, (status, moe.lib.moe_last_error())
    assert bool(moe.lib.moe_last_error()) == (expect != OK)


def heads(h, d, data=0x10000, ts=None, hs=None):
    return moe.Heads(data, h * d if ts is None else ts, d if hs is None else hs)


def slots(B=2, free=4, page=16, blocks=4, stride=4, base=0, most=8, ptr=P, out=P, table=P, pool=P):
    return moe.lib.moe_kv_slots(ptr, P, B, pool, free, page, table, stride, blocks, base, most, out, P, P, P, None)


def test_kv_slots_refuses():
    for kw in (dict(B=-1), dict(free=-1), dict(most=-1), dict(base=-1), dict(page=0), dict(page=24), dict(page=2048),
               dict(blocks=0), dict(stride=3), dict(blocks=1 << 28, stride=1 << 28), dict(most=1 << 31), dict(ptr=None),
               dict(out=None), dict(table=None), dict(pool=None)):
        refuses(slots(**kw), INVALID)
    refuses(slots(B=4097), UNSUPPORTED)


def rope(T=4, p=None, q=None, k=None, v=None, qo=None, ko=None, cache=None, slots=P, pos=P, cs=P, qw=P, **kw):
    fields = dict(q_heads=4, kv_heads=2, head_dim=128, v_dim=128, rot_dim=64, interleaved=0, max_position=100, eps=1e-6)
    fields.update(kw)
    D = fields["head_dim"]
    prm = moe.RopeParams(*fields.values()) if p is None else p
    return moe.lib.moe_qk_norm_rope(heads(4, D) if q is None else q, heads(2, D) if k is None else k,
                                    heads(2, 128) if v is None else v, T, prm, pos, cs, qw, None,
                                    heads(4, D) if qo is None else qo, heads(2, D) if ko is None else ko or None, cache,
                                    slots, None)


def cache(k=0x10000, v=0x10000, pages=8, page=16):
    return moe.KvCache(k, v, pages, page)


def test_qk_norm_rope_refuses():
    for kw in (dict(T=-1), dict(q_heads=0), dict(kv_heads=0), dict(eps=-1.0), dict(eps=float("nan")), dict(rot_dim=-16),
               dict(rot_dim=24), dict(rot_dim=144), dict(pos=None), dict(cs=None), dict(max_position=0), dict(qw=ODD),
               dict(q=heads(4, 128, None)), dict(q=heads(4, 128, 0x10002)), dict(q=heads(4, 128, ts=515)),
               dict(k=heads(2, 128, hs=-128)), dict(qo=heads(4, 128, ts=504)), dict(qo=heads(4, 128, hs=120)),
               dict(ko=False), dict(cache=cache(k=None)), dict(cache=cache(page=12)), dict(cache=cache(pages=0)),
               dict(cache=cache(pages=1 << 30)), dict(cache=cache(), slots=None), dict(cache=cache(), v_dim=12),
               dict(cache=cache(), v=heads(2, 128, None)), dict(cache=cache(v=0x10008)), dict(T=1 << 30)):
        refuses(rope(**kw), INVALID)
    refuses(rope(head_dim=96), UNSUPPORTED)
    refuses(rope(T=0), OK)


def prompt(seqs=2, tq=8, tk=8, q=None, k=None, out=None, cu=P, lse=None, hq=4, hkv=2, D=128, Dv=128, scale=0.1,
           ws=None, nbytes=0):
    p = moe.AttnParams(hq, hkv, D, Dv, scale)
    return moe.lib.moe_attn_prompt(heads(hq, D) if q is None else q, heads(hkv, D) if k is None else k, heads(hkv, Dv), cu, P,
                                   seqs, tq, tk, p, heads(hq, Dv) if out is None else out, lse, ws, nbytes, None)


def test_attn_prompt_refuses():
    for kw in (dict(seqs=-1), dict(tq=-1), dict(tk=-1), dict(tq=1 << 31), dict(hq=3), dict(hkv=0), dict(hq=1, hkv=2),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(cu=None),
               dict(q=heads(4, 128, None)), dict(k=heads(2, 128, 0x10004)), dict(out=heads(4, 128, ts=128)),
               dict(lse=ctypes.c_void_p(0x10002)), dict(tq=(1 << 31) - 1, hq=4096, hkv=1)):
        refuses(prompt(**kw), INVALID)
    for D, Dv in ((96, 96), (128, 64), (192, 192), (256, 256)):
        refuses(prompt(D=D, Dv=Dv), UNSUPPORTED)
    refuses(prompt(k=heads(2, 128, ts=(1 << 23) + 8)), UNSUPPORTED)
    need = moe.attn_prompt_workspace_bytes(2, 8, 8000, 4, 2, 128, 128)
    assert need > 0                                                  # few rows, many keys: parts to join
    for kw in (dict(), dict(ws=P, nbytes=need - 1), dict(ws=ODD, nbytes=need)):
        refuses(prompt(tk=8000, **kw), WORKSPACE)
    refuses(prompt(seqs=0), OK)
    refuses(prompt(tq=0), OK)


def decode(B=4, c=None, table=P, stride=16, blocks=16, lens=P, most=100, ptab=P, pblocks=4, prefix=40, q=None, out=None,
           lse=None, ws=P, nbytes=1 << 40, hq=8, hkv=2, D=128, Dv=128, scale=0.1):
    p = moe.AttnParams(hq, hkv, D, Dv, scale)
    return moe.lib.moe_attn_decode(heads(hq, D) if q is None else q, cache() if c is None else c, table, stride, blocks, lens,
                                   B, most, ptab, pblocks, prefix, p, heads(hq, Dv) if out is None else out, lse, ws, nbytes,
                                   None)


def test_attn_decode_refuses():
    for kw in (dict(B=-1), dict(most=-1), dict(prefix=-1), dict(blocks=-1), dict(most=257), dict(stride=15), dict(table=None),
               dict(lens=None), dict(prefix=65), dict(ptab=None), dict(hq=9), dict(scale=0.0), dict(c=cache(page=48)),
               dict(c=cache(k=0x10008)), dict(c=cache(pages=1 << 28)), dict(q=heads(8, 128, None)),
               dict(out=heads(8, 128, hs=64)), dict(lse=ctypes.c_void_p(0x10001))):
        refuses(decode(**kw), INVALID)
    refuses(decode(D=192, Dv=192), UNSUPPORTED)
    assert moe.attn_decode_workspace_bytes(4, 40, 100, 8, 2, 128, 128) == 0     # few keys: no parts to join
    need = moe.attn_decode_workspace_bytes(4, 40, 4000, 8, 2, 128, 128)
    assert need > 0
    for kw in (dict(ws=None), dict(nbytes=need - 1), dict(ws=ODD)):
        refuses(decode(most=4000, blocks=256, stride=256, **kw), WORKSPACE)
    refuses(decode(B=0), OK)


def test_workspace_size():
    f = moe.attn_decode_workspace_bytes
    assert f(0, 40, 100, 8, 2, 128, 128) == 0 and f(4, -1, 100, 8, 2, 128, 128) == 0 and f(4, 40, 100, 7, 2, 128, 128) == 0
    assert f(1, 0, 0, 8, 2, 128, 128) == 0                          # nothing to join
    assert f(1, 0, 131072, 32, 8, 128, 128) > 0
    g = moe.attn_prompt_workspace_bytes
    assert g(0, 8, 8000, 4, 2, 128, 128) == 0 and g(2, 8, 8000, 5, 2, 128, 128) == 0 and g(2, 0, 8000, 4, 2, 128, 128) == 0
    assert g(16, 64, 512 * 16 - 1, 4, 2, 128, 128) == 0             # under 512 keys each: never
    assert g(1, 16384, 16384, 32, 4, 128, 128) == 0                 # rows for the whole chip


def test_python_wrappers_refuse_before_the_library():
    x = torch.zeros((2, 2, 128), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.attn_prompt(x, x, x, i)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.attn_decode(x, x[None], x[None], i[None], i, 1)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.qk_norm_rope(x, x, None, None)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.kv_slots(i, i, i, i[None], 16, 1)


def test_calls_parse_like_python_functions():
    x = torch.zeros((2, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="missing required argument 'cu_q'"):
        moe.attn_prompt(x, x, x)
    with pytest.raises(TypeError, match="unexpected keyword argument 'cuq'"):
        moe.attn_prompt(x, x, x, x, cuq=x)
    with pytest.raises(TypeError, match="multiple values for argument 'q'"):
        moe.attn_prompt(x, x, x, x, q=x)
    with pytest.raises(TypeError, match="at most 12"):
        moe.kv_slots(*[x] * 13)
    with pytest.raises(ValueError, match="q must be a GPU tensor"):
        moe.attn_decode(None, x, x, x, x, 1)
    import inspect
    assert list(inspect.signature(moe.attn_decode).parameters)[:4] == ["q", "k_cache", "v_cache", "block_table"]
    assert inspect.signature(moe.qk_norm_rope).parameters["eps"].default == 1e-6
    assert "paged cache" in moe.attn_decode.__doc__
