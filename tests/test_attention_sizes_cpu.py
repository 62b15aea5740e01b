"""Sizes whose products pass 64 bits are refused like others that are too large (no GPU needed)."""
import os
import subprocess
import sys

import pytest

from test_attention_abi_cpu import INVALID, moe, prompt, decode, refuses, rope


@pytest.mark.parametrize("T", [1 << 31, 1 << 60, 1 << 61, 1 << 62, (1 << 63) - 1])
def test_qk_norm_rope_refuses_any_number_of_tokens_that_is_too_large(T):
    """T x heads (8 here, and 10 for odd ones) wraps to 0 or to a small number at some of these."""
    for kw in (dict(), dict(q_heads=6), dict(kv_heads=6)):
        refuses(rope(T=T, **kw), INVALID)


@pytest.mark.parametrize("n", [1 << 31, 1 << 60, 1 << 62, (1 << 63) - 1])
def test_attention_refuses_any_number_of_rows_or_keys_that_is_too_large(n):
    refuses(prompt(tq=n), INVALID)
    refuses(prompt(tk=n), INVALID)
    refuses(decode(most=n), INVALID)
    refuses(decode(prefix=n), INVALID)
    assert moe.attn_prompt_workspace_bytes(1, n, n, 8, 2, 128, 128) == 0
    assert moe.attn_decode_workspace_bytes(1, n, n, 8, 2, 128, 128) == 0


@pytest.mark.parametrize("B,Hq,Hkv", [(1 << 23, 1 << 16, 1), ((1 << 31) - 1, 1 << 16, 1 << 16), (1 << 24, 1 << 15, 1), (1 << 15, 1 << 16, 1)])
def test_decode_refuses_rows_past_31_bits(B, Hq, Hkv):
    """In a process of its own: the plan's row blocks wrapped to 0, and a division by them ended the process."""
    code = (f"import test_attention_abi_cpu as t\n"
            f"assert t.moe.attn_decode_workspace_bytes({B}, 100, 4000, {Hq}, {Hkv}, 128, 128) == 0\n"
            f"t.refuses(t.decode(B={B}, hq={Hq}, hkv={Hkv}), t.INVALID)\n")
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=here,
                       env={**os.environ, "PYTHONPATH": os.path.dirname(here)})
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
