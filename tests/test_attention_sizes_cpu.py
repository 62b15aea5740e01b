"""Sizes whose products pass 64 bits are refused like others that are too large (no GPU needed)."""
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
