"""How the decode call shares the chip, read off the workspace that it asks for (no GPU needed)."""
import pytest

moe = pytest.importorskip("block_scaled_fp4_group_amd")


def runs(B, prefix, longest, Hq, Hkv, D=128):
    """Workgroups per key head that share the own keys of all requests, for a prefix of one part and up to 32 heads of a
    key head: each leaves two parts of G rows for each request that it meets, of which there are runs + B in all, and
    the prefix's part one row for each head."""
    G = Hq // Hkv
    assert G <= 32 and prefix <= 128 and B * G > 64
    entries, rest = divmod(moe.attn_decode_workspace_bytes(B, prefix, longest, Hq, Hkv, D, D) - 4 * (B + 1), 4 * D + 8)
    entries -= B * Hq if prefix else 0
    assert rest == 0 and entries % (Hkv * 2 * G) == 0
    return entries // (Hkv * 2 * G) - B


@pytest.mark.parametrize("B,Hq,Hkv,longest", [(512, 64, 8, 2048), (700, 64, 8, 2048), (1000, 64, 8, 2048), (512, 128, 16, 1024),
                                              (2048, 32, 8, 512), (256, 64, 8, 4000)])
def test_own_keys_of_many_requests_have_the_chip_behind_a_short_prefix(B, Hq, Hkv, longest):
    """A short prefix is done early however many rows it has: it must not leave the own keys a few workgroups."""
    alone = runs(B, 0, longest, Hq, Hkv)
    assert alone * Hkv >= 512 or Hkv > 512
    assert runs(B, 100, longest, Hq, Hkv) * Hkv >= 0.7 * 512


def test_own_keys_beside_a_long_prefix_keep_to_the_chip():
    """64 requests behind 8192 tokens: the two kinds run side by side, no workgroup waits for a place."""
    B, Hq, Hkv, D = 64, 64, 8, 128
    nbytes = moe.attn_decode_workspace_bytes(B, 8192, 2048, Hq, Hkv, D, D) - 4 * (B + 1)
    assert nbytes % (4 * D + 8) == 0
    entries = nbytes // (4 * D + 8)
    found = [(parts, own // (Hkv * 2 * 8) - B) for parts in range(1, 65)
             for own in [entries - parts * B * Hq] if own > 0 and own % (Hkv * 2 * 8) == 0]
    assert any(r > 0 and parts * 4 * Hkv + r * Hkv <= 512 for parts, r in found)
