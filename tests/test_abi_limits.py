"""Counts next to 2^31 of the window and decode calls: their kernels step 32-bit counters by the number of
blocks, so the last 2^16 counts are refused.  Every call here returns before its first CUDA call."""
import ctypes

import sparse_attention_long_head_b200 as vs


def _fake(addr):
    return ctypes.c_void_p(addr)


def test_window_units_next_to_32_bits():
    def call(B, pairs, Hq=6, Hkv=2, d=64):
        return vs.lib().vs_window_attn_fwd_varlen(
            _fake(0x1000), _fake(0x2000), _fake(0x3000), 0, 1000, B, _fake(0x9000), 256 * pairs, Hq, Hkv, d, Hq * d,
            Hkv * d, 0.0, 64, 4, _fake(0x8000), None, _fake(0x10010), 256, None)

    assert 7161 * 6 * 49981 == 2 ** 31 - 2
    assert call(7161, 49981) == vs.VS_ERR_UNSUPPORTED
    assert call(7162, 49981) == vs.VS_ERR_UNSUPPORTED
    # well below the border only the workspace, 16 bytes off its alignment, is wrong
    assert call(7000, 49981) == vs.VS_ERR_WORKSPACE


def test_decode_pages_next_to_32_bits():
    def call(B, pages, ws_bytes):
        return vs.lib().vs_kv4_decode_attn_fwd(
            _fake(0x10000), 0, 256, _fake(0x100000), 100, _fake(0x2000), 1 << 18, _fake(0x3000), B, 64 * pages, 4, 1,
            64, 0.0, 0, 0, None, None, 0, _fake(0x20000), None, _fake(0x40000), ws_bytes, None)

    assert 42966 * 49981 == 2 ** 31 - 2
    assert call(42966, 49981, 1 << 40) == vs.VS_ERR_UNSUPPORTED
    assert call(42967, 49981, 1 << 40) == vs.VS_ERR_UNSUPPORTED
    assert call(42000, 49981, 256) == vs.VS_ERR_WORKSPACE
