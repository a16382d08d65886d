"""The largest placements that dak_attn_tree takes: what dak.h says, decided before any CUDA call."""
import ctypes

import pytest

from test_cache_ops import CUDA, UNSUPPORTED, _kv, dak, no_gpu  # noqa: F401

pytestmark = pytest.mark.cpu


def _line(B, H, L, T, G):
    return (6 + 2 * -(-L // 64)) * -(-T // (128 // G)) * B * H


@pytest.mark.parametrize("B,H,L,T,G", [
    (2000, 8, 64, 1, 1), (1 << 20, 8, 64, 256, 16), (1 << 20, 16, 64, 256, 8), (4096, 8, 1 << 20, 1, 1), (4096, 8, 1 << 20, 4, 1),
    (2, 1, 2_000_000_000, 1, 1), (32, 8, 1 << 20, 256, 16), (1, 1, 1 << 30, 256, 16), (1 << 23, 1, 64, 256, 1)])
def test_the_line_fits_or_is_refused(dak, no_gpu, B, H, L, T, G):
    kv, W = _kv(B=B, H=H, L=L), -(-T // 64)
    fits = _line(B, H, L, T, G) < 2 ** 31 - 2 ** 24 and B * H * -(-L // 64) < 2 ** 31 and B * T < 2 ** 31
    n = dak.lib.dak_attn_tree_workspace_bytes(ctypes.byref(kv), T, H * G)
    assert (n > 0) == fits
    st = dak.lib.dak_attn_tree(0x1000, ctypes.byref(kv), 0x2000, T, 0x3000, T * W, None, H * G, 0.0, 1 << 60, 0, 0x4000, 1 << 50,
                               None, None)
    assert st == (CUDA if fits else UNSUPPORTED)
