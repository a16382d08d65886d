"""What the cache operators' calls refuse or promise beyond tests/test_cache_ops.py, without a GPU."""
import ctypes

import pytest

from test_cache_ops import ALIGN, CUDA, INVALID, _kv, dak, no_gpu  # noqa: F401 (fixtures)

pytestmark = pytest.mark.cpu


def test_append_rope_acc_refusals(dak, no_gpu):  # noqa: F811
    kv, rope = _kv(), dak.dak_rope_make(128)
    good = dict(KV=ctypes.byref(kv), rope=ctypes.byref(rope), q=0x100000, k=0x200000, v=0x300000, fp32=0, T=3, Hq=8,
                qp=8 * 128, kp=4 * 128, vp=4 * 128, slots=0x4000, pos=0x5000, n_new=0x6000, q_out=0x400000,
                slot_pos=0x7000, acc=0x8000, stream=None)

    def call(**kw):
        a = dict(good, **kw)
        return dak.lib.dak_kv_append_rope_acc(*[a[k] for k in good])

    assert call() == CUDA and call(acc=None) == CUDA and call(slot_pos=None) == CUDA
    assert call(acc=0x8002) == ALIGN
    assert call(KV=None) == INVALID and call(slots=None) == INVALID and call(T=0) == INVALID
