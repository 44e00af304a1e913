"""Refusals of pa_cross_attention (CPU)."""
import ctypes

import pagedattention_kv_cache_pa_b200 as pa
from pagedattention_kv_cache_pa_b200 import binding

FAKE = ctypes.c_void_p(0x10000)          # never dereferenced: validation fails first
MIS = ctypes.c_void_p(0x10008)


def _desc(**kw):
    base = dict(num_blocks=8, block_size=16, num_kv_heads=2, num_q_heads=4, head_dim=64, max_blocks_per_seq=4)
    return pa.CacheDesc.make(**{**base, **kw})


def _call(desc, q=FAKE, cu=FAKE, n=1, rows=4, longest=16, scale=0.1, ws=FAKE, size=256, out=FAKE):
    return binding.lib.pa_cross_attention(q, FAKE, FAKE, FAKE, cu, FAKE, n, rows, longest, ctypes.c_float(scale), out, ws,
                                          size, ctypes.byref(desc) if desc is not None else None, None)


def test_refusals():
    d = _desc()
    assert _call(None) == -1 and _call(d, n=-1) == -1 and _call(d, rows=-1) == -1 and _call(d, longest=-1) == -1
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _call(d, scale=scale) == -1
    assert _call(d, q=None) == -1 and _call(d, q=MIS) == -1 and _call(d, out=MIS) == -1
    assert _call(_desc(num_q_heads=5)) == -1
    assert _call(_desc(head_dim=96)) == -2 and _call(_desc(block_size=24)) == -2
    assert _call(d, rows=64 * 65535) == -2
    assert _call(d, ws=None) == -4 and _call(d, size=255) == -4 and _call(d, ws=MIS) == -4
    assert _call(d, n=0) == 0 and _call(d, rows=0) == 0
    # the single-row form takes no offsets, and exactly one row a sequence
    assert _call(d, cu=None, rows=2) == -1 and _call(d, cu=None, rows=0) == -1
    assert _call(d, cu=None, rows=1, n=0) == 0
    assert _call(_desc(num_q_heads=34), cu=None, rows=1) == -2


def test_workspace_size_of_many_rows():
    assert pa.pa_cross_attention_workspace_size(3, 5, 100, _desc()) >= 256
    assert binding.lib.pa_cross_attention_workspace_size(-1, 5, 100, ctypes.byref(_desc())) == 0
