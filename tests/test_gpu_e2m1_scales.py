"""4-bit attention with cache scales at the ends of their range (needs a B200 but for the refusals).

Tolerances as in test_gpu_e2m1.py: |got - ref| <= 2^-8 |ref| + 2^-9 max|V|.  The scales multiply fp32
sums once more (2^-24), and an output below 2^-126 is rounded by 2^-134 at most, under 2^-9 max|V| here.
"""
import ctypes

import numpy as np
import pytest
import torch

import pagedattention_kv_cache_pa_b200 as pa
from pagedattention_kv_cache_pa_b200 import binding


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tests import gpu_harness
    return gpu_harness


@pytest.mark.gpu
@pytest.mark.parametrize("gs", [(1.0, 2.0 ** -126), (1.0, 2.0 ** 110), (2.0 ** -126, 1.0), (2.0 ** 100, 1.0)])
@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 64), (8, 1, 128)])
def test_decode(h, hq, hkv, d, gs):
    from tests.test_gpu_e2m1 import Case
    c = Case(5, [4000, 17, 900], hq, hkv, d, 16, gs=gs)
    c.scale = 2.0 ** -12 / gs[0]                           # (K saturates at 2688 of its small scale)
    for ctas in (1, 0):                                   # whole sequences; pieces
        c.check(h, max_ctas=ctas)


@pytest.mark.gpu
@pytest.mark.parametrize("gs", [(1.0, 2.0 ** -126), (1.0, 2.0 ** 110), (2.0 ** -126, 1.0), (2.0 ** 100, 1.0)])
@pytest.mark.parametrize("kernel", [pa.PA_PREFILL_ROWS, pa.PA_PREFILL_TCGEN05_WS])
@pytest.mark.parametrize("lens,rows,d", [([4000, 60, 900], [3, 60, 130], 64), ([4000, 60, 900], [3, 60, 130], 128),
                                         ([9000], [300], 64)])
def test_prefill(h, kernel, lens, rows, d, gs):
    from tests.test_gpu_e2m1_prefill import _case, _check
    c = _case(6, lens, rows, 8, 2, d, 16, gs=gs)
    c.scale, c.kernel = 2.0 ** -12 / gs[0], kernel
    _check(c, h)


def test_scores_past_fp32_are_refused():
    # scale k_scale log2(e) is what multiplies a score: where it is no finite float no score is
    fake = ctypes.c_void_p(0x10000)
    d = pa.CacheDesc.make(num_blocks=8, block_size=16, num_kv_heads=2, num_q_heads=4, head_dim=64, max_blocks_per_seq=4)
    for scale, ks, want in ((2.0 ** 20, 2.0 ** 110, -1), (3.0, 1e38, -1), (float("nan"), 1.0, -1),
                            (float("inf"), 1.0, -1), (-float("inf"), 1.0, -1), (-3.0, 1e38, -1)):
        o = pa.DecodeOptions(kv_dtype=pa.PA_KV_E2M1, k_scale=ks, v_scale=1.0)
        args = (fake, fake, fake, fake, fake, 1, 16, ctypes.c_float(scale), fake)
        rest = (fake, 1 << 30, ctypes.byref(d), ctypes.byref(o), None)
        assert binding.lib.pa_decode_ex(*args, *rest) == want
        assert binding.lib.pa_append_decode(fake, fake, *args, *rest) == want
        assert binding.lib.pa_decode_noalloc(*args, ctypes.byref(d), ctypes.byref(o), None) == want
        if scale > 0:
            p = pa.PrefillOptions(kv_dtype=pa.PA_KV_E2M1, k_scale=ks, v_scale=1.0)
            assert binding.lib.pa_prefill_ex(fake, fake, fake, fake, fake, fake, 1, 1, 16, ctypes.c_float(scale), fake,
                                             fake, 1 << 30, ctypes.byref(d), ctypes.byref(p), None) == want
