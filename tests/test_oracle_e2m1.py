"""The 4-bit format's oracle against closed forms, and the refusals of its entry points (CPU)."""
import ctypes

import numpy as np
import pytest

import pagedattention_kv_cache_pa_b200 as pa
from oracle import e2m1
from pagedattention_kv_cache_pa_b200 import binding


def bits(x):
    return (np.asarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def test_codes_of_a_group_with_scale_one():
    # amax 6 gives scale 1: every midpoint goes to the even code, signs kept
    x = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.26]
    codes, s = e2m1.quantize(bits(x), 1.0)
    got = e2m1.values(codes, s)
    np.testing.assert_array_equal(got, [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, 0.5])


def test_scale_ties_and_saturation():
    row = np.zeros(16, dtype=np.float32)
    for amax, want in ((51.0, 8.0), (57.0, 10.0), (6 * 448.0, 448.0), (1e6, 448.0), (6 * 2.0 ** -9, 2.0 ** -9),
                       (6 * 2.0 ** -11, 0.0)):
        row[3] = -amax                                  # 51 / 6 = 8.5 and 57 / 6 = 9.5: half way, to the even code
        codes, s = e2m1.quantize(bits(row), 1.0)
        assert e2m1._E4M3[s[0]] == want, amax
        got = e2m1.values(codes, s)
        assert got[3] <= 0 and np.all(got[np.arange(16) != 3] == 0)
    row[3] = np.inf
    assert e2m1.values(*e2m1.quantize(bits(row), 1.0))[3] == 6 * 448
    row[3] = np.nan
    assert np.isnan(e2m1.values(*e2m1.quantize(bits(row), 1.0))).all()


def test_pack_round_trip_and_exact_bf16_values():
    rng = np.random.default_rng(1)
    x = bits(rng.standard_normal((3, 2, 16, 64)) * 4)
    codes, s = e2m1.quantize(x, 0.5)
    pages = e2m1.pack(codes, s)
    assert pages.shape == (3, 2, 16 * 36)
    c2, s2 = e2m1.unpack(pages, 16, 64)
    np.testing.assert_array_equal(codes, c2)
    np.testing.assert_array_equal(s, s2)
    v = e2m1.to_float(e2m1.pool_bits(pages, 16, 64)).astype(np.float64) * 0.5
    # each value is within half the widest gap (2 scales) plus the scale's rounding (2^-4) of its own
    amax = np.abs(e2m1.to_float(x)).reshape(3, 2, 16, 4, 16).max(-1).repeat(16, -1)
    assert np.all(np.abs(v - e2m1.to_float(x)) <= amax * (1 / 6 + 2.0 ** -4) * 1.01)


def _desc(**kw):
    base = dict(num_blocks=8, block_size=16, num_kv_heads=3, num_q_heads=6, head_dim=64, max_blocks_per_seq=4)
    return pa.CacheDesc.make(**{**base, **kw})


def test_cache_bytes():
    assert pa.pa_kv_cache_bytes(_desc(), pa.PA_KV_BF16) == 8 * 3 * 16 * 128
    assert pa.pa_kv_cache_bytes(_desc(), pa.PA_KV_E4M3) == 8 * 3 * 16 * 64
    assert pa.pa_kv_cache_bytes(_desc(), pa.PA_KV_E2M1) == 8 * 3 * 16 * 36
    for bad in (_desc(block_size=24), _desc(head_dim=96), _desc(num_blocks=0)):
        with pytest.raises(pa.PaError):
            pa.pa_kv_cache_bytes(bad, pa.PA_KV_E2M1)
    with pytest.raises(pa.PaError):
        pa.pa_kv_cache_bytes(_desc(), 7)


FAKE = ctypes.c_void_p(0x10000)          # never dereferenced: validation fails first
F = ctypes.c_float


def _append(desc, n=1, ks=1.0, vs=1.0, k=FAKE, kc=FAKE):
    return binding.lib.pa_append_kv_e2m1(k, FAKE, FAKE, n, F(ks), F(vs), kc, FAKE, ctypes.byref(desc), None)


def _rope(desc, n=1, theta=1e4, ks=1.0, q=FAKE):
    return binding.lib.pa_rope_append_kv_e2m1(q, FAKE, FAKE, FAKE, FAKE, FAKE, n, F(theta), F(ks), F(1.0), FAKE,
                                              FAKE, ctypes.byref(desc), None)


def _gather(desc, n=1, ks=1.0, k=FAKE):
    return binding.lib.pa_gather_kv_e2m1(FAKE, FAKE, FAKE, n, F(ks), F(1.0), k, FAKE, ctypes.byref(desc), None)


def test_append_and_gather_refusals():
    d = _desc()
    for call in (_append, _rope, _gather):
        assert call(d, n=0) == 0 and call(d, n=-1) == -1
        for ks in (0.0, -1.0, float("nan"), float("inf"), 1e-39):     # 1e-39: its reciprocal overflows
            assert call(d, ks=ks) == -1, ks
        assert call(_desc(head_dim=96)) == -2 and call(_desc(block_size=24)) == -2
        assert call(_desc(num_q_heads=7)) == -1
        # a row index of the pool that passes 32 bits
        assert call(_desc(num_blocks=2 ** 30, num_kv_heads=8, num_q_heads=8)) == -2
    mis = ctypes.c_void_p(0x10008)
    assert _append(d, k=mis) == -1 and _append(d, kc=mis) == -1 and _append(d, k=None) == -1
    assert _gather(d, k=mis) == -1 and _rope(d, q=mis) == -1 and _rope(d, q=None) == -1
    for theta in (0.0, -1.0, float("nan"), float("inf")):
        assert _rope(d, theta=theta) == -1
    lib = binding.lib
    assert lib.pa_copy_blocks_e2m1(FAKE, FAKE, FAKE, -1, ctypes.byref(d), None) == -1
    assert lib.pa_copy_blocks_e2m1(FAKE, FAKE, None, 1, ctypes.byref(d), None) == -1
    assert lib.pa_copy_blocks_e2m1(FAKE, FAKE, FAKE, 0, ctypes.byref(d), None) == 0
    bad = _desc(block_size=24)
    assert lib.pa_copy_blocks_e2m1(FAKE, FAKE, FAKE, 1, ctypes.byref(bad), None) == -2


def test_decode_refusals():
    lib = binding.lib

    def call(d, **kw):
        o = pa.DecodeOptions(**{**dict(kv_dtype=pa.PA_KV_E2M1, k_scale=1.0, v_scale=1.0), **kw})
        return lib.pa_decode_ex(FAKE, FAKE, FAKE, FAKE, FAKE, 1, 16, F(0.1), FAKE, FAKE, 1 << 20, ctypes.byref(d),
                                ctypes.byref(o), None)

    assert call(_desc(), k_scale=0.0) == -1 and call(_desc(), v_scale=float("nan")) == -1
    assert call(_desc(), kernel=pa.PA_KERNEL_SIMT) == -2 and call(_desc(), kernel=pa.PA_KERNEL_TENSOR_SPLIT) == -2
    assert call(_desc(num_q_heads=51)) == -2              # 17 query heads a kv head
    assert call(_desc(head_dim=96)) == -2 and call(_desc(block_size=24)) == -2
    assert call(_desc(), kv_dtype=3) == -1
    assert call(_desc(), rope_theta=1e4) == -1            # rotation needs the new rows
