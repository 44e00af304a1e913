"""Long contexts of many small weights behind one large one, over 4-bit pools, against fp64 (needs a B200).

One key takes nearly all of the softmax and its V is zero (a sink), so the output is what the other
weights bring.  |got - ref| <= 2^-8 |ref| + n 2^-x max|V|: the output's rounding to bf16 (2^-9); P's
rounding to f16, which is 2^-12 of a weight where that is normal and 2^-x of the largest for any smaller
one, x = 36 in the decode kernel (weights times 2^11) and 32 in the prefill tiles (times 2^7), half a step of
2^-24 either way; the products' sums in fp32 (n / 16 steps of at most 2^-23: 2^-10); scores of up to 30 in
fp32 (2^-18).
"""
import functools

import numpy as np
import pytest
import torch

import oracle
import pagedattention_kv_cache_pa_b200 as pa
from oracle import e2m1

pytestmark = pytest.mark.gpu
N, BS = 131072, 64


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tests import gpu_harness
    return gpu_harness


@functools.lru_cache(maxsize=1)
def pools(heads, d, at):
    """The 4-bit pools, and their values as bf16 pools."""
    rng = np.random.default_rng(heads + d)
    codes = np.zeros((N // BS, heads, BS, d), dtype=np.uint8)
    scales = np.full((N // BS, heads, BS, d // 16), 0x38, dtype=np.uint8)          # 1.0
    vcodes = rng.integers(1, 8, codes.shape).astype(np.uint8)
    codes[at // BS, :, at % BS], vcodes[at // BS, :, at % BS] = 2, 0               # 1.0; zero
    bits = e2m1.bf16_bits(e2m1.MAGNITUDES)
    return [e2m1.pack(x, scales) for x in (codes, vcodes)], [bits[x] for x in (codes, vcodes)]


class Sink:
    """One sequence's blocks in order; q all ones, K zero but the sink's, a score of gap ln 2."""

    def __init__(self, heads, d, gap, at, seqs, small=2.0 ** -36):
        self.pools, values = pools(heads, d, at)
        self.scale = float(np.float32(gap * np.log(2.0) / d))
        self.q = np.full((seqs, heads, d), 0x3F80, dtype=np.uint16)
        self.table = np.arange(N // BS, dtype=np.int32)[None]
        self.ref = oracle.paged_decode(self.q[:1], *values, self.table, np.array([N], np.int32), self.scale)
        self.tol = 2.0 ** -8 * np.abs(self.ref) + N * small * 6.0
        self.seqs = seqs
        self.desc = pa.CacheDesc.make(num_blocks=N // BS, block_size=BS, num_kv_heads=heads, num_q_heads=heads,
                                      head_dim=d, max_blocks_per_seq=N // BS)

    def device(self, h):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(h.DEV)
        return (h.to_dev(self.q), dev(self.pools[0]), dev(self.pools[1]), dev(np.repeat(self.table, self.seqs, 0)),
                dev(np.full(self.seqs, N, dtype=np.int32)))

    def check(self, out):
        torch.cuda.synchronize()
        err = np.abs(out.double().cpu().numpy() - self.ref) - self.tol
        assert err.max() <= 0, "outside the tolerance by %g, the largest output %g" % (err.max(), self.ref.max())


# (the pools of one (d, at) are made once for the gaps)
@pytest.mark.parametrize("d,at,gap", [(d, at, gap) for d in (64, 128) for at in (0, N - 1) for gap in (24.5, 25.5, 30.0)])
def test_decode(h, d, at, gap):
    c = Sink(8, d, gap, at, 1)
    opts = pa.DecodeOptions(kv_dtype=pa.PA_KV_E2M1, k_scale=1.0, v_scale=1.0, max_ctas=1, flags=pa.PA_FLAG_CHECK)
    q, k, v, tables, lens = c.device(h)
    out = torch.empty_like(q)
    ws = torch.zeros(pa.pa_decode_workspace_size(1, N, c.desc, opts), dtype=torch.uint8, device=h.DEV)
    pa.pa_decode(q, k, v, tables, lens, N, c.scale, out, ws, c.desc, opts)
    c.check(out)


@pytest.mark.parametrize("kernel,d,gap", [(k, d, gap) for k in (pa.PA_PREFILL_ROWS, pa.PA_PREFILL_TCGEN05_WS)
                                          for d in (64, 128) for gap in (24.5, 25.5, 30.0)])
def test_prefill(h, kernel, d, gap):
    # one row a sequence, the sequences over the same blocks: as many items as SMs, so that none is cut
    if kernel == pa.PA_PREFILL_TCGEN05_WS:
        c = Sink(1, d, gap, 0, torch.cuda.get_device_properties(0).multi_processor_count, 2.0 ** -32)
    else:
        c = Sink(8, d, gap, 0, 40)
    opts = pa.PrefillOptions(kernel=kernel, kv_dtype=pa.PA_KV_E2M1, k_scale=1.0, v_scale=1.0)
    q, k, v, tables, lens = c.device(h)
    out, cu = torch.empty_like(q), torch.arange(c.seqs + 1, dtype=torch.int32, device=h.DEV)
    ws = torch.zeros(pa.pa_prefill_workspace_size(c.seqs, 1, N, c.desc, opts), dtype=torch.uint8, device=h.DEV)
    pa.pa_prefill_ex(q, k, v, tables, cu, lens, 1, N, c.scale, out, ws, c.desc, opts)
    c.check(out)
    assert pa.pa_decode_status(ws) == 0
