"""The 4-bit KV cache through the C ABI against its oracle (needs a B200).

Appends must leave exactly the oracle's bytes (the codes are decided by correctly rounded float
operations) and touch no other.  Decodes are compared with fp64 attention over the same codes:
|got - ref| <= 2^-8 |ref| + 2^-9 max|V|.  The first term is the output's rounding to bf16; the
second covers P's rounding to f16 (2^-11 of sum p |V|), what f16 P loses below its normal range
(2^-25 a token, at most 2^-10 of the sum's weight at these lengths) and fp32 scores (a few 2^-24 of
sum |q k|, below 2^-13 here).
"""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
import pagedattention_kv_cache_pa_b200 as pa
from oracle import e2m1

pytestmark = pytest.mark.gpu

# (Hq, Hkv, D, Bs): groups of 8, 1, 3, 2, 4 kv heads a team; G from 1 to 16; every block size
SHAPES = [(32, 8, 64, 16), (8, 8, 64, 8), (16, 1, 128, 16), (64, 8, 128, 32), (6, 3, 64, 256), (2, 2, 128, 64),
          (20, 4, 128, 128), (40, 40, 64, 8), (36, 3, 64, 32), (10, 2, 128, 8)]


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tests import gpu_harness
    return gpu_harness


def dev(a, h):
    return torch.from_numpy(np.ascontiguousarray(a)).to(h.DEV)


def same_bytes(got, want, bs, d):
    """Equal pages, a code of -0 counting as 0."""
    gc, gs = e2m1.unpack(got, bs, d)
    wc, ws = e2m1.unpack(want, bs, d)
    np.testing.assert_array_equal(gs, ws)
    np.testing.assert_array_equal(np.where(gc == 8, 0, gc), np.where(wc == 8, 0, wc))


def normal(rng, *shape, scale=1.0):
    x = (rng.standard_normal(shape) * scale).astype(np.float32)
    return (x.view(np.uint32) >> 16).astype(np.uint16)


def pool(rng, n, hkv, bs, d, gs):
    return e2m1.pack(*e2m1.quantize(normal(rng, n, hkv, bs, d, scale=2.0), gs))


def tolerance(ref, vmax):
    return 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * vmax


# ---- append and read back -------------------------------------------------------------------
@pytest.mark.parametrize("gs", [(1.0, 1.0), (0.37, 1.7)], ids=["unit", "scaled"])
@pytest.mark.parametrize("tokens", [1, 37, 700])
@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES[:7])
def test_append_bytes(h, hq, hkv, d, bs, tokens, gs):
    rng = np.random.default_rng(tokens + d + bs)
    n = -(-tokens // bs) + 2
    k, v = normal(rng, tokens, hkv, d, scale=3.0), normal(rng, tokens, hkv, d)
    slots = rng.permutation(n * bs)[:tokens].astype(np.int64)
    slots[::7] = -1
    if tokens > 3:
        slots[3] = n * bs                                 # past the pool
        slots[2] = 1 << 40
    k0, v0 = rng.integers(0, 256, (2, n, hkv, bs * d * 9 // 16), dtype=np.uint8)
    kc, vc = dev(k0, h), dev(v0, h)
    desc = pa.CacheDesc.make(num_blocks=n, block_size=bs, num_kv_heads=hkv, num_q_heads=hq, head_dim=d,
                             max_blocks_per_seq=n)
    pa.pa_append_kv_e2m1(h.to_dev(k), h.to_dev(v), dev(slots, h), *gs, kc, vc, desc)
    torch.cuda.synchronize()
    want_k, want_v = e2m1.append(k0, k, gs[0], slots, bs), e2m1.append(v0, v, gs[1], slots, bs)
    live = [int(s) for s in slots if 0 <= s < n * bs]
    for got, want, before in ((kc, want_k, k0), (vc, want_v, v0)):
        got = got.cpu().numpy()
        gc, gsc = e2m1.unpack(got, bs, d)
        bc, bsc = e2m1.unpack(before, bs, d)
        touched = np.zeros((n, bs), dtype=bool)
        touched.reshape(-1)[live] = True
        np.testing.assert_array_equal(gc.transpose(0, 2, 1, 3)[~touched], bc.transpose(0, 2, 1, 3)[~touched])
        np.testing.assert_array_equal(gsc.transpose(0, 2, 1, 3)[~touched], bsc.transpose(0, 2, 1, 3)[~touched])
        same_bytes(got, want, bs, d)
    # read back: code * s * gs in float, rounded to bf16; zeros where there is no slot
    kb, vb = (torch.full((tokens, hkv, d), 9.0, dtype=torch.bfloat16, device=h.DEV) for _ in range(2))
    pa.pa_gather_kv_e2m1(kc, vc, dev(slots, h), *gs, kb, vb, desc)
    torch.cuda.synchronize()
    for back, rows, g in ((kb, k, gs[0]), (vb, v, gs[1])):
        x = e2m1.values(*e2m1.quantize(rows, g)).astype(np.float32) * np.float32(g)
        u = x.view(np.uint32).astype(np.uint64)
        want = e2m1.to_float(((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16))
        bad = (slots < 0) | (slots >= n * bs)
        np.testing.assert_array_equal(back.float().cpu().numpy(), np.where(bad[:, None, None], 0.0, want))


def test_append_extremes(h):
    row = np.zeros((12, 64), dtype=np.float32)
    row[0] = np.linspace(-6, 6, 64)
    row[1, :16] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6]
    row[2, 5] = 51.0                                      # a scale half way between two codes
    row[3, 5], row[3, 6] = np.inf, 1.0
    row[4, 5], row[4, 20] = np.nan, 1.0
    row[5, ::3] = 1e30
    row[6] = 2.0 ** -12                                   # scale 0
    row[7] = 2.0 ** -8.5
    row[8, 17] = -np.inf
    row[9] = -0.0
    row[10] = np.float32(3.3e38)
    row[11] = np.float32(1e-40)
    bits = (row.view(np.uint32) >> 16).astype(np.uint16)[:, None]
    desc = pa.CacheDesc.make(num_blocks=2, block_size=8, num_kv_heads=1, num_q_heads=1, head_dim=64,
                             max_blocks_per_seq=2)
    zero = np.zeros((2, 1, 8 * 36), dtype=np.uint8)
    for gs in ((1.0, 0.25), (1e-30, 1e30)):
        kc, vc = dev(zero, h), dev(zero, h)
        slots = np.arange(12, dtype=np.int64)
        pa.pa_append_kv_e2m1(h.to_dev(bits), h.to_dev(bits), dev(slots, h), *gs, kc, vc, desc)
        torch.cuda.synchronize()
        for got, g in ((kc, gs[0]), (vc, gs[1])):
            gv = e2m1.values(*e2m1.unpack(got.cpu().numpy(), 8, 64))
            wv = e2m1.values(*e2m1.unpack(e2m1.append(zero, bits, g, slots, 8), 8, 64))
            np.testing.assert_array_equal(gv, wv)


@pytest.mark.parametrize("far", [64, 131072])
@pytest.mark.parametrize("tokens", [1, 300])
@pytest.mark.parametrize("hq,hkv,d,bs", [(32, 8, 64, 16), (7, 1, 128, 8), (6, 3, 64, 256), (16, 16, 128, 32)])
def test_rope_append_bytes(h, hq, hkv, d, bs, tokens, far):
    rng = np.random.default_rng(tokens + far + d)
    n = -(-tokens // bs) + 1
    q, k, v = normal(rng, tokens, hq, d), normal(rng, tokens, hkv, d, scale=3.0), normal(rng, tokens, hkv, d)
    pos = rng.integers(0, far, tokens).astype(np.int32)
    pos[-1] = far - 1
    slots = rng.permutation(n * bs)[:tokens].astype(np.int64)
    slots[1::5] = -1
    zero = np.zeros((n, hkv, bs * d * 9 // 16), dtype=np.uint8)
    kc, vc, qd = dev(zero, h), dev(zero, h), h.to_dev(q)
    out = torch.empty_like(qd)
    desc = pa.CacheDesc.make(num_blocks=n, block_size=bs, num_kv_heads=hkv, num_q_heads=hq, head_dim=d,
                             max_blocks_per_seq=n)
    args = (h.to_dev(k), h.to_dev(v), dev(pos, h), dev(slots, h), 500000.0, 0.5, 2.0)
    pa.pa_rope_append_kv_e2m1(qd, out, *args, kc, vc, desc)
    torch.cuda.synchronize()
    same_bytes(kc.cpu().numpy(), e2m1.append(zero, e2m1.rope_rows(k, pos, 500000.0), 0.5, slots, bs), bs, d)
    same_bytes(vc.cpu().numpy(), e2m1.append(zero, v, 2.0, slots, bs), bs, d)
    ok, worst = h.rope_close(h.to_host_bits(out), q, pos, 500000.0)
    assert ok, worst
    kc2, vc2 = dev(zero, h), dev(zero, h)                 # in place, and the same bytes again
    pa.pa_rope_append_kv_e2m1(qd, qd, *args, kc2, vc2, desc)
    torch.cuda.synchronize()
    assert torch.equal(qd, out) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_copy_blocks(h):
    rng = np.random.default_rng(5)
    n, hkv, bs, d = 9, 3, 8, 64
    k0, v0 = rng.integers(0, 256, (2, n, hkv, bs * d * 9 // 16), dtype=np.uint8)
    kc, vc = dev(k0, h), dev(v0, h)
    desc = pa.CacheDesc.make(num_blocks=n, block_size=bs, num_kv_heads=hkv, num_q_heads=hkv, head_dim=d,
                             max_blocks_per_seq=4)
    pairs = np.array([[0, 5], [1, 8], [-1, 3], [2, 9], [7, 4]], dtype=np.int32)
    pa.pa_copy_blocks_e2m1(kc, vc, dev(pairs, h), desc)
    torch.cuda.synchronize()
    for got, want in ((kc, k0.copy()), (vc, v0.copy())):
        want[5], want[8], want[4] = want[0], want[1], want[7]
        np.testing.assert_array_equal(got.cpu().numpy(), want)


# ---- decode -----------------------------------------------------------------------------------
class Case:
    """Sequences of the given lengths over a 4-bit pool in random order, NaN scales and random
    codes in every row that no sequence holds."""

    def __init__(self, seed, lens, hq, hkv, d, bs, gs=(1.0, 0.5), spare=2, q_scale=1.0):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, dtype=np.int32)
        self.hq, self.hkv, self.d, self.bs, self.gs = hq, hkv, d, bs, gs
        need = [-(-int(x) // bs) for x in lens]
        self.n = sum(need) + spare
        self.mb = max(1, max(need)) + 1
        order = rng.permutation(self.n).astype(np.int32)
        self.tables = np.full((len(lens), self.mb), -1, dtype=np.int32)
        held = np.zeros((self.n, bs), dtype=bool)
        at = 0
        for i, m in enumerate(need):
            self.tables[i, :m] = order[at:at + m]
            for j in range(m):
                held[order[at + j], :min(bs, int(lens[i]) - j * bs)] = True
            at += m
        self.pools = []
        for g in gs:
            codes, scales = e2m1.quantize(normal(rng, self.n, hkv, bs, d, scale=2.0), g)
            codes = np.where(held[:, None, :, None], codes, rng.integers(0, 16, codes.shape).astype(np.uint8))
            scales = np.where(held[:, None, :, None], scales, 0x7F).astype(np.uint8)
            self.pools.append(e2m1.pack(codes, scales))
        self.q = normal(rng, len(lens), hq, d, scale=q_scale)
        self.scale = d ** -0.5
        self.desc = pa.CacheDesc.make(num_blocks=self.n, block_size=bs, num_kv_heads=hkv, num_q_heads=hq, head_dim=d,
                                      max_blocks_per_seq=self.mb)

    def values(self):
        """bf16 pools of code * scale, rows that no sequence holds as zeros."""
        out = []
        for pages in self.pools:
            codes, scales = e2m1.unpack(pages, self.bs, self.d)
            dead = (scales == 0x7F).all(-1, keepdims=True)
            out.append(e2m1.bf16_bits(e2m1.values(codes, np.where(dead, 0, scales).astype(np.uint8))))
        return out

    def reference(self):
        k, v = self.values()
        ref = oracle.paged_decode(self.q, k, v, self.tables, self.lens, self.scale * self.gs[0]) * self.gs[1]
        return ref, np.abs(e2m1.to_float(v)).max() * self.gs[1]

    def options(self, **kw):
        return pa.DecodeOptions(kv_dtype=pa.PA_KV_E2M1, k_scale=self.gs[0], v_scale=self.gs[1], **kw)

    def run(self, h, stream=None, **kw):
        opts = self.options(**{"flags": pa.PA_FLAG_CHECK, **kw})
        longest = int(self.lens.max()) if self.lens.size else 0
        q = h.to_dev(self.q)
        out = torch.full_like(q, 7.0)
        ws = torch.zeros(pa.pa_decode_workspace_size(len(self.lens), longest, self.desc, opts), dtype=torch.uint8,
                         device=h.DEV)
        pa.pa_decode(q, *(dev(x, h) for x in self.pools), dev(self.tables, h), dev(self.lens, h), longest, self.scale,
                     out, ws, self.desc, opts, stream=stream)
        torch.cuda.synchronize()
        return out.float().cpu().numpy().astype(np.float64)

    def check(self, h, **kw):
        got = self.run(h, **kw)
        ref, vmax = self.reference()
        err = np.abs(got - ref) - tolerance(ref, vmax)
        assert np.isfinite(got).all() and err.max() <= 0, "outside the tolerance by %g" % err.max()
        return got


@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES)
def test_decode_shapes(h, hq, hkv, d, bs):
    Case(hq + d + bs, [1, bs - 1, bs, bs + 1, 0, 15, 33, 517, 130], hq, hkv, d, bs).check(h)


@pytest.mark.parametrize("max_ctas", [1, 2, 7, 0])
@pytest.mark.parametrize("hq,hkv,d,bs", [(32, 8, 64, 16), (8, 1, 128, 8), (32, 2, 64, 32)])
def test_decode_partitions(h, hq, hkv, d, bs, max_ctas):
    # few slices: many sequences a slice; more: sequences cut between them, at any slab
    Case(7, [300, 0, 1, 64, 999, 31, 32, 0], hq, hkv, d, bs, gs=(0.37, 1.7)).check(h, max_ctas=max_ctas)


def test_decode_all_empty_and_one_token(h):
    c = Case(3, [0, 0, 0], 8, 8, 64, 16)
    assert np.array_equal(c.run(h), np.zeros((3, 8, 64)))
    c = Case(4, [1], 8, 8, 64, 16)
    got = c.check(h)                                      # one token: its V row
    v = e2m1.to_float(c.values()[1])[c.tables[0, 0], :, 0] * 0.5
    np.testing.assert_array_equal(got[0], v)


def test_decode_long_batch_and_many_sequences(h):
    Case(11, [40000, 3, 20011], 16, 2, 128, 16).check(h)
    rng = np.random.default_rng(1)
    Case(12, rng.integers(0, 200, 300), 8, 8, 64, 16).check(h)     # 300 sequences: 10 lengths a lane


@pytest.mark.parametrize("q_scale", [2.0 ** -100, 2.0 ** -20, 40.0, 2.0 ** 20])
def test_decode_q_of_any_size(h, q_scale):
    # q beyond f16's range: brought there by its power of two; the scale undoes it for large ones
    c = Case(21, [200, 77], 16, 4, 64, 16, q_scale=q_scale)
    if q_scale == 2.0 ** 20:
        c.scale = 2.0 ** -20
    c.check(h)


@pytest.mark.parametrize("scale", [-0.25, 0.0, -1e-3])
def test_decode_scale_of_any_sign(h, scale):
    c = Case(23, [200, 77, 1], 16, 4, 64, 16, q_scale=2.0)
    c.scale = scale
    c.check(h)


def test_decode_rising_and_far_scores(h):
    # K rows that grow along the sequence raise the running max at every slab; others fall far below it
    c = Case(31, [640], 8, 8, 64, 16, q_scale=4.0)
    codes, scales = e2m1.unpack(c.pools[0], 16, 64)
    scales = scales.copy()
    for j, blk in enumerate(c.tables[0, :40]):
        scales[blk] = min(0x50, 0x20 + 2 * j)
    c.pools[0] = e2m1.pack(codes, scales)
    c.check(h)


def test_decode_nan_values_reach_the_output(h):
    c = Case(41, [50, 60], 8, 8, 64, 16)
    codes, scales = e2m1.unpack(c.pools[1], 16, 64)
    scales = scales.copy()
    scales[c.tables[0, 1], 2, 3, 1] = 0x7F                # a NaN in V of sequence 0, kv head 2, dims 16 .. 31
    c.pools[1] = e2m1.pack(codes, scales)
    got = c.run(h)
    bad = np.isnan(got)
    assert bad[0, 2, 16:32].all() and bad.sum() == 16


def test_decode_bad_blocks_and_lengths(h):
    c = Case(51, [100, 100], 8, 8, 64, 16)
    for bad in (-5, c.n, 2 ** 30):
        keep = c.tables[1, 2]
        c.tables[1, 2] = bad
        with pytest.raises(pa.PaError) as e:
            c.run(h)
        assert e.value.status == -7
        c.tables[1, 2] = keep
    c.lens[0] = (c.mb + 1) * 16                           # past the table: clipped and reported; the entries
    with pytest.raises(pa.PaError) as e:                  # behind the sequence's blocks are no blocks, which
        c.run(h)                                          # is the status that comes first
    assert e.value.status == -7
    c.lens[0] = -3
    with pytest.raises(pa.PaError) as e:
        c.run(h)
    assert e.value.status == -8
    c.lens[0] = 100
    c.check(h)


def test_decode_other_stream_graph_and_noalloc(h):
    c = Case(61, [300, 0, 5, 1000], 32, 8, 64, 16)
    ref, vmax = c.reference()
    opts = c.options()
    q, out = h.to_dev(c.q), torch.zeros((4, 32, 64), dtype=torch.bfloat16, device=h.DEV)
    pools, tables, lens = [dev(x, h) for x in c.pools], dev(c.tables, h), dev(c.lens, h)
    ws = torch.zeros(pa.pa_decode_workspace_size(4, 1000, c.desc, opts), dtype=torch.uint8, device=h.DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        pa.pa_decode(q, *pools, tables, lens, 1000, c.scale, out, ws, c.desc, opts)
    side.synchronize()
    first = out.clone()
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tolerance(ref, vmax))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_decode(q, *pools, tables, lens, 1000, c.scale, out, ws, c.desc, opts)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)                    # no atomics: the same bits every time
    # a replay with other lengths in place: the plan is made on the device
    lens.copy_(dev(np.array([299, 16, 0, 640], dtype=np.int32), h))
    tables[1, 0] = tables[0, 0]
    g.replay()
    torch.cuda.synchronize()
    c.lens, c.tables = np.array([299, 16, 0, 640], dtype=np.int32), tables.cpu().numpy()
    ref, vmax = c.reference()
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tolerance(ref, vmax))
    same = out.clone()
    pa.pa_decode_noalloc(q, *pools, tables, lens, 1000, c.scale, out, c.desc, c.options(flags=pa.PA_FLAG_CHECK))
    torch.cuda.synchronize()
    assert torch.equal(out, same)


def test_decode_two_calls_at_once_and_early_start(h):
    cs = [Case(71 + i, [900, 33, 2000], 32, 8, 64, 16) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    held, outs = [], []
    for c in cs:
        opts = c.options(flags=pa.PA_FLAG_PDL)
        held.append((h.to_dev(c.q), [dev(x, h) for x in c.pools], dev(c.tables, h), dev(c.lens, h), opts,
                     torch.zeros(pa.pa_decode_workspace_size(3, 2000, c.desc, opts), dtype=torch.uint8, device=h.DEV)))
        outs.append(torch.zeros((3, 32, 64), dtype=torch.bfloat16, device=h.DEV))
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, x, out in zip(cs, streams, held, outs):
            with torch.cuda.stream(s):
                pa.pa_decode(x[0], *x[1], x[2], x[3], 2000, c.scale, out, x[5], c.desc, x[4])
    torch.cuda.synchronize()
    for c, x, out in zip(cs, held, outs):
        assert pa.pa_decode_status(x[5]) == 0
        ref, vmax = c.reference()
        assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tolerance(ref, vmax))


def test_describe(h):
    desc = pa.CacheDesc.make(num_blocks=8, block_size=16, num_kv_heads=12, num_q_heads=12, head_dim=64,
                             max_blocks_per_seq=4)
    opts = pa.DecodeOptions(kv_dtype=pa.PA_KV_E2M1, k_scale=1.0, v_scale=1.0, max_ctas=3)
    info = pa.pa_decode_describe(2, 64, desc, opts)
    assert info.kernel == pa.PA_KERNEL_TENSOR and info.ctas == 3 * 2 and info.split_tokens % 16 == 0


# ---- append and decode together -----------------------------------------------------------------
@pytest.mark.parametrize("theta", [0.0, 10000.0], ids=["plain", "rope"])
@pytest.mark.parametrize("hq,hkv,d,bs", [(32, 8, 64, 16), (4, 1, 128, 8), (6, 3, 64, 256)])
def test_append_decode(h, hq, hkv, d, bs, theta):
    c = Case(81, [17, 1, bs, 0, bs + 1, 400], hq, hkv, d, bs)
    rng = np.random.default_rng(5)
    k, v = normal(rng, 6, hkv, d, scale=2.0), normal(rng, 6, hkv, d)
    pos = np.maximum(c.lens - 1, 0)
    slots = np.array([c.tables[i, p // bs] * bs + p % bs if c.lens[i] else -1 for i, p in enumerate(pos)])
    kr = e2m1.rope_rows(k, pos, theta) if theta else k
    want = [e2m1.append(c.pools[0], kr, c.gs[0], slots, bs), e2m1.append(c.pools[1], v, c.gs[1], slots, bs)]
    opts = c.options(flags=pa.PA_FLAG_CHECK, rope_theta=theta)
    pools, q = [dev(x, h) for x in c.pools], h.to_dev(c.q)
    out = torch.empty_like(q)
    ws = torch.zeros(pa.pa_decode_workspace_size(6, 400, c.desc, opts), dtype=torch.uint8, device=h.DEV)
    pa.pa_append_decode(q, h.to_dev(k), h.to_dev(v), *pools, dev(c.tables, h), dev(c.lens, h), 400, c.scale, out, ws,
                        c.desc, opts)
    torch.cuda.synchronize()
    for got, w in zip(pools, want):
        same_bytes(got.cpu().numpy(), w, bs, d)
    q_before, c.pools = c.q, want
    if theta:
        c.q = oracle.rope_bf16(c.q, pos.astype(np.int32), theta)
    ref, vmax = c.reference()
    # a rotated q value may round to the neighbouring bf16: scores move by 2^-8 of |q k| at one dim
    extra = 2.0 ** -8 * vmax if theta else 0.0
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= tolerance(ref, vmax) + extra)
    assert np.array_equal(h.to_host_bits(q), q_before)


@pytest.mark.parametrize("theta", [0.0, 10000.0], ids=["plain", "rope"])
def test_append_decode_layers_started_early_in_a_graph(h, theta):
    # layers of a step back to back over one workspace, each decode started early: the bits of plain calls
    layers = [Case(91 + i, [700, 1, 33, 0, 1500], 32, 8, 64, 16) for i in range(3)]
    rng = np.random.default_rng(6)
    new = [(h.to_dev(normal(rng, 5, 8, 64)), h.to_dev(normal(rng, 5, 8, 64))) for _ in layers]
    got = []
    for flags in (0, pa.PA_FLAG_PDL):
        opts = layers[0].options(flags=flags, rope_theta=theta)
        ws = torch.zeros(pa.pa_decode_workspace_size(5, 1500, layers[0].desc, opts), dtype=torch.uint8, device=h.DEV)
        held = [(h.to_dev(c.q), *kv, *(dev(x, h) for x in c.pools), dev(c.tables, h), dev(c.lens, h))
                for c, kv in zip(layers, new)]
        outs = [torch.zeros((5, 32, 64), dtype=torch.bfloat16, device=h.DEV) for _ in layers]
        torch.cuda.synchronize()

        def step():
            for c, x, out in zip(layers, held, outs):
                pa.pa_append_decode(*x, 1500, c.scale, out, ws, c.desc, opts)
        if flags:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            for _ in range(3):
                g.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert pa.pa_decode_status(ws) == 0
        got.append(outs + [x for y in held for x in y[3:5]])
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_serving_steps(h):
    """Prompts appended, then steps of one token a sequence with the block manager: the same tokens
    read back and attended to as the whole history quantized at once."""
    rng = np.random.default_rng(9)
    hq, hkv, d, bs, B = 8, 2, 64, 8, 3
    prompts, steps = [13, 1, 24], 12
    n, mb = 40, 12
    bm = pa.BlockManager(n, bs, B, mb, rng.permutation(n).astype(np.int32))
    desc = pa.CacheDesc.make(num_blocks=n, block_size=bs, num_kv_heads=hkv, num_q_heads=hq, head_dim=d,
                             max_blocks_per_seq=mb)
    size = pa.pa_kv_cache_bytes(desc, pa.PA_KV_E2M1)
    kc, vc = (torch.full((size,), 0xFF, dtype=torch.uint8, device=h.DEV) for _ in range(2))
    opts = pa.DecodeOptions(kv_dtype=pa.PA_KV_E2M1, k_scale=1.0, v_scale=1.0, rope_theta=1e4)
    hist = [[], [], []]
    for s, p in enumerate(prompts):
        bm.add_seq(s, p)
        q, k, v = normal(rng, p, hq, d), normal(rng, p, hkv, d), normal(rng, p, hkv, d)
        pos = np.arange(p, dtype=np.int32)
        slots = bm.block_tables()[s, pos // bs].astype(np.int64) * bs + pos % bs
        qd = h.to_dev(q)
        pa.pa_rope_append_kv_e2m1(qd, qd, h.to_dev(k), h.to_dev(v), dev(pos, h), dev(slots, h), 1e4, 1.0, 1.0, kc, vc,
                                  desc)
        hist[s] += list(zip(e2m1.rope_rows(k, pos, 1e4), v))
    ws = torch.zeros(pa.pa_decode_workspace_size(B, mb * bs, desc, opts), dtype=torch.uint8, device=h.DEV)
    for _ in range(steps):
        bm.append_tokens(np.arange(B))
        lens, tables = bm.context_lens().copy(), bm.block_tables().copy()
        q, k, v = normal(rng, B, hq, d), normal(rng, B, hkv, d), normal(rng, B, hkv, d)
        out = torch.empty((B, hq, d), dtype=torch.bfloat16, device=h.DEV)
        pa.pa_append_decode(h.to_dev(q), h.to_dev(k), h.to_dev(v), kc, vc, dev(tables, h), dev(lens, h), mb * bs,
                            d ** -0.5, out, ws, desc, opts)
        turned = e2m1.rope_rows(k, lens - 1, 1e4)
        for s in range(B):
            hist[s].append((turned[s], v[s]))
        assert pa.pa_decode_status(ws) == 0
        qr = oracle.rope_bf16(q, (lens - 1).astype(np.int32), 1e4)
        for s in range(B):
            L = int(lens[s])
            kk, vv = (np.stack([x[i] for x in hist[s]])[None].transpose(0, 2, 1, 3) for i in range(2))
            kv = [e2m1.bf16_bits(e2m1.values(*e2m1.quantize(x, 1.0))) for x in (kk, vv)]
            ref = oracle.paged_decode(qr[s:s + 1], *kv, np.zeros((1, 1), np.int32), np.array([L], np.int32), d ** -0.5)
            vmax = np.abs(e2m1.to_float(kv[1])).max()
            err = np.abs(out[s].double().cpu().numpy() - ref[0])
            assert np.all(err <= tolerance(ref[0], vmax) + 2.0 ** -8 * vmax)
    bm.close()
