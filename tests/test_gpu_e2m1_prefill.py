"""Chunked prefill over the 4-bit KV cache against the fp64 oracle (needs a B200).

|got - ref| <= 2^-8 |ref| + 2^-9 max|V|: the output's rounding to bf16; P's rounding to f16 (2^-11 of
sum p |V|, and 2^-25 a token below f16's normal range) and fp32 scores (a few 2^-24 of sum |q k|).
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import pagedattention_kv_cache_pa_b200 as pa
from oracle import e2m1
from pagedattention_kv_cache_pa_b200 import binding


def _desc(**kw):
    base = dict(num_blocks=8, block_size=16, num_kv_heads=2, num_q_heads=4, head_dim=64, max_blocks_per_seq=4)
    return pa.CacheDesc.make(**{**base, **kw})


def test_refusals():
    fake, mis = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)

    def call(d=_desc(), q=fake, n=1, rows=4, longest=16, scale=0.1, ws=fake, size=1 << 30, **kw):
        o = pa.PrefillOptions(**{**dict(kv_dtype=pa.PA_KV_E2M1, k_scale=1.0, v_scale=1.0), **kw})
        return binding.lib.pa_prefill_ex(q, fake, fake, fake, fake, fake, n, rows, longest, ctypes.c_float(scale), fake,
                                         ws, size, ctypes.byref(d), ctypes.byref(o), None)

    for bad in (dict(k_scale=0.0), dict(v_scale=-1.0), dict(k_scale=float("nan")), dict(v_scale=1e-39),
                dict(kv_dtype=9), dict(kernel=5), dict(kernel=-1), dict(n=-1), dict(rows=-1), dict(longest=-1),
                dict(scale=0.0), dict(scale=float("inf")), dict(q=None), dict(q=mis), dict(d=_desc(num_q_heads=5))):
        assert call(**bad) == -1, bad
    for bad in (dict(kv_dtype=pa.PA_KV_E4M3), dict(kernel=pa.PA_PREFILL_MMA), dict(kernel=pa.PA_PREFILL_TCGEN05),
                dict(d=_desc(head_dim=96)), dict(d=_desc(block_size=24)), dict(d=_desc(block_size=192)),
                dict(rows=64 * 65535), dict(kernel=pa.PA_PREFILL_ROWS, n=65535, rows=2000000),
                dict(kernel=pa.PA_PREFILL_ROWS, d=_desc(num_q_heads=34))):
        assert call(**bad) == -2, bad
    assert call(ws=None) == -4 and call(size=0) == -4 and call(ws=mis) == -4
    assert call(n=0) == 0 and call(rows=0) == 0
    assert binding.lib.pa_prefill_workspace_size(1, -1, 1, ctypes.byref(_desc()), None) == 0
    assert pa.pa_prefill_workspace_size(1, 1, 1, _desc()) >= 256


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tests import gpu_harness
    return gpu_harness


def _case(seed, lens, rows, hq, hkv, d, bs, **kw):
    from tests.test_gpu_e2m1 import Case, normal
    c = Case(seed, lens, hq, hkv, d, bs, **kw)
    c.rows, c.kernel = list(rows), pa.PA_PREFILL_AUTO
    c.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    c.q = normal(np.random.default_rng(seed + 1), int(c.cu[-1]), hq, d, scale=kw.get("q_scale", 1.0))
    return c


def _reference(c):
    k, v = c.values()
    ref = oracle.paged_prefill(c.q, k, v, c.tables, c.cu, c.lens, c.scale * c.gs[0]) * c.gs[1]
    vmax = np.abs(e2m1.to_float(v)).max() * c.gs[1]
    return ref, 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * vmax


def _device(c, h):
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(h.DEV)
    return (h.to_dev(c.q), dev(c.pools[0]), dev(c.pools[1]), dev(c.tables), dev(c.cu), dev(c.lens))


def _options(c):
    return pa.PrefillOptions(kernel=c.kernel, kv_dtype=pa.PA_KV_E2M1, k_scale=c.gs[0], v_scale=c.gs[1])


def _workspace(c, most, h):
    longest = int(c.lens.max())
    size = pa.pa_prefill_workspace_size(len(c.rows), most, longest, c.desc, _options(c))
    return longest, torch.zeros(size, dtype=torch.uint8, device=h.DEV)


def _run(c, h, max_rows=None, longest=None):
    most = max(c.rows) if max_rows is None else max_rows
    args = _device(c, h)
    out = torch.full((args[0].shape[0] + 3, *args[0].shape[1:]), 9.0, dtype=torch.bfloat16, device=h.DEV)
    real, ws = _workspace(c, most, h)
    pa.pa_prefill_ex(*args, most, real if longest is None else longest, c.scale, out, ws, c.desc, _options(c))
    torch.cuda.synchronize()
    assert bool((out[args[0].shape[0]:] == 9.0).all())     # rows behind the last sequence stay
    return out[:args[0].shape[0]].double().cpu().numpy(), pa.pa_decode_status(ws)


def _check(c, h, **kw):
    got, status = _run(c, h, **kw)
    assert status == 0
    ref, tol = _reference(c)
    err = np.abs(got - ref) - tol
    assert np.isfinite(got).all() and err.max() <= 0, "outside the tolerance by %g" % err.max()
    return got


SHAPES = [(32, 8, 64, 16), (8, 8, 64, 8), (16, 1, 128, 16), (64, 8, 128, 32), (6, 3, 64, 256), (2, 2, 128, 64),
          (20, 4, 128, 128), (17, 1, 64, 32), (10, 2, 128, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES)
def test_shapes(h, hq, hkv, d, bs):
    # whole prompts, chunks, single rows, no rows, lengths at the tile edges
    _check(_case(hq + d + bs, [1, 63, 64, 65, 200, 129, 300, 0], [1, 63, 1, 65, 33, 100, 0, 0], hq, hkv, d, bs,
                 gs=(0.37, 1.7)), h)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d,bs", [(32, 8, 64, 16), (4, 4, 128, 8), (16, 1, 64, 64), (7, 1, 128, 32), (40, 2, 64, 16)])
@pytest.mark.parametrize("most", [1, 2, 3, 5, 9, 16])
def test_few_rows(h, hq, hkv, d, bs, most):
    rows = [most, 1, max(1, most - 1), 0, most, 1, most]
    lens = [most, 1, 40 + most, 9, 517, 1000, 64]
    _check(_case(most + hq, lens, rows, hq, hkv, d, bs), h)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [pa.PA_PREFILL_ROWS, pa.PA_PREFILL_TCGEN05_WS])
@pytest.mark.parametrize("hq,hkv,d,bs", [(32, 8, 64, 16), (16, 1, 128, 8), (7, 1, 64, 64), (3, 3, 128, 256)])
def test_either_kernel(h, kernel, hq, hkv, d, bs):
    # whatever an automatic call would take: one row up to several chunks of rows, and several tiles of them
    c = _case(kernel + hq, [1, 18, 40, 300, 700, 64, 129], [1, 18, 3, 0, 130, 64, 1], hq, hkv, d, bs, gs=(1.3, 0.21))
    c.kernel = kernel
    _check(c, h)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,rows,hq,hkv,d,bs", [
    ([9000], [300], 8, 2, 64, 16),                        # few items, many pieces each
    ([5000, 9900, 100, 6000, 0], [60, 200, 100, 1, 0], 16, 1, 128, 64),   # ragged, short ones among them
    ([2600], [2600], 2, 2, 64, 16),                       # pieces behind a row's (or a row tile's) last key
    ([6300], [6300], 1, 1, 128, 16),
    ([2700, 130], [2690, 130], 1, 1, 64, 8),
    ([1300, 1290, 40, 1200, 9, 1, 3500, 1280], [3, 7, 0, 2, 9, 1, 1280, 4], 4, 4, 64, 32),   # whole rounds before
    ([1300, 1290, 40, 1200, 9, 1, 7000, 1280], [3, 7, 0, 2, 9, 1, 1280, 4], 4, 4, 128, 32),
])
def test_last_round_cut_between_ctas(h, lens, rows, hq, hkv, d, bs):
    c = _case(len(lens) + hq + d, lens, rows, hq, hkv, d, bs, gs=(0.6, 2.3))
    c.kernel = pa.PA_PREFILL_TCGEN05_WS
    assert pa.pa_prefill_workspace_size(len(rows), max(rows), max(lens), c.desc, _options(c)) > 256
    _check(c, h)
    _check(c, h)


@pytest.mark.gpu
def test_cut_calls_report_and_repeat(h):
    c = _case(31, [4000, 3500, 3900], [140, 150, 130], 8, 4, 64, 16)
    c.kernel = pa.PA_PREFILL_TCGEN05_WS
    ref, tol = _reference(c)
    live = np.r_[0:140, 290:420]
    keep, c.lens[1] = c.lens[1], 149
    got, st = _run(c, h, longest=4000)
    c.lens[1] = keep
    assert st == -8 and (got[140:290] == 9.0).all() and np.all(np.abs(got - ref)[live] <= tol[live])
    keep, c.tables[1, 3] = c.tables[1, 3], c.n
    got, st = _run(c, h)
    c.tables[1, 3] = keep
    assert st == -7 and np.all(np.abs(got - ref)[live] <= tol[live])
    x = _device(c, h)                                     # back to back in a graph, over one workspace
    longest, ws = _workspace(c, max(c.rows), h)
    outs = [torch.zeros_like(x[0]) for _ in range(2)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for out in outs * 3:
            pa.pa_prefill_ex(*x, max(c.rows), longest, c.scale, out, ws, c.desc, _options(c))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(*outs) and pa.pa_decode_status(ws) == 0
    assert np.all(np.abs(outs[0].double().cpu().numpy() - ref) <= tol)


@pytest.mark.gpu
def test_long_and_many(h):
    _check(_case(3, [9000], [300], 8, 2, 64, 16), h)
    _check(_case(4, [20000, 1], [7, 1], 8, 1, 128, 16), h)
    rng = np.random.default_rng(5)
    rows = rng.integers(0, 150, 40)
    _check(_case(5, rows + rng.integers(0, 200, 40), [int(x) for x in rows], 24, 8, 64, 16), h)
    _check(_case(6, [700], [520], 8, 8, 64, 16, q_scale=6.0), h)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [[4, 5, 6], [40, 50, 60]])
def test_reported_lengths_leave_rows_unwritten(h, rows):
    c = _case(11, [80, 90, 100], rows, 8, 8, 64, 16)
    ref, tol = _reference(c)
    a, b = rows[0], rows[0] + rows[1]
    for value in (c.mb * 16 + 1, rows[1] - 1, -1):         # past the table; fewer tokens than rows
        keep, c.lens[1] = c.lens[1], value
        got, st = _run(c, h, longest=c.mb * 16 + 1)
        c.lens[1] = keep
        live = np.r_[0:a, b:b + rows[2]]
        assert st == -8 and (got[a:b] == 9.0).all() and np.all(np.abs(got - ref)[live] <= tol[live])
    keep, c.tables[1, 0] = c.tables[1, 0], c.n
    got, st = _run(c, h)
    c.tables[1, 0] = keep
    assert st == -7
    got, st = _run(c, h, max_rows=rows[1])                 # a sequence with more rows than announced
    assert st == -8 and (got[b:] == 9.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [[3, 0, 2], [40, 3, 129]])
def test_graph_streams_and_repeats(h, rows):
    cs = [_case(21 + i, [300, 5, 277], rows, 16, 8, 64, 16) for i in range(2)]
    held = [(*_device(c, h), _workspace(c, max(rows), h)[1]) for c in cs]
    outs = [torch.zeros_like(x[0]) for x in held]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    graphs = []
    for c, x, out, s in zip(cs, held, outs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pa.pa_prefill_ex(*x[:6], max(rows), 300, c.scale, out, x[6], c.desc, _options(c))
        graphs.append(g)
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, x, out in zip(cs, held, outs):
        ref, tol = _reference(c)
        assert pa.pa_decode_status(x[6]) == 0 and np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 64), (16, 1, 128), (7, 7, 64), (10, 2, 128)])
@pytest.mark.parametrize("kernel", [pa.PA_PREFILL_AUTO, pa.PA_PREFILL_ROWS, pa.PA_PREFILL_TCGEN05_WS])
def test_a_workspace_serves_smaller_calls(h, hq, hkv, d, kernel):
    rng = np.random.default_rng(hq + kernel)
    desc = _desc(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, max_blocks_per_seq=4000)
    opt = pa.PrefillOptions(kernel=kernel, kv_dtype=pa.PA_KV_E2M1, k_scale=1.0, v_scale=1.0)
    most = (40, 1500, 50000)
    size = pa.pa_prefill_workspace_size(*most, desc, opt)
    cross = pa.pa_cross_attention_workspace_size(*most, desc)
    for _ in range(40):
        small = [int(np.exp(rng.uniform(0, np.log(m)))) for m in most]
        assert pa.pa_prefill_workspace_size(*small, desc, opt) <= size
        small[1] = max(2, small[1])                       # (one row a sequence without offsets has the decode's size)
        assert pa.pa_cross_attention_workspace_size(*small, desc) <= cross


@pytest.mark.gpu
def test_one_workspace_for_calls_of_every_path(h):
    cs = [_case(41, [700, 4000], [3, 1], 16, 4, 64, 16), _case(42, [5000], [300], 16, 4, 64, 16),
          _case(43, [900, 20, 600], [400, 20, 300], 16, 4, 64, 16)]
    size = max(pa.pa_prefill_workspace_size(3, 400, 5000, c.desc, _options(c)) for c in cs)
    ws = torch.zeros(size, dtype=torch.uint8, device=h.DEV)
    for c in cs * 2:
        args = _device(c, h)
        out = torch.zeros_like(args[0])
        pa.pa_prefill_ex(*args, max(c.rows), int(c.lens.max()), c.scale, out, ws, c.desc, _options(c))
        ref, tol = _reference(c)
        assert pa.pa_decode_status(ws) == 0 and np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)


@pytest.mark.gpu
def test_bf16_options_are_pa_prefill(h):
    rng = np.random.default_rng(2)
    from tests.test_gpu_e2m1 import normal
    k, v, q = normal(rng, 6, 2, 16, 64), normal(rng, 6, 2, 16, 64), normal(rng, 40, 4, 64)
    t = torch.arange(6, dtype=torch.int32, device=h.DEV)[None]
    desc = _desc(num_blocks=6, max_blocks_per_seq=6)
    cu, lens = (torch.tensor(x, dtype=torch.int32, device=h.DEV) for x in ([0, 40], [90]))
    outs = [torch.zeros((40, 4, 64), dtype=torch.bfloat16, device=h.DEV) for _ in range(2)]
    ws = torch.zeros(256, dtype=torch.uint8, device=h.DEV)
    a = (h.to_dev(q), h.to_dev(k), h.to_dev(v), t, cu, lens, 40)
    pa.pa_prefill(*a, 0.125, outs[0], ws, desc)
    pa.pa_prefill_ex(*a, 90, 0.125, outs[1], ws, desc)
    torch.cuda.synchronize()
    assert torch.equal(*outs)
