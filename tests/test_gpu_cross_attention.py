"""Cross attention to a paged encoder's states against the fp64 oracle (needs a B200).

The oracle's decode of each row over the encoder's tokens is the operation's definition.
|got - ref| <= 2^-8 |ref| + (2^-8 + 2^-10) max|V|: the output's rounding to bf16; P's rounding to
bf16 (2^-8 of sum p |V|) and fp32 scores and exponentials (far below 2^-10 of it).
"""
import numpy as np
import pytest
import torch

import oracle
import pagedattention_kv_cache_pa_b200 as pa
from oracle import e2m1

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tests import gpu_harness
    return gpu_harness


def normal(rng, *shape, scale=1.0):
    return ((rng.standard_normal(shape) * scale).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


class Case:
    """Encoder states in a pool in random order, NaN patterns in every row that no sequence holds."""

    def __init__(self, seed, lens, rows, hq, hkv, d, bs, q_scale=1.0):
        rng = np.random.default_rng(seed)
        self.rows, self.lens = rows, np.asarray(lens, dtype=np.int32)
        need = [-(-int(x) // bs) for x in lens]
        self.n, self.mb = sum(need) + 2, max(1, max(need)) + 1
        order, at = rng.permutation(self.n).astype(np.int32), 0
        self.tables = np.full((len(lens), self.mb), -1, dtype=np.int32)
        held = np.zeros((self.n, bs), dtype=bool)
        for i, m in enumerate(need):
            self.tables[i, :m] = order[at:at + m]
            for j in range(m):
                held[order[at + j], :min(bs, int(lens[i]) - j * bs)] = True
            at += m
        self.clean = [normal(rng, self.n, hkv, bs, d) * held[:, None, :, None].astype(np.uint16) for _ in range(2)]
        self.pools = [np.where(held[:, None, :, None], x, 0x7FC1).astype(np.uint16) for x in self.clean]
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.q = normal(rng, int(self.cu[-1]), hq, d, scale=q_scale)
        self.scale, self.longest = d ** -0.5, int(self.lens.max())
        self.desc = pa.CacheDesc.make(num_blocks=self.n, block_size=bs, num_kv_heads=hkv, num_q_heads=hq, head_dim=d,
                                      max_blocks_per_seq=self.mb)

    def reference(self):
        seq = np.repeat(np.arange(len(self.rows)), self.rows)
        ref = oracle.paged_decode(self.q, *self.clean, self.tables[seq], self.lens[seq], self.scale)
        return ref, 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * np.abs(e2m1.to_float(np.stack(self.clean)[1])).max()

    def device(self, h):
        return (h.to_dev(self.q), h.to_dev(self.pools[0]), h.to_dev(self.pools[1]),
                torch.from_numpy(self.tables).to(h.DEV), torch.from_numpy(self.cu).to(h.DEV),
                torch.from_numpy(self.lens).to(h.DEV))

    def run(self, h, step=False, max_rows=None):
        q, k, v, t, cu, lens = self.device(h)
        most = max(self.rows) if max_rows is None else max_rows
        out = torch.full((q.shape[0] + 3, *q.shape[1:]), 9.0, dtype=torch.bfloat16, device=h.DEV)
        size = pa.pa_cross_attention_workspace_size(len(self.rows), most, self.longest, self.desc)
        ws = torch.zeros(size, dtype=torch.uint8, device=h.DEV)
        pa.pa_cross_attention(q, k, v, t, None if step else cu, lens, most, self.longest, self.scale, out, ws, self.desc)
        torch.cuda.synchronize()
        assert bool((out[q.shape[0]:] == 9.0).all())      # rows behind the last sequence stay
        return out[:q.shape[0]].double().cpu().numpy(), pa.pa_decode_status(ws)

    def check(self, h, **kw):
        got, status = self.run(h, **kw)
        assert status == 0
        ref, tol = self.reference()
        err = np.abs(got - ref) - tol
        assert np.isfinite(got).all() and err.max() <= 0, "outside the tolerance by %g" % err.max()
        return got


SHAPES = [(16, 16, 64, 16), (32, 8, 64, 64), (8, 1, 128, 8), (6, 3, 128, 256), (20, 4, 64, 32), (7, 1, 64, 128),
          (4, 4, 128, 192)]


@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES)
def test_shapes(h, hq, hkv, d, bs):
    # more rows than tokens, one token, none, tile edges, a sequence with no rows
    Case(hq + d + bs, [1, 63, 64, 65, 0, 200, 129, 7], [5, 130, 1, 64, 33, 0, 17, 300], hq, hkv, d, bs).check(h)


def test_more_tiles_than_the_grid_and_masks(h):
    rng = np.random.default_rng(3)
    Case(3, rng.integers(0, 150, 40), [int(x) for x in rng.integers(0, 200, 40)], 24, 8, 64, 16).check(h)
    Case(4, [0, 0], [70, 200], 8, 2, 64, 16).check(h)     # nothing to attend to anywhere
    Case(5, [1000], [3], 8, 8, 128, 16, q_scale=6.0).check(h)


@pytest.mark.parametrize("lens,rows,hq,hkv,bs", [
    ([9000], [5], 4, 2, 16),                              # one item cut into many slices
    ([3001, 0, 70, 1500, 5000], [3, 7, 0, 200, 129], 6, 2, 64),   # empty, without rows, ragged, whole ones among them
    ([1024, 1025, 1], [128, 128, 128], 3, 3, 128),        # slices that end with items
    ([2000] * 40, [1, 2] * 20, 2, 1, 8),                  # more sequences than a warp's lanes
])
@pytest.mark.parametrize("d", [64, 128])
def test_few_items_cut_between_slices(h, lens, rows, hq, hkv, bs, d):
    c = Case(len(lens) + hq, lens, rows, hq, hkv, d, bs)
    size = pa.pa_cross_attention_workspace_size(len(rows), max(rows), c.longest, c.desc)
    assert size > 256                                     # the call keeps pieces' states there
    c.check(h)


def test_few_items_report_bad_lengths(h):
    c = Case(5, [2000, 1900, 2500], [4, 5, 6], 4, 4, 64, 16)
    ref, tol = c.reference()
    c.lens[1] = c.mb * 16 + 1
    got, st = c.run(h)
    live = np.r_[0:4, 9:15]
    assert st == -8 and (got[4:9] == 9.0).all() and np.all(np.abs(got - ref)[live] <= tol[live])
    got, st = c.run(h, max_rows=5)
    assert st == -8 and (got[4:] == 9.0).all() and np.all(np.abs(got - ref)[:4] <= tol[:4])


@pytest.mark.parametrize("hq,hkv,d,bs", [(16, 16, 64, 16), (8, 1, 128, 8), (12, 6, 64, 128)])
def test_single_rows(h, hq, hkv, d, bs):
    c = Case(9, [1, 64, 0, 300, 77], [1] * 5, hq, hkv, d, bs)
    a, b = c.check(h, step=True), c.check(h)              # with and without row offsets
    assert np.abs(a - b).max() <= 2 * c.reference()[1].max()


def test_reported_lengths_leave_rows_unwritten(h):
    c = Case(11, [50, 60, 70], [4, 5, 6], 8, 8, 64, 16)
    ref, tol = c.reference()
    for what, value, status in (("lens", c.mb * 16 + 1, -8), ("lens", -1, -8), ("tables", c.n, -7)):
        keep = c.lens[1] if what == "lens" else c.tables[1, 0]
        (c.lens if what == "lens" else c.tables[1])[1 if what == "lens" else 0] = value
        got, st = c.run(h)
        assert st == status
        live = np.r_[0:4, 9:15]
        assert np.all(np.abs(got - ref)[live] <= (tol if np.isscalar(tol) else tol[live]))
        if what == "lens":
            assert (got[4:9] == 9.0).all()
        (c.lens if what == "lens" else c.tables[1])[1 if what == "lens" else 0] = keep
    got, st = c.run(h, max_rows=5)                        # a sequence with more rows than announced
    assert st == -8 and (got[9:] == 9.0).all()


def test_graph_streams_and_repeats(h):
    cs = [Case(21 + i, [300, 0, 77], [40, 3, 129], 16, 8, 64, 16) for i in range(2)]
    held = [(*c.device(h), torch.zeros(pa.pa_cross_attention_workspace_size(3, 129, 300, c.desc), dtype=torch.uint8,
                                       device=h.DEV)) for c in cs]
    outs = [torch.zeros_like(x[0]) for x in held]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    graphs = []
    for c, x, out, s in zip(cs, held, outs, streams):
        q, k, v, t, cu, lens, ws = x
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pa.pa_cross_attention(q, k, v, t, cu, lens, 129, 300, c.scale, out, ws, c.desc)
        graphs.append(g)
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, x, out in zip(cs, held, outs):
        ref, tol = c.reference()
        assert pa.pa_decode_status(x[-1]) == 0 and np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)
