"""pa_append_decode over 4-bit pools with lengths that it reports (needs a B200): no byte of such a
sequence's tokens changes, the others' new rows are written."""
import numpy as np
import pytest
import torch

import pagedattention_kv_cache_pa_b200 as pa
from oracle import e2m1

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tests import gpu_harness
    return gpu_harness


@pytest.mark.parametrize("theta", [0.0, 10000.0], ids=["plain", "rope"])
@pytest.mark.parametrize("given,longest", [(120, 100), (100 + 3 * 16, 10000), (-7, 100)],
                         ids=["bound", "table", "negative"])
@pytest.mark.parametrize("d", [64, 128])
def test_reported_lengths_append_nothing(h, d, given, longest, theta):
    from tests.test_gpu_e2m1 import Case, dev, normal, same_bytes
    c = Case(13, [100, 37], 8, 2, d, 16)
    c.tables[0, c.mb - 1] = c.tables[0, 0]                 # every entry a block: only the length is reported
    rng = np.random.default_rng(1)
    k, v = normal(rng, 2, 2, d, scale=2.0), normal(rng, 2, 2, d)
    lens = np.array([given, 37], dtype=np.int32)
    slots = np.array([-1, c.tables[1, 36 // 16] * 16 + 36 % 16])
    kr = e2m1.rope_rows(k, np.array([0, 36]), theta) if theta else k
    want = [e2m1.append(c.pools[0], kr, c.gs[0], slots, 16), e2m1.append(c.pools[1], v, c.gs[1], slots, 16)]
    opts = c.options(rope_theta=theta)
    pools, q = [dev(x, h) for x in c.pools], h.to_dev(c.q)
    ws = torch.zeros(pa.pa_decode_workspace_size(2, longest, c.desc, opts), dtype=torch.uint8, device=h.DEV)
    pa.pa_append_decode(q, h.to_dev(k), h.to_dev(v), *pools, dev(c.tables, h), dev(lens, h), longest, c.scale,
                        torch.empty_like(q), ws, c.desc, opts)
    assert pa.pa_decode_status(ws) == -8
    for got, w in zip(pools, want):
        same_bytes(got.cpu().numpy(), w, 16, d)
