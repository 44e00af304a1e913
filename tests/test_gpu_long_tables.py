"""Block tables whose row could hold 2^31 tokens and more: every attention call gives the bits that it
gives over a table of the few blocks in use (needs a B200)."""
import numpy as np
import pytest
import torch

import pagedattention_kv_cache_pa_b200 as pa

pytestmark = pytest.mark.gpu
BS, LENS, ROWS = 256, [700, 130], [40, 3]


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tests import gpu_harness
    return gpu_harness


class Pool:
    def __init__(self, hkv, d, e2m1):
        g = torch.Generator(device="cuda").manual_seed(hkv + d)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
        self.hkv, self.d, self.e2m1 = hkv, d, e2m1
        self.k, self.v = r(5, hkv, BS, d), r(5, hkv, BS, d)
        self.q, self.step, self.new = r(43, 8, d), r(2, 8, d), (r(2, hkv, d), r(2, hkv, d))
        if e2m1:
            desc = self.desc(3)
            rows = [x.transpose(1, 2).reshape(5 * BS, hkv, d).contiguous() for x in (self.k, self.v)]
            self.k, self.v = (torch.zeros(pa.pa_kv_cache_bytes(desc, pa.PA_KV_E2M1), dtype=torch.uint8, device="cuda")
                              for _ in range(2))
            pa.pa_append_kv_e2m1(*rows, torch.arange(5 * BS, device="cuda"), 1.0, 1.0, self.k, self.v, desc)
        self.cu = torch.tensor([0, 40, 43], dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(LENS, dtype=torch.int32, device="cuda")

    def desc(self, mb):
        return pa.CacheDesc.make(num_blocks=5, block_size=BS, num_kv_heads=self.hkv, num_q_heads=8, head_dim=self.d,
                                 max_blocks_per_seq=mb)

    def run(self, mb, call, kernel):
        desc, q = self.desc(mb), self.q if call in ("prefill", "cross") else self.step
        tables = torch.zeros((2, mb), dtype=torch.int32, device="cuda")
        tables[0, :3], tables[1, :1] = torch.tensor([4, 0, 2], device="cuda"), 1
        k, v, out = self.k.clone(), self.v.clone(), torch.full_like(q, 9.0)
        ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
        kv = dict(kv_dtype=pa.PA_KV_E2M1, k_scale=1.0, v_scale=1.0) if self.e2m1 else {}
        scale = self.d ** -0.5
        if call == "prefill" and self.e2m1:
            pa.pa_prefill_ex(q, k, v, tables, self.cu, self.lens, 40, 700, scale, out, ws, desc,
                             pa.PrefillOptions(kernel=kernel, **kv))
        elif call == "prefill":
            pa.pa_prefill(q, k, v, tables, self.cu, self.lens, 40, scale, out, ws, desc, kernel=kernel)
        elif call.startswith("cross"):
            step = call == "cross_step"
            pa.pa_cross_attention(q, k, v, tables, None if step else self.cu, self.lens, 1 if step else 40, 700, scale,
                                  out, ws, desc)
        elif call == "decode":
            pa.pa_decode(q, k, v, tables, self.lens, 700, scale, out, ws, desc, pa.DecodeOptions(kernel=kernel, **kv))
        else:
            pa.pa_append_decode(q, *self.new, k, v, tables, self.lens, 700, scale, out, ws, desc,
                                pa.DecodeOptions(kernel=kernel, rope_theta=1e4 if call == "append_rope" else 0.0, **kv))
        assert pa.pa_decode_status(ws) == 0
        return out, k, v


CALLS = [(True, "prefill", pa.PA_PREFILL_ROWS), (True, "prefill", pa.PA_PREFILL_TCGEN05_WS),
         (False, "prefill", "tcgen05"), (False, "prefill", "tcgen05_ws"), (False, "prefill", "mma"),
         (False, "cross", 0), (False, "cross_step", 0)] + \
        [(True, c, pa.PA_KERNEL_TENSOR) for c in ("decode", "append", "append_rope")] + \
        [(False, c, k) for c in ("decode", "append", "append_rope")
         for k in (pa.PA_KERNEL_SIMT, pa.PA_KERNEL_TENSOR, pa.PA_KERNEL_TENSOR_SPLIT)]


@pytest.mark.parametrize("e2m1,call,kernel", CALLS)
@pytest.mark.parametrize("hkv,d", [(8, 64), (2, 128)])
def test_rows_of_2_to_the_31_tokens(h, hkv, d, e2m1, call, kernel):
    p = Pool(hkv, d, e2m1)
    want = p.run(3, call, kernel)
    for mb in (2 ** 23, 2 ** 24 + 4):                      # 2^31 tokens; 2^32 and four blocks
        for a, b in zip(p.run(mb, call, kernel), want):
            assert torch.equal(a, b)
    assert bool(torch.isfinite(want[0].float()).all()) and not bool((want[0] == 9.0).all())
