"""Pools past 4 GB and the most sequences a call takes, over 4-bit pools and in cross attention (needs a B200).

The bits are those of the same rows in a small pool, or of the same sequences in smaller calls.
"""
import pytest
import torch

import pagedattention_kv_cache_pa_b200 as pa

pytestmark = pytest.mark.gpu
HKV, HQ, D, BS = 8, 16, 128, 256
E2M1 = dict(kv_dtype=pa.PA_KV_E2M1, k_scale=1.0, v_scale=0.5)


def rand(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def desc(blocks, mb, bs=BS, hkv=HKV, hq=HQ, d=D):
    return pa.CacheDesc.make(num_blocks=blocks, block_size=bs, num_kv_heads=hkv, num_q_heads=hq, head_dim=d,
                             max_blocks_per_seq=mb)


def test_4bit_pools_past_32_bits():
    k, v, q = rand(1, 4 * BS, HKV, D), rand(2, 4 * BS, HKV, D), rand(3, 300, HQ, D)
    lens, cu = i32(900), i32(0, 300)
    outs = []
    for blocks in (5, 40000):
        dd = desc(blocks, 4)
        size = pa.pa_kv_cache_bytes(dd, pa.PA_KV_E2M1)
        assert blocks == 5 or size > 2 ** 32
        kc, vc = (torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2))
        ids = torch.tensor([blocks - 1, blocks - 3, blocks - 2, blocks - 4], device="cuda")
        slots = (ids[:, None] * BS + torch.arange(BS, device="cuda")).reshape(-1)
        pa.pa_append_kv_e2m1(k[:700], v[:700], slots[:700], 1.0, 0.5, kc, vc, dd)
        pos, qr = torch.arange(700, 1024, dtype=torch.int32, device="cuda"), torch.empty(324, HQ, D, dtype=torch.bfloat16,
                                                                                        device="cuda")
        pa.pa_rope_append_kv_e2m1(torch.cat([q, q[:24]]), qr, k[700:], v[700:], pos, slots[700:], 1e4, 1.0, 0.5, kc, vc, dd)
        kb, vb = torch.empty_like(k), torch.empty_like(v)
        pa.pa_gather_kv_e2m1(kc, vc, slots, 1.0, 0.5, kb, vb, dd)
        tables = ids.to(torch.int32)[None].contiguous()
        got = [qr, kb, vb]
        for kernel in (pa.PA_PREFILL_ROWS, pa.PA_PREFILL_TCGEN05_WS):
            o = pa.PrefillOptions(kernel=kernel, **E2M1)
            ws = torch.zeros(pa.pa_prefill_workspace_size(1, 300, 900, dd, o), dtype=torch.uint8, device="cuda")
            out = torch.empty_like(q)
            pa.pa_prefill_ex(q, kc, vc, tables, cu, lens, 300, 900, D ** -0.5, out, ws, dd, o)
            assert pa.pa_decode_status(ws) == 0
            got.append(out)
        o = pa.DecodeOptions(rope_theta=1e4, **E2M1)
        ws = torch.zeros(pa.pa_decode_workspace_size(1, 900, dd, o), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q[:1])
        pa.pa_append_decode(q[:1], k[:1], v[:1], kc, vc, tables, lens, 900, D ** -0.5, out, ws, dd, o)
        assert pa.pa_decode_status(ws) == 0
        pa.pa_copy_blocks_e2m1(kc, vc, torch.stack([ids[1], ids[3] - 1])[None].to(torch.int32),
                               dd)
        page = size // blocks
        got += [out] + [x[page * (blocks - 5):].clone() for x in (kc, vc)]
        outs.append(got)
        torch.cuda.synchronize()
        del kc, vc
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows,d", [(300, 128), (300, 64), (5, 64), (5, 128), (0, 64)])
def test_cross_attention_pools_past_32_bits(rows, d):
    k, v = rand(4, 4, HKV, BS, d), rand(5, 4, HKV, BS, d)
    q = rand(6, rows or 1, HQ, d)
    outs = []
    for blocks in (4, 9000 * 128 // d):
        dd = desc(blocks, 4, d=d)
        kc, vc = (torch.zeros(blocks, HKV, BS, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        assert blocks == 4 or kc.numel() * 2 > 2 ** 32
        kc[-4:], vc[-4:] = k, v
        tables = i32(blocks - 2, blocks - 4, blocks - 1, blocks - 3)[None].contiguous()
        ws = torch.zeros(pa.pa_cross_attention_workspace_size(1, rows or 1, 1000, dd), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        pa.pa_cross_attention(q, kc, vc, tables, i32(0, rows) if rows else None, i32(1000), rows or 1, 1000, d ** -0.5, out,
                              ws, dd)
        assert pa.pa_decode_status(ws) == 0
        outs.append(out)
        del kc, vc
    assert torch.equal(*outs)


@pytest.mark.parametrize("call", ["decode", "append", "rows", "tiles", "cross", "cross_step"])
def test_most_sequences(call):
    n, bs, d = 65535, 8, 64
    dd = desc(64, 2, bs, 2, 4, d)
    g = torch.Generator(device="cuda").manual_seed(7)
    lens = torch.randint(1, 17, (n,), generator=g, device="cuda", dtype=torch.int32)
    tables = torch.randint(0, 64, (n, 2), generator=g, device="cuda", dtype=torch.int32)
    if call == "append":                                   # every sequence writes a block of its own
        dd = desc(n + 1, 1, bs, 2, 4, d)
        lens, tables = lens.clamp(max=8), torch.randperm(n, generator=g, device="cuda").to(torch.int32)[:, None].contiguous()
    q, new = rand(8, n, 4, d), (rand(9, n, 2, d), rand(10, n, 2, d))
    bf16 = call.startswith("cross")
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    if bf16:
        pools = [rand(11, 64, 2, bs, d), rand(12, 64, 2, bs, d)]
    else:
        pools = [torch.zeros(pa.pa_kv_cache_bytes(dd, pa.PA_KV_E2M1), dtype=torch.uint8, device="cuda") for _ in range(2)]
        t = dd.num_blocks * bs
        pa.pa_append_kv_e2m1(rand(11, t, 2, d), rand(12, t, 2, d), torch.arange(t, device="cuda"), 1.0, 0.5, *pools, dd)

    def run(lo, hi):
        m, kv, out = hi - lo, [x.clone() for x in pools], torch.empty_like(q[lo:hi])
        a = (q[lo:hi], *kv, tables[lo:hi], cu[:m + 1], lens[lo:hi])
        if call in ("rows", "tiles"):
            o = pa.PrefillOptions(kernel=pa.PA_PREFILL_ROWS if call == "rows" else pa.PA_PREFILL_TCGEN05_WS, **E2M1)
            ws = torch.zeros(pa.pa_prefill_workspace_size(m, 1, 16, dd, o), dtype=torch.uint8, device="cuda")
            pa.pa_prefill_ex(*a, 1, 16, d ** -0.5, out, ws, dd, o)
        elif bf16:
            ws = torch.zeros(pa.pa_cross_attention_workspace_size(m, 1, 16, dd), dtype=torch.uint8, device="cuda")
            pa.pa_cross_attention(*a[:4], None if call == "cross_step" else a[4], a[5], 1, 16, d ** -0.5, out, ws, dd)
        else:
            o = pa.DecodeOptions(**E2M1)
            ws = torch.zeros(pa.pa_decode_workspace_size(m, 16, dd, o), dtype=torch.uint8, device="cuda")
            if call == "decode":
                pa.pa_decode(*a[:4], a[5], 16, d ** -0.5, out, ws, dd, o)
            else:
                pa.pa_append_decode(a[0], *(x[lo:hi] for x in new), *kv, a[3], a[5], 16, d ** -0.5, out, ws, dd, o)
        assert pa.pa_decode_status(ws) == 0
        return out

    whole = run(0, n).float()
    for lo, hi in ((0, 100), (32000, 32300), (n - 50, n)):
        # a sequence that one call cuts between CTAs and the other does not is rounded elsewhere: one bf16 step
        part = run(lo, hi).float()
        assert bool(((whole[lo:hi] - part).abs() <= 2.0 ** -7 * part.abs() + 2.0 ** -9 * 3.0).all())
