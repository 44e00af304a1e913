"""The measured operators: a paged KV cache held in 4 bits (append with the position rotation,
single-token attention, chunked prefill) and cross attention to an encoder's paged states.

The 4-bit format: a row of D values (one token, one kv head) is cut into groups of 16.  With
y = x / gs (gs: one scale per cache tensor), a group keeps s = E4M3(max|y| / 6) in one byte and
E2M1(y / s) for each value in 4 bits, both nearest even and saturating.  A page (block, kv head)
holds Bs rows of D / 2 code bytes, the even dim in the low nibble, then D / 16 rows of Bs scale
bytes.
"""
import math

import torch

own = False

DEV = "cuda:0"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ----------------------------------------------------------------------------------
def _append(t, hq, hkv, d, bs, rope, far):
    return {"op": "append", "tokens": t, "hq": hq, "hkv": hkv, "d": d, "bs": bs, "rope": rope, "far": far}


def _decode(b, lo, hi, hq, hkv, d, bs, empty=False):
    return {"op": "decode", "seqs": b, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "d": d, "bs": bs, "empty": empty}


def _prefill(b, qlo, qhi, clo, chi, hq, hkv, d, bs):
    return {"op": "prefill", "seqs": b, "qlo": qlo, "qhi": qhi, "clo": clo, "chi": chi, "hq": hq, "hkv": hkv, "d": d,
            "bs": bs}


def _cross(b, qlo, qhi, lo, hi, hq, hkv, d, bs, empty=False):
    return {"op": "cross", "seqs": b, "qlo": qlo, "qhi": qhi, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "d": d,
            "bs": bs, "empty": empty}


def listed():
    named = [
        # one new token of one stream, rotated and cached: latency
        ("append_step_1", _append(1, 32, 8, 64, 16, True, 2048)),
        # a prompt chunk of a 32-head, 64-dim layer, an odd number of tokens
        ("append_chunk_2047", _append(2047, 32, 8, 64, 16, True, 16384)),
        # many prompts at once in a 64-head, 128-dim layer, positions of a long context
        ("append_prompts_16384", _append(16384, 64, 8, 128, 16, True, 131072)),
        # one interactive stream
        ("decode_one_777", _decode(1, 777, 777, 32, 8, 64, 16)),
        # a batch of chats: one layer, 64 sequences of 128 to 2048 tokens
        ("decode_batch_64", _decode(64, 128, 2048, 32, 8, 64, 16)),
        # large pages, longer contexts
        ("decode_pages_256", _decode(32, 1280, 8192, 32, 8, 64, 256)),
        # four documents of 32 to 128 thousand tokens, 8 query heads a kv head
        ("decode_long_131072", _decode(4, 32768, 131072, 64, 8, 128, 16)),
        # a few tokens a sequence (a draft being verified, the tail of a prompt)
        ("prefill_tail_7", _prefill(6, 1, 7, 300, 1700, 32, 8, 64, 16)),
        # whole prompts of 2048 tokens
        ("prefill_prompts_2048", _prefill(4, 2048, 2048, 0, 0, 32, 8, 64, 16)),
        # one chunk of a long prompt over what is cached already
        ("prefill_chunk_1021", _prefill(1, 1021, 1021, 15000, 15000, 64, 8, 128, 16)),
        # decoder prompts against encoder states (30 seconds of audio: 1500 frames), no shared heads
        ("cross_prompts_448", _cross(8, 200, 448, 1100, 1500, 16, 16, 64, 16)),
        # one token a sequence against its encoder states
        ("cross_step_64", _cross(64, 1, 1, 300, 1500, 16, 16, 64, 16)),
    ]
    return [dict(c, name=n) for n, c in named]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill", "cross"])
    d = rng.choice([64, 128])
    bs = rng.choice([8, 16, 32, 64, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8, 16])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if op == "append":
        t = min(_log_int(rng, 1, 16384), 160_000_000 // ((g + 2) * hkv * d))
        return _append(t, g * hkv, hkv, d, bs, rng.random() < 0.7, rng.choice([256, 16384, 131072]))
    if op == "decode":
        b = _log_int(rng, 1, 128)
        hi = max(1, min(_log_int(rng, 1, 131072), 330_000_000 // (b * hkv * d)))
        return _decode(b, rng.randint(1, hi), hi, g * hkv, hkv, d, bs, rng.random() < 0.3)
    if op == "prefill":
        b = _log_int(rng, 1, 8)
        qhi, chi = _log_int(rng, 1, 2048), _log_int(rng, 1, 16384) - 1
        most = 60_000_000_000 // (b * g * hkv * d * 4)          # pairs of a query row and a key
        chi = min(chi, max(0, most // qhi - qhi))
        qhi = min(qhi, int(math.isqrt(max(1, most))))
        return _prefill(b, rng.randint(1, qhi), qhi, rng.randint(0, chi), chi, g * hkv, hkv, d, bs)
    b = _log_int(rng, 1, 64)
    qhi = 1 if rng.random() < 0.3 else _log_int(rng, 1, 448)
    hi = _log_int(rng, 1, 4096)
    hi = max(1, min(hi, 60_000_000_000 // (b * g * hkv * d * 4 * qhi), 260_000_000 // (b * hkv * d)))
    return _cross(b, 1 if qhi == 1 else rng.randint(1, qhi), qhi, rng.randint(1, hi), hi, g * hkv, hkv, d, bs,
                  rng.random() < 0.3)


def _spread(n, lo, hi, by=0.6180339887498949):
    """n lengths over [lo, hi], both ends among them: the same for every seed."""
    u = [((i * by) % 1.0) for i in range(n)]
    out = [lo + int(x * (hi - lo + 1)) for x in u]
    out[0] = hi
    if n > 1:
        out[-1] = lo
    return out


def _lengths(case):
    """Query rows and cached tokens of each sequence."""
    n = case["seqs"]
    if case["op"] == "decode":
        lens = _spread(n, case["lo"], case["hi"])
        rows = [1] * n
    elif case["op"] == "prefill":
        rows = _spread(n, case["qlo"], case["qhi"])
        lens = [q + c for q, c in zip(rows, _spread(n, case["clo"], case["chi"], 0.7548776662466927))]
    else:
        rows = _spread(n, case["qlo"], case["qhi"])
        lens = _spread(n, case["lo"], case["hi"], 0.7548776662466927)
    if case.get("empty"):
        lens = [0 if i % 5 == 3 else x for i, x in enumerate(lens)]
    return rows, lens


# ---- inputs ----------------------------------------------------------------------------------
def _bf16(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).bfloat16()


def _quantize(x, inv):
    """Codes [..., D] (0..15) and scale bytes [..., D / 16] of bf16 rows."""
    y = x.float() * inv
    y = y.unflatten(-1, (-1, 16))
    s8 = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float().unsqueeze(-1)
    t = torch.where(s == 0, torch.zeros_like(y), y / s)
    a = t.abs()
    # nearest of the eight magnitudes; a value half way goes to the even code
    up = torch.stack([a > 0.25, a >= 0.75, a > 1.25, a >= 1.75, a > 2.5, a >= 3.5, a > 5.0]).sum(0)
    code = torch.where(s == 0, torch.zeros_like(up), up + 8 * torch.signbit(t))
    return code.flatten(-2).to(torch.uint8), s8.view(torch.uint8)


def _page_bytes(case):
    return case["bs"] * case["d"] * 9 // 16


def _pool4(case, gen, blocks, inv):
    """A cache tensor of normal values with a few strong channels, as keys have them: [blocks, Hkv, page bytes]."""
    hkv, bs, d = case["hkv"], case["bs"], case["d"]
    pool = torch.empty(blocks, hkv, _page_bytes(case), dtype=torch.uint8, device=DEV)
    gain = 1.0 + 3.0 * (torch.rand(hkv, 1, d, generator=gen, device=DEV) < 0.05)
    step = max(1, (1 << 26) // (hkv * bs * d))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        x = (torch.randn(n, hkv, bs, d, generator=gen, device=DEV) * gain).bfloat16()
        code, s = _quantize(x, inv)
        pool[i:i + n, :, :bs * d // 2] = (code[..., 0::2] | (code[..., 1::2] << 4)).flatten(-2)
        pool[i:i + n, :, bs * d // 2:] = s.transpose(-1, -2).flatten(-2)
    return pool


def _tables(gen, lens, bs):
    """Block tables of the sequences over a pool in random order with a few blocks to spare."""
    need = [-(-x // bs) for x in lens]
    blocks = sum(need) + 3
    order = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
    mb = max(1, max(need))
    tables = torch.zeros(len(lens), mb, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = order[at:at + n]
        at += n
    return tables, blocks


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    st = {"case": case, "k_scale": 1.0, "v_scale": 0.5, "theta": 500000.0}
    if case["op"] == "append":
        t = case["tokens"]
        blocks = -(-t // bs) + 3
        slots = torch.randperm(blocks * bs, generator=gen, device=DEV)[:t].clone()
        slots[torch.arange(t, device=DEV) % 61 == 60] = -1           # padding rows of a batch
        st |= {"blocks": blocks, "table_width": blocks, "slots": slots,
               "positions": torch.randint(0, case["far"], (t,), generator=gen, device=DEV, dtype=torch.int32),
               "q": _bf16(gen, t, hq, d), "k": _bf16(gen, t, hkv, d, scale=2.0), "v": _bf16(gen, t, hkv, d)}
        for name in ("k_cache", "v_cache"):
            st[name] = torch.zeros(blocks, hkv, _page_bytes(case), dtype=torch.uint8, device=DEV)
        st |= {"q_out": torch.empty_like(st["q"]), "k_back": torch.empty_like(st["k"]),
               "v_back": torch.empty_like(st["v"])}
        return st
    rows, lens = _lengths(case)
    tables, blocks = _tables(gen, lens, bs)
    total = sum(rows)
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    st |= {"blocks": blocks, "table_width": tables.shape[1], "tables": tables, "rows": max(rows), "longest": max(lens),
           "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
           "cu": torch.tensor(cu, dtype=torch.int32, device=DEV),
           "q": _bf16(gen, total, hq, d, scale=1.5), "scale": d ** -0.5}
    if case["op"] == "cross":
        st["k_cache"], st["v_cache"] = _bf16(gen, blocks, hkv, bs, d), _bf16(gen, blocks, hkv, bs, d)
    else:
        st["k_cache"] = _pool4(case, gen, blocks, 1.0 / st["k_scale"])
        st["v_cache"] = _pool4(case, gen, blocks, 1.0 / st["v_scale"])
    st["out"] = torch.empty_like(st["q"])
    return st


# ---- the plain forms -------------------------------------------------------------------------
def _values(pages, bs, d, scale):
    """Pages [..., page bytes] as the values they stand for: [..., Bs, D] in 32 bits."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=pages.device)
    codes = pages[..., :bs * d // 2].unflatten(-1, (bs, d // 2))
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    s = pages[..., bs * d // 2:].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (d // 16, bs))
    return (lut[both.int()].unflatten(-1, (-1, 16)) * s.transpose(-1, -2).unsqueeze(-1)).flatten(-2) * scale


def _rotate(x, positions, theta):
    half = x.shape[-1] // 2
    freq = theta ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    a = (positions.double()[:, None] * freq)[:, None]
    x1, x2 = x.double().chunk(2, -1)
    return torch.cat([x1 * a.cos() - x2 * a.sin(), x1 * a.sin() + x2 * a.cos()], -1).float().bfloat16()


def _plain_append(st):
    case = st["case"]
    hkv, d, bs = case["hkv"], case["d"], case["bs"]
    q, k = st["q"], st["k"]
    if case["rope"]:
        q, k = _rotate(q, st["positions"], st["theta"]), _rotate(k, st["positions"], st["theta"])
    live = st["slots"] >= 0
    slots = st["slots"][live]
    blk, off = slots // bs, slots % bs
    back = []
    for x, cache, scale in ((k, st["k_cache"], st["k_scale"]), (st["v"], st["v_cache"], st["v_scale"])):
        code, s = _quantize(x[live], 1.0 / scale)
        rows = cache[..., :bs * d // 2].unflatten(-1, (bs, d // 2))
        rows[blk, :, off] = code[..., 0::2] | (code[..., 1::2] << 4)
        scales = cache[..., bs * d // 2:].unflatten(-1, (d // 16, bs))
        scales[blk, :, :, off] = s
        one = torch.cat([rows[blk, :, off], scales[blk, :, :, off]], -1)          # pages of one token
        out = torch.zeros(x.shape, device=x.device)
        out[live] = _values(one, 1, d, scale).squeeze(-2)
        back.append(out.bfloat16())
    return {"q": q, "k": back[0], "v": back[1]} if case["rope"] else {"k": back[0], "v": back[1]}


def _plain_attention(st, k, v, causal):
    """Rows of every sequence against its tokens: k, v [B, Hkv, L, D] in 32 bits."""
    case = st["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    b, _, length, _ = k.shape
    cu, lens = st["cu"].long(), st["lens"].long()
    seq = (torch.arange(st["q"].shape[0], device=DEV)[:, None] >= cu[None, 1:]).sum(1)
    at = torch.arange(st["q"].shape[0], device=DEV) - cu[seq]
    q = torch.zeros(b, st["rows"], hq, d, device=DEV)
    q[seq, at] = st["q"].float()
    q = q.view(b, st["rows"], hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    s = (q @ k.transpose(-1, -2) * st["scale"]).view(b, hkv, hq // hkv, st["rows"], length)
    last = (lens - 1)[:, None].expand(b, st["rows"])
    if causal:
        last = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(st["rows"], device=DEV)[None]
        last = torch.minimum(last, (lens - 1)[:, None])
    seen = torch.arange(length, device=DEV)[None, None] <= last[..., None]                 # [B, rows, L]
    s = s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = (s - torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    den = p.sum(-1, keepdim=True)
    o = p.view(b, hkv, -1, length) @ v
    o = o.view(b, hkv, hq // hkv, st["rows"], d) / torch.where(den == 0, torch.ones_like(den), den)
    return o.permute(0, 3, 1, 2, 4).reshape(b, st["rows"], hq, d)[seq, at].bfloat16()


def _seen_pages(st, cache):
    """The sequences' pages side by side, [B, width, Hkv, ...]; what lies behind a sequence's last token reads as zero."""
    case = st["case"]
    bs = case["bs"]
    pages = cache[st["tables"].long()]
    if case["op"] == "cross":
        x = pages.float()
    else:
        x = _values(pages, bs, case["d"], st["k_scale"] if cache is st["k_cache"] else st["v_scale"])
    x = x.transpose(1, 2).flatten(2, 3)[:, :, :max(1, st["longest"])]
    live = torch.arange(x.shape[2], device=DEV)[None] < st["lens"].long()[:, None]
    return x.masked_fill_(~live[:, None, :, None], 0.0)


# ---- the framework's calls -------------------------------------------------------------------
def _package():
    import pagedattention_kv_cache_pa_b200 as pa
    return pa


def _handle(st):
    """What a program keeps beside its cache: the pool's description, the options and the workspace."""
    if "desc" not in st:
        pa, case = _package(), st["case"]
        st["desc"] = pa.CacheDesc.make(num_blocks=st["blocks"], block_size=case["bs"], num_kv_heads=case["hkv"],
                                       num_q_heads=case["hq"], head_dim=case["d"],
                                       max_blocks_per_seq=st["table_width"])
        size = 256
        if case["op"] == "decode":
            st["options"] = pa.DecodeOptions(kv_dtype=pa.PA_KV_E2M1, k_scale=st["k_scale"], v_scale=st["v_scale"])
            size = pa.pa_decode_workspace_size(case["seqs"], st["longest"], st["desc"], st["options"])
        elif case["op"] == "prefill":
            st["options"] = pa.PrefillOptions(kv_dtype=pa.PA_KV_E2M1, k_scale=st["k_scale"], v_scale=st["v_scale"])
            size = pa.pa_prefill_workspace_size(case["seqs"], st["rows"], st["longest"], st["desc"], st["options"])
        elif case["op"] == "cross":
            size = pa.pa_cross_attention_workspace_size(case["seqs"], st["rows"], st["longest"], st["desc"])
        st["workspace"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
    return st["desc"]


def _own_append(st):
    pa, case, desc = _package(), st["case"], _handle(st)
    if case["rope"]:
        pa.pa_rope_append_kv_e2m1(st["q"], st["q_out"], st["k"], st["v"], st["positions"], st["slots"], st["theta"],
                                  st["k_scale"], st["v_scale"], st["k_cache"], st["v_cache"], desc)
    else:
        pa.pa_append_kv_e2m1(st["k"], st["v"], st["slots"], st["k_scale"], st["v_scale"], st["k_cache"],
                             st["v_cache"], desc)
    pa.pa_gather_kv_e2m1(st["k_cache"], st["v_cache"], st["slots"], st["k_scale"], st["v_scale"], st["k_back"],
                         st["v_back"], desc)
    back = {"k": st["k_back"], "v": st["v_back"]}
    return {"q": st["q_out"], **back} if case["rope"] else back


def _own_attention(st):
    pa, case, desc = _package(), st["case"], _handle(st)
    if case["op"] == "decode":
        pa.pa_decode(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["longest"], st["scale"],
                     st["out"], st["workspace"], desc, st["options"])
    elif case["op"] == "prefill":
        pa.pa_prefill_ex(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["cu"], st["lens"], st["rows"],
                         st["longest"], st["scale"], st["out"], st["workspace"], desc, st["options"])
    else:
        # one row a sequence: the single-token form, which takes no row offsets
        pa.pa_cross_attention(st["q"], st["k_cache"], st["v_cache"], st["tables"],
                              st["cu"] if st["rows"] > 1 else None, st["lens"], st["rows"], st["longest"],
                              st["scale"], st["out"], st["workspace"], desc)
    return st["out"]


def run(state):
    if state["case"]["op"] == "append":
        return _own_append(state) if own else _plain_append(state)
    if own:
        return _own_attention(state)
    return _plain_attention(state, _seen_pages(state, state["k_cache"]), _seen_pages(state, state["v_cache"]),
                            state["case"]["op"] == "prefill")


# ---- what a pass cannot do without -----------------------------------------------------------
def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        t = case["tokens"]
        rotated = (hq + hkv) * d if case["rope"] else 0
        # k and v in, their rows in the pool, the values read back; q in and out
        per = 2 * hkv * (2 * d + d * 9 // 16 + 2 * d) + (4 * hq * d + 4 if case["rope"] else 0) + 8
        return {"bytes": t * per, "flops": t * (3 * rotated + 2 * hkv * d * 4)}
    rows, lens = _lengths(case)
    row = 4 * d if case["op"] == "cross" else 2 * (d * 9 // 16)              # K and V of a token and head
    nbytes = sum(lens) * hkv * row + sum(rows) * hq * d * 4 + sum(-(-x // case["bs"]) for x in lens) * 4
    if case["op"] == "prefill":
        pairs = sum(q * (n - q) + q * (q + 1) // 2 for q, n in zip(rows, lens))
    else:
        pairs = sum(q * n for q, n in zip(rows, lens))
    return {"bytes": nbytes, "flops": 4 * hq * d * pairs}


# ---- from the definition, in 64 bits ---------------------------------------------------------
def _e2m1_of(x):
    """Nearest E2M1 value of each x (64 bits), half way to the even code, saturating."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    gap = (x.abs().unsqueeze(-1) - grid).abs()
    near = gap.amin(-1, keepdim=True)
    index = torch.arange(8, device=x.device)
    # the candidates at the least distance: an even code before an odd one
    pick = torch.where(gap == near, index % 2, torch.full_like(index, 2)).argmin(-1)
    return torch.copysign(grid[pick], x)


def _e4m3_of(x):
    """Nearest E4M3 value of each x >= 0 (64 bits), half way to the even one, saturating at 448."""
    e = torch.floor(torch.log2(x.clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(max=448.0)


def _bf16_of(x):
    """Nearest bf16 value of each x (64 bits)."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256.0), e - 8)


def _stands_for(page, bs, d, scale):
    """One sequence's pages [n, page bytes] as rows [n Bs, D] in 64 bits, from the bits' meaning."""
    raw = page[:, :bs * d // 2].reshape(-1, d // 2).to(torch.int32)
    nib = torch.empty(raw.shape[0], d, dtype=torch.int32, device=page.device)
    nib[:, 0::2], nib[:, 1::2] = raw % 16, raw // 16
    e, m = (nib // 2) % 4, (nib % 2).double()
    mag = torch.where(e == 0, m / 2, torch.exp2(e.double() - 1) * (1 + m / 2))
    val = torch.where(nib >= 8, -mag, mag)
    sb = page[:, bs * d // 2:].reshape(-1, d // 16, bs).permute(0, 2, 1).reshape(-1, d // 16).to(torch.int32)
    se, sm = (sb // 8) % 16, (sb % 8).double() / 8
    s = torch.where(se == 0, sm * 2.0 ** -6, torch.exp2(se.double() - 7) * (1 + sm))
    return val * s.repeat_interleave(16, dim=1) * scale


def _exact_append(st):
    case = st["case"]
    d = case["d"]
    half = d // 2

    def turn(x):
        x = x.double()
        i = torch.arange(half, dtype=torch.float64, device=DEV)
        angle = torch.outer(st["positions"].double(), torch.pow(torch.tensor(st["theta"], dtype=torch.float64, device=DEV),
                                                                -2 * i / d)).unsqueeze(1)
        c, s = torch.cos(angle), torch.sin(angle)
        y = torch.empty_like(x)
        y[..., :half] = c * x[..., :half] - s * x[..., half:]
        y[..., half:] = s * x[..., :half] + c * x[..., half:]
        return y

    k = _bf16_of(turn(st["k"])) if case["rope"] else st["k"].double()
    found = {"q": turn(st["q"])} if case["rope"] else {}
    for name, x, gs in (("k", k, st["k_scale"]), ("v", st["v"].double(), st["v_scale"])):
        parts = []
        for part in x.split(4096):
            y = (part / gs).reshape(*part.shape[:-1], d // 16, 16)
            s = _e4m3_of(y.abs().amax(-1, keepdim=True) / 6)
            codes = torch.where(s > 0, _e2m1_of(y / s.clamp(min=2.0 ** -9)), torch.zeros_like(y))
            parts.append((codes * s * gs).reshape(part.shape))
        found[name] = torch.cat(parts) * (st["slots"] >= 0).double()[:, None, None]
    return found


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    if work(case)["flops"] > 2e12:
        return None
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    rows, lens = _lengths(case)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, length) in enumerate(zip(rows, lens)):
        ids = st["tables"][b, :-(-length // bs)].long()
        for h in range(hkv if length else 0):
            if case["op"] == "cross":
                k, v = (st[c][ids, h].reshape(-1, d)[:length].double() for c in ("k_cache", "v_cache"))
            else:
                k = _stands_for(st["k_cache"][ids, h], bs, d, st["k_scale"])[:length]
                v = _stands_for(st["v_cache"][ids, h], bs, d, st["v_scale"])[:length]
            for g in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                s = (st["q"][at:at + n, g].double() @ k.T) * st["scale"]
                if case["op"] == "prefill":
                    future = torch.arange(length, device=DEV)[None] > torch.arange(length - n, length, device=DEV)[:, None]
                    s[future] = -math.inf
                out[at:at + n, g] = torch.softmax(s, -1) @ v
        at += n
    return out
