"""Measured cases of the paged-cache operators and of the few-row 4-bit product.

Four operators of a serving step whose sequences come and go: ``append`` writes
new keys and values into a paged cache (rotated by their positions where the
model asks for it, quantized to 4 bits where the cache is), ``read`` brings
cached keys and values back as fp16 rows, ``attention`` lets a ragged batch of
new tokens (single tokens, chunks, or both) attend over the paged cache, and
``gemv`` multiplies a few rows by a 4-bit weight in the tiled layout.

``own`` chooses between the plain torch form of each operator and the calls a
user makes of the library.  Sizes follow this repository's configurations
(hidden sizes 2048 to 7168, head widths 64 and 128, prompts of 512 and 1024)
and generic serving batches; a shape with fewer key/value heads than query
heads is generic.
"""
import math

import torch

own = False

DEV = "cuda"
EPI_BIAS, EPI_GELU, EPI_RESIDUAL, EPI_F32 = 1, 2, 4, 8


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _cache_case(op, bits, heads, kv_heads, d, page, b, chunks, new, past, rope=0, interleaved=False):
    """`chunks` of the b sequences bring new[0]..new[1] tokens, the others one;
    all have past[0]..past[1] tokens in the cache before that."""
    return dict(op=op, bits=bits, heads=heads, kv_heads=kv_heads, d=d, page=page, b=b, chunks=chunks,
                new_lo=new[0], new_hi=new[1], past_lo=past[0], past_hi=past[1], rope=rope, interleaved=interleaved)


def _gemv_case(m, n, k, epi):
    return dict(op="gemv", m=m, n=n, k=k, epi=epi)


def listed():
    return [
        # every sequence of a decode block appends its token (learned positions: no rotation), and it is read back
        dict(_cache_case("append", 4, 56, 56, 128, 16, 144, 0, (1, 1), (500, 1040)), name="append q4 decode"),
        # prompts in chunks, rotated, four query heads to a key head; read back
        dict(_cache_case("append", 4, 32, 8, 128, 64, 8, 8, (511, 1500), (0, 2000), 128), name="append q4 chunks rope"),
        # fp16 cache, a mixed batch, partial rotation of neighbouring pairs; the pools and the rotated queries are the outputs
        dict(_cache_case("append", 16, 32, 32, 64, 32, 24, 12, (1, 300), (0, 700), 32, True), name="append f16 mixed rope"),
        # whole histories out of the cache, as for moving a sequence or for a kernel that wants plain rows
        dict(_cache_case("read", 4, 32, 32, 128, 16, 6, 6, (1000, 5001), (0, 0)), name="read q4 histories"),
        # one token for each sequence of a block: the ordinary decode step
        dict(_cache_case("attention", 4, 56, 56, 128, 16, 144, 0, (1, 1), (300, 1040)), name="attention q4 decode"),
        # a few long conversations, grouped heads
        dict(_cache_case("attention", 4, 32, 8, 128, 64, 5, 0, (1, 1), (9000, 32700)), name="attention q4 decode long"),
        # one user, fp16 cache: latency counts
        dict(_cache_case("attention", 16, 32, 32, 64, 16, 1, 0, (1, 1), (901, 901)), name="attention f16 decode one"),
        # long prompts, chunk by chunk
        dict(_cache_case("attention", 4, 32, 32, 128, 64, 2, 2, (1900, 2048), (1000, 4096)), name="attention q4 chunks"),
        # chunks of some prompts riding with the single tokens of the others
        dict(_cache_case("attention", 4, 56, 56, 128, 16, 32, 4, (100, 301), (20, 1500)), name="attention q4 mixed"),
        # one token through a small model's output projection: latency counts
        dict(_gemv_case(1, 2048, 2048, EPI_BIAS | EPI_RESIDUAL), name="gemv one"),
        # five sequences through the first MLP projection
        dict(_gemv_case(5, 28672, 7168, EPI_BIAS | EPI_GELU), name="gemv mlp"),
        # sixteen rows onto the vocabulary, fp32 logits
        dict(_gemv_case(16, 50272, 4096, EPI_F32), name="gemv head"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _draw_once(rng):
    op = rng.choice(["append", "read", "attention", "attention", "gemv", "gemv"])
    if op == "gemv":
        n = _log_int(rng, 64, 50272)
        k = 64 * _log_int(rng, 4, 448)
        epi = rng.choice([0, EPI_BIAS, EPI_BIAS | EPI_GELU, EPI_BIAS | EPI_RESIDUAL, EPI_BIAS | EPI_GELU | EPI_RESIDUAL, EPI_F32])
        return _gemv_case(rng.randint(1, 16), n, k, epi)
    d = rng.choice([64, 128])
    group = rng.choice([1, 1, 1, 2, 4, 7, 8])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 12, 16, 32])
    heads = kv_heads * group
    while heads * d > 7168 or heads * d % 128:
        kv_heads = rng.choice([2, 4, 8])
        group = rng.choice([1, 2, 4, 7])
        heads = kv_heads * group
    b = _log_int(rng, 1, 160)
    bits = rng.choice([4, 4, 16])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    chunks = rng.choice([0, 0, rng.randint(0, b), b])
    new_hi = _log_int(rng, 1, 2048)
    past_hi = _log_int(rng, 1, 32000)
    new = (_log_int(rng, 1, new_hi) - rng.choice([0, 1]), new_hi)
    past = (_log_int(rng, 1, past_hi) - 1, past_hi)
    rope, inter = 0, False
    if op == "append":
        rope = rng.choice([0, d, d, d // 2, 48])
        inter = rng.random() < 0.5
        past = (min(past[0], 4000), min(past[1], 4000))
    if op == "read":
        past, new, chunks = (0, 0), (min(new[0], past[1]), past[1]), b
    return _cache_case(op, bits, heads, kv_heads, d, page, b, chunks, new, past, rope, inter)


def _affordable(case):
    w = work(case)
    if case["op"] == "gemv":
        return w["bytes"] < 1.2e8
    new, past = _lens(case)
    longest = max(n + p for n, p in zip(new, past))
    padded = case["b"] * longest * case["kv_heads"] * case["d"]  # elements of a padded K
    scores = case["b"] * max(max(new), 1) * case["heads"] * longest if case["op"] == "attention" else 0
    return w["bytes"] < 8e8 and w["flops"] < 3e11 and padded < 1.2e9 and scores < 1.5e9 and sum(new) > 0


def draw(rng):
    case = _draw_once(rng)
    while not _affordable(case):
        case = _draw_once(rng)
    return case


def _spread(i, lo, hi):
    """Entry i of a sequence spread evenly over lo..hi, hi first."""
    f = (1.0 - 1e-9 + i * 0.6180339887498949) % 1.0
    return lo + int(f * (hi - lo + 1))


def _lens(case):
    """New and past tokens of each sequence."""
    b, c = case["b"], case["chunks"]
    new = [_spread(i, case["new_lo"], case["new_hi"]) if i < c else 1 for i in range(b)]
    past = [_spread(3 * i, case["past_lo"], case["past_hi"]) for i in range(b)]
    return new, past


def work(case):
    if case["op"] == "gemv":
        m, n, k, epi = case["m"], case["n"], case["k"], case["epi"]
        by = n * k / 2 + n * k / 64 * 4 + m * k * 2 + m * n * (4 if epi & EPI_F32 else 2)
        by += n * 2 if epi & EPI_BIAS else 0
        by += m * n * 2 if epi & EPI_RESIDUAL else 0
        return {"bytes": by, "flops": 2 * m * n * k}
    new, past = _lens(case)
    d, kvh, h = case["d"], case["kv_heads"], case["heads"]
    slot = 2 * kvh * (d * 2 if case["bits"] == 16 else d // 2 + d // 64 * 4)  # bytes of one token in the cache
    rows = sum(new)
    row16 = 2 * kvh * d * 2  # its keys and values as fp16 rows
    if case["op"] == "append":
        by = rows * (row16 + slot)
        by += (rows * h * d * 2 * 2 + sum(new) * case["rope"] * 4) if case["rope"] else 0
        by += rows * row16 if case["bits"] == 4 else 0  # read back
        return {"bytes": by, "flops": rows * (2 * kvh * d * 4 + (h + kvh) * case["rope"] * 3)}
    if case["op"] == "read":
        return {"bytes": rows * (row16 + slot), "flops": rows * kvh * d * 4}
    seen = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    by = 2 * rows * h * d * 2 + sum((n + p) * slot for n, p in zip(new, past) if n)
    return {"bytes": by, "flops": 4 * d * h * seen}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
_LUT = {}


def _code_bytes(shape, gen):
    """Bytes of two 4-bit codes, bell-shaped around the middle of the range as
    those of a quantized group are."""
    if not _LUT:
        u = (torch.arange(256, dtype=torch.float64) + 0.5) / 256
        nib = (7.5 + 3.3 * math.sqrt(2.0) * torch.erfinv(2 * u - 1)).round().clamp(0, 15).to(torch.uint8)
        w = torch.arange(65536)
        _LUT["lut"] = (nib[w & 255] | (nib[w >> 8] << 4)).to(DEV)
    r = torch.randint(0, 65536, shape, device=DEV, generator=gen, dtype=torch.int32)
    return _LUT["lut"][r]


def _meta(shape, size, gen):
    """(min, scale) fp16 pairs of groups whose values have about the given size."""
    s = size * (0.25 + 0.1 * torch.rand(shape, device=DEV, generator=gen))
    m = -s * (6.5 + 2.0 * torch.rand(shape, device=DEV, generator=gen))
    return torch.stack([m, s], -1).half()


def _prepare_gemv(case, gen):
    m, n, k = case["m"], case["n"], case["k"]
    tiles = -(-n // 128)
    packed = torch.zeros(tiles, k // 64, 4608, device=DEV, dtype=torch.uint8)
    packed[:, :, :4096] = _code_bytes((tiles, k // 64, 4096), gen)
    meta = _meta((tiles, k // 64, 128), 0.03, gen)
    packed[:, :, 4096:] = meta.view(torch.uint8).reshape(tiles, k // 64, 512)
    if n % 128:  # rows past n are zero in the layout
        tail = packed[-1]
        tail[:, :4096].view(k // 64, 128, 32)[:, n % 128:] = 0
        tail[:, 4096:].view(k // 64, 128, 4)[:, n % 128:] = 0
    rnd = lambda *s: torch.randn(s, device=DEV, generator=gen).half()  # noqa: E731
    y = torch.empty(m, n, device=DEV, dtype=torch.float32 if case["epi"] & EPI_F32 else torch.float16)
    return dict(case=case, x=rnd(m, k), w=packed, bias=rnd(n) * 0.1, res=rnd(m, n), y=y)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "gemv":
        return _prepare_gemv(case, gen)
    bits, d, kvh, h, ps, b = (case[x] for x in ("bits", "d", "kv_heads", "heads", "page", "b"))
    new, past = _lens(case)
    lens = [n + p for n, p in zip(new, past)]
    per = [-(-x // ps) for x in lens]
    ld = max(max(per), 1)
    pages = sum(per) + 3
    st = dict(case=case, rows=sum(new), max_new=max(max(new), 1), max_len=max(max(lens), 1), pages=pages)
    if bits == 4:
        st["k"] = _code_bytes((pages, kvh, ps, d // 2), gen)
        st["v"] = _code_bytes((pages, kvh, ps // 8, d * 4), gen).view(torch.int32)
        st["k_meta"] = _meta((pages, kvh, ps, d // 64), 1.0, gen)
        st["v_meta"] = _meta((pages, kvh, ps, d // 64), 1.0, gen)
    else:
        st["k"] = torch.randn(pages, kvh, ps, d, device=DEV, generator=gen, dtype=torch.float16)
        st["v"] = torch.randn(pages, kvh, ps, d, device=DEV, generator=gen, dtype=torch.float16)
    # the pages of a sequence lie anywhere in the pool
    order = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32)
    first = torch.tensor([0] + per[:-1]).cumsum(0)
    at = (first[:, None] + torch.arange(ld)[None]).clamp(max=pages - 1)
    inside = torch.arange(ld)[None] < torch.tensor(per)[:, None]
    st["table"] = torch.where(inside.to(DEV), order[at.to(DEV)], torch.zeros((), dtype=torch.int32, device=DEV)).contiguous()
    st["row_start"] = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(DEV)
    st["kv_len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    rows = st["rows"]
    rnd = lambda *s: torch.randn(s, device=DEV, generator=gen)  # noqa: E731
    if case["op"] == "append":
        # keys have a few wide channels, as keys do
        wide = 1.0 + 3.0 * (torch.rand(kvh * d, device=DEV, generator=gen) < 0.03)
        st["k_new"] = (rnd(rows, kvh * d) * wide).half()
        st["v_new"] = rnd(rows, kvh * d).half()
        if case["rope"]:
            st["q"] = rnd(rows, h * d).half()
            st["q_out"] = torch.empty_like(st["q"])
            rot = case["rope"]
            freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
            ang = torch.arange(st["max_len"], dtype=torch.float64)[:, None] * freq[None]
            st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().to(DEV)
    if case["op"] == "attention":
        st["q"] = (1.5 * rnd(rows, h * d)).half()
        st["out"] = torch.empty(rows, h * d, device=DEV, dtype=torch.float16)
    if case["op"] == "read" or (case["op"] == "append" and bits == 4):
        st["k_out"] = torch.empty(rows, kvh * d, device=DEV, dtype=torch.float16)
        st["v_out"] = torch.empty(rows, kvh * d, device=DEV, dtype=torch.float16)
    return st


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _handles(st):
    """The descriptors a user's program keeps beside its cache."""
    from quantized_opt_decode_b200 import flexq as fq
    c = st["case"]
    cfg = fq.flexq_config(h=c["heads"] * c["d"], heads=c["heads"], ffn=4 * c["heads"] * c["d"], w_bits=4,
                          kv_bits=c["bits"], ln_eps=1e-5)
    ptr = lambda x: st[x].data_ptr() if x in st else None  # noqa: E731
    kv = fq.flexq_paged_kv(ptr("k"), ptr("v"), ptr("k_meta"), ptr("v_meta"), c["kv_heads"], st["pages"], c["page"],
                           ptr("table"), st["table"].shape[1])
    batch = fq.flexq_ragged(c["b"], st["rows"], st["max_new"], st["max_len"], ptr("row_start"), ptr("kv_len"))
    rope = None
    if c["rope"]:
        rope = fq.flexq_rope(ptr("cos_sin"), st["cos_sin"].shape[0], c["rope"], int(c["interleaved"]))
    return fq, cfg, kv, batch, rope


def _run_own(st):
    c = st["case"]
    if c["op"] == "gemv":
        if "fq" not in st:
            from quantized_opt_decode_b200 import flexq
            st["fq"] = flexq
        st["fq"].flexq_gemv_q4(st["x"], c["k"], st["w"], c["m"], c["n"], c["k"], st["bias"], st["res"], c["n"],
                               c["epi"], st["y"], c["n"])
        return st["y"]
    if "handles" not in st:
        st["handles"] = _handles(st)
    fq, cfg, kv, batch, rope = st["handles"]
    row = c["kv_heads"] * c["d"]
    if c["op"] == "attention":
        ld = c["heads"] * c["d"]
        fq.flexq_attention_paged(cfg, kv, batch, st["q"], ld, st["out"], ld)
        return st["out"]
    if c["op"] == "append":
        ld = c["heads"] * c["d"]
        fq.flexq_paged_append(cfg, kv, batch, rope, st["k_new"], st["v_new"], row, st.get("q"), ld, st.get("q_out"), ld)
    if c["op"] == "read" or c["bits"] == 4:
        fq.flexq_paged_read(cfg, kv, batch, st["k_out"], st["v_out"], row)
    return _outputs(st)


def _outputs(st):
    """What append and read leave: the rows read back (or the fp16 pools) and the rotated queries."""
    c = st["case"]
    out = dict(k=st["k_out"], v=st["v_out"]) if "k_out" in st else dict(k=st["k"], v=st["v"])
    if c["rope"]:
        out["q"] = st["q_out"]
    return out


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _row_owner(st):
    """Sequence and position of every row."""
    rows = torch.arange(st["rows"], device=DEV)
    start = st["row_start"].long()
    seq = (rows[:, None] >= start[None, 1:]).sum(1)
    new = start[1:] - start[:-1]
    pos = st["kv_len"].long()[seq] - new[seq] + rows - start[seq]
    return seq, pos


def _slots(st, seq, pos):
    """(page, slot in the page) of positions of sequences."""
    ps = st["case"]["page"]
    return st["table"].long()[seq, pos // ps], pos % ps


def _dequant(code, meta):
    """fp16 values (as fp32) of codes [..., d] with pairs [..., d / 64, 2]."""
    d = code.shape[-1]
    x = code.float().view(*code.shape[:-1], d // 64, 64)
    x = x * meta[..., 1:].float() + meta[..., :1].float()
    return x.half().float().reshape(code.shape)


def _cached(st, page, slot):
    """Keys and values (fp32, [..., kv_heads, d]) of cached tokens."""
    if st["case"]["bits"] == 16:
        return st["k"][page, :, slot].float(), st["v"][page, :, slot].float()
    kb = st["k"][page, :, slot]
    kc = torch.stack([kb & 15, kb >> 4], -1).flatten(-2)
    vw = st["v"][page, :, slot // 8]
    vc = (vw >> (4 * (slot % 8))[..., None, None]) & 15
    return _dequant(kc, st["k_meta"][page, :, slot]), _dequant(vc, st["v_meta"][page, :, slot])


def _rotate(st, x, pos, heads):
    """Rows [rows, heads * d] rotated by their positions, as fp16."""
    c = st["case"]
    rot, d = c["rope"], c["d"]
    x = x.view(x.shape[0], heads, d).float()
    cos, sin = st["cos_sin"][pos][:, None, :rot // 2], st["cos_sin"][pos][:, None, rot // 2:]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if c["interleaved"] else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., rot:]], -1).half().reshape(x.shape[0], heads * d)


def _quantize(x):
    """Codes and (min, scale) pairs of fp16 rows [..., d]."""
    g = x.float().view(*x.shape[:-1], x.shape[-1] // 64, 64)
    lo, hi = g.amin(-1) + 0.0, g.amax(-1) + 0.0
    scale, low = ((hi - lo) / 15.0).half(), lo.half()
    s = scale.float()[..., None]
    code = ((g - low.float()[..., None]) / torch.where(s == 0, torch.ones_like(s), s)).round().clamp(0, 15)
    code = torch.where(s == 0, torch.zeros_like(code), code).to(torch.int32)
    return code.reshape(x.shape), torch.stack([low, scale], -1)


def _append_plain(st):
    c = st["case"]
    kvh, d = c["kv_heads"], c["d"]
    seq, pos = _row_owner(st)
    page, slot = _slots(st, seq, pos)
    k, v = st["k_new"], st["v_new"]
    if c["rope"]:
        k = _rotate(st, k, pos, kvh)
        st["q_out"].copy_(_rotate(st, st["q"], pos, c["heads"]))
    k, v = k.view(-1, kvh, d), v.view(-1, kvh, d)
    if c["bits"] == 16:
        st["k"][page, :, slot] = k
        st["v"][page, :, slot] = v
        return
    code, meta = _quantize(k)
    st["k"][page, :, slot] = (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8)
    st["k_meta"][page, :, slot] = meta
    code, meta = _quantize(v)
    st["v_meta"][page, :, slot] = meta
    # a word holds eight tokens' codes: clear the new tokens' nibbles, then add them in
    shift = 4 * (slot % 8)
    ps8, pages = c["page"] // 8, st["pages"]
    at = page * ps8 + slot // 8
    words = st["v"].permute(0, 2, 1, 3).reshape(pages * ps8, kvh, d)
    bits = torch.zeros(pages * ps8, dtype=torch.int64, device=DEV).index_add_(0, at, torch.ones_like(shift) * (15 << shift))
    fresh = torch.zeros(pages * ps8, kvh, d, dtype=torch.int64, device=DEV)
    fresh.index_add_(0, at, code.long() << shift[:, None, None])
    keep = (words.long() & 0xFFFFFFFF) & ~bits[:, None, None]
    joined = keep | fresh
    joined = torch.where(joined >= 1 << 31, joined - (1 << 32), joined).to(torch.int32)
    st["v"].copy_(joined.view(pages, ps8, kvh, d).permute(0, 2, 1, 3))


def _attention_plain(st):
    c = st["case"]
    h, kvh, d, b = c["heads"], c["kv_heads"], c["d"], c["b"]
    g, t, n = h // kvh, st["max_len"], st["max_new"]
    seq, pos = _row_owner(st)
    every = torch.arange(t, device=DEV)
    alive = every[None] < st["kv_len"][:, None]
    where = torch.where(alive, every[None], torch.zeros_like(every)[None])
    page, slot = _slots(st, torch.arange(b, device=DEV)[:, None], where)
    k, v = _cached(st, page, slot)  # [b, t, kvh, d]
    local = torch.arange(st["rows"], device=DEV) - st["row_start"].long()[seq]
    q = torch.zeros(b, n, h, d, device=DEV)
    q[seq, local] = st["q"].view(-1, h, d).float()
    at = torch.full((b, n), -1, dtype=torch.int64, device=DEV)
    at[seq, local] = pos
    q = q.view(b, n, kvh, g, d).permute(0, 2, 1, 3, 4).reshape(b, kvh, n * g, d)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(d)
    s = s.view(b, kvh, n, g, t).masked_fill((every[None, None] > at[:, :, None])[:, None, :, None], -math.inf)
    s -= s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = s.exp_()
    p = (p / p.sum(-1, keepdim=True)).view(b, kvh, n * g, t)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)).view(b, kvh, n, g, d).permute(0, 2, 1, 3, 4).reshape(b, n, h * d)
    st["out"].copy_(o[seq, local])


def _weight(st):
    """The tiled 4-bit weight as fp16 values (fp32) [n, k]."""
    c = st["case"]
    n, k = c["n"], c["k"]
    w = st["w"]
    words = w[:, :, :4096].contiguous().view(torch.int32).view(-1, k // 64, 128, 8)
    meta = w[:, :, 4096:].contiguous().view(torch.float16).view(-1, k // 64, 128, 2)
    e = torch.arange(8, device=DEV, dtype=torch.int32)
    code = (words[..., None] >> (4 * ((e >> 1) + 4 * (e & 1)))) & 15  # [tile, block, row, word, element]
    x = code.float().flatten(-2) * meta[..., 1:].float() + meta[..., :1].float()
    return x.half().float().permute(0, 2, 1, 3).reshape(-1, k)[:n]


def _gemv_plain(st):
    epi = st["case"]["epi"]
    y = torch.matmul(st["x"].float(), _weight(st).t())
    if epi & EPI_BIAS:
        y = y + st["bias"].float()
    if epi & EPI_GELU:
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    if epi & EPI_RESIDUAL:
        y = y + st["res"].float()
    st["y"].copy_(y)
    return st["y"]


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    if c["op"] == "gemv":
        return _gemv_plain(st)
    if c["op"] == "attention":
        _attention_plain(st)
        return st["out"]
    if c["op"] == "append":
        _append_plain(st)
    if "k_out" in st:
        seq, pos = _row_owner(st)
        k, v = _cached(st, *_slots(st, seq, pos))
        st["k_out"].copy_(k.flatten(1))
        st["v_out"].copy_(v.flatten(1))
    return _outputs(st)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------
def _history64(st, i, length):
    """Keys and values of the first `length` tokens of sequence i: [length, kv_heads, d] doubles."""
    c = st["case"]
    ps, kvh, d = c["page"], c["kv_heads"], c["d"]
    ids = st["table"][i, : -(-length // ps)].long()
    if c["bits"] == 16:
        take = lambda x: st[x][ids].transpose(1, 2).reshape(-1, kvh, d)[:length].double()  # noqa: E731
        return take("k"), take("v")
    kb = st["k"][ids].transpose(1, 2).reshape(-1, kvh, d // 2)[:length]
    kc = torch.empty(length, kvh, d, dtype=torch.float64, device=DEV)
    kc[..., 0::2] = (kb % 16).double()
    kc[..., 1::2] = torch.div(kb, 16, rounding_mode="floor").double()
    vw = st["v"][ids].long() % (1 << 32)  # [pages, kvh, ps / 8, d]
    vc = torch.stack([torch.div(vw, 16 ** t, rounding_mode="floor") % 16 for t in range(8)], 3)
    vc = vc.reshape(len(ids), kvh, ps, d).transpose(1, 2).reshape(-1, kvh, d)[:length].double()

    def value(code, name):
        m = st[name][ids].transpose(1, 2).reshape(-1, kvh, d // 64, 2)[:length].double()
        return (code * m[..., 1].repeat_interleave(64, -1) + m[..., 0].repeat_interleave(64, -1)).half().double()
    return value(kc, "k_meta"), value(vc, "v_meta")


def _exact_quantized(x):
    """What a 4-bit cache holds for rows [..., d] of fp16 values."""
    g = x.double().unflatten(-1, (-1, 64))
    lo = g.min(-1, keepdim=True).values
    scale = ((g.max(-1, keepdim=True).values - lo) / 15).half().double()
    code = ((g - lo) / scale.clamp(min=2.0 ** -24)).round().clamp(0, 15) * (scale > 0)
    return (code * scale + lo).flatten(-2)


def _exact_rotation(st, x, heads, pos):
    c = st["case"]
    rot, d = c["rope"], c["d"]
    x = x.double().view(-1, heads, d).clone()
    first = torch.arange(0, rot, 2, device=DEV) if c["interleaved"] else torch.arange(rot // 2, device=DEV)
    second = first + (1 if c["interleaved"] else rot // 2)
    z = torch.complex(x[..., first], x[..., second])
    turn = torch.complex(st["cos_sin"][pos, : rot // 2].double(), st["cos_sin"][pos, rot // 2:].double())
    z = z * turn[:, None]
    x[..., first], x[..., second] = z.real, z.imag
    return x.reshape(-1, heads * d)


def _exact_append(st):
    c = st["case"]
    kvh, d, ps = c["kv_heads"], c["d"], c["page"]
    new, past = _lens(c)
    pos = torch.cat([torch.arange(p, p + n) for n, p in zip(new, past)]).to(DEV)
    k, out = st["k_new"], {}
    if c["rope"]:
        k = _exact_rotation(st, k, kvh, pos).half()
        out["q"] = _exact_rotation(st, st["q"], c["heads"], pos)
    k, v = k.view(-1, kvh, d), st["v_new"].view(-1, kvh, d)
    if c["bits"] == 4:
        return dict(out, k=_exact_quantized(k).flatten(1), v=_exact_quantized(v).flatten(1))
    pools = dict(k=st["k"].double(), v=st["v"].double())
    row = 0
    for i, n in enumerate(new):
        at = torch.arange(past[i], past[i] + n, device=DEV)
        ids = st["table"][i].long()[at // ps]
        for name, x in (("k", k), ("v", v)):
            pools[name][ids, :, at % ps] = x[row:row + n].double()
        row += n
    return dict(out, **pools)


def _exact_attention(st):
    c = st["case"]
    h, kvh, d = c["heads"], c["kv_heads"], c["d"]
    new, past = _lens(c)
    out = torch.empty(st["rows"], h, d, dtype=torch.float64, device=DEV)
    row = 0
    for n, p, i in zip(new, past, range(c["b"])):
        if n == 0:
            continue
        k, v = _history64(st, i, n + p)
        mask = torch.ones(n, n + p, dtype=torch.bool, device=DEV).tril(p)
        for j in range(kvh):
            heads = slice(j * (h // kvh), (j + 1) * (h // kvh))
            q = st["q"].view(-1, h, d)[row:row + n, heads].double().transpose(0, 1)
            s = (q @ k[:, j].T) * d ** -0.5
            out[row:row + n, heads] = (s.masked_fill(~mask, -math.inf).softmax(-1) @ v[:, j]).transpose(0, 1)
        row += n
    return out.flatten(1)


def _exact_gemv(st):
    c = st["case"]
    n, k, epi = c["n"], c["k"], c["epi"]
    y = torch.empty(c["m"], n, dtype=torch.float64, device=DEV)
    x = st["x"].double()
    nib = [0, 4, 1, 5, 2, 6, 3, 7]  # nibble of a word's element 0..7
    for t in range(-(-n // 128)):
        tile = st["w"][t]
        b = tile[:, :4096].reshape(k // 64, 128, 8, 4).long()
        word = b[..., 0] + b[..., 1] * 256 + b[..., 2] * 65536 + b[..., 3] * 16777216
        code = torch.stack([torch.div(word, 16 ** q, rounding_mode="floor") % 16 for q in nib], -1)
        m = tile[:, 4096:].contiguous().view(torch.float16).view(k // 64, 128, 2).double()
        w = (code.flatten(2).double() * m[..., 1:] + m[..., :1]).half().double()
        w = w.transpose(0, 1).reshape(128, k)[: min(128, n - 128 * t)]
        y[:, 128 * t:128 * t + w.shape[0]] = x @ w.T
    if epi & EPI_BIAS:
        y += st["bias"].double()
    if epi & EPI_GELU:
        y = y * 0.5 * torch.special.erfc(-y / math.sqrt(2.0))
    if epi & EPI_RESIDUAL:
        y += st["res"].double()
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "gemv":
        return _exact_gemv(st)
    if case["op"] == "attention":
        return _exact_attention(st)
    if case["op"] == "append":
        return _exact_append(st)
    new, past = _lens(case)
    rows = [_history64(st, i, n + p) for i, (n, p) in enumerate(zip(new, past)) if n]
    return dict(k=torch.cat([r[0].flatten(1) for r in rows]), v=torch.cat([r[1].flatten(1) for r in rows]))
