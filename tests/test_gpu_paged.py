"""Paged KV cache on the GPU: append (with rotation and quantization), read-back
and attention of ragged batches against plain references: bit for bit where the
operation is defined bit for bit, 64-bit attention with bounds counted element
by element (paged_helpers.attention_reference) elsewhere."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import paged_helpers as ph  # noqa: E402
from gpu_helpers import f16_groups, fq, to_dev, to_host  # noqa: E402


class Dev:
    """A Paged case on the device with the library's descriptors."""

    def __init__(self, pg, max_new=None, max_len=None, rows=None):
        self.pg = pg
        self.k, self.v = to_dev(pg.k), to_dev(pg.v)
        self.km = to_dev(pg.km) if pg.bits == 4 else None
        self.vm = to_dev(pg.vm) if pg.bits == 4 else None
        self.table, self.row_start, self.kv_len = to_dev(pg.table), to_dev(pg.row_start), to_dev(pg.kv_len)
        h = pg.heads * pg.d
        self.cfg = fq.flexq_config(h=h, heads=pg.heads, ffn=4 * h, w_bits=4, kv_bits=pg.bits, ln_eps=1e-5)
        p = lambda x: None if x is None else x.data_ptr()  # noqa: E731
        self.kv = fq.flexq_paged_kv(p(self.k), p(self.v), p(self.km), p(self.vm), pg.kv_heads, pg.pages, pg.page,
                                    p(self.table), pg.table_ld)
        self.batch = fq.flexq_ragged(pg.b, pg.rows if rows is None else rows, max_new or max(max(pg.new), 1),
                                     max_len or max(max(pg.lens), 1), p(self.row_start), p(self.kv_len))


def same_bits(got, want):
    got, want = np.ascontiguousarray(got), np.ascontiguousarray(want)
    assert got.dtype == want.dtype and got.shape == want.shape
    np.testing.assert_array_equal(got.view(np.uint8), want.view(np.uint8))


def check_attention(pg, q, out, **pools):
    """Every row of the batch within its bound; rows outside as they were (NaN)."""
    assert np.isnan(out[: pg.row_start[0]]).all() and np.isnan(out[pg.row_start[-1]:]).all()
    for i in range(pg.b):
        if pg.new[i] == 0:
            continue
        ref, tol = ph.attention_reference(pg, q, i, **pools)
        got = out[pg.row_start[i]:pg.row_start[i] + pg.new[i]].astype(np.float64)
        assert np.isfinite(got).all(), f"sequence {i}: non-finite output"
        over = np.abs(got - ref) / tol
        at = np.unravel_index(np.argmax(over), over.shape)
        assert over[at] <= 1, (f"sequence {i} (new {pg.new[i]}, past {pg.past[i]}): element {at} is {got[at]:.6f}, "
                               f"reference {ref[at]:.6f}, {over[at]:.2f} of the bound")


APPEND = [
    # bits, heads, kv_heads, d, page, new, past, rot, interleaved
    (4, 2, 2, 128, 16, (1, 1, 1), (0, 7, 40), 0, 0),
    (4, 4, 2, 64, 8, (1, 0, 1, 1), (8, 3, 15, 16), 64, 0),
    (4, 6, 2, 128, 32, (3, 17, 0, 40, 1), (5, 0, 9, 30, 63), 128, 0),
    (4, 4, 4, 64, 16, (9, 8, 1, 7), (7, 8, 0, 25), 32, 1),
    (4, 2, 1, 128, 64, (130,), (3,), 48, 1),
    (16, 2, 2, 64, 8, (1, 1), (0, 9), 0, 0),
    (16, 8, 2, 128, 16, (5, 0, 33), (2, 6, 15), 128, 1),
    (16, 3, 3, 128, 256, (1, 20, 300), (255, 250, 0), 16, 0),
]


@pytest.mark.parametrize("bits,heads,kv_heads,d,page,new,past,rot,inter", APPEND)
def test_append_matches_the_codec_bit_for_bit(bits, heads, kv_heads, d, page, new, past, rot, inter):
    pg = ph.Paged(bits, heads, kv_heads, d, page, new, past, seed=len(new) * page + rot, front=2, pad=3)
    dv = Dev(pg)
    k, v, q = pg.new_rows()
    cs = ph.rope_table(max(pg.lens), max(rot, 16))
    csd = to_dev(cs)
    rope = fq.flexq_rope(csd.data_ptr(), cs.shape[0], rot, inter) if rot else None
    q_out = torch.full((pg.rows, heads * d), float("nan"), dtype=torch.float16, device="cuda")
    with_q = rope is not None
    fq.flexq_paged_append(dv.cfg, dv.kv, dv.batch, rope, to_dev(k), to_dev(v), kv_heads * d,
                          to_dev(q) if with_q else None, heads * d, q_out if with_q else None, heads * d)
    fq.flexq_device_status()
    pools, q_ref = ph.append_reference(pg, k, v, q if with_q else None, cs, rot, inter)
    for got, want in zip((dv.k, dv.v, dv.km, dv.vm), pools):
        if want is not None:
            same_bits(to_host(got), want)
    if with_q:
        qo = to_host(q_out)
        live = ~np.isnan(q_ref)
        same_bits(qo[live], q_ref[live])
        assert np.isnan(qo[~live]).all()


def test_append_rotates_queries_in_place():
    pg = ph.Paged(4, 4, 2, 128, 16, (5, 1, 9), (3, 0, 20), seed=3)
    dv = Dev(pg)
    k, v, q = pg.new_rows()
    cs = ph.rope_table(64, 128)
    csd, qd = to_dev(cs), to_dev(q)
    rope = fq.flexq_rope(csd.data_ptr(), 64, 128, 0)
    fq.flexq_paged_append(dv.cfg, dv.kv, dv.batch, rope, to_dev(k), to_dev(v), 256, qd, 512, qd, 512)
    fq.flexq_device_status()
    same_bits(to_host(qd), ph.append_reference(pg, k, v, q, cs, 128, 0)[1])


def test_append_from_a_fused_projection_buffer():
    """K and V as columns of one [rows][3h] buffer, the way the QKV projection leaves them."""
    pg = ph.Paged(4, 2, 2, 64, 16, (4, 11), (6, 0), seed=9)
    dv = Dev(pg)
    h = 128
    buf = (pg.rng.standard_normal((pg.rows, 3 * h + 8))).astype(np.float16)
    bd = to_dev(buf)
    p = bd.data_ptr()
    fq.flexq_paged_append(dv.cfg, dv.kv, dv.batch, None, p + 2 * h, p + 4 * h, 3 * h + 8)
    fq.flexq_device_status()
    pools, _ = ph.append_reference(pg, buf[:, h:2 * h], buf[:, 2 * h:3 * h])
    for got, want in zip((dv.k, dv.v, dv.km, dv.vm), pools):
        same_bits(to_host(got), want)


def test_append_special_values_follow_the_codec():
    """Constant groups, signed zeros, subnormals and the input range's ends."""
    pg = ph.Paged(4, 2, 2, 128, 16, (12,), (5,), seed=4)
    dv = Dev(pg)
    k, v, _ = pg.new_rows()
    rows = [np.full(64, 0.75), np.array([-0.0, 0.0] * 32), np.arange(64) * 2.0 ** -24, np.linspace(-32768, 32768, 64),
            np.full(64, -0.0), np.array([0.3, -1.7] * 32), np.full(64, 32768.0)]
    for r, x in enumerate(rows):
        k[r, 64:128], v[r, 0:64] = x.astype(np.float16), x.astype(np.float16)
    fq.flexq_paged_append(dv.cfg, dv.kv, dv.batch, None, to_dev(k), to_dev(v), 256)
    fq.flexq_device_status()
    for got, want in zip((dv.k, dv.v, dv.km, dv.vm), ph.append_reference(pg, k, v)[0]):
        same_bits(to_host(got), want)


@pytest.mark.parametrize("d,kv_heads", [(128, 4), (64, 6)])
def test_append_codes_at_every_magnitude_and_next_to_rounding_boundaries(d, kv_heads):
    """Groups of 1e-6 to 1e4 with the codec's special ones, subnormal scales, and groups whose
    elements sit on, just below and just above code + 1/2 steps of their scale."""
    n = 700
    pg = ph.Paged(4, kv_heads, kv_heads, d, 64, (n,), (3,), seed=12)
    dv = Dev(pg)
    rng = np.random.default_rng(5)
    width = kv_heads * d
    k = f16_groups(rng, n * width // 64).reshape(n, width)
    sc = rng.integers(1, 0x6000, n * width // 64).astype(np.uint16).view(np.float16).astype(np.float64)[:, None]
    lo = rng.choice([0.0, -7.5, 3.0, -15.0], (len(sc), 1)) * sc
    x = (lo + (rng.integers(0, 16, (len(sc), 64)) + rng.choice([0.0, 0.5], (len(sc), 64))) * sc)
    x[:, 0], x[:, 1] = lo[:, 0], lo[:, 0] + 15 * sc[:, 0]
    x = np.clip(x, -32768, 32768).astype(np.float16)
    nudge = rng.integers(-2, 3, x.shape).astype(np.int16) * (np.abs(x) > 1e-6) * (np.abs(x) < 3e4)
    v = np.ascontiguousarray((x.view(np.int16) + nudge.astype(np.int16)).view(np.float16)).reshape(n, width)
    fq.flexq_paged_append(dv.cfg, dv.kv, dv.batch, None, to_dev(k), to_dev(v), width)
    fq.flexq_device_status()
    for got, want in zip((dv.k, dv.v, dv.km, dv.vm), ph.append_reference(pg, k, v)[0]):
        same_bits(to_host(got), want)


@pytest.mark.parametrize("bits,heads,kv_heads,d,page,new,past", [
    (4, 2, 2, 128, 16, (1, 1, 1), (0, 7, 40)), (4, 2, 2, 64, 8, (3, 0, 30), (5, 2, 1)),
    (4, 2, 1, 128, 64, (200, 1), (0, 70)), (16, 4, 4, 64, 32, (1, 64, 5), (31, 0, 30)),
    (16, 2, 2, 128, 8, (1, 1), (9, 0)), (4, 5, 5, 128, 1024, (70, 1025), (0, 0))])
def test_read_returns_the_cached_values(bits, heads, kv_heads, d, page, new, past):
    pg = ph.Paged(bits, heads, kv_heads, d, page, new, past, seed=page, front=1, pad=2)
    dv = Dev(pg)
    outs = [torch.full((pg.rows, kv_heads * d + 8), float("nan"), dtype=torch.float16, device="cuda") for _ in "kv"]
    fq.flexq_paged_read(dv.cfg, dv.kv, dv.batch, *outs, kv_heads * d + 8)
    fq.flexq_device_status()
    want = [np.full((pg.rows, kv_heads * d + 8), np.nan, np.float16) for _ in "kv"]
    for i in range(pg.b):
        for w, hist in zip(want, pg.history(i)):
            w[pg.row_start[i]:pg.row_start[i] + new[i], :kv_heads * d] = (
                hist[past[i]:].reshape(new[i], kv_heads * d).astype(np.float16))
    for got, w in zip(outs, want):
        g = to_host(got)
        live = ~np.isnan(w)
        same_bits(g[live], w[live])
        assert np.isnan(g[~live]).all()


ATTN = [
    # bits, heads, kv_heads, d, page, new, past
    (4, 2, 2, 128, 16, (1,), (0,)),
    (4, 2, 2, 128, 16, (1, 1, 1, 1), (0, 6, 15, 16)),
    (4, 2, 2, 64, 8, (1, 1, 0, 1), (31, 100, 5, 517)),
    (4, 8, 2, 128, 32, (1, 1, 1), (33, 700, 64)),
    (4, 7, 1, 128, 64, (1, 1), (1300, 3)),
    (4, 32, 2, 64, 128, (1, 1), (300, 5)),
    (4, 4, 4, 128, 16, (1,), (5000,)),
    (16, 2, 2, 128, 16, (1, 1, 1), (0, 40, 333)),
    (16, 4, 1, 64, 8, (1, 0, 1), (127, 3, 900)),
    (16, 24, 2, 128, 256, (1,), (2000,)),
    (4, 2, 2, 128, 16, (5, 1, 0, 70), (11, 64, 9, 0)),
    (4, 8, 2, 128, 64, (33, 130, 1), (100, 7, 400)),
    (4, 2, 2, 64, 8, (129, 64, 2), (0, 63, 65)),
    (4, 7, 7, 128, 32, (65,), (190,)),
    (4, 3, 1, 128, 16, (50, 3, 1, 1), (1, 260, 8, 0)),
    (4, 16, 1, 64, 128, (40, 17), (0, 333)),
    (16, 2, 2, 128, 16, (100, 1, 31), (0, 64, 33)),
    (16, 10, 2, 64, 64, (77, 128), (51, 0)),
    (16, 6, 2, 128, 8, (260,), (129,)),
    (4, 2, 2, 128, 1024, (300, 200), (900, 0)),
]


@pytest.mark.parametrize("bits,heads,kv_heads,d,page,new,past", ATTN)
def test_attention_against_64_bits(bits, heads, kv_heads, d, page, new, past):
    pg = ph.Paged(bits, heads, kv_heads, d, page, new, past, seed=sum(past) + heads, front=1, pad=2)
    dv = Dev(pg)
    q = pg.new_rows()[2]
    out = torch.full((pg.rows, heads * d), float("nan"), dtype=torch.float16, device="cuda")
    fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, to_dev(q), heads * d, out, heads * d)
    fq.flexq_device_status()
    check_attention(pg, q, to_host(out))


SHARED = [
    # long histories of few units, which are shared out over a cluster; groups of more than 16
    # heads; both row tiles and one, of a unit; sequences on either side of the few-row limit
    (4, 24, 1, 128, 16, (1,), (3000,)),
    (16, 32, 1, 64, 32, (3, 1), (5000, 70)),
    (4, 2, 2, 64, 256, (40,), (9000,)),
    (4, 2, 2, 128, 64, (9, 8, 1), (4100, 2000, 7000)),
    (16, 4, 2, 128, 128, (300,), (2500,)),
    (16, 2, 2, 128, 16, (130, 1), (3000, 6000)),
    (4, 20, 1, 64, 8, (1, 2, 0, 13), (129, 640, 50, 0)),
    (4, 14, 2, 128, 32, (2, 3, 1), (500, 31, 64)),
    (4, 12, 1, 128, 16, (1, 1), (15000, 10)),
    (4, 70, 1, 64, 64, (1, 30), (700, 3)),
    (16, 17, 1, 128, 8, (1, 1), (64, 63)),
]


@pytest.mark.parametrize("bits,heads,kv_heads,d,page,new,past", SHARED)
def test_attention_of_shared_out_histories_and_wide_groups(bits, heads, kv_heads, d, page, new, past):
    test_attention_against_64_bits(bits, heads, kv_heads, d, page, new, past)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("scale", [0.0, 1e-4, 12.0])
@pytest.mark.parametrize("new,past", [((1, 1), (300, 17)), ((70, 3), (90, 5))])
def test_attention_of_flat_tiny_and_peaked_scores(bits, scale, new, past):
    """Equal weights over a history, queries near fp16's subnormals, one key that takes all."""
    pg = ph.Paged(bits, 4, 2, 128, 16, new, past, seed=7)
    dv = Dev(pg)
    q = pg.new_rows(scale)[2]
    out = torch.full((pg.rows, 512), float("nan"), dtype=torch.float16, device="cuda")
    fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, to_dev(q), 512, out, 512)
    fq.flexq_device_status()
    check_attention(pg, q, to_host(out))


@pytest.mark.parametrize("new,past", [((1, 1, 1), (200, 90, 64)), ((40, 3, 1), (100, 80, 64))])
def test_shared_prefix_pages_and_row_strides(new, past):
    """Sequences that share read-only pages; q and out inside wider rows."""
    pg = ph.Paged(4, 4, 4, 64, 16, new, past, seed=11, share=4)
    dv = Dev(pg)
    q = pg.new_rows()[2]
    wide = np.full((pg.rows, 256 + 24), np.nan, np.float16)
    wide[:, 8:264] = q
    out = torch.full((pg.rows, 256 + 40), float("nan"), dtype=torch.float16, device="cuda")
    qd = to_dev(wide)
    fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, qd.data_ptr() + 16, 280, out.data_ptr() + 32, 296)
    fq.flexq_device_status()
    o = to_host(out)
    assert np.isnan(o[:, :16]).all() and np.isnan(o[:, 272:]).all()
    check_attention(pg, q, o[:, 16:272])


@pytest.mark.parametrize("max_new,max_len", [(1, 4000), (64, 600), (600, 4000)])
def test_loose_bounds_give_the_same_rows(max_new, max_len):
    """Bounds far above the batch's own, as a captured graph has them."""
    pg = ph.Paged(4, 4, 2, 128, 16, (1, 1, 1, 0), (99, 0, 260, 3), seed=5, pad=100)
    pg.table = np.concatenate([pg.table, np.full((4, 300), -1, np.int32)], 1)
    pg.table_ld = pg.table.shape[1]
    dv = Dev(pg, max_new=max_new, max_len=max_len)
    k, v, q = pg.new_rows()
    out = torch.full((pg.rows, 512), float("nan"), dtype=torch.float16, device="cuda")
    fq.flexq_paged_append(dv.cfg, dv.kv, dv.batch, None, to_dev(k), to_dev(v), 256)
    fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, to_dev(q), 512, out, 512)
    fq.flexq_device_status()
    pools, _ = ph.append_reference(pg, k, v)
    for got, want in zip((dv.k, dv.v, dv.km, dv.vm), pools):
        same_bits(to_host(got), want)
    check_attention(pg, q, to_host(out), k=pools[0], v=pools[1], km=pools[2], vm=pools[3])


@pytest.mark.parametrize("bits,heads,kv_heads,d", [(4, 16, 8, 128), (4, 12, 12, 64), (16, 8, 8, 128)])
def test_short_units_under_the_bound_of_a_very_long_one(bits, heads, kv_heads, d):
    """A cluster then shares out each of the several units it has, most with fewer tiles than CTAs:
    units of one and two row tiles, empty and single-token sequences between them."""
    new = (300, 1, 20, 0, 140, 64, 1, 9, 260, 100)
    past = (0, 40, 900, 7, 500, 0, 1300, 3000, 70, 260)
    pg = ph.Paged(bits, heads, kv_heads, d, 128, new, past, seed=heads, front=2, pad=9)
    pg.table = np.concatenate([pg.table, np.full((pg.b, 256), -1, np.int32)], 1)
    pg.table_ld = pg.table.shape[1]
    dv = Dev(pg, max_len=256 * 128)
    q = pg.new_rows()[2]
    qd = to_dev(q)
    outs = [torch.full((pg.rows, heads * d), float("nan"), dtype=torch.float16, device="cuda") for _ in range(3)]
    for out in outs:
        fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, qd, heads * d, out, heads * d)
    fq.flexq_device_status()
    check_attention(pg, q, to_host(outs[0]))
    for out in outs[1:]:
        same_bits(to_host(out), to_host(outs[0]))


def test_many_sequences():
    """More sequences than one probe round of the owner search covers."""
    rng = np.random.default_rng(0)
    b = 1100
    new = rng.integers(0, 4, b)
    new[::97] = 30
    past = rng.integers(0, 20, b)
    pg = ph.Paged(4, 2, 2, 64, 8, new, past, seed=1, pad=5)
    dv = Dev(pg)
    k, v, q = pg.new_rows()
    out = torch.full((pg.rows, 128), float("nan"), dtype=torch.float16, device="cuda")
    fq.flexq_paged_append(dv.cfg, dv.kv, dv.batch, None, to_dev(k), to_dev(v), 128)
    fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, to_dev(q), 128, out, 128)
    fq.flexq_device_status()
    pools, _ = ph.append_reference(pg, k, v)
    for got, want in zip((dv.k, dv.v, dv.km, dv.vm), pools):
        same_bits(to_host(got), want)
    check_attention(pg, q, to_host(out), k=pools[0], v=pools[1], km=pools[2], vm=pools[3])


def test_one_page_per_sequence_equals_the_block_cache():
    """Pages as long as the block cache's sequences: the appended bytes are those of
    flexq_kv_append, and decode attention agrees with flexq_attention_decode."""
    b, heads, d, L, n0 = 3, 2, 128, 64, 37
    h = heads * d
    rng = np.random.default_rng(2)
    cfg = fq.flexq_config(h=h, heads=heads, ffn=4 * h, w_bits=4, kv_bits=4, ln_eps=1e-5)
    nb = fq.flexq_kv_bytes(cfg, b, L)
    assert nb == fq.flexq_paged_kv_bytes(cfg, heads, b, L)
    def pool():
        return [torch.zeros(n, dtype=torch.uint8, device="cuda")
                for n in (b * L * h // 2, b * L * h // 2, b * L * h // 16, b * L * h // 16)]
    one, two = pool(), pool()
    slab = fq.flexq_kv(*[x.data_ptr() for x in one], b, L)
    table = torch.arange(b, dtype=torch.int32, device="cuda")
    paged = fq.flexq_paged_kv(*[x.data_ptr() for x in two], heads, b, L, table.data_ptr(), 1)
    x = to_dev(rng.standard_normal((2, b * n0, h)).astype(np.float16))
    start = torch.arange(0, (b + 1) * n0, n0, dtype=torch.int32, device="cuda")
    lens = torch.full((b,), n0, dtype=torch.int32, device="cuda")
    fq.flexq_kv_append(cfg, slab, x[0], x[1], h, b, 0, n0)
    fq.flexq_paged_append(cfg, paged, fq.flexq_ragged(b, b * n0, n0, L, start.data_ptr(), lens.data_ptr()), None,
                          x[0], x[1], h)
    for a, c in zip(one, two):
        same_bits(to_host(a), to_host(c))
    q = to_dev(rng.standard_normal((b, h)).astype(np.float16))
    o1, o2 = torch.empty_like(q), torch.empty_like(q)
    start1 = torch.arange(b + 1, dtype=torch.int32, device="cuda")
    fq.flexq_attention_decode(cfg, slab, q, h, b, n0, o1, h)
    fq.flexq_attention_paged(cfg, paged, fq.flexq_ragged(b, b, 1, L, start1.data_ptr(), lens.data_ptr()), q, h, o2, h)
    fq.flexq_device_status()
    assert np.linalg.norm(to_host(o1).astype(float) - to_host(o2).astype(float)) < 2e-3 * np.linalg.norm(to_host(o1).astype(float))


def _bad(kind):
    pg = ph.Paged(4, 2, 2, 64, 16, (3, 1, 4), (20, 9, 5), seed=6)
    if kind == "page below the pool":
        pg.table[1, 0] = -1
    elif kind == "page above the pool":
        pg.table[1, 0] = pg.pages
    elif kind == "length below the new tokens":
        pg.kv_len[1] = 0
    elif kind == "length above the bound":
        pg.kv_len[1] = 10 ** 6
    elif kind == "rows past the buffer":
        pg.row_start[3] = pg.rows + 5
    return pg


@pytest.mark.parametrize("kind", ["page below the pool", "page above the pool", "length below the new tokens",
                                  "length above the bound", "rows past the buffer"])
@pytest.mark.parametrize("op", ["append", "read", "attention"])
def test_bad_device_side_inputs_are_reported_and_contained(kind, op):
    """The bad sequence is reported; the first one's rows come out as they should."""
    pg = _bad(kind)
    dv = Dev(pg)
    k, v, q = pg.new_rows()
    out = torch.full((pg.rows, 128), float("nan"), dtype=torch.float16, device="cuda")
    out2 = torch.empty_like(out)
    if op == "append":
        fq.flexq_paged_append(dv.cfg, dv.kv, dv.batch, None, to_dev(k), to_dev(v), 128)
    elif op == "read":
        fq.flexq_paged_read(dv.cfg, dv.kv, dv.batch, out, out2, 128)
    else:
        fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, to_dev(q), 128, out, 128)
    with pytest.raises(fq.FlexqError) as ei:
        fq.flexq_device_status()
    assert ei.value.status == 6
    fq.flexq_device_status()  # read and cleared
    if op == "attention":
        ref, tol = ph.attention_reference(pg, q, 0)
        assert (np.abs(to_host(out)[:3].astype(float) - ref) <= tol).all()
    elif op == "read":
        assert np.array_equal(to_host(out)[:3].astype(float), pg.history(0)[0][20:].reshape(3, -1))


def test_rotation_past_the_table_is_reported():
    pg = ph.Paged(4, 2, 2, 64, 16, (3, 1), (20, 9), seed=6)
    dv = Dev(pg)
    k, v, _ = pg.new_rows()
    csd = to_dev(ph.rope_table(22, 64))
    fq.flexq_paged_append(dv.cfg, dv.kv, dv.batch, fq.flexq_rope(csd.data_ptr(), 22, 64, 0), to_dev(k), to_dev(v), 128)
    with pytest.raises(fq.FlexqError) as ei:
        fq.flexq_device_status()
    assert ei.value.status == 6


@pytest.mark.parametrize("bits", [4, 16])
def test_offsets_past_32_bits(bits):
    """A pool whose last pages lie behind 4 GiB (and, for fp16, 2^31 elements)."""
    heads, d, page = 2, 128, 1024
    h = heads * d
    per = page * h // 2 if bits == 4 else page * h * 2  # bytes of a page of K
    pages = (5 << 30) // per
    kb = torch.zeros(pages * per, dtype=torch.uint8, device="cuda")
    vb = torch.zeros(pages * per, dtype=torch.uint8, device="cuda")
    metas = [torch.zeros(pages * page * h // 16, dtype=torch.uint8, device="cuda") for _ in "kv"] if bits == 4 else None
    cfg = fq.flexq_config(h=h, heads=heads, ffn=4 * h, w_bits=4, kv_bits=bits, ln_eps=1e-5)
    table = torch.tensor([[pages - 1, 0], [1, pages - 2]], dtype=torch.int32, device="cuda")
    kv = fq.flexq_paged_kv(kb.data_ptr(), vb.data_ptr(), metas[0].data_ptr() if metas else None,
                           metas[1].data_ptr() if metas else None, heads, pages, page, table.data_ptr(), 2)
    new = [70, 1030]
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, sum(new), h)).astype(np.float16)
    xd = to_dev(x)
    start = to_dev(np.array([0, 70, 1100], np.int32))
    lens = to_dev(np.array(new, np.int32))
    batch = fq.flexq_ragged(2, 1100, 1030, 1030, start.data_ptr(), lens.data_ptr())
    out = torch.empty(3, 1100, h, dtype=torch.float16, device="cuda")
    fq.flexq_paged_append(cfg, kv, batch, None, xd[0], xd[1], h)
    fq.flexq_paged_read(cfg, kv, batch, out[0], out[1], h)
    fq.flexq_attention_paged(cfg, kv, batch, xd[2], h, out[2], h)
    fq.flexq_device_status()
    got = to_host(out)
    pg = ph.Paged(bits, heads, heads, d, page, new, (0, 0), seed=1, spare=0)
    pools, _ = ph.append_reference(pg, x[0], x[1])
    names = dict(zip(("k", "v", "km", "vm"), pools))
    row = 0
    for i, n in enumerate(new):
        kh, vh = pg.history(i, **names)
        assert np.array_equal(got[0, row:row + n].astype(float), kh.reshape(n, -1))
        assert np.array_equal(got[1, row:row + n].astype(float), vh.reshape(n, -1))
        ref, tol = ph.attention_reference(pg, x[2], i, **names)
        assert (np.abs(got[2, row:row + n].astype(float) - ref) <= tol).all()
        row += n
    del kb, vb
    torch.cuda.empty_cache()


def test_results_repeat_and_streams_are_honoured():
    """The same call on another stream gives the same bits, ordered after work queued there."""
    pg = ph.Paged(4, 8, 2, 128, 16, (1, 1, 50), (3000, 77, 200), seed=8)
    dv = Dev(pg)
    q = pg.new_rows()[2]
    qd = to_dev(q)
    outs = []
    side = torch.cuda.Stream()
    for s in (None, side, side):
        late = torch.zeros_like(qd)
        out = torch.full((pg.rows, 1024), float("nan"), dtype=torch.float16, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(side if s else torch.cuda.current_stream()):
            big = torch.randn(4096, 4096, device="cuda")
            for _ in range(4):
                big = big @ big * 1e-3
            late.copy_(qd)
            fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, late, 1024, out, 1024, stream=s)
        outs.append(to_host(out))
    same_bits(outs[0], outs[1])
    same_bits(outs[0], outs[2])
    check_attention(pg, q, outs[0])
