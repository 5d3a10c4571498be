"""Paged attention where its running softmax and its sums can go wrong: scores that outgrow
the exponent base inside a key tile, weights far below the largest, and long histories of
values of one sign, against 64 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import paged_helpers as ph  # noqa: E402
from paged_bounds import attention_rows  # noqa: E402
from gpu_helpers import fq, to_dev, to_host  # noqa: E402
from test_gpu_paged import Dev, check_attention  # noqa: E402


def set_levels(pg, i, level, boost):
    """Key p of sequence i becomes the constant vector level[p] (exact in both caches); its value
    is multiplied by 2^boost[p] (exact too)."""
    p = np.arange(pg.lens[i])
    at, sl = pg.table[i, p // pg.page], p % pg.page
    level, boost = np.asarray(level), np.asarray(boost, int)
    if pg.bits == 16:
        pg.k[at, :, sl] = level[:, None, None]
        pg.v[at, :, sl] = np.ldexp(pg.v[at, :, sl], boost[:, None, None])
    else:
        pg.k[at, :, sl] = 0
        pg.km[at, :, sl, :, 0], pg.km[at, :, sl, :, 1] = level[:, None, None], 0
        pg.vm[at, :, sl] = np.ldexp(pg.vm[at, :, sl], boost[:, None, None, None])


# base-2 logarithms of the weights of 32-key pieces: they outgrow 2^8 at each piece of a tile,
# in the first tile and later ones, twice and three times in one, by more than fp16 can scale by
STEPS = [
    (0, 9, 9, 9, 9, 9, 9, 9),
    (0, 0, 9, 9, 9, 9, 9, 9),
    (0, 0, 0, 9, 9, 9, 9, 9),
    (0, 0, 0, 0, 9, 9, 9, 9),
    (0, 0, 0, 0, 0, 9, 18, 18),
    (0, 9, 18, 27, 27, 27, 27, 27),
    (0, 0, 0, 0, 0, 9, 18, 27),
    (0, 0, 0, 0, 26, 26, 26, 52),
    (0, 26, 26, 26, 26, 52, 52, 52),
    (40, 0, 49, 0, 10, 58, 0, 67),
]


@pytest.mark.parametrize("steps", STEPS)
@pytest.mark.parametrize("bits,d", [(4, 128), (4, 64), (16, 128), (16, 64)])
@pytest.mark.parametrize("new", [1, 40, 300])
def test_scores_that_outgrow_the_base_inside_a_tile(steps, bits, d, new):
    """Every piece's values are so much larger than the later ones' that each counts in the
    result: a piece whose weights are not scaled with the base shows."""
    past = 32 * len(steps)
    pg = ph.Paged(bits, 4, 2, d, 16, (new,), (past,), seed=len(steps) + sum(steps))
    log2 = np.concatenate([np.repeat(steps, 32), np.full(new, steps[-1])]).astype(float)
    boost = np.clip(max(steps) - log2, 0, 13)
    # scores q k / sqrt d of q = 1: a step of `log2` in base 2
    level = (log2 / np.log2(np.e) / np.sqrt(d)).astype(np.float16)
    set_levels(pg, 0, level, boost)
    q = np.ones((pg.rows, 4 * d), np.float16)
    # some rows see half or none of the growth, or its reverse: their bases move elsewhere or not at all
    q *= np.array([1, 0.5, 1, 0, 1, -0.25], np.float16)[np.arange(pg.rows) % 6][:, None]
    dv = Dev(pg)
    out = torch.full((pg.rows, 4 * d), float("nan"), dtype=torch.float16, device="cuda")
    fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, to_dev(q), 4 * d, out, 4 * d)
    fq.flexq_device_status()
    check_attention(pg, q, to_host(out))


@pytest.mark.parametrize("bits,d", [(4, 128), (4, 64), (16, 128), (16, 64)])
@pytest.mark.parametrize("jump", [22, 24.5, 26, 30])
@pytest.mark.parametrize("new", [1, 40, 300])
def test_weights_above_their_base_outlive_a_move_of_it(bits, d, jump, new):
    """The second and third piece of a tile reach 2^7.5 of the first one's base without moving
    it; the fourth moves it by 2^22 to 2^30.  Their weights are then 2^-14.5 to 2^-22.5 of the largest,
    and their values, of one sign, make up for it."""
    steps = [-20, -20, -20, -20, 0, 7.5, 7.5, jump]
    pg = ph.Paged(bits, 4, 2, d, 16, (new,), (256,), seed=int(2 * jump) + new)
    if bits == 16:
        pg.v = np.abs(pg.v)
    else:
        pg.vm[..., 0] = np.where(np.isnan(pg.vm[..., 0]), np.nan, 0)  # values: code * scale
    log2 = np.concatenate([np.repeat(steps, 32), np.full(new, jump)])
    boost = np.repeat([0, 0, 0, 0, 0, 12, 12, 0], 32).tolist() + [0] * new
    set_levels(pg, 0, (log2 / np.log2(np.e) / np.sqrt(d)).astype(np.float16), boost)
    q = np.ones((pg.rows, 4 * d), np.float16)
    dv = Dev(pg)
    out = torch.full((pg.rows, 4 * d), float("nan"), dtype=torch.float16, device="cuda")
    fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, to_dev(q), 4 * d, out, 4 * d)
    fq.flexq_device_status()
    check_attention(pg, q, to_host(out))


@pytest.mark.parametrize("bits,new", [(4, 1), (4, 20), (16, 1), (16, 20)])
@pytest.mark.parametrize("n,sink", [(32, 0), (33, 3), (128, 100), (131072, 70000)])
def test_a_flat_history_behind_one_large_weight(bits, new, n, sink):
    """Equal weights, 2^20 to 2^28 below that of one key whose value is zero: the result is what
    they sum up to, however many there are."""
    d = 128
    pg = ph.Paged(bits, 1, 1, d, 1024, (new,), (n - new,), seed=new, spare=1)
    if bits == 16:
        pg.v = np.abs(pg.v)
    else:
        pg.vm[..., 0] = np.where(np.isnan(pg.vm[..., 0]), np.nan, 0)  # values: code * scale
    at, sl = pg.where(0, sink)
    (pg.v if bits == 16 else pg.vm)[at, :, sl] = 0
    boost = 12 if n < 1000 else 0  # (else the result is below fp16)
    q = np.ones((new, d), np.float16)
    for below in (20, 25.25, 28):
        log2 = np.zeros(n)
        log2[sink] = below
        set_levels(pg, 0, (log2 / np.log2(np.e) / np.sqrt(d)).astype(np.float16), np.full(n, boost))
        boost = 0  # (the values keep it)
        dv = Dev(pg)
        out = torch.full((new, d), float("nan"), dtype=torch.float16, device="cuda")
        fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, to_dev(q), d, out, d)
        fq.flexq_device_status()
        k, v = pg.history(0)
        ref, tol = attention_rows(q, k[:, 0], v[:, 0], n - new)
        over = np.abs(to_host(out).astype(np.float64) - ref) / tol
        assert over.max() <= 1, (below, over.max())


def _positive_pool(bits, n, d, page=1024):
    """A pool whose pages 0, 1, .. hold n keys in (-1/2, 1/2) and values in (1/2, 3/2), on the device."""
    pages = -(-n // page)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n + bits)
    if bits == 16:
        k = (torch.rand(pages, 1, page, d, device="cuda", generator=gen) - 0.5).half()
        v = (torch.rand(pages, 1, page, d, device="cuda", generator=gen) + 0.5).half()
        return (k, v, None, None), k.view(-1, d)[:n].double(), v.view(-1, d)[:n].double()
    k = torch.randint(0, 256, (pages, 1, page, d // 2), device="cuda", generator=gen, dtype=torch.uint8)
    v = torch.randint(-2 ** 31, 2 ** 31 - 1, (pages, 1, page // 8, d), device="cuda", generator=gen, dtype=torch.int32)
    km, vm = (torch.tensor([lo, 1 / 15], device="cuda").half().repeat(pages, 1, page, d // 64, 1) for lo in (-0.5, 0.5))
    kc = torch.stack([k & 15, k >> 4], -1).reshape(-1, d)[:n]
    vc = ((v.view(pages, page // 8, 1, d) >> (4 * torch.arange(8, device="cuda").view(8, 1))) & 15).reshape(-1, d)[:n]
    value = lambda c, m: (c.float() * m[0, 0, 0, 0, 1].float() + m[0, 0, 0, 0, 0].float()).half().double()  # noqa: E731
    return (k, v, km, vm), value(kc, km), value(vc, vm)


def _long_history(bits, n, d, b, new, looked_at):
    """Signed relative errors of `looked_at` rows of b sequences of `new` tokens that share one history
    of n keys (the new tokens' among them)."""
    page = 1024
    bufs, k, v = _positive_pool(bits, n, d, page)
    pages = bufs[0].shape[0]
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(b, 1).contiguous()
    start = torch.arange(0, (b + 1) * new, new, dtype=torch.int32, device="cuda")
    lens = torch.full((b,), n, dtype=torch.int32, device="cuda")
    cfg = fq.flexq_config(h=2 * d, heads=2, ffn=8 * d, w_bits=4, kv_bits=bits, ln_eps=1e-5)
    kv = fq.flexq_paged_kv(*[t if t is None else t.data_ptr() for t in bufs], 1, pages, page, table.data_ptr(), pages)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    q = (0.3 * torch.randn(b * new, 2 * d, device="cuda", generator=gen)).half()
    out = torch.full_like(q, float("nan"))
    fq.flexq_attention_paged(cfg, kv, fq.flexq_ragged(b, b * new, new, n, start.data_ptr(), lens.data_ptr()), q, 2 * d, out,
                             2 * d)
    fq.flexq_device_status()
    rows = torch.linspace(0, b * new - 1, looked_at, device="cuda").long()
    s = q[rows].double().view(looked_at, 2, d) @ k.T / d ** 0.5
    s.masked_fill_(torch.arange(n, device="cuda") > (n - new + rows % new)[:, None, None], float("-inf"))
    ref = torch.softmax(s, -1) @ v
    return (out[rows].double().view(looked_at, 2, d) / ref - 1).cpu().numpy()


def check_drift(err):
    """Each error is that of one output: its rounding to fp16 (2^-11), the weights' (2^-11 at the most)
    and the sums' (2^-12), and a little for exponents of scores below 8 in size.  Their mean has
    no roundings to fp16 in it, which go up as often as down (a mean of N of them is below
    2^-11 * 4 / sqrt(3 N), four standard deviations, and the weights' are smaller still): what is left is what sums
    lose or gain in one direction, 2^-13 at the most."""
    assert np.abs(err).max() <= 2.0 ** -10 + 2.0 ** -12 + 2.0 ** -16, np.abs(err).max()
    noise = 2 * 2.0 ** -11 * 4 / np.sqrt(3 * err.size)
    assert abs(err.mean()) <= 2.0 ** -13 + noise, (err.mean(), noise)


@pytest.mark.parametrize("bits,n,d,b", [(4, 262144, 128, 4800), (16, 200000, 64, 4800), (4, 16385, 64, 4800),
                                        (4, 600000, 128, 3), (16, 17, 128, 300), (4, 300001, 64, 300)])
def test_single_tokens_over_long_histories_do_not_drift(bits, n, d, b):
    """Values of one sign, so that what a sum loses at each step shows; many sequences (few warps
    a history) and few."""
    check_drift(_long_history(bits, n, d, b, 1, min(b, 48)))


CHUNKS = [  # bits, keys, d, sequences, new tokens
    (4, 16384, 128, 3, 150), (4, 16385, 64, 160, 130), (16, 30000, 128, 300, 64), (16, 40000, 64, 2, 40),
    (4, 65537, 128, 90, 140), (4, 131072, 64, 2, 129), (16, 131073, 128, 1, 20), (4, 131082, 128, 2, 30),
    (4, 140000, 128, 20, 300), (16, 300000, 64, 1, 9), (4, 530000, 128, 1, 40), (4, 40000, 128, 160, 512),
    (16, 33000, 64, 170, 480), (4, 16500, 64, 200, 400)]


@pytest.mark.parametrize("bits,n,d,b,new", CHUNKS)
def test_chunks_over_long_histories_do_not_drift(bits, n, d, b, new):
    """The same for chunks: histories that one accumulator takes, that a cluster does, that it takes in
    pieces, the last of which some rows see nothing of, and that each of many CTAs takes alone."""
    check_drift(_long_history(bits, n, d, b, new, 48))


@pytest.mark.parametrize("bits,d", [(4, 128), (16, 64)])
def test_pieces_of_a_history_with_different_bases(bits, d):
    """Scores that grow and fall from piece to piece of 131072 keys, each of which counts."""
    n, new = 300000, 24
    pg = ph.Paged(bits, 1, 1, d, 1024, (new,), (n - new,), seed=2, spare=1) if d == 128 else \
        ph.Paged(bits, 2, 1, d, 1024, (new,), (n - new,), seed=2, spare=1)
    for level, boost in (((0, 9, 15), (9, 0, 0)), ((20, 0, 9), (0, 12, 3)), ((0, 3, -6), (0, 0, 4))):
        piece = np.minimum(np.arange(n) // 131072, 2)
        set_levels(pg, 0, (np.array(level, float)[piece] / np.log2(np.e) / np.sqrt(d)).astype(np.float16), np.array(boost)[piece])
        dv = Dev(pg)
        q = np.ones((new, pg.heads * d), np.float16)
        q[::3] *= -0.5
        out = torch.full((new, pg.heads * d), float("nan"), dtype=torch.float16, device="cuda")
        fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, to_dev(q), pg.heads * d, out, pg.heads * d)
        fq.flexq_device_status()
        k, v = pg.history(0)
        ref, tol = attention_rows(q[:, :d], k[:, 0], v[:, 0], n - new)
        over = np.abs(to_host(out)[:, :d].astype(np.float64) - ref) / tol
        assert over.max() <= 1, (level, over.max())
        set_levels(pg, 0, np.zeros(n), -np.array(boost)[piece])


@pytest.mark.parametrize("bits", [4, 16])
def test_long_histories_of_many_units_with_different_bases(bits):
    """The same where the units are many and each is one CTA's: scores that grow and fall every 16384
    keys, by more than fp32's range too, values that make up for it, and a bound far above the batch."""
    n, new, d, heads = 40000, 2400, 64, 64
    pg = ph.Paged(bits, heads, 1, d, 1024, (new,), (n - new,), seed=3, spare=1)
    pg.table = np.concatenate([pg.table, np.full((1, 100), -1, np.int32)], 1)
    pg.table_ld = pg.table.shape[1]
    rows = [0, 1, 2, 255, 256, 700, 1600, 1601, new - 1]
    for level, boost in (((0, 9, 15), (9, 0, 0)), ((20, 0, 9), (0, 12, 3)), ((0, 3, -6), (0, 0, 4)), ((0, 140, 131), (0, 0, 9)),
                         ((150, 0, 0), (0, 0, 0))):
        piece = np.minimum(np.arange(n) // 16384, 2)
        set_levels(pg, 0, (np.array(level, float)[piece] / np.log2(np.e) / np.sqrt(d)).astype(np.float16), np.array(boost)[piece])
        dv = Dev(pg, max_len=100000)
        q = np.ones((new, heads * d), np.float16)
        q[::3] *= -0.5
        out = torch.full((new, heads * d), float("nan"), dtype=torch.float16, device="cuda")
        fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, to_dev(q), heads * d, out, heads * d)
        fq.flexq_device_status()
        out = to_host(out).astype(np.float64).reshape(new, heads, d)
        assert (out == out[:, :1]).all()  # (the heads' queries are alike)
        k, v = pg.history(0)
        for t in rows:
            ref, tol = attention_rows(q[t:t + 1, :d], k[:, 0], v[:, 0], n - new + t)
            over = np.abs(out[t, 0] - ref[0]) / tol[0]
            assert over.max() <= 1, (level, t, over.max())
        set_levels(pg, 0, np.zeros(n), -np.array(boost)[piece])


def test_a_wait_that_runs_out_in_a_piece_is_reported_and_the_next_call_is_right():
    n, new, d, page = 270000, 20, 64, 1024
    bufs, k, v = _positive_pool(4, n, d, page)
    pages = bufs[0].shape[0]
    table = torch.arange(pages, dtype=torch.int32, device="cuda")
    start, lens = to_dev(np.array([0, new], np.int32)), to_dev(np.array([n], np.int32))
    cfg = fq.flexq_config(h=2 * d, heads=2, ffn=8 * d, w_bits=4, kv_bits=4, ln_eps=1e-5)
    kv = fq.flexq_paged_kv(*[t.data_ptr() for t in bufs], 1, pages, page, table.data_ptr(), pages)
    q = torch.randn(new, 2 * d, device="cuda").half()
    outs = [torch.full_like(q, float("nan")) for _ in range(2)]

    def run(out):
        fq.flexq_attention_paged(cfg, kv, fq.flexq_ragged(1, new, new, n, start.data_ptr(), lens.data_ptr()), q, 2 * d, out, 2 * d)
    run(outs[0])
    fq.flexq_device_status()
    try:
        fq.flexq_set_wait_limit_ns(1)
        run(outs[1])
        with pytest.raises(fq.FlexqError) as ei:
            fq.flexq_device_status()
        assert ei.value.status == 4
    finally:
        fq.flexq_set_wait_limit_ns(0)
    run(outs[1])
    fq.flexq_device_status()
    np.testing.assert_array_equal(to_host(outs[0]).view(np.uint16), to_host(outs[1]).view(np.uint16))


@pytest.mark.parametrize("bits,d", [(16, 128), (16, 64)])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_at_the_documented_limit_give_averages_of_values(bits, d, new, sign):
    """Scores of nearly 2^22, whose last bit is half a power of two of a weight and more: the weights' own
    size is anyone's, but no weight leaves fp16's range and each result lies among the values (up to the
    weights' rounding and the output's, 2^-11 each)."""
    n = 700
    pg = ph.Paged(bits, 2, 1, d, 16, (new,), (n - new,), seed=d + new)
    p = np.arange(n)
    at, sl = pg.table[0, p // 16], p % 16
    q = np.full((new, 2 * d), 1000.0, np.float16)
    q[:, 0] = q[:, d] = 64  # one dimension that tells the keys apart: steps of 2 to 3 in the weights' exponent
    size = 2.0 ** 21.9 * np.sqrt(d) / (1000.0 * (d - 1))
    pg.k[at, :, sl] = np.float16(sign * size)
    pg.k[at, :, sl, 0] = (sign * size + np.random.default_rng(0).integers(0, 4, n) * 0.25).astype(np.float16)[:, None]
    dv = Dev(pg)
    out = torch.full((new, 2 * d), float("nan"), dtype=torch.float16, device="cuda")
    fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, to_dev(q), 2 * d, out, 2 * d)
    fq.flexq_device_status()
    k, v = pg.history(0)
    s = np.abs(q[0, :d].astype(float) @ k[0, 0]) / np.sqrt(d)
    assert 2.0 ** 21.5 < s < 2.0 ** 22
    got = to_host(out).astype(float).reshape(new, 2, d)
    lo, hi = v[:, 0].min(0), v[:, 0].max(0)
    slack = 2.0 ** -10 * np.maximum(np.abs(lo), np.abs(hi))
    assert np.isfinite(got).all() and (got >= lo - slack).all() and (got <= hi + slack).all()


@pytest.mark.parametrize("level", [0.03, 0.05, 0.08])
@pytest.mark.parametrize("n,b,new", [(1600000, 200, 400), (1600000, 1, 20), (1600000, 2, 1), (400000, 4800, 1), (16384, 200, 400)])
def test_equal_weights_over_long_histories_do_not_drift(level, n, b, new):
    """Equal weights are the hardest for a running sum: each addition is rounded the same way.  The
    means over a history's dimensions, in which the outputs' roundings cancel, are off by the weight's
    one rounding to fp16 (2^-11) and the sums' 2^-12 at the most."""
    d, page = 64, 1024
    (k, v, km, vm), _, vd = _positive_pool(4, n, d, page)
    k.zero_()
    km.copy_(torch.tensor([level, 0.0], device="cuda").expand_as(km))
    pages = k.shape[0]
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(b, 1).contiguous()
    start = torch.arange(0, (b + 1) * new, new, dtype=torch.int32, device="cuda")
    lens = torch.full((b,), n, dtype=torch.int32, device="cuda")
    cfg = fq.flexq_config(h=2 * d, heads=2, ffn=8 * d, w_bits=4, kv_bits=4, ln_eps=1e-5)
    kv = fq.flexq_paged_kv(k.data_ptr(), v.data_ptr(), km.data_ptr(), vm.data_ptr(), 1, pages, page, table.data_ptr(), pages)
    q = torch.ones(b * new, 2 * d, device="cuda").half()
    out = torch.full_like(q, float("nan"))
    fq.flexq_attention_paged(cfg, kv, fq.flexq_ragged(b, b * new, new, n, start.data_ptr(), lens.data_ptr()), q, 2 * d, out,
                             2 * d)
    fq.flexq_device_status()
    for t in {0, new // 2, new - 1}:
        ref = vd[:n - new + t + 1].mean(0)
        err = (out[t].double().view(2, d) / ref - 1).cpu().numpy()
        assert np.abs(err).max() <= 2.0 ** -10 + 2.0 ** -12, np.abs(err).max()
        assert abs(err.mean()) <= 2.0 ** -11 + 2.0 ** -12, err.mean()
