"""Keys and values that are not finite, or beyond the codec's range, in a paged append: they
stay in their own 64-element group, as in the block cache's append."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import paged_helpers as ph  # noqa: E402
from gpu_helpers import fq, to_dev, to_host  # noqa: E402
from test_gpu_paged import Dev, same_bits  # noqa: E402

INF, NAN = np.inf, np.nan
GROUPS = {
    "a NaN": {17: NAN}, "an infinity": {40: INF}, "minus infinity": {3: -INF}, "both infinities": {0: INF, 63: -INF},
    "NaN and infinity": {8: NAN, 9: INF}, "NaN in a constant group": {None: 0.75, 5: NAN}, "NaN among zeros": {None: 0, 31: NAN},
    "all NaN": {None: NAN}, "all infinite": {None: INF}, "all minus infinity": {None: -INF}, "all but one NaN": {None: NAN, 50: 2.5},
    "the ends of fp16": {0: 65504, 1: -65504}, "NaN in a group of subnormals": {None: 2.0 ** -24, 1: 2.0 ** -20, 2: NAN},
}


@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("d,group", [(64, 0), (128, 0), (128, 1)])
def test_non_finite_groups_are_stored_as_the_block_append_stores_them(name, d, group):
    """One such group of K and of V in the middle of an 8-token block: every byte as
    flexq_kv_append leaves it, and all but that group's as without it."""
    heads, b, L, n0, tok = 2, 1, 32, 21, 11
    h = heads * d
    cfg = fq.flexq_config(h=h, heads=heads, ffn=4 * h, w_bits=4, kv_bits=4, ln_eps=1e-5)
    x = np.random.default_rng(d).standard_normal((2, n0, h)).astype(np.float16)
    y = x.copy()
    at = slice(d + 64 * group, d + 64 * group + 64)  # of head 1
    for s in (0, 1):
        for e, value in GROUPS[name].items():
            y[s, tok, at][slice(None) if e is None else e] = value
    start, lens = to_dev(np.array([0, n0], np.int32)), to_dev(np.array([n0], np.int32))
    table = torch.zeros(1, dtype=torch.int32, device="cuda")
    sizes = (b * L * h // 2, b * L * h // 2, b * L * h // 16, b * L * h // 16)

    def stored(rows, paged):
        bufs = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes]
        xd = to_dev(rows)
        if paged:
            kv = fq.flexq_paged_kv(*[t.data_ptr() for t in bufs], heads, 1, L, table.data_ptr(), 1)
            fq.flexq_paged_append(cfg, kv, fq.flexq_ragged(1, n0, n0, L, start.data_ptr(), lens.data_ptr()), None,
                                  xd[0], xd[1], h)
        else:
            fq.flexq_kv_append(cfg, fq.flexq_kv(*[t.data_ptr() for t in bufs], b, L), xd[0], xd[1], h, b, 0, n0)
        fq.flexq_device_status()
        k, v, km, vm = [to_host(t) for t in bufs]
        v = v.view(np.uint32).reshape(heads, L // 8, 1, d) >> (4 * np.arange(8, dtype=np.uint32))[:, None] & 15
        return (k.reshape(heads, L, d // 2), v.reshape(heads, L, d), km.view(np.uint32).reshape(heads, L, d // 64),
                vm.view(np.uint32).reshape(heads, L, d // 64))
    got, want, clean = stored(y, True), stored(y, False), stored(x, True)
    for a, w in zip(got, want):
        same_bits(a, w)
    for a, c, wide in zip(got, clean, (32, 64, 1, 1)):
        a, c = a.copy(), c.copy()
        own = slice(wide * group, wide * (group + 1))
        a[1, tok, own] = c[1, tok, own] = 0
        same_bits(a, c)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("slot", range(8))
def test_a_non_finite_value_leaves_the_slots_around_it(bad, slot):
    """Slot `slot` of a partly filled block gets a group with a value that is not finite: the tokens
    that were there and the slots that no token owns keep their codes."""
    pg = ph.Paged(4, 2, 2, 128, 16, (1,), (8 + slot,), seed=slot)
    dv = Dev(pg)
    k, v, _ = pg.new_rows()
    pools, _ = ph.append_reference(pg, k, v)
    k[0, 70], v[0, 70] = bad, bad
    fq.flexq_paged_append(dv.cfg, dv.kv, dv.batch, None, to_dev(k), to_dev(v), 256)
    fq.flexq_device_status()
    page, at = pg.where(0, 8 + slot)
    for got, want in zip((dv.k, dv.v, dv.km, dv.vm), pools):
        got, want = to_host(got).copy(), want.copy()
        for a in (got, want):  # head 0, group 1 is the value's own
            if a.dtype == np.int32:
                a.view(np.uint32)[page, 0, at // 8, 64:] &= ~np.uint32(15 << 4 * (at % 8))
            else:
                a[page, 0, at, (32 if a.dtype == np.uint8 else 1):] = 0
        same_bits(got, want)


def test_rotated_keys_with_infinities():
    """An infinity becomes NaN in the rotation's pair; the rest of the row is what it was."""
    d, n0 = 128, 9
    pg = ph.Paged(4, 2, 2, d, 16, (n0,), (3,), seed=1)
    dv = Dev(pg)
    k, v, q = pg.new_rows()
    cs = ph.rope_table(64, 32)
    pools, _ = ph.append_reference(pg, k, v, None, cs, 32, 0)
    k[4, d + 5] = np.inf  # head 1, pair (5, 21)
    csd = to_dev(cs)
    fq.flexq_paged_append(dv.cfg, dv.kv, dv.batch, fq.flexq_rope(csd.data_ptr(), 64, 32, 0), to_dev(k), to_dev(v), 2 * d)
    fq.flexq_device_status()
    page, at = pg.where(0, 7)
    for name, got, want in zip(("k", "v", "km", "vm"), (dv.k, dv.v, dv.km, dv.vm), pools):
        got, want = to_host(got).copy(), want.copy()
        if name in ("k", "km"):  # head 1, group 0 is the pair's own
            own = slice(32 if name == "k" else 1)
            got[page, 1, at, own] = want[page, 1, at, own] = 0
        same_bits(got, want)
