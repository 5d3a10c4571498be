"""Device-side inputs that break a ragged batch's promises (starts that decrease or are negative, more
new tokens than the bound): reported, and nothing is written outside the sequences that break them."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import paged_helpers as ph  # noqa: E402
from gpu_helpers import fq, to_dev, to_host  # noqa: E402
from test_gpu_paged import Dev, same_bits  # noqa: E402

NEW, PAST = (3, 1, 40), (20, 9, 300)
KINDS = {  # what changes in row_start, max_new, the sequences that stay as they should be (none where a start decreases)
    "a start that decreases": ({2: 2}, 64, ()),
    "a start far below": ({1: -2 ** 31}, 64, ()),
    "a last start that decreases": ({3: 0}, 64, ()),
    "a negative first start": ({0: -2}, 64, (1, 2)),
    "a first start behind the second": ({0: 4}, 64, ()),
    "more tokens than the bound": ({}, 4, (0, 1)),
    "more tokens than one": ({}, 1, (1,)),
}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bits,heads,kv_heads,d", [(4, 4, 2, 64), (16, 2, 2, 128), (4, 40, 2, 64)])
@pytest.mark.parametrize("op", ["append", "read", "attention"])
def test_broken_batches_are_reported_and_contained(kind, bits, heads, kv_heads, d, op):
    change, max_new, fine = KINDS[kind]
    good = ph.Paged(bits, heads, kv_heads, d, 16, NEW, PAST, seed=7, pad=5)
    dv = Dev(good, max_new=max_new)
    for at, value in change.items():
        dv.row_start[at] = value
    k, v, q = good.new_rows()
    kd, vd, qd = to_dev(k), to_dev(v), to_dev(q)
    width = heads * d if op == "attention" else kv_heads * d
    out, out2 = (torch.full((good.rows, width), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    before = [None if x is None else to_host(x).copy() for x in (dv.k, dv.v, dv.km, dv.vm)]
    torch.cuda.synchronize()
    if op == "append":
        fq.flexq_paged_append(dv.cfg, dv.kv, dv.batch, None, kd, vd, width)
    elif op == "read":
        fq.flexq_paged_read(dv.cfg, dv.kv, dv.batch, out, out2, width)
    else:
        fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, qd, width, out, width)
    with pytest.raises(fq.FlexqError) as ei:
        fq.flexq_device_status()
    assert ei.value.status == 6
    fq.flexq_device_status()  # read and cleared
    after = [None if x is None else to_host(x) for x in (dv.k, dv.v, dv.km, dv.vm)]
    # rows behind the batch, and pages of no sequence (or, but for an append, of any)
    rows = to_host(out)
    assert np.isnan(rows[good.row_start[-1]:]).all()
    owned = np.zeros(good.pages, bool)
    if op == "append":
        for i in range(good.b):
            owned[good.table[i][good.table[i] >= 0]] = True
    for a, b in zip(after, before):
        if a is not None:
            same_bits(a[~owned], b[~owned])
    pools, _ = ph.append_reference(good, k, v)
    for i in fine:
        r = slice(good.row_start[i], good.row_start[i + 1])
        if op == "append":
            mine = good.table[i][good.table[i] >= 0]
            for a, w in zip(after, pools):
                if a is not None:
                    same_bits(a[mine], w[mine])
        elif op == "read":
            kh, vh = good.history(i)
            for got, want in ((out, kh), (out2, vh)):
                same_bits(to_host(got)[r], want[good.past[i]:].reshape(NEW[i], -1).astype(np.float16))
        else:
            ref, tol = ph.attention_reference(good, q, i)
            assert (np.abs(rows[r].astype(np.float64) - ref) <= tol).all()
