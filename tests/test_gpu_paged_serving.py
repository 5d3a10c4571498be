"""The paged-cache operators and the few-row product together, as a server of
sequences that come and go runs them: whole layer steps over a changing ragged
batch against the oracle, captured graphs replayed with other lengths and
tables, two streams at once, and waits that run out."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import synth  # noqa: E402
import paged_helpers as ph  # noqa: E402
from oracle import opt  # noqa: E402
from gpu_helpers import assert_close, fq, to_dev, to_host  # noqa: E402
from quantized_opt_decode_b200.device_model import DeviceModel  # noqa: E402
from test_gpu_gemv import case as gemv_case, check as gemv_check  # noqa: E402
from test_gpu_paged import Dev, check_attention, same_bits  # noqa: E402

TOL = 2e-3  # the bar of the layer tests


class Server:
    """One layer's paged pool with a table that hands out pages as sequences grow."""

    def __init__(self, dm, kv_bits, page, pages, slots):
        self.dm, self.cfg, self.page, self.slots = dm, dm.cfg, page, slots
        h, heads = self.cfg.h, self.cfg.heads
        per = page * h
        u8 = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.bufs = [u8(pages * per // 2), u8(pages * per // 2), u8(pages * per // 16), u8(pages * per // 16)] \
            if kv_bits == 4 else [u8(pages * per * 2), u8(pages * per * 2)]
        assert sum(b.numel() for b in self.bufs) == fq.flexq_paged_kv_bytes(self.cfg, heads, pages, page)
        self.free = list(np.random.default_rng(page).permutation(pages))
        self.table = np.full((slots, 8), -1, np.int32)
        self.len = np.zeros(slots, np.int32)
        self.table_dev = to_dev(self.table)
        ptr = [b.data_ptr() for b in self.bufs] + [None] * (4 - len(self.bufs))
        self.kv = fq.flexq_paged_kv(*ptr, heads, pages, page, self.table_dev.data_ptr(), 8)

    def step(self, new, x):
        """Layer output rows for new[i] tokens of every slot, inputs x [rows][h]."""
        h, ffn, heads = self.cfg.h, self.cfg.ffn, self.cfg.heads
        self.len += np.array(new, np.int32)
        for i, n in enumerate(self.len):
            for p in range(-(-int(n) // self.page)):
                if self.table[i, p] < 0:
                    self.table[i, p] = self.free.pop()
        self.table_dev.copy_(torch.from_numpy(self.table))
        start = to_dev(np.cumsum([0] + list(new)).astype(np.int32))
        lens = to_dev(self.len)
        rows = len(x)
        batch = fq.flexq_ragged(self.slots, rows, max(new), int(self.len.max()), start.data_ptr(), lens.data_ptr())
        t = self.dm.layers[0].t
        w_bits = self.cfg.w_bits

        def linear(inp, w, n, k, bias, res, epi):
            y = torch.empty(rows, n, dtype=torch.float16, device="cuda")
            if rows <= 16 and w_bits == 4:
                fq.flexq_gemv_q4(inp, k, w, rows, n, k, bias, res, n, epi, y, n)
            else:
                nb = max(fq.flexq_linear_workspace(rows, n, k, w_bits, 0), 1)
                ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
                fq.flexq_linear(inp, k, w, w_bits, rows, n, k, bias, res, n, epi, y, n, ws, nb)
            return y

        xd = to_dev(x)
        u = torch.empty_like(xd)
        fq.flexq_layernorm(xd, h, t["ln1_g"], t["ln1_b"], u, h, rows, h)
        qkv = linear(u, t["w_qkv"], 3 * h, h, t["b_qkv"], None, 1)
        p = qkv.data_ptr()
        fq.flexq_paged_append(self.cfg, self.kv, batch, None, p + 2 * h, p + 4 * h, 3 * h)
        o = torch.empty_like(xd)
        fq.flexq_attention_paged(self.cfg, self.kv, batch, p, 3 * h, o, h)
        out = linear(o, t["w_o"], h, h, t["b_o"], xd, 5)
        v = torch.empty_like(xd)
        fq.flexq_layernorm(out, h, t["ln2_g"], t["ln2_b"], v, h, rows, h)
        mid = linear(v, t["w_fc1"], ffn, h, t["b_fc1"], None, 3)
        y = linear(mid, t["w_fc2"], h, ffn, t["b_fc2"], out, 5)
        fq.flexq_device_status()
        return to_host(y)

    def drop(self, i):
        self.free += [int(p) for p in self.table[i] if p >= 0]
        self.table[i] = -1
        self.len[i] = 0


@pytest.mark.parametrize("name,over,page", [
    ("tiny", {}, 16), ("tiny", dict(h=512, heads=4, ffn=2048), 32), ("tiny16", {}, 8),
    ("tiny16", dict(h=512, heads=4, ffn=2048), 64)])
def test_layer_steps_of_sequences_that_come_and_go(name, over, page):
    """Prompts, chunks, single tokens and idle slots by turns; a slot is given to a new
    sequence half way.  Every row against the oracle's prefill over its own sequence."""
    p = dict(synth.CONFIGS[name])
    p.update(over, prefill_kv_cache=True)
    dm = DeviceModel(p, b=1, max_len=8, layers=1)
    cfg = opt.Config.from_preset(p, ln1_f16=True)
    W = opt.effective_layer(cfg, opt.raw_layer(cfg, synth.config_seed(p), 0))
    rng = np.random.default_rng(7)
    srv = Server(dm, p["kv_bits"], page, 40, 4)
    seqs = [[] for _ in range(4)]  # (inputs, outputs) of every live sequence
    done = []
    plan = [(7, 19, 0, 1), (1, 1, 0, 1), (1, 0, 23, 1), (5, 30, 1, 0), "drop 1", (1, 1, 1, 1), (1, 9, 1, 0), (0, 1, 0, 0),
            (1, 1, 1, 1)]
    for new in plan:
        if new == "drop 1":
            done.append(seqs[1])
            seqs[1] = []
            srv.drop(1)
            continue
        x = rng.standard_normal((sum(new), cfg.h)).astype(np.float16)
        y = srv.step(new, x)
        at = 0
        for i, n in enumerate(new):
            if n:
                seqs[i].append((x[at:at + n], y[at:at + n]))
            at += n
    for s in seqs + done:
        x = np.concatenate([a for a, _ in s])
        y = np.concatenate([b for _, b in s])
        ref, _, _ = opt.layer_prefill(cfg, W, x[None].astype(np.float64))
        assert_close(y, ref[0], TOL)


def test_captured_step_replays_with_other_lengths_and_tables():
    """Append, both attention forms and the product in one graph, captured once
    under loose bounds and replayed over new tokens, lengths and pages; two graphs of the same
    calls replayed by turns."""
    heads, kvh, d, page, b, rows, L = 8, 2, 128, 16, 4, 96, 512
    h = heads * d
    pages = b * L // page + 3
    x, w, bias, res, wq, _ = gemv_case(6, 512, 1024, 1)
    xd, bd = to_dev(x), to_dev(bias)
    graphs = []
    for g in range(2):
        pg = ph.Paged(4, heads, kvh, d, page, (1,) * b, (0,) * b, seed=g, pad=rows - b)
        pg.pages = pages
        pools = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in
                 (pages * page * kvh * d // 2, pages * page * kvh * d // 2, pages * page * kvh * 8, pages * page * kvh * 8)]
        table = torch.full((b, L // page), -1, dtype=torch.int32, device="cuda")
        start = torch.zeros(b + 1, dtype=torch.int32, device="cuda")
        lens = torch.zeros(b, dtype=torch.int32, device="cuda")
        cfg = fq.flexq_config(h=h, heads=heads, ffn=4 * h, w_bits=4, kv_bits=4, ln_eps=1e-5)
        kv = fq.flexq_paged_kv(*[t.data_ptr() for t in pools], kvh, pages, page, table.data_ptr(), L // page)
        batch = fq.flexq_ragged(b, rows, 64, L, start.data_ptr(), lens.data_ptr())
        k, v = (torch.zeros(rows, kvh * d, dtype=torch.float16, device="cuda") for _ in "kv")
        q, o = (torch.zeros(rows, h, dtype=torch.float16, device="cuda") for _ in "qo")
        y = torch.zeros(6, 512, dtype=torch.float16, device="cuda")

        def step(s):
            fq.flexq_paged_append(cfg, kv, batch, None, k, v, kvh * d, stream=s)
            fq.flexq_attention_paged(cfg, kv, batch, q, h, o, h, stream=s)
            fq.flexq_gemv_q4(xd, 1024, wq, 6, 512, 1024, bd, None, 0, 1, y, 512, stream=s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(torch.cuda.current_stream())
        graphs.append((graph, pools, table, start, lens, k, v, q, o, y, cfg, kv, batch))
    rng = np.random.default_rng(3)
    perm = [rng.permutation(pages)[: b * L // page].reshape(b, -1).astype(np.int32) for _ in range(2)]
    past = np.zeros((2, b), int)
    hist = [[[[], []] for _ in range(b)] for _ in range(2)]
    for new in ((30, 1, 0, 64), (1, 1, 1, 1), (0, 40, 7, 1), (1, 0, 50, 1), (1, 1, 1, 1)):
        inputs = []
        for g, (graph, pools, table, start, lens, k, v, q, o, y, *_rest) in enumerate(graphs):
            n = np.array(new) if g == 0 else np.array(new)[::-1]
            kx, vx, qx = (rng.standard_normal((rows, wd)).astype(np.float16) for wd in (kvh * d, kvh * d, h))
            for t, a in ((k, kx), (v, vx), (q, qx), (table, perm[g])):
                t.copy_(torch.from_numpy(a))
            past[g] += n
            start.copy_(torch.from_numpy(np.cumsum([0] + list(n)).astype(np.int32)))
            lens.copy_(torch.from_numpy(past[g].astype(np.int32)))
            o.fill_(float("nan"))
            y.fill_(float("nan"))
            inputs.append((n, kx, vx, qx))
        for g in (0, 1):
            graphs[g][0].replay()
        torch.cuda.synchronize()
        fq.flexq_device_status()
        for g in (0, 1):
            n, kx, vx, qx = inputs[g]
            out = to_host(graphs[g][8])
            assert np.isnan(out[n.sum():]).all()
            row = 0
            for i in range(b):
                for s, a in enumerate((kx, vx)):
                    hist[g][i][s].append(a[row:row + n[i]])
                if n[i]:
                    kh, vh = (opt.cached_rows(_kv4(), np.concatenate(hist[g][i][s])) for s in (0, 1))
                    _check_rows(qx[row:row + n[i]], kh, vh, past[g][i] - n[i], heads, kvh, out[row:row + n[i]])
                row += n[i]
            gemv_check(x, w, bias, res, 6, 512, 1024, 1, to_host(graphs[g][9]))


def _kv4():
    p = dict(synth.CONFIGS["tiny"])
    return opt.Config.from_preset(p)


def _check_rows(q, kh, vh, past, heads, kvh, out):
    """attention_reference's bound for one sequence given its cached rows."""
    d = q.shape[1] // heads
    pg = ph.Paged(16, heads, kvh, d, 8, (len(q),), (past,), seed=0, spare=0)

    class One:
        pass
    one = One()
    one.__dict__.update(heads=heads, kv_heads=kvh, d=d, new=[len(q)], past=[past], row_start=[0])
    one.history = lambda i, **kw: (kh.reshape(-1, kvh, d).astype(np.float64), vh.reshape(-1, kvh, d).astype(np.float64))
    assert len(kh) == past + len(q) == pg.lens[0]
    ref, tol = ph.attention_reference(one, q, 0)
    assert (np.abs(out.astype(np.float64) - ref) <= tol).all()


def test_two_streams_at_once():
    """No call keeps anything that another one could disturb: the same bits alone and side by side."""
    jobs = []
    for seed, (heads, kvh, new, past) in enumerate([(8, 2, (1, 1, 80), (4000, 90, 300)), (4, 4, (200, 1), (700, 2500))]):
        pg = ph.Paged(4, heads, kvh, 128, 32, new, past, seed=seed)
        dv = Dev(pg)
        q = pg.new_rows()[2]
        qd, out = to_dev(q), torch.empty(pg.rows, heads * 128, dtype=torch.float16, device="cuda")
        x, w, bias, res, wq, _ = gemv_case(9, 640, 4096, 0, seed=seed)
        xd, y = to_dev(x), torch.empty(9, 640, dtype=torch.float16, device="cuda")
        jobs.append((pg, dv, q, qd, out, heads * 128, xd, wq, y, torch.cuda.Stream()))

    def run(job, stream):
        pg, dv, q, qd, out, h, xd, wq, y, _ = job
        fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, qd, h, out, h, stream=stream)
        fq.flexq_gemv_q4(xd, 4096, wq, 9, 640, 4096, None, None, 0, 0, y, 640, stream=stream)
    alone = []
    for job in jobs:
        run(job, None)
        alone.append((to_host(job[4]).copy(), to_host(job[8]).copy()))
        check_attention(job[0], job[2], alone[-1][0])
        job[4].fill_(float("nan"))
        job[8].fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(20):
        for job in jobs:
            run(job, job[9])
    torch.cuda.synchronize()
    fq.flexq_device_status()
    for job, (o, y) in zip(jobs, alone):
        same_bits(to_host(job[4]), o)
        same_bits(to_host(job[8]), y)


@pytest.mark.parametrize("op", ["product", "chunks", "chunks of a shared-out history", "many shared-out units"])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(op):
    if op == "product":
        x, w, bias, res, wq, _ = gemv_case(5, 640, 4096, 0)
        xd, out = to_dev(x), torch.empty(5, 640, dtype=torch.float16, device="cuda")
        run = lambda: fq.flexq_gemv_q4(xd, 4096, wq, 5, 640, 4096, None, None, 0, 0, out, 640)  # noqa: E731
    else:
        new, past = {"chunks": ((300, 150), (100, 20)), "many shared-out units": ((40,) * 30, (200,) * 30)}.get(
            op, ((20,), (6000,)))
        pg = ph.Paged(4, 2, 2, 128, 32, new, past, seed=2)
        if op == "many shared-out units":
            pg.table = np.concatenate([pg.table, np.full((pg.b, 1024), -1, np.int32)], 1)
            pg.table_ld = pg.table.shape[1]
        dv = Dev(pg, max_len=32768 if op == "many shared-out units" else None)
        q = pg.new_rows()[2]
        qd, out = to_dev(q), torch.empty(pg.rows, 256, dtype=torch.float16, device="cuda")
        run = lambda: fq.flexq_attention_paged(dv.cfg, dv.kv, dv.batch, qd, 256, out, 256)  # noqa: E731
    fq.flexq_device_status()
    try:
        fq.flexq_set_wait_limit_ns(1)
        run()
        with pytest.raises(fq.FlexqError) as ei:
            fq.flexq_device_status()
        assert ei.value.status == 4
    finally:
        fq.flexq_set_wait_limit_ns(0)
    out.fill_(float("nan"))
    run()
    fq.flexq_device_status()
    if op == "product":
        gemv_check(x, w, bias, res, 5, 640, 4096, 0, to_host(out))
    else:
        check_attention(pg, q, to_host(out))
