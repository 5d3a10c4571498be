"""The paged cache's and the few-row product's refusals, and the index
arithmetic their kernels rest on (compiled for the host); no GPU."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x100000  # aligned placeholder; a refused call launches nothing


@pytest.fixture(scope="module")
def fq():
    from quantized_opt_decode_b200 import build
    build.build()
    from quantized_opt_decode_b200 import flexq
    return flexq


def parts(fq, **over):
    v = dict(h=512, heads=4, kv_bits=4, k=A, v=A, k_meta=A, v_meta=A, kv_heads=2, num_pages=8, page_size=16, table=A,
             table_ld=4, b=2, rows=8, max_new=4, max_len=64, row_start=A, kv_len=A)
    v.update(over)
    cfg = fq.flexq_config(h=v["h"], heads=v["heads"], ffn=1024, w_bits=4, kv_bits=v["kv_bits"], ln_eps=1e-5)
    kv = fq.flexq_paged_kv(v["k"], v["v"], v["k_meta"], v["v_meta"], v["kv_heads"], v["num_pages"], v["page_size"],
                           v["table"], v["table_ld"])
    batch = fq.flexq_ragged(v["b"], v["rows"], v["max_new"], v["max_len"], v["row_start"], v["kv_len"])
    return cfg, kv, batch


COMMON = [(dict(kv_heads=3), "kv_heads"), (dict(kv_heads=0), "kv_heads"), (dict(page_size=24), "page_size"),
          (dict(page_size=4), "page_size"), (dict(page_size=2048), "page_size"), (dict(num_pages=0), "num_pages"),
          (dict(k=None), "NULL"), (dict(v=A + 8), "aligned"), (dict(k_meta=None), "k_meta"),
          (dict(v_meta=A + 4), "k_meta"), (dict(b=-1), "b and rows"), (dict(rows=-1), "b and rows"),
          (dict(b=70000), "65535"), (dict(table=None), "table"), (dict(row_start=None), "row_start"),
          (dict(kv_len=A + 2), "kv_len"), (dict(max_new=0), "max_new"), (dict(max_len=0), "max_len"),
          (dict(rows=1 << 24, h=8192, heads=128), "rows * heads"), (dict(max_len=65), "exceeds a table row"), (dict(table_ld=0), "exceeds a table row"), (dict(heads=3), "heads")]


@pytest.mark.parametrize("over,word", COMMON)
def test_every_paged_call_checks_cache_and_batch(fq, over, word):
    cfg, kv, batch = parts(fq, **over)
    for call in (lambda: fq.flexq_paged_append(cfg, kv, batch, None, A, A, 256),
                 lambda: fq.flexq_paged_read(cfg, kv, batch, A, A, 256),
                 lambda: fq.flexq_attention_paged(cfg, kv, batch, A, 512, A + 4096, 512)):
        with pytest.raises(fq.FlexqError) as ei:
            call()
        assert ei.value.status == 1 and word in str(ei.value)


def test_null_descriptors_are_refused(fq):
    cfg, kv, batch = parts(fq)
    lib = fq._lib
    assert lib.flexq_attention_paged(None, C.byref(kv), C.byref(batch), A, 512, A, 512, None) == 1
    assert lib.flexq_attention_paged(C.byref(cfg), None, C.byref(batch), A, 512, A, 512, None) == 1
    assert lib.flexq_attention_paged(C.byref(cfg), C.byref(kv), None, A, 512, A, 512, None) == 1
    assert "batch" in fq.flexq_last_error()


def test_row_buffers_are_checked(fq):
    cfg, kv, batch = parts(fq)
    bad = [lambda: fq.flexq_paged_append(cfg, kv, batch, None, None, A, 256),
           lambda: fq.flexq_paged_append(cfg, kv, batch, None, A, A, 248),
           lambda: fq.flexq_paged_append(cfg, kv, batch, None, A, A + 2, 256),
           lambda: fq.flexq_paged_append(cfg, kv, batch, None, A, A, 260),
           lambda: fq.flexq_paged_append(cfg, kv, batch, None, A, A, 256, A, 512, A, 512),  # q without rope
           lambda: fq.flexq_paged_read(cfg, kv, batch, A, None, 256),
           lambda: fq.flexq_paged_read(cfg, kv, batch, A, A, 128),
           lambda: fq.flexq_attention_paged(cfg, kv, batch, A, 504, A + 4096, 512),
           lambda: fq.flexq_attention_paged(cfg, kv, batch, A, 512, None, 512),
           lambda: fq.flexq_attention_paged(cfg, kv, batch, A, 512, A + 4, 512),
           lambda: fq.flexq_attention_paged(cfg, kv, batch, A, 512, A, 512)]  # out over q
    for call in bad:
        with pytest.raises(fq.FlexqError) as ei:
            call()
        assert ei.value.status == 1


def test_rope_is_checked(fq):
    cfg, kv, batch = parts(fq)
    for args, word in (((A, 64, 24, 0), "rot_dim"), ((A, 64, 256, 0), "rot_dim"), ((A, 64, 0, 0), "rot_dim"),
                       ((None, 64, 64, 0), "table"), ((A + 4, 64, 64, 0), "table"), ((A, 0, 64, 0), "max_pos"),
                       ((A, 64, 64, 2), "interleaved")):
        with pytest.raises(fq.FlexqError) as ei:
            fq.flexq_paged_append(cfg, kv, batch, fq.flexq_rope(*args), A, A, 256)
        assert ei.value.status == 1 and word in str(ei.value)
    rope = fq.flexq_rope(A, 64, 64, 0)
    for q, ldq, qo, ldqo in ((A, 504, A + 4096, 512), (A, 512, None, 512), (A, 512, A, 520)):
        with pytest.raises(fq.FlexqError):
            fq.flexq_paged_append(cfg, kv, batch, rope, A, A, 256, q, ldq, qo, ldqo)


def test_empty_batches_do_nothing(fq):
    for over in (dict(b=0, row_start=None, kv_len=None, table=None), dict(rows=0, max_new=0, max_len=0)):
        cfg, kv, batch = parts(fq, **over)
        fq.flexq_paged_append(cfg, kv, batch, None, None, None, 0)
        fq.flexq_paged_read(cfg, kv, batch, None, None, 0)
        fq.flexq_attention_paged(cfg, kv, batch, None, 0, None, 0)


def test_pool_bytes(fq):
    for bits, per in ((4, 0.5 + 4 / 64), (16, 2.0)):
        cfg, _, _ = parts(fq, kv_bits=bits)
        assert fq.flexq_paged_kv_bytes(cfg, 2, 10, 16) == int(2 * per * 10 * 16 * 2 * 128)
    cfg, _, _ = parts(fq)
    assert fq.flexq_paged_kv_bytes(cfg, 3, 10, 16) == 0
    assert fq.flexq_paged_kv_bytes(cfg, 2, 0, 16) == 0
    assert fq.flexq_paged_kv_bytes(cfg, 2, 10, 12) == 0


def test_gemv_refusals(fq):
    ok = dict(x=A, ldx=128, w=A, m=4, n=256, k=128, bias=None, res=None, ld_res=0, epi=0, y=A, ldy=256)
    bad = [(dict(m=-1), 1, "m >= 0"), (dict(n=0), 1, "n > 0"), (dict(k=96), 1, "multiple of 64"),
           (dict(m=17), 5, "at most 16"), (dict(x=None), 1, "NULL"), (dict(w=None), 1, "NULL"), (dict(y=None), 1, "NULL"),
           (dict(ldx=120), 1, "ldx"), (dict(ldx=132), 1, "ldx"), (dict(x=A + 2), 1, "alignment"), (dict(w=A + 8), 1, "w must"),
           (dict(ldy=255), 1, "ldy"), (dict(epi=1), 1, "bias"), (dict(epi=4), 1, "residual"),
           (dict(epi=4, res=A, ld_res=255), 1, "residual"), (dict(epi=9, bias=A), 1, "fp32 output"),
           (dict(epi=16), 1, "flags"), (dict(y=A + 1), 1, "aligned"), (dict(y=A + 2, epi=8), 1, "aligned")]
    for over, status, word in bad:
        with pytest.raises(fq.FlexqError) as ei:
            fq.flexq_gemv_q4(*{**ok, **over}.values())
        assert ei.value.status == status and word in str(ei.value), over
    fq.flexq_gemv_q4(*{**ok, "m": 0, "x": None, "y": None}.values())


@pytest.fixture(scope="module")
def math_lib(tmp_path_factory):
    """csrc/paged_math.h compiled for the host."""
    d = tmp_path_factory.mktemp("paged_math")
    src = d / "m.cpp"
    src.write_text('#include "paged_math.h"\nusing namespace flexq;\nextern "C" {\n'
                   "int span(int a, int b, int c, int d, int e, int f) { return span_ok(a, b, c, d, e, f); }\n"
                   "int page(int p, int n) { return page_ok(p, n); }\n"
                   "long long base(int r, int i, int s, int h, int e) { return unit_base_at(r, i, s, h, e); }\n"
                   "long long total(int r, int b, int s, int h, int e) { return unit_total(r, b, s, h, e); }\n}\n")
    so = d / "m.so"
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I" + os.path.join(ROOT, "quantized_opt_decode_b200", "csrc"), str(src), "-o", str(so)], check=True)
    lib = C.CDLL(str(so))
    lib.base.restype = lib.total.restype = C.c_longlong
    return lib


def test_spans_and_pages_that_are_accepted_stay_in_range(math_lib):
    edge = [-2 ** 31, -5, -1, 0, 1, 3, 8, 9, 100, 2 ** 24, 2 ** 31 - 1]
    rows, max_new, max_len = 9, 8, 100
    for row0 in edge:
        for n in edge:
            for length in edge:
                ok = bool(math_lib.span(row0, n, length, rows, max_new, max_len))
                want = row0 >= 0 and 0 < n <= max_new and row0 + n <= rows and n <= length <= max_len
                assert ok == want, (row0, n, length)
    for p in edge:
        assert bool(math_lib.page(p, 100)) == (0 <= p < 100)


@pytest.mark.parametrize("scale,shift,extra", [(1, 3, 2), (1, 0, 0), (1, 7, 1), (7, 7, 1), (8, 6, 1), (56, 7, 1)])
def test_units_cover_every_sequence(math_lib, scale, shift, extra):
    """Sequence i's own unit numbers hold all its items, at any phase for the 8-token blocks."""
    rng = np.random.default_rng(scale * 100 + shift)
    size = 1 << shift
    for _ in range(200):
        b = int(rng.integers(1, 40))
        new = rng.integers(0, 3 * size + 2, b) * (rng.random(b) < 0.8)
        start = np.concatenate([[int(rng.integers(0, 5))], new]).cumsum()
        rows = int(start[-1]) + int(rng.integers(0, 4))
        base = [math_lib.base(int(s), i, scale, shift, extra) for i, s in enumerate(start)]
        assert base[0] >= 0
        assert math_lib.total(rows, b, scale, shift, extra) >= base[-1]
        for i in range(b):
            room = base[i + 1] - base[i]
            assert room >= 0
            if extra == 2:  # blocks of 8 positions from any first position
                need = max(((p0 + int(new[i]) - 1) // 8 - p0 // 8 + 1) if new[i] else 0 for p0 in range(8))
            else:
                need = -(-int(new[i]) * scale // size)
            assert room >= need, (i, new[i])
