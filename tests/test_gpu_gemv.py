"""flexq_gemv_q4 against a plain 64-bit product with the codec's fp16 weights.

The bound of an element counts: the fp32 sums of products, in any order and
tree of depth at most k/32 + 64 with each addition off by at most a step of
2^-23 (a truncating adder), (k/32 + 64) 2^-23 sum |w x|; bias, GELU (whose slope
is below 1.13 and whose erf is good to a few steps) and residual in fp32; and the
output's rounding, 2^-11 |y| in fp16 (2^-25 below its normal range) or 2^-24
|y| in fp32."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from gpu_helpers import fq, to_dev, to_host  # noqa: E402
from oracle import opt, q64  # noqa: E402


def case(m, n, k, epi, seed=0, ldx=None, ldy=None, ld_res=None, wscale=0.05, xscale=1.0):
    rng = np.random.default_rng(seed + m * 7 + n + k)
    ldx, ldy, ld_res = ldx or k, ldy or n, ld_res or n
    x = np.full((m, ldx), np.nan, np.float16)
    x[:, :k] = rng.standard_normal((m, k)) * xscale
    w = (rng.standard_normal((n, k)) * wscale + 0.01).astype(np.float16)
    bias = (rng.standard_normal(n) * 0.1).astype(np.float16)
    res = np.full((m, ld_res), np.nan, np.float16)
    res[:, :n] = rng.standard_normal((m, n))
    wq = torch.empty(fq.flexq_packed_weight_bytes(n, k), dtype=torch.uint8, device="cuda")
    fq.flexq_quantize_weight_q4(to_dev(w), n, k, wq)
    return x, w, bias, res, wq, (ldx, ldy, ld_res)


def check(x, w, bias, res, m, n, k, epi, got):
    we = q64.roundtrip(w).astype(np.float64)
    xe = x[:, :k].astype(np.float64)
    ref = xe @ we.T
    tol = (k / 32 + 64) * 2.0 ** -23 * (np.abs(xe) @ np.abs(we).T)
    size = np.abs(ref)
    if epi & 1:
        ref = ref + bias.astype(np.float64)
        size = size + np.abs(ref)
    if epi & 2:
        tol = 1.13 * tol + 2.0 ** -21 * np.abs(ref)
        ref = opt.gelu(ref)
    if epi & 4:
        ref = ref + res[:, :n].astype(np.float64)
        size = size + np.abs(ref)
    tol = tol + 2.0 ** -22 * size
    tol = tol + (2.0 ** -24 * np.abs(ref) if epi & 8 else 2.0 ** -11 * np.abs(ref) + 2.0 ** -25)
    g = got.astype(np.float64)
    assert np.isfinite(g).all()
    over = np.abs(g - ref) / tol
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 1, f"element {at}: {g[at]} against {ref[at]}, {over[at]:.2f} of the bound"


CASES = [(m, n, k, e) for m, n, k, e in [
    (1, 128, 64, 1), (1, 1, 64, 0), (2, 2048, 2048, 5), (3, 130, 192, 8), (4, 200, 4096, 3), (5, 1000, 320, 7),
    (7, 257, 8192, 1), (8, 512, 128, 5), (9, 384, 640, 8), (12, 50, 1024, 2), (15, 640, 2112, 1), (16, 1281, 256, 5),
    (16, 128, 28672, 4), (1, 7168, 7168, 1), (6, 50272, 256, 8), (1, 64, 49152, 0), (16, 5000, 704, 3),
    (1, 16384, 4096, 3), (2, 17, 128, 7), (13, 2048, 64, 8)]]


@pytest.mark.parametrize("m,n,k,epi", CASES)
def test_gemv_against_64_bits(m, n, k, epi):
    x, w, bias, res, wq, (ldx, ldy, ld_res) = case(m, n, k, epi)
    y = torch.full((m, n), float("nan"), dtype=torch.float32 if epi & 8 else torch.float16, device="cuda")
    fq.flexq_gemv_q4(to_dev(x), k, wq, m, n, k, to_dev(bias) if epi & 1 else None, to_dev(res) if epi & 4 else None,
                     n, epi, y, n)
    fq.flexq_device_status()
    check(x, w, bias, res, m, n, k, epi, to_host(y))


@pytest.mark.parametrize("m", range(1, 17))
def test_every_row_count(m):
    n, k, epi = 321, 448, 5
    x, w, bias, res, wq, _ = case(m, n, k, epi)
    y = torch.full((m + 1, n), float("nan"), dtype=torch.float16, device="cuda")
    fq.flexq_gemv_q4(to_dev(x), k, wq, m, n, k, to_dev(bias), to_dev(res), n, epi, y, n)
    got = to_host(y)
    assert np.isnan(got[m:]).all()
    check(x, w, bias, res, m, n, k, epi, got[:m])


@pytest.mark.parametrize("epi", [5, 8])
def test_row_strides_odd_bases_and_untouched_surroundings(epi):
    """x, residual and y inside wider rows, y and bias at odd element offsets."""
    m, n, k = 5, 203, 256
    x, w, bias, res, wq, (ldx, ldy, ld_res) = case(m, n, k, epi, ldx=264, ldy=211, ld_res=207)
    dt = torch.float32 if epi & 8 else torch.float16
    buf = torch.full((m * ldy + 1,), float("nan"), dtype=dt, device="cuda")
    bbuf = to_dev(np.concatenate([[np.float16(0)], bias]))
    fq.flexq_gemv_q4(to_dev(x), ldx, wq, m, n, k, bbuf[1:], to_dev(res), ld_res, epi, buf[1:], ldy)
    fq.flexq_device_status()
    got = to_host(buf)
    assert np.isnan(got[0])
    got = got[1:].reshape(m, ldy)
    assert np.isnan(got[:, n:]).all()
    check(x, w, bias, res, m, n, k, epi, got[:, :n])


def test_output_over_the_residual():
    m, n, k, epi = 3, 512, 1024, 4
    x, w, bias, res, wq, _ = case(m, n, k, epi)
    y = to_dev(res)
    fq.flexq_gemv_q4(to_dev(x), k, wq, m, n, k, None, y, n, epi, y, n)
    check(x, w, bias, res, m, n, k, epi, to_host(y))


@pytest.mark.parametrize("xscale,wscale", [(1e-6, 0.05), (1000.0, 8.0), (1.0, 1e-5)])
def test_ranges(xscale, wscale):
    """fp16 subnormal activations and weights, and large ones, into fp32."""
    m, n, k = 4, 300, 512
    x, w, bias, res, wq, _ = case(m, n, k, 8, xscale=xscale, wscale=wscale)
    y = torch.full((m, n), float("nan"), dtype=torch.float32, device="cuda")
    fq.flexq_gemv_q4(to_dev(x), k, wq, m, n, k, None, None, 0, 8, y, n)
    check(x, w, bias, res, m, n, k, 8, to_host(y))


def test_agrees_with_the_gemm_and_repeats():
    m, n, k, epi = 7, 1024, 2048, 1
    x, w, bias, res, wq, _ = case(m, n, k, epi)
    xd, bd = to_dev(x), to_dev(bias)
    ys = [torch.empty(m, n, dtype=torch.float16, device="cuda") for _ in range(3)]
    for y in ys[:2]:
        fq.flexq_gemv_q4(xd, k, wq, m, n, k, bd, None, 0, epi, y, n)
    nb = max(fq.flexq_linear_workspace(m, n, k, 4, 0), 1)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    fq.flexq_linear(xd, k, wq, 4, m, n, k, bd, None, 0, epi, ys[2], n, ws, nb)
    a, b, c = (to_host(y) for y in ys)
    assert np.array_equal(a.view(np.uint16), b.view(np.uint16))
    check(x, w, bias, res, m, n, k, epi, c)
    check(x, w, bias, res, m, n, k, epi, a)
