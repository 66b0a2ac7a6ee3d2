"""Product of 8-bit operands (lf_matmul_f8) on the GPU against 64 bits.

Tolerances: a product of two e4m3 values is exact in fp32 (8 bits of mantissa).  The
tensor core adds 32 of them to the accumulator in one step, whose sum it may cut:
2^-23 of the magnitude sum |a b| per step; the two scalings add 2^-24 each, then comes
one rounding."""
import math

import numpy as np
import pytest

import paged_reference as ref

pytestmark = pytest.mark.gpu
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def operands(m, n, k, seed, scale=100.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    a, b = ((scale * r(x, k)).clamp(-448, 448).to(torch.float8_e4m3fn) for x in (m, n))
    return a, b, 0.01 * r(m).abs() + 1e-3, 0.01 * r(n).abs() + 1e-3


def run(a, b, sa, sb, out_dtype, out=None, stream=None):
    import torch
    import decode_persistent_sm_gb300 as lf
    m, k = a.shape
    n = b.shape[0]
    c = torch.full((m, n), 9.0, dtype=ref.torch_dtype(out_dtype), device="cuda") if out is None else out
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    lf.matmul_f8(a.data_ptr(), p(sa), b.data_ptr(), p(sb), c.data_ptr(), out_dtype, m, n, k, err.data_ptr(), stream)
    if stream is None:
        torch.cuda.synchronize()
        assert err.item() == 0
    return c


def check(a, b, sa, sb, out_dtype, c):
    import torch
    k = a.shape[1]
    sc = 1.0
    for s, at in ((sa, (slice(None), None)), (sb, (None, slice(None)))):
        if s is not None:
            sc = sc * s.double()[at]
    ad, bd = a.double(), b.double()
    want, mag = (ad @ bd.t()) * sc, (ad.abs() @ bd.abs().t()) * sc
    tol = mag * (2.0 ** -23 * (math.ceil(k / 32) + 2) + 2.0 ** -23)
    tol = tol + HALF[out_dtype] * (want.abs() + tol) + (2.0 ** -25 if out_dtype == "f16" else 0.0)
    got = c.double()
    bad = ~((got - want).abs() <= tol)
    worst = ((got - want).abs() / mag.clamp(min=1e-300)).max().item()
    assert not bad.any(), (bad.sum().item(), worst, bad.nonzero()[:5].tolist())


@pytest.mark.parametrize("out_dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (1, 64, 128), (5, 7, 48), (16, 8192, 4096), (17, 300, 144), (128, 256, 128),
                                   (129, 257, 272), (255, 130, 1024), (300, 1000, 4096), (1000, 5000, 512), (8, 70, 2048),
                                   (120, 4000, 96), (2000, 4100, 16)])
def test_products(m, n, k, out_dtype):
    a, b, sa, sb = operands(m, n, k, m + n + k)
    check(a, b, sa, sb, out_dtype, run(a, b, sa, sb, out_dtype))


def test_exact_integers():
    # whole numbers whose sums fp32 holds: every bit counts, and every element is the right one
    import torch
    m, n, k = 200, 520, 256
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = (torch.randint(-8, 9, (x, k), device="cuda", generator=g).float().to(torch.float8_e4m3fn) for x in (m, n))
    c = run(a, b, None, None, "f32")
    assert torch.equal(c.double(), a.double() @ b.double().t())


def test_without_scales_and_with_one():
    a, b, sa, sb = operands(40, 90, 208, 3, 1.0)
    for x, y in ((None, None), (sa, None), (None, sb)):
        check(a, b, x, y, "f32", run(a, b, x, y, "f32"))


def test_nothing_behind_the_result_is_written():
    import torch
    m, n, k = 130, 261, 160
    a, b, sa, sb = operands(m, n, k, 4)
    for dt in ("f32", "f16"):
        c = torch.full((m * n + 999,), 9.0, dtype=ref.torch_dtype(dt), device="cuda")
        run(a, b, sa, sb, dt, out=c)
        assert (c[m * n:] == 9.0).all()
        check(a, b, sa, sb, dt, c[:m * n].view(m, n))


def test_not_a_number_stays_in_its_row_and_column():
    import torch
    a, b, sa, sb = operands(140, 300, 320, 5)
    clean = run(a, b, sa, sb, "f32")
    a.view(torch.uint8)[3, 7] = 0x7f
    b.view(torch.uint8)[290, 319] = 0x7f
    sa[100] = math.inf
    c = run(a, b, sa, sb, "f32")
    hit = torch.zeros_like(c, dtype=torch.bool)
    hit[3], hit[:, 290] = True, True
    assert torch.isnan(c[hit]).all()
    hit[100] = True
    assert torch.equal(c[~hit], clean[~hit])


def test_results_beyond_the_type_become_infinite():
    import torch
    a, b = (torch.full((x, 64), 448.0, device="cuda").to(torch.float8_e4m3fn) for x in (4, 9))
    c = run(a, b, None, None, "f16")
    assert torch.isposinf(c).all()


def test_chained_on_a_stream_captured_and_repeated():
    import torch
    a, b, sa, sb = operands(300, 700, 1024, 6)
    first = run(a, b, sa, sb, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(first) for _ in range(4)]
    for o in outs:
        run(a, b, sa, sb, "bf16", out=o, stream=s.cuda_stream)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    third = torch.empty_like(first)
    with torch.cuda.graph(gr):
        run(a, b, sa, sb, "bf16", out=third, stream=torch.cuda.current_stream().cuda_stream)
    gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs + [third])


@pytest.mark.parametrize("m,n,k", [(70001, 65600, 16), (5, 1 << 20, 4224)])
def test_offsets_past_32_bits(m, n, k):
    # a result, and a weight matrix, of more than 2^32 places: their last rows and some between
    import torch
    g = torch.Generator(device="cuda").manual_seed(11)
    a, b = (torch.randint(0, 120, (x, k), device="cuda", generator=g, dtype=torch.uint8).view(torch.float8_e4m3fn) for x in (m, n))
    c = run(a, b, None, None, "bf16")
    for rows, cols in ((slice(max(0, m - 70), m), slice(n - 300, n)), (slice(m // 2, m // 2 + 9), slice(n // 2, n // 2 + 99))):
        check(a[rows], b[cols], None, None, "bf16", c[rows, cols])
