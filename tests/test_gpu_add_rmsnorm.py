"""RMSNorm with the residual's addition (lf_add_rmsnorm) on the GPU against the
formula in 64 bits.

Tolerances: s is one fp32 addition (2^-24) and one rounding.  mean(s^2) is a sum of
positive terms, 2^-24 for each of a thread's up to 32 steps and of the 10 joins, so
within 2^-18 of itself; root, reciprocal and the two products add 2^-22: y is within
2^-18 of itself before its one rounding.  An 8-bit value is off by half a step, 2^-4
of itself or 2^-10 (half the smallest step) times the scale, and by 2^-18 more."""
import math

import numpy as np
import pytest

import paged_reference as ref

pytestmark = pytest.mark.gpu
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}


def run(x, res, gain, dtypes, out_dtype, eps=1e-5, want_sum=True, lds=None, out=None, sum_to=None, stream=None):
    import torch
    import decode_persistent_sm_gb300 as lf
    rows, cols = x.shape
    dt = dict(e4m3=torch.float8_e4m3fn)
    s = sum_to if sum_to is not None else (torch.empty_like(res) if want_sum and res is not None else None)
    y = torch.empty(rows, cols, dtype=dt.get(out_dtype) or ref.torch_dtype(out_dtype), device="cuda") if out is None else out
    scale = torch.full((rows,), 7.0, device="cuda")
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    ld = lambda t: cols if t is None else t.stride(0)  # noqa: E731
    lf.add_rmsnorm(x.data_ptr(), dtypes[0], ld(x), p(res), p(s), dtypes[1], ld(res), ld(s), p(gain), dtypes[2], rows,
                   cols, eps, y.data_ptr(), out_dtype, y.stride(0), scale.data_ptr() if out_dtype == "e4m3" else None,
                   stream)
    torch.cuda.synchronize()
    return s, y, scale


def check(x, res, gain, dtypes, out_dtype, eps, s, y, scale):
    xs = x.double().cpu().numpy() + (0.0 if res is None else res.double().cpu().numpy())
    g = 1.0 if gain is None else gain.double().cpu().numpy()
    want = g * xs / np.sqrt((xs * xs).mean(-1, keepdims=True) + eps)
    if s is not None:
        tol = (HALF[dtypes[1]] + 2.0 ** -24) * np.abs(xs) * (1 + 2.0 ** -8) + TINY[dtypes[1]]
        assert (np.abs(s.double().cpu().numpy() - xs) <= tol).all()
    got = y.float().double().cpu().numpy()
    if out_dtype != "e4m3":
        tol = (HALF[out_dtype] * (1 + 2.0 ** -8) + 2.0 ** -18) * np.abs(want) + TINY[out_dtype]
        assert (np.abs(got - want) <= tol).all()
        return
    sc = scale.double().cpu().numpy()[:, None]
    top = np.abs(want).max(-1, keepdims=True) / 448.0
    assert (np.abs(sc - np.where(top > 0, top, 1.0)) <= 2.0 ** -18 * np.where(top > 0, top, 1.0)).all()
    assert (np.abs(got) <= 448.0).all()
    tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * sc) * (1 + 2.0 ** -10) + 2.0 ** -17 * np.abs(want)
    assert (np.abs(got * sc - want) <= tol).all()


def inputs(rows, cols, dtypes, seed, ld=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = lambda scale, d, n=rows: (scale * torch.randn(n, cols + ld, device="cuda", generator=g)).to(ref.torch_dtype(d))[:, :cols]  # noqa: E731
    x, res = make(0.7, dtypes[0]), make(3.0, dtypes[1])
    return x, res, (1 + 0.2 * torch.randn(cols, device="cuda", generator=g)).to(ref.torch_dtype(dtypes[2]))


@pytest.mark.parametrize("out_dtype", ["f32", "f16", "bf16", "e4m3"])
@pytest.mark.parametrize("dtypes", [("f32", "f32", "f16"), ("f16", "f16", "f16"), ("bf16", "bf16", "bf16"),
                                    ("f16", "f32", "f32"), ("f32", "bf16", "bf16"), ("bf16", "f16", "f32")])
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 1), (5, 33), (300, 256), (7, 520), (3, 4096), (2, 7168), (9, 16384),
                                       (2, 32768), (1, 20000), (4, 1001), (2, 16389)])
def test_rows(rows, cols, dtypes, out_dtype):
    x, res, gain = inputs(rows, cols, dtypes, rows + cols)
    check(x, res, gain, dtypes, out_dtype, 1e-5, *run(x, res, gain, dtypes, out_dtype))


@pytest.mark.parametrize("out_dtype", ["f16", "e4m3"])
@pytest.mark.parametrize("pad", [1, 4, 8])
def test_strides_and_rows_of_padding_untouched(pad, out_dtype):
    import torch
    dtypes = ("f16", "f32", "f32")
    x, res, gain = inputs(6, 512, dtypes, pad, ld=pad)
    dt = torch.float8_e4m3fn if out_dtype == "e4m3" else torch.float16
    out = torch.full((7, 512 + 2 * pad), 1.5, device="cuda").to(dt)
    s = torch.full((7, 512 + 3 * pad), 1.5, device="cuda")
    s_, y, scale = run(x, res, gain, dtypes, out_dtype, out=out[:6, :512], sum_to=s[:6, :512])
    check(x, res, gain, dtypes, out_dtype, 1e-5, s_, y, scale)
    assert (out[6].float() == 1.5).all() and (out[:, 512:].float() == 1.5).all()
    assert (s[6] == 1.5).all() and (s[:, 512:] == 1.5).all()


def test_without_residual_gain_or_sum():
    dtypes = ("bf16", "f16", "f32")
    x, res, gain = inputs(4, 640, dtypes, 1)
    check(x, None, gain, dtypes, "f16", 1e-5, *run(x, None, gain, dtypes, "f16"))
    check(x, res, None, dtypes, "e4m3", 1e-5, *run(x, res, None, dtypes, "e4m3"))
    check(x, res, gain, dtypes, "f32", 1e-5, *run(x, res, gain, dtypes, "f32", want_sum=False))
    import torch
    s = torch.empty(4, 640, dtype=torch.float16, device="cuda")
    check(x, None, gain, dtypes, "f16", 1e-5, *run(x, None, gain, dtypes, "f16", sum_to=s))


def test_in_place():
    import torch
    dtypes = ("f16", "f16", "f32")
    x, res, gain = inputs(50, 1024, dtypes, 2)
    s, y, _ = run(x, res, gain, dtypes, "f16")
    for where in ("residual", "x"):
        a, b = x.clone(), res.clone()
        s2, y2, _ = run(a, b, gain, dtypes, "f16", sum_to=b if where == "residual" else a, out=a if where == "residual" else b)
        assert torch.equal(s, s2) and torch.equal(y, y2)


def test_rows_of_zeros_tiny_and_large_values():
    import torch
    dtypes = ("f32", "f32", "f32")
    x = torch.zeros(6, 256, device="cuda")
    x[1] = 1e-30
    x[2, 5] = 1e-38
    x[3] = 1e18
    x[4] = torch.linspace(-1, 1, 256, device="cuda") * 1e-20
    x[5, 0] = 1e10
    res = torch.zeros_like(x)
    for out_dtype in ("f32", "e4m3"):
        check(x, res, None, dtypes, out_dtype, 1e-5, *run(x, res, None, dtypes, out_dtype))


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_what_is_not_finite_stays_in_its_row(bad):
    import torch
    dtypes = ("f16", "f32", "f32")
    x, res, gain = inputs(5, 768, dtypes, 3)
    clean = run(x, res, gain, dtypes, "e4m3")
    res[2, 100] = bad
    s, y, scale = run(x, res, gain, dtypes, "e4m3")
    keep = [0, 1, 3, 4]
    assert torch.equal(y[keep].view(torch.uint8), clean[1][keep].view(torch.uint8)) and torch.equal(scale[keep], clean[2][keep])
    assert torch.isnan(y[2, 100].float()) and scale[2] == 1.0
    assert torch.isnan(y[2].float()).all() == math.isnan(bad)  # an infinite mean square leaves zeros besides
    _, y, _ = run(x, res, gain, dtypes, "f32")
    assert torch.isnan(y[2, 100]) and torch.isfinite(y[keep]).all()


def test_8_bit_rounding_is_to_nearest_even():
    # a row whose scale is 1: 448 beside every border between two neighbouring values
    import torch
    grid = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (grid[1:] + grid[:-1]) / 2
    x = torch.zeros(1, 1024, dtype=torch.float64)
    x[0, :126], x[0, 126:252], x[0, 252:378] = mid, -mid, grid[1:]
    x[0, 378] = 448.0
    rms = math.sqrt(float((x * x).mean()))
    # y = x exactly where the mean square is a power of four
    x[0, 379] = math.sqrt((4.0 ** 4 - rms * rms) * 1024) if rms < 16 else 0.0
    gain = torch.full((1024,), 1.0, dtype=torch.float32)
    xs = x.float().cuda()
    s, y, scale = run(xs, torch.zeros_like(xs), gain.cuda(), ("f32", "f32", "f32"), "e4m3")
    want = (xs.double() / math.sqrt(float((xs.double() ** 2).mean()) + 1e-5)).cpu()
    check(xs, torch.zeros_like(xs), gain, ("f32", "f32", "f32"), "e4m3", 1e-5, s, y, scale)
    q = (want / scale.double().cpu()[:, None]).float().to(torch.float8_e4m3fn)
    differ = (q.view(torch.uint8) != y.cpu().view(torch.uint8)).float().mean()
    assert differ < 0.3  # only values within 2^-18 of a border may fall to the other side


def test_on_another_stream_and_captured():
    import torch
    import decode_persistent_sm_gb300 as lf  # noqa: F401
    dtypes = ("f32", "f32", "f16")
    x, res, gain = inputs(40, 4096, dtypes, 5)
    first = run(x, res, gain, dtypes, "e4m3")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    again = run(x, res, gain, dtypes, "e4m3", stream=st.cuda_stream)
    y, s, scale = torch.empty_like(first[1]), torch.empty_like(res), torch.empty(40, device="cuda")
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        lf.add_rmsnorm(x.data_ptr(), "f32", 4096, res.data_ptr(), s.data_ptr(), "f32", 4096, 4096, gain.data_ptr(), "f16",
                       40, 4096, 1e-5, y.data_ptr(), "e4m3", 4096, scale.data_ptr(),
                       torch.cuda.current_stream().cuda_stream)
    gr.replay()
    torch.cuda.synchronize()
    for a, b in ((again[0], s), (again[1].view(torch.uint8), y.view(torch.uint8)), (again[2], scale)):
        assert torch.equal(a, b)
    assert torch.equal(first[1].view(torch.uint8), y.view(torch.uint8))


def test_rows_past_32_bits():
    import torch
    rows, cols = (1 << 32) // 8192 + 5, 8192
    x = torch.zeros(rows, cols, dtype=torch.float16, device="cuda")
    x[-1] = 2.0
    _, y, _ = run(x, None, None, ("f16", "f16", "f16"), "f16")
    assert (y[-1] == 1.0).all() and not y[-2].any()


@pytest.mark.parametrize("dtypes", [("f16", "f16", "f16"), ("bf16", "bf16", "f32"), ("f16", "bf16", "bf16")])
@pytest.mark.parametrize("rows,cols,out_dtype", [(1300, 4096, "e4m3"), (1301, 8192, "f16"), (700, 7168, "bf16"),
                                                 (640, 4104, "e4m3"), (2000, 5000, "f32")])
def test_many_rows_of_16_bits(rows, cols, out_dtype, dtypes):
    x, res, gain = inputs(rows, cols, dtypes, cols)
    check(x, res, gain, dtypes, out_dtype, 1e-5, *run(x, res, gain, dtypes, out_dtype))
    check(x, None, None, dtypes, out_dtype, 1e-5, *run(x, None, None, dtypes, out_dtype))


def test_many_rows_in_place_strided_and_not_finite():
    import torch
    dtypes = ("f16", "f16", "f16")
    x, res, gain = inputs(1000, 4608, dtypes, 5, ld=24)
    s, y, scale = run(x, res, gain, dtypes, "e4m3")
    a, b = x.clone(), res.clone()
    s2, y2, scale2 = run(a, b, gain, dtypes, "e4m3", sum_to=b)
    assert torch.equal(s, s2) and torch.equal(y.view(torch.uint8), y2.view(torch.uint8)) and torch.equal(scale, scale2)
    s3, y3, _ = run(a, res, gain, dtypes, "f16", sum_to=a, out=res.clone())
    assert torch.equal(s, s3)
    x[999, 7] = math.nan
    _, y4, scale4 = run(x, res, gain, dtypes, "e4m3")
    assert torch.equal(y4[:999].view(torch.uint8), y[:999].view(torch.uint8)) and torch.isnan(y4[999].float()).all() and scale4[999] == 1


@pytest.mark.parametrize("rows", [607, 608, 609])
def test_both_ways_agree_at_their_border(rows):
    import torch
    dtypes = ("bf16", "bf16", "bf16")
    x, res, gain = inputs(rows, 6144, dtypes, 9)
    s, y, _ = run(x, res, gain, dtypes, "bf16")
    s2, y2, _ = run(x[:100], res[:100], gain, dtypes, "bf16")
    assert torch.equal(s[:100], s2)
    check(x, res, gain, dtypes, "bf16", 1e-5, s, y, torch.ones(rows))
    assert (y[:100] != y2).float().mean() < 1e-3  # the sums of squares may differ in their last bit
