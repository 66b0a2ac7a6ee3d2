"""Rounding of lf_add_rmsnorm's 8-bit output, bit for bit.  s is 1 or -1 everywhere and
eps is 3, so the mean square plus eps is 4 and 1 / rms 1/2, all exact; the gain carries
the values, its largest 2 * 448 times a power of two, so the scale is that power, exact
too, and out is what one rounding of gain * s / 2 / scale gives: to nearest, the even
neighbour of a value in the middle of two."""
import numpy as np
import pytest


def e4m3_nearest_even(x):
    """The nearest of the 256 values by the definition in 64 bits, as bytes."""
    codes = np.arange(127)
    e, m = codes >> 3, codes & 7
    grid = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    a = np.abs(x)
    i = np.clip(np.searchsorted(grid, a, side="right") - 1, 0, 125)  # grid[i] <= a
    up, down = grid[i + 1] - a, a - grid[i]
    code = np.where(up < down, i + 1, np.where(up > down, i, i + (i & 1)))  # (a code is even with its last mantissa bit)
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def values():
    """Every value of the grid, every middle of two, and both fp32 neighbours of each middle."""
    codes = np.arange(127)
    grid = np.where(codes >> 3 == 0, (codes & 7) * 2.0 ** -9, (8 + (codes & 7)) * 2.0 ** ((codes >> 3) - 10.0))
    mid = ((grid[1:] + grid[:-1]) / 2).astype(np.float32)
    assert (mid.astype(np.float64) * 2 == grid[1:] + grid[:-1]).all()  # exact in fp32
    return np.concatenate([grid.astype(np.float32), mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(999))])


def test_the_rounding_that_is_expected():
    # the oracle itself: what one wrong neighbour would change
    x = values().astype(np.float64)
    code = e4m3_nearest_even(x)
    n = len(x) - 3 * 126
    assert (code[:n] == np.arange(127)).all()
    assert (code[n:n + 126] % 2 == 0).all()                                   # middles: the even neighbour
    assert (code[n + 126:n + 252] == np.arange(126)).all() and (code[n + 252:] == np.arange(1, 127)).all()


@pytest.mark.gpu  # one block to a row, in vectors and not, and (16-bit rows, many of them) the walk over rows
@pytest.mark.parametrize("power", [0, -7, 9, -100])  # of the scale; the last one's values divide instead of multiply
@pytest.mark.parametrize("dtype,rows,cols", [("f32", 3, 1024), ("bf16", 3, 1024), ("f32", 2, 1021), ("f16", 2000, 4096),
                                             ("bf16", 1300, 8192)])
def test_values_between_two_round_to_the_nearest_and_the_even(dtype, rows, cols, power):
    import torch
    import decode_persistent_sm_gb300 as lf
    v = values()
    y = np.resize(v, cols)                    # each row: the values in turn
    y[-1] = 448.0
    g = np.random.default_rng(cols)
    gain = torch.from_numpy(y * np.float32(2.0) ** (power + 1)).cuda()
    sign = g.choice([-1.0, 1.0], (rows, cols))
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    res = torch.from_numpy(g.integers(-3, 4, (rows, cols)).astype(np.float32)).cuda().to(dt)
    x = torch.from_numpy(sign).cuda().to(dt) - res        # small whole numbers: exact
    out = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(rows, device="cuda")
    lf.add_rmsnorm(x.data_ptr(), dtype, cols, res.data_ptr(), None, dtype, cols, cols, gain.data_ptr(), "f32", rows, cols, 3.0,
                   out.data_ptr(), "e4m3", cols, scale.data_ptr())
    torch.cuda.synchronize()
    assert (scale == 2.0 ** power).all()
    want = e4m3_nearest_even(sign * y.astype(np.float64))
    got = out.cpu().numpy()
    assert (got == want).all(), (np.argwhere(got != want)[:5], got[got != want][:5], want[got != want][:5])
