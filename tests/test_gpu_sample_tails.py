"""The filtered draw (lf_sample_filtered) on rows whose mass lies in many tiny
weights, against its definition in extended precision.

A weight is the integer ceil(2^58 w), so the mass of a row of V logits is off by
less than V 2^-58 <= 2^-40 (the maximum's weight is 1), besides 2^-40 of every
weight: the token is the definition's wherever u times the kept mass lies further
than 2^-39 of that mass from a border, which every row here asserts of its own
inputs.  A weight that is not zero in 64 bits (above 2^-1075) is at least one
unit, so u = 0 draws the first kept index.  The log share is off by 2^-21 of it
(fp32, as in the other tests of the draw) and by the mass's 2^-40 and 2^-40."""
import numpy as np
import pytest

import paged_reference as ref

pytestmark = pytest.mark.gpu
SLACK = 2.0 ** -39


def running(w):
    """Running sums of weights of at most 1 without a long sum's rounding: multiples
    of 2^-30 add up exactly, the rests below that in steps of 2^-53 2^-12."""
    high = np.floor(w * 2.0 ** 30) / 2.0 ** 30
    return np.cumsum(high) + np.cumsum(w - high)


def define(z, us, t=1.0, k=0, p=1.0, mp=0.0):
    """For each u the token, the log share and the distance of u from the nearest
    border, as shares of the kept mass."""
    z = np.asarray(z, dtype=np.float64)
    w = np.exp((z - z.max()) / t)
    kept = np.ones(len(z), dtype=bool)
    if 0 < k < len(z):
        kept &= z >= np.sort(z)[-k]
    if p < 1:
        order = np.argsort(-z, kind="stable")
        c = running(np.where(kept, w, 0.0)[order])
        edge = z[order[np.searchsorted(c, p * c[-1])]]
        # what lies above the border falls short of the target, with the border's own it reaches it
        below, reached = c[(z[order] > edge).sum() - 1] if edge < z.max() else 0.0, c[(z[order] >= edge).sum() - 1]
        gap = min(p - below / c[-1], reached / c[-1] - p)
        assert gap > SLACK, gap
        kept &= z >= edge
    if mp > 0:
        kept &= w >= mp
    c = running(np.where(kept, w, 0.0))
    out = []
    for u in us:
        i = int(np.searchsorted(c, u * c[-1], side="right"))
        edge = np.abs(c - u * c[-1]).min() / c[-1] if u > 0 else np.inf
        out.append((i, float(np.log(w[i] / c[-1]) if w[i] < 1 else -np.log1p(c[-1] - 1)), float(edge)))
    return out


def check(z, dtype="f32", **kw):
    """z: one row; kw as define's, u a list.  Every u is a row of one call."""
    import torch
    import decode_persistent_sm_gb300 as lf
    us = np.asarray(kw.pop("u"), dtype=np.float32)
    n, v = len(us), len(z)
    zd = torch.from_numpy(np.asarray(z, dtype=np.float32)).cuda().to(ref.torch_dtype(dtype))
    rows = zd.repeat(n, 1)
    par = {"t": (1.0, torch.float32), "k": (0, torch.int32), "p": (1.0, torch.float32), "mp": (0.0, torch.float32)}
    dev = {x: torch.full((n,), kw.get(x, d), dtype=dt, device="cuda") for x, (d, dt) in par.items()}
    ud = torch.from_numpy(us).cuda()
    tok = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((n,), 7.0, device="cuda")
    lf.sample_filtered(rows.data_ptr(), dtype, n, v, v, dev["t"].data_ptr(), dev["k"].data_ptr(), dev["p"].data_ptr(),
                       dev["mp"].data_ptr(), ud.data_ptr(), tok.data_ptr(), lp.data_ptr())
    torch.cuda.synchronize()
    exact = {x: dev[x][0].item() for x in kw}
    got, share = tok.tolist(), lp.double().cpu().numpy()
    for i, (want, ls, edge) in enumerate(define(zd.double().cpu().numpy(), [float(u) for u in us], **exact)):
        assert edge > SLACK, (i, edge)
        assert got[i] == want, (i, got[i], want)
        assert abs(share[i] - ls) <= 2.0 ** -21 * abs(ls) + 2.0 ** -39, (i, share[i], ls)
    return got


def tail(v, level, heads):
    z = np.full(v, level, dtype=np.float32)
    for at, x in heads.items():
        z[at] = x
    return z


@pytest.mark.parametrize("dtype,level", [("f32", -31.3), ("f32", -30.0), ("bf16", -31.25), ("f16", -31.25)])
@pytest.mark.parametrize("v", [30000, 131074, 262144])
def test_half_of_two_maxima_behind_a_tail(v, level, dtype):
    # the tail's mass of 2^-30 .. 2^-27 moves the middle onto the first of the two
    assert check(tail(v, level, {v - 2: 0.0, v - 1: 0.0}), dtype, u=[0.5]) == [v - 2]


@pytest.mark.parametrize("level", [-31.3, -31.1916, -30.0, -25.0, -18.0])
def test_log_share_of_a_maximum_above_a_tail(level):
    for v in (5000, 131073, 262144):
        check(tail(v, level, {v - 1: 0.0}), u=[0.5, 0.999])


@pytest.mark.parametrize("rows", [1, 12, 40, 200])
@pytest.mark.parametrize("v,t", [(32000, 0.3), (32000, 1.0), (3000, 0.05), (262144, 0.5)])
def test_u_of_zero_draws_the_first_kept_index(v, t, rows):
    if rows * v > 12_000_000:
        rows = 40
    g = np.random.default_rng(v)
    z = (2.5 * g.standard_normal(v)).astype(np.float32)
    z[0] = -9.0
    assert check(z, t=t, u=[0.0] * rows) == [0] * rows
    z[:7] = -np.inf
    assert check(z, t=t, u=[0.0] * rows) == [7] * rows
    top = int(np.flatnonzero(z >= np.sort(z)[-50])[0])
    assert check(z, t=t, k=50, u=[0.0] * rows) == [top] * rows


def test_what_is_zero_in_64_bits_is_never_drawn():
    # the type's lowest value as a mask, and 800 below the maximum; -700 is not zero
    for dtype in ("f32", "f16", "bf16"):
        import torch
        low = torch.finfo(ref.torch_dtype(dtype)).min
        for v in (100, 40000):
            assert check(tail(v, low, {v - 3: 2.0, v - 9: 1.0}), dtype, u=[0.0, 0.9]) == [v - 9, v - 3]
    assert check(tail(9000, -800.0, {8000: 0.0}), u=[0.0, 0.7]) == [8000, 8000]
    assert check(tail(9000, -700.0, {8000: 0.0}), u=[0.0, 0.7]) == [0, 8000]
    assert check(tail(9000, -400.0, {8000: 0.0}), t=0.5, u=[0.0, 0.7]) == [8000, 8000]


@pytest.mark.parametrize("v", [20000, 131072, 262144])
def test_nucleus_that_ends_in_a_tail(v):
    # one maximum, three levels of tiny weights whose masses lie around the nucleus' last 2^-20, in every type
    g = np.random.default_rng(v)
    z = np.empty(v, dtype=np.float32)
    z[:] = g.choice(np.array([-22.0, -22.75, -23.5], dtype=np.float32), v)
    z[v // 3] = 0.0
    w = np.exp(z.astype(np.float64))
    for keep in ([0.0], [0.0, -22.0], [0.0, -22.0, -22.75]):
        # a border in the middle of the next level's mass
        have = w[np.isin(z, np.array(keep, dtype=np.float32))].sum()
        nxt = {1: -22.0, 2: -22.75, 3: -23.5}[len(keep)]
        p = np.float32((have + w[z == np.float32(nxt)].sum() / 2) / w.sum())
        if not p < 1:
            continue
        for dtype in ("f32", "bf16"):
            check(z, dtype, p=p, u=[0.0, 0.25, 0.5, 1 - 2.0 ** -24])


@pytest.mark.parametrize("rows", [1, 24, 90])
@pytest.mark.parametrize("spread,t", [(4.0, 0.3), (8.0, 1.0), (1.0, 3.0), (0.001, 1.0), (2.0, 0.6)])
def test_nucleus_over_many_magnitudes(spread, t, rows):
    # weights from 1 down past 2^-58, or hardly different: every width of the mass histogram's steps
    g = np.random.default_rng(int(spread * 100) + rows)
    z = (spread * g.standard_normal(37003)).astype(np.float32)
    u = g.random(rows, dtype=np.float32)
    for p in (0.3, 0.9, 0.9999, 1 - 2.0 ** -24):
        check(z, t=t, p=np.float32(p), u=u)
    check(z, t=t, p=np.float32(0.95), k=700, u=u)
    check(z, t=t, p=np.float32(0.95), k=5000, u=u)


def test_nucleus_of_ties_that_fill_no_list():
    # thousands of equal values on the border, tiny ones and large ones
    for level in (-0.5, -12.0, -20.0):
        z = tail(60000, level, {i: 0.0 for i in range(0, 60000, 4000)})
        z[1::7] = level - 1.0
        w = np.exp(z.astype(np.float64))
        p = np.float32((w[z == 0].sum() + w[z == np.float32(level)].sum() / 2) / w.sum())
        if p < 1:
            check(z, p=p, u=[0.0, 0.3, 0.99])
            check(z, p=p, k=59000, u=[0.0, 0.3, 0.99])
