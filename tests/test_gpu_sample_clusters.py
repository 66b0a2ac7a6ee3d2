"""The filtered draw's special rows (no draw, infinite, masked, extreme
temperatures) where a row is shared by 1, 2, 4 and 8 CTAs: the number follows
from the rows and the vocabulary (40000 entries: 8 for 1 and 12 rows, 4 for 40, 1
for 120 rows; 262144: 8 for 9 rows; 20011: 2 for 90 rows)."""
import numpy as np
import pytest

from test_gpu_sample_filtered import check

pytestmark = pytest.mark.gpu
SIZES = [(1, 40000), (12, 40000), (40, 40000), (120, 40000), (9, 262144), (90, 20011)]


def spots(v):
    """The first and the last index, and some in the middle CTAs' ranges."""
    return [0, v // 8, v // 2 - 1, v // 2, 3 * v // 4 + 5, v - 1]


@pytest.mark.parametrize("rows,v", SIZES)
def test_nan_anywhere(rows, v):
    z = np.random.default_rng(rows).standard_normal((rows, v)).astype(np.float32)
    for at in spots(v):
        y = z.copy()
        y[::2, at] = np.nan
        tok = check(y, "f32", t=np.where(np.arange(rows) % 4 < 2, 1.0, 0.0), k=np.arange(rows) % 3 * 20, p=0.9, u=0.4)
        assert (tok[::2] == -1).all() and (tok[1::2] >= 0).all()


@pytest.mark.parametrize("rows,v", SIZES)
def test_bad_parameters(rows, v):
    z = np.random.default_rng(rows + 1).standard_normal((rows, v)).astype(np.float32)
    good = dict(t=1.0, p=0.9, mp=0.01, u=0.5)
    for bad in (dict(t=-1.0), dict(t=np.inf), dict(t=np.nan), dict(p=0.0), dict(p=1.5), dict(mp=-0.1), dict(mp=1.1), dict(u=1.0),
                dict(u=np.nan)):
        par = {x: np.full(rows, y) for x, y in good.items()}
        for x, y in bad.items():
            par[x][::2] = y
        tok = check(z, "f32", **par)
        assert (tok[::2] == -1).all() and (tok[1::2] >= 0).all()


@pytest.mark.parametrize("rows,v", SIZES)
def test_masked_and_infinite(rows, v):
    none = np.full((rows, v), -np.inf, dtype=np.float32)
    assert (check(none, "f32", t=1.0, k=3, p=0.5, u=0.5) == -1).all()
    for at in spots(v):
        y = none.copy()
        y[:, at] = -7.0  # one logit in one CTA's range
        for par in (dict(t=1.0), dict(t=0.0), dict(t=0.5, k=50, p=0.9, mp=0.1)):
            assert (check(y, "f32", u=0.999, **par) == at).all()
    z = np.random.default_rng(rows + 2).standard_normal((rows, v)).astype(np.float32)
    for at in spots(v):
        y = z.copy()
        y[:, at] = np.inf
        for par in (dict(t=1.0), dict(t=0.0), dict(t=2.0, k=5, p=0.3, mp=0.5)):
            assert (check(y, "f32", u=0.77, **par) == at).all()
    y = z.copy()
    y[:, spots(v)] = np.inf  # several, in several CTAs' ranges
    tok = check(y, "f32", t=1.0, k=2, u=(np.arange(rows) % 12 + 0.5) / 12)
    assert all(t == spots(v)[i % 12 // 2] for i, t in enumerate(tok))


@pytest.mark.parametrize("rows,v", SIZES)
def test_extreme_temperatures(rows, v):
    z = np.random.default_rng(rows + 3).standard_normal((rows, v)).astype(np.float32)
    big = z / np.abs(z).max() * np.float32(3.4e38)
    for t in (1e-30, 1e-5, 1e5, 1e30):
        check(z, "f32", t=t, p=0.9, u=0.7)
        check(big, "f32", t=t, k=30, u=0.7)
    assert (check(z, "f32", t=1e-38, u=0.7) == -1).all()


@pytest.mark.parametrize("rows,v", SIZES)
def test_equal_logits_over_every_part(rows, v):
    z = np.full((rows, v), 1.5, dtype=np.float32)
    u = (np.arange(rows) + 0.5) / rows
    for par in (dict(), dict(k=9), dict(p=0.4), dict(k=9, p=0.4, mp=0.9), dict(t=0.0)):
        check(z, "f32", u=u, **par)
