"""What the binding hands to the batch calls (no GPU needed: a stand-in for the
library records the arguments): uniform numbers rounded to fp32 stay below what they
were, so a valid one is never refused; and a call with more or fewer tokens than
the batch has samples does not reach the library."""
import ctypes

import numpy as np
import pytest


class Library:
    """A batch of `n` samples that takes every call."""

    def __init__(self, n):
        self.n, self.calls = n, []

    def lf_batch_info(self, h, nb, pos):
        nb._obj.value, pos._obj.value = self.n, 5
        return 0 if self.n >= 0 else 1

    def lf_batch_generate_filtered(self, h, first, steps, t, k, p, mp, u, out, lp):
        assert self.n > 0
        self.calls.append(np.ctypeslib.as_array(ctypes.cast(u, ctypes.POINTER(ctypes.c_float)), (self.n, steps)).copy())
        return 0

    def lf_batch_step(self, *a):
        self.calls.append("step")
        return 0

    def lf_batch_generate(self, *a):
        self.calls.append("generate")
        return 0

    def lf_destroy(self, h):
        return 0


def engine(n):
    from decode_persistent_sm_gb300 import Engine
    e = object.__new__(Engine)
    e._lib, e._h, e.vocab = Library(n), 1, 100
    return e


@pytest.mark.parametrize("u", [1 - 2.0 ** -25, 1 - 2.0 ** -30, np.nextafter(1.0, 0.0), 0.3, 1 / 3, 0.0, 2.0 ** -160, 1 - 2.0 ** -24,
                               5e-324])
def test_u_is_rounded_down(u):
    e = engine(2)
    e.batch_generate_filtered([1, 2], np.array([[u, 0.25], [0.5, u]]))
    got = e._lib.calls[0].astype(np.float64)
    for g in (got[0, 0], got[1, 1]):
        assert 0 <= g <= u and g < 1
        assert np.nextafter(np.float32(g), np.float32(2)).astype(np.float64) > u  # the next one up is above u
    assert got[0, 1] == 0.25 and got[1, 0] == 0.5


def test_what_is_out_of_range_stays_out_of_range():
    # (the library refuses it)
    for u in (1.0, 1.5, 1e300, np.inf, -1e-300, -0.5, -np.inf, np.nan):
        e = engine(1)
        e.batch_generate_filtered([1], np.array([[u]]))
        assert not 0 <= e._lib.calls[0][0, 0] < 1


def test_fp32_is_passed_as_it_is():
    e = engine(1)
    u = np.random.default_rng(0).random((1, 1000), dtype=np.float32)
    e.batch_generate_filtered([1], u)
    assert np.array_equal(e._lib.calls[0], u)


def test_any_layout_of_u():
    u = np.random.default_rng(1).random((7, 5))
    for view in (np.asfortranarray(u), u[::1, ::-1], np.repeat(u, 2, 1)[:, ::2]):
        e = engine(7)
        e.batch_generate_filtered([1] * 7, view)
        got = e._lib.calls[0].astype(np.float64)
        assert (got <= view).all() and np.abs(got - view).max() < 2.0 ** -23


@pytest.mark.parametrize("have,given", [(3, 2), (3, 4), (1, 0), (16, 1)])
def test_a_token_for_each_sample_of_the_batch(have, given):
    # the library reads and writes as many as the batch has samples
    tokens = [1] * given
    for call in (lambda e: e.batch_step(tokens), lambda e: e.batch_step(tokens, logits=False),
                 lambda e: e.batch_generate(tokens, 4, 0.8, 0.9, 1),
                 lambda e: e.batch_generate_filtered(tokens, np.full((given, 4), 0.5))):
        e = engine(have)
        with pytest.raises(ValueError, match=f"{have} samples"):
            call(e)
        assert not e._lib.calls


def test_without_a_batch_the_library_answers():
    from decode_persistent_sm_gb300 import LaneformerError
    e = engine(0)
    e._lib.lf_batch_step = lambda *a: 4
    with pytest.raises(LaneformerError, match="NOT_LOADED"):
        e.batch_step([1, 2])
