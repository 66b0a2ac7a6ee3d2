"""The waits between the CTAs that share a row of the filtered draw, run out on
purpose (debug library): a chosen CTA gives up in its nth wait without waiting,
the others run out of theirs after a limit of a millisecond.  The row then gets
token -1 (or its token, where the last wait ran out and every CTA's part is there
after all), no CTA ends before the others are done with its shared memory, and the
next call is as if nothing had happened."""
import numpy as np
import pytest

import paged_reference as ref
import synth

pytestmark = pytest.mark.gpu
LIMIT, NEVER = 1_000_000, 2_000_000_000


@pytest.fixture
def lib():
    import decode_persistent_sm_gb300 as lf
    d = lf.load_library(debug=True)
    yield d
    assert d.lf_debug_sample_wait(NEVER, -1, 0) == 0


def draw(lib, z, t, k, p, mp, u):
    import torch
    rows, v = z.shape
    dev = lambda x, dt: torch.full((rows,), x, dtype=dt, device="cuda")  # noqa: E731
    zd, td, kd, pd, md = torch.from_numpy(z).cuda(), dev(t, torch.float32), dev(k, torch.int32), dev(p, torch.float32), dev(mp, torch.float32)
    ud, tok, lp = dev(u, torch.float32), dev(-7, torch.int32), dev(7.0, torch.float32)
    assert lib.lf_sample_filtered(zd.data_ptr(), 0, rows, v, v, td.data_ptr(), kd.data_ptr(), pd.data_ptr(), md.data_ptr(),
                                  ud.data_ptr(), tok.data_ptr(), lp.data_ptr(), None) == 0
    torch.cuda.synchronize()
    return tok.cpu().numpy(), lp.cpu().numpy()


# flows with few and with many waits: no filter, greedy, a nucleus, a top-k by its groups' bound, by the histogram,
# one that fills the lists (ties), and both
FLOWS = [dict(t=1.0), dict(t=0.0), dict(t=0.8, p=0.95), dict(t=0.8, k=50), dict(t=0.8, k=2500, p=0.9), dict(t=1.0, k=5, p=0.4)]


@pytest.mark.parametrize("flow", range(len(FLOWS)))
@pytest.mark.parametrize("rows,v,rank", [(3, 40000, -1), (3, 40000, 0), (3, 40000, 7), (40, 40000, 2), (90, 20011, 1), (90, 20011, -1)])
def test_a_wait_that_runs_out(lib, rows, v, rank, flow):
    g = np.random.default_rng(flow)
    z = (2.0 * g.standard_normal((rows, v))).astype(np.float32)
    if flow == len(FLOWS) - 1:
        z = np.round(z / 4)
    par = dict(dict(t=1.0, k=0, p=1.0, mp=0.0), **FLOWS[flow])
    f = lambda x: float(np.float32(x))  # noqa: E731
    want = [ref.draw(z[i], f(par["t"]), par["k"], f(par["p"]), 0.0, 0.4375)[0] for i in range(rows)]
    lost = np.ones(rows, dtype=bool)
    for nth in range(1, 40):
        assert lib.lf_debug_sample_wait(LIMIT, rank, nth) == 0
        tok, lp = draw(lib, z, u=0.4375, **par)
        assert not ((tok == -1) & ~lost).any()  # a row that has no nth wait has no later one
        lost = tok == -1
        assert lost.all() or nth > 1  # every flow has a wait before its last
        assert np.isnan(lp[lost]).all() and np.array_equal(tok[~lost], np.array(want)[~lost])
        if not lost.any():
            break
    assert not lost.any()
    assert lib.lf_debug_sample_wait(NEVER, -1, 0) == 0
    assert list(draw(lib, z, u=0.4375, **par)[0]) == want


def test_a_row_of_one_cta_waits_for_nobody(lib):
    assert lib.lf_debug_sample_wait(LIMIT, -1, 1) == 0
    z = np.random.default_rng(3).standard_normal((5, 3000)).astype(np.float32)
    tok, _ = draw(lib, z, 1.0, 0, 0.9, 0.0, 0.3)
    assert list(tok) == [ref.draw(r, 1.0, 0, float(np.float32(0.9)), 0.0, float(np.float32(0.3)))[0] for r in z]


def test_the_batched_generation_reports_a_timeout(lib):
    from decode_persistent_sm_gb300 import Engine, LaneformerError
    shape = synth.TINY.replace(vocab=16384)
    with Engine.from_shape(shape, debug=True) as eng:
        eng.load_weights(synth.make_weights(shape, 3))
        eng.prefill(synth.make_tokens(3, 10, shape.vocab), logits=False)
        eng.batch_begin_shared(2)
        toks, _ = eng.batch_generate_filtered([3, 9], np.full((2, 3), 0.5), top_p=0.9)
        assert (toks >= 0).all()
        assert lib.lf_debug_sample_wait(LIMIT, 1, 2) == 0
        with pytest.raises(LaneformerError, match="TIMEOUT"):
            eng.batch_generate_filtered([3, 9], np.full((2, 3), 0.5), top_p=0.9)
        assert lib.lf_debug_sample_wait(NEVER, -1, 0) == 0
        eng.reset()
        eng.prefill(synth.make_tokens(3, 10, shape.vocab), logits=False)
        eng.batch_begin_shared(2)
        again, _ = eng.batch_generate_filtered([3, 9], np.full((2, 3), 0.5), top_p=0.9)
        assert np.array_equal(again, toks)
