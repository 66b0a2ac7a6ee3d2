"""The waits of the chunk attention's tensor-core kernel, given up on purpose (debug
library): a warp of one CTA, or of each, gives up in its nth wait, with copies and
products under way.  The error word then says so, every CTA (of a cluster too) ends
with nothing running behind it, and the next call is as if nothing had happened."""
import ctypes

import pytest

from test_gpu_paged_chunk import Case

pytestmark = pytest.mark.gpu


@pytest.fixture
def lib():
    import decode_persistent_sm_gb300 as lf
    d = lf.load_library(debug=True)
    yield d
    assert d.lf_debug_chunk_wait(-1, 0, 0) == 0


# the list with shared items, clusters of four, of two and of one CTA; masked tiles, a window, one row tile to an item
@pytest.mark.parametrize("new,ctx,nq,nkv,dim,window", [
    ([700] * 6, [3000 + 100 * i for i in range(6)], 32, 8, 128, 0), ([256], [3840], 32, 16, 128, 0),
    ([512], [3584], 32, 16, 128, 0), ([500] + [90] * 12, [1000] * 13, 24, 8, 64, 600), ([150], [20], 8, 8, 128, 0)])
def test_a_warp_that_gives_up(lib, new, ctx, nq, nkv, dim, window):
    import torch
    c = Case(new, ctx, nq, nkv, dim, 64, "f16", window, seed=len(new))
    ws = torch.full((lib.lf_attn_paged_chunk_workspace(ctypes.byref(c.kv), nq, c.rows),), 255, dtype=torch.uint8, device="cuda")
    most = max(c.lens)

    def run():
        out = torch.full((c.rows, nq * dim), 9.0, dtype=torch.float16, device="cuda")
        c.err.zero_()
        assert lib.lf_attn_paged_chunk(ctypes.byref(c.kv), c.q.data_ptr(), nq * dim, out.data_ptr(), nq * dim, None, nq,
                                       c.starts.data_ptr(), c.rows, c.ln.data_ptr(), most, window, c.scale, ws.data_ptr(),
                                       ws.numel(), c.err.data_ptr(), None) == 0
        torch.cuda.synchronize()
        return out, c.err.item()

    want, err = run()
    assert err == 0 and torch.isfinite(want).all()
    gave_up = 0
    for cta in (-1, 0, 1):
        for warp in range(10):
            for nth in (1, 2, 3, 5, 8, 13, 30):
                assert lib.lf_debug_chunk_wait(cta, warp, nth) == 0
                got, err = run()
                assert err in (0, 2)
                assert err == 2 or torch.equal(got, want)  # (a warp without that many waits)
                assert err == 2 or cta >= 0 or nth > 1 or warp in (0, 6, 7, 8, 9)  # (no wait of the copies; one row tile)
                gave_up += err == 2
                assert lib.lf_debug_chunk_wait(-1, 0, 0) == 0
                got, err = run()
                assert err == 0 and torch.equal(got, want)
    assert gave_up > 30
