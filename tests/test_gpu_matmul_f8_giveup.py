"""The waits of the 8-bit product, run out on purpose (debug library): a limit of a
nanosecond, which the wait for a long tile's accumulator passes while copies and
products are under way.  The error word then says so, the CTAs leave nothing
running behind them, and the next calls are as if nothing had happened."""
import pytest

pytestmark = pytest.mark.gpu
NEVER = 2_000_000_000


@pytest.fixture
def lib():
    import decode_persistent_sm_gb300 as lf
    d = lf.load_library(debug=True)
    yield d
    assert d.lf_debug_matmul_f8_wait(NEVER) == 0


# every form of the kernel: tiles of 64 columns with 32 and with 128 rows of A to a stage, of 128 and of 256 columns, one
# and several tiles to a CTA
@pytest.mark.parametrize("m,n,k", [(5, 70, 1 << 18), (64, 3000, 1 << 16), (300, 6000, 1 << 16), (130, 19400, 1 << 15),
                                   (1000, 20000, 1 << 14)])
def test_a_wait_that_runs_out(lib, m, n, k):
    import torch
    g = torch.Generator(device="cuda").manual_seed(m)
    a, b = (torch.randint(0, 120, (x, k), device="cuda", generator=g, dtype=torch.uint8) for x in (m, n))

    def run():
        c = torch.full((m, n), 9.0, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert lib.lf_matmul_f8(a.data_ptr(), None, b.data_ptr(), None, c.data_ptr(), 2, m, n, k, err.data_ptr(), None) == 0
        torch.cuda.synchronize()
        return c, err.item()

    want, err = run()
    assert err == 0 and not (want == 9.0).all()
    for _ in range(5):
        assert lib.lf_debug_matmul_f8_wait(1) == 0
        _, err = run()
        assert err == 2
        assert lib.lf_debug_matmul_f8_wait(NEVER) == 0
        got, err = run()
        assert err == 0 and torch.equal(got, want)
