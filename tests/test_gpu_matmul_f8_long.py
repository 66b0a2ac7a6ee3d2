"""Products of 8-bit operands that take longer in all than one of their waits may:
the limit is a single wait's without progress, not a call's.  Operands of whole
numbers in a few columns and zeros elsewhere, so that every result is exact."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture
def memory():
    yield
    import torch
    torch.cuda.empty_cache()  # up to 137 GB, for allocations that are not torch's


def sparse(rows, k, seed):
    """[rows][k] e4m3 as bytes, and its columns that are not zero, among them the first and the last."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    at = torch.cat([torch.tensor([0, k - 1], device="cuda"), torch.randint(1, k - 1, (60,), device="cuda", generator=g)]).unique()
    v = torch.randint(-4, 5, (rows, len(at)), device="cuda", generator=g).float()
    a = torch.zeros(rows, k, dtype=torch.uint8, device="cuda")
    for i, j in enumerate(at.tolist()):
        a[:, j] = v[:, i].to(torch.float8_e4m3fn).view(torch.uint8)
    return a, v


# 12e15 operations over many tiles of a CTA (4.5 s); one tile whose result comes behind 2^31 places of K (2.6 s)
@pytest.mark.parametrize("rows,k", [(1 << 17, 360448), (64, (1 << 31) - 512)])
def test_longer_than_the_limit_of_a_wait(rows, k, memory):
    import torch
    import decode_persistent_sm_gb300 as lf
    a, v = sparse(rows, k, rows)
    c = torch.full((rows, rows), 999.0, dtype=torch.float16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lf.matmul_f8(a.data_ptr(), None, a.data_ptr(), None, c.data_ptr(), "f16", rows, rows, k, err.data_ptr(),
                 torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert err.item() == 0
    for i in (slice(0, 128), slice(rows // 2, rows // 2 + 128), slice(max(0, rows - 300), rows)):
        assert torch.equal(c[i].float(), v[i] @ v.t())
