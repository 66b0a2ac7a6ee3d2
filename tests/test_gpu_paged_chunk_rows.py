"""lf_attn_paged_chunk on queries as a fused projection leaves them: rows further apart
than their heads, keys and values (or NaN) between them, NaN in rows that are nobody's;
and on batches whose lengths leave nothing to see."""
import math

import pytest

from test_gpu_paged_chunk import Case

pytestmark = pytest.mark.gpu

# warp-level products of 16, 32 and 64 rows in clusters and by the list, tensor cores in clusters and by the list
SHAPES = [([5] * 8, [300 + 40 * i for i in range(8)], 8, 4, 128, 0), ([1] * 70, [90] * 70, 8, 8, 64, 0),
          ([30, 2], [500, 900], 16, 4, 32, 0), ([40] * 12, [2000] * 12, 8, 8, 64, 50), ([130], [70], 6, 2, 64, 0),
          ([333, 1], [1000, 5], 5, 1, 128, 0), ([700] * 6, [3000] * 6, 8, 2, 128, 0), ([257, 64], [0, 900], 16, 1, 64, 128)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new,ctx,nq,nkv,dim,window", SHAPES)
def test_rows_of_a_fused_projection(new, ctx, nq, nkv, dim, window, dtype):
    import torch
    import decode_persistent_sm_gb300 as lf
    c = Case(new, ctx, nq, nkv, dim, 32, dtype, window, seed=nq + dim, pad=3, lead=2)
    d, ld = nq * dim, (nq + 2 * nkv) * dim + 8
    c.q[:2], c.q[c.tokens:] = math.nan, math.nan
    fused = torch.full((c.rows, ld), math.nan, dtype=c.q.dtype, device="cuda")
    fused[:, :d] = c.q.view(c.rows, d)
    ws, most = c.workspace(), max(c.lens)
    plain, lse = c.run(ws=ws, max_len=most)
    c.check(plain, lse)

    def run(out, ld_out):
        ls = torch.full((c.rows, nq), 9.0, device="cuda")
        lf.attn_paged_chunk(c.kv, fused.data_ptr(), ld, out.data_ptr(), ld_out, ls.data_ptr(), nq, c.starts.data_ptr(), c.rows,
                            c.ln.data_ptr(), most, window, c.scale, ws.data_ptr(), ws.numel(), c.err.data_ptr())
        torch.cuda.synchronize()
        assert c.err.item() == 0 and torch.equal(ls, lse)

    out = torch.full((c.rows, d), 9.0, dtype=c.q.dtype, device="cuda")
    run(out, d)
    assert torch.equal(out, plain)
    run(fused, ld)  # in place, between the keys and values
    assert torch.equal(fused[2:c.tokens, :d], plain[2:c.tokens])
    assert fused[:2].isnan().all() and fused[c.tokens:].isnan().all() and fused[:, d:].isnan().all()


@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("new", [[1], [5, 0, 9], [200], [300, 7]])
def test_nothing_to_see_at_all(new, dim):
    import torch
    c = Case(new, [-x for x in new], 8, 4, dim, 16, "f16", pad=1)
    for most in (0, 4096 if c.table.shape[1] * 16 >= 4096 else c.table.shape[1] * 16):
        out, lse = c.run(max_len=most)
        torch.cuda.synchronize()
        assert c.err.item() == 0 and not out[:-1].any() and torch.isneginf(lse[:-1]).all()
        assert (out[-1] == 9.0).all() and (lse[-1] == 9.0).all()
