"""lf_attn_paged_chunk at the lengths of long documents, where hundreds of key tiles to
an item are shared among CTAs and joined: rows spread over the chunks against 64
bits.  Tolerances as in test_gpu_paged_chunk.py, from the magnitudes of each row."""
import numpy as np
import pytest

import paged_reference as ref
from test_gpu_paged_chunk import Case, f64

pytestmark = pytest.mark.gpu


def check_rows(c, out, lse, picks):
    """Rows `picks` (of a sequence's new tokens) of each sequence."""
    import torch
    torch.cuda.synchronize()
    assert c.err.item() == 0
    nq, nkv, d = c.nq, c.nkv, c.dim
    eps, at = ref.EPS[c.dtype], c.lead
    for b, (new, ctx) in enumerate(zip(c.new, c.ctx)):
        j = np.arange(c.lens[b])
        pg, row = torch.from_numpy(c.table[b][j // c.page]).cuda().long(), torch.from_numpy(j % c.page).cuda()
        k, v = c.k[pg, :, row].double().transpose(0, 1), c.v[pg, :, row].double().transpose(0, 1)  # [kv][j][d]
        for i in sorted({min(new - 1, int(p * new)) for p in picks}):
            lo, hi = (max(0, ctx + i + 1 - c.window) if c.window else 0), ctx + i + 1
            q = c.q[at + i].double().view(nkv, nq // nkv, d)
            s = c.scale * (q @ k[:, lo:hi].transpose(1, 2))
            m = s.amax(-1, keepdim=True)
            e = (s - m).exp()
            total = e.sum(-1, keepdim=True)
            want, mag = (e @ v[:, lo:hi]) / total, (e @ v[:, lo:hi].abs()) / total
            qk = c.scale * (q.abs() @ k[:, lo:hi].abs().transpose(1, 2)).amax(-1, keepdim=True)
            ds = 2.0 ** -23 * (d / 16 + 4) * qk
            keys = hi - lo
            tol = (eps / 2 + 2 * ds + 2.0 ** -18 + keys * 2.0 ** -27) * mag
            tol = tol + ref.TINY_HALF[c.dtype] * (keys / total * v[:, lo:hi].abs().amax() + 1)
            tol = tol + eps / 2 * (want.abs() + tol)
            got = out[at + i].double().view(nkv, nq // nkv, d)
            assert ((got - want).abs() <= tol).all(), (b, i, ((got - want).abs() / tol).max().item())
            wl, gl = (m + total.log()).reshape(-1), lse[at + i].double()
            tl = (2 * ds + 2.0 ** -18 + keys * 2.0 ** -24).reshape(-1) + 2.0 ** -22 * wl.abs()
            assert ((gl - wl).abs() <= tl).all(), (b, i)
        at += new
    got = f64(out)
    assert np.isfinite(got[c.lead:c.tokens]).all() and (got[c.tokens:] == 9.0).all()


@pytest.mark.parametrize("new,ctx,nq,nkv,dim,page,dtype,window", [
    ([1777, 2048], [9001, 14336], 64, 8, 128, 32, "bf16", 0),
    ([2048], [14336], 32, 16, 128, 64, "f16", 0),
    ([1500, 1, 700], [20000, 30000, 1], 12, 4, 64, 16, "f16", 0),
    ([3000, 64], [12000, 16000], 16, 4, 128, 128, "bf16", 4096),
    ([600, 9], [15000, 8000], 8, 2, 32, 16, "f16", 0),       # warp-level products
    ([1000], [30000], 4, 4, 64, 4, "bf16", 0),               # pages too small for a copy of boxes
])
def test_rows_of_long_chunks(new, ctx, nq, nkv, dim, page, dtype, window):
    c = Case(new, ctx, nq, nkv, dim, page, dtype, window, seed=len(new), pad=3)
    out, lse = c.run(max_len=max(c.lens))
    check_rows(c, out, lse, [0, 0.01, 0.13, 0.34, 0.5, 0.62, 0.77, 0.9, 0.995, 1])
