"""The attention of many rows (three kernels in a row) right behind the kernels that
write what it reads: queries, lengths, page table, keys and values change before
every call, without a pause, and every result equals the one after a pause."""
import numpy as np
import pytest

from test_gpu_paged import Case, lens_of
from test_gpu_serving_chain import STEPS, Loop

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,page,dtype", [(128, 16, "f16"), (64, 64, "bf16")])
def test_everything_the_call_reads_is_written_just_before(dim, page, dtype):
    import torch
    n, nkv, shared, own = 64, 8, 8064, 40
    c = Case(lens_of(shared, [own] * n), shared, 2 * nkv if dim == 128 else 4 * nkv, nkv, dim, page, dtype)
    g = torch.Generator(device="cuda").manual_seed(7)
    dt = c.q.dtype
    steps = 12
    qs = torch.randn(steps, *c.q.shape, device="cuda", generator=g).to(dt)
    lens = torch.randint(shared + 1, shared + own + 1, (steps, n), device="cuda", generator=g, dtype=torch.int32)
    tables = []
    order = np.random.default_rng(1)
    for _ in range(steps):  # the common pages and the own ones in another order each time
        t, w = c.table.copy(), shared // page
        t[:, :w] = order.permutation(t[0, :w])
        t[:, w:] = t[order.permutation(n), w:]
        tables.append(t)
    tables = torch.from_numpy(np.stack(tables)).cuda()
    c.k.nan_to_num_(0.25)  # any order of the own pages may be read
    c.v.nan_to_num_(0.25)
    k0, v0 = c.k.clone(), c.v.clone()
    ws = c.workspace()
    torch.cuda.synchronize()

    def run(pause):
        c.k.copy_(k0)
        c.v.copy_(v0)
        outs = []
        for i in range(steps):
            c.k.mul_(-1)
            c.v.mul_(-1)
            c.tb.copy_(tables[i])
            c.ln.copy_(lens[i])
            c.q.copy_(qs[i])
            if pause:
                torch.cuda.synchronize()
            outs.append(c.run(ws=ws))
            if pause:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert c.err.item() == 0
        return outs

    want = run(True)
    assert len({float(o.float().abs().sum()) for o, _ in want}) == steps  # every step's input counts
    for _ in range(4):
        for (a, la), (b, lb) in zip(run(False), want):
            assert torch.equal(a, b) and torch.equal(la, lb)


class LongLoop(Loop):
    SHAPES = {"many rows": (64, 16, 8, 128, 64, 8064, 10, 8192)}


def test_append_attention_and_draw_back_to_back():
    import torch
    for dtype in ("f16", "bf16"):
        loops = [LongLoop("many rows", dtype) for _ in range(2)]
        for loop, pause in zip(loops, (torch.cuda.synchronize, lambda: None)):
            for i in range(STEPS):
                loop.feed(i)
                pause()
                loop.step(pause)
                loop.keep(i)
        loops[1].same_as(loops[0])
