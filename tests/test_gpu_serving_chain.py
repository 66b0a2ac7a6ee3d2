"""The serving operators one behind the other, as a decode loop runs them:
append, attention, draw; every step's input new in the
same buffers.  The operators' sums have a fixed order, so every way of running
the loop (with a pause behind each call, back to back, fed from another stream,
two loops at once, as a replayed graph) gives the same bits."""
import numpy as np
import pytest

import paged_reference as ref

pytestmark = pytest.mark.gpu
STEPS = 5


class Loop:
    """Its own cache, buffers and workspace over the same numbers."""

    # seqs, query heads, KV heads, dim, page, common positions, own positions before the first step, bound of the lengths
    SHAPES = {"direct": (3, 8, 4, 64, 16, 48, 20, 96), "list": (5, 8, 4, 64, 16, 700, 30, 8192),
              "many rows": (64, 16, 8, 128, 64, 6016, 10, 6144)}

    def __init__(self, shape, dtype):
        import torch
        import decode_persistent_sm_gb300 as lf
        self.n, self.nq, self.nkv, self.d, self.page, self.shared, own, self.most = self.SHAPES[shape]
        g = np.random.default_rng(5)
        gen = torch.Generator(device="cuda").manual_seed(5)
        dt, cols = ref.torch_dtype(dtype), (self.nq + 2 * self.nkv) * self.d
        max_pages = -(-self.most // self.page)
        whole = self.shared // self.page
        live = -(-(self.shared + own + STEPS) // self.page)  # pages that are reached
        table, n_pages = ref.page_tables(g, self.n, live, whole)
        full = np.full((self.n, max_pages), -1, dtype=np.int32)
        full[:, :live] = table
        self.table = torch.from_numpy(full).cuda()
        self.k = torch.randn(n_pages, self.nkv, self.page, self.d, device="cuda", generator=gen).to(dt)
        self.v = torch.randn(n_pages, self.nkv, self.page, self.d, device="cuda", generator=gen).to(dt)
        self.inputs = torch.randn(STEPS, self.n, cols, device="cuda", generator=gen)
        self.us = torch.rand(STEPS, self.n, device="cuda", generator=gen)
        self.rope = torch.from_numpy(ref.rope_table(self.most, self.d)).cuda()
        self.kv = lf.paged_kv(self.k.data_ptr(), self.v.data_ptr(), self.table.data_ptr(), n_pages=n_pages,
                              n_kv_heads=self.nkv, page_size=self.page, head_dim=self.d, n_seqs=self.n,
                              max_pages=max_pages, dtype=dtype)
        self.x = torch.zeros(self.n, cols, device="cuda")
        self.u = torch.zeros(self.n, device="cuda")
        self.pos = torch.full((self.n,), self.shared + own, dtype=torch.int32, device="cuda")
        self.len = self.pos + 1
        self.q = torch.zeros(self.n, self.nq * self.d, dtype=dt, device="cuda")
        self.out = torch.zeros_like(self.q)
        self.logits = torch.zeros(self.n, 512, dtype=dt, device="cuda")
        self.tok = torch.zeros(self.n, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.full((lf.attn_paged_shared_workspace(self.kv, self.nq),), 255, dtype=torch.uint8, device="cuda")
        self.got = [torch.zeros(STEPS, *t.shape, dtype=t.dtype, device="cuda") for t in (self.out, self.tok)]
        self.dtype = dtype
        torch.cuda.synchronize()

    def feed(self, i):
        self.x.copy_(self.inputs[i])
        self.u.copy_(self.us[i])

    def step(self, pause=lambda: None):
        import torch
        import decode_persistent_sm_gb300 as lf
        st, nq, nkv, d, cols = torch.cuda.current_stream().cuda_stream, self.nq, self.nkv, self.d, self.x.shape[1]
        at = self.x.data_ptr()
        lf.kv_append_paged(self.kv, at, at + 4 * nq * d, at + 4 * (nq + nkv) * d, "f32", cols, cols, cols, nq,
                           self.q.data_ptr(), nq * d, None, self.pos.data_ptr(), self.n, self.rope.data_ptr(), self.most,
                           self.err.data_ptr(), st)
        pause()
        lf.attn_paged_shared(self.kv, self.q.data_ptr(), nq * d, self.out.data_ptr(), nq * d, None, nq, self.len.data_ptr(),
                             self.most, self.shared, 0, d ** -0.5, self.ws.data_ptr(), self.ws.numel(),
                             self.err.data_ptr(), st)
        pause()
        torch.mul(self.out[:, :512], 32, out=self.logits)
        pause()
        lf.sample_filtered(self.logits.data_ptr(), self.dtype, self.n, 512, 512, None, None, None, None,
                           self.u.data_ptr(), self.tok.data_ptr(), None, st)
        pause()
        self.pos.add_(1)
        self.len.add_(1)

    def keep(self, i):
        self.got[0][i].copy_(self.out)
        self.got[1][i].copy_(self.tok)

    def same_as(self, other):
        import torch
        torch.cuda.synchronize()
        assert self.err.item() == 0 and (self.got[1] >= 0).all()
        for a, b in ((self.got[0], other.got[0]), (self.got[1], other.got[1]), (self.k, other.k), (self.v, other.v)):
            assert torch.equal(a, b)


@pytest.fixture(scope="module", params=[(s, d) for s in Loop.SHAPES for d in ("f16", "bf16")], ids=str)
def paused(request):
    """The loop with a pause behind each call."""
    import torch
    loop = Loop(*request.param)
    for i in range(STEPS):
        loop.feed(i)
        torch.cuda.synchronize()
        loop.step(torch.cuda.synchronize)
        loop.keep(i)
    loop.shape = request.param
    assert len({tuple(t.tolist()) for t in loop.got[1]}) == STEPS  # the inputs differ and are used
    return loop


def test_back_to_back(paused):
    loop = Loop(*paused.shape)
    for i in range(STEPS):
        loop.feed(i)
        loop.step()
        loop.keep(i)
    loop.same_as(paused)


def test_fed_from_another_stream_and_two_loops_at_once(paused):
    import torch
    loops = [Loop(*paused.shape) for _ in range(2)]
    work = [torch.cuda.Stream() for _ in loops]
    feeds = [torch.cuda.Stream() for _ in loops]
    for i in range(STEPS):
        for loop, w, f in zip(loops, work, feeds):
            f.wait_stream(w)  # the step before has read its input
            with torch.cuda.stream(f):
                loop.feed(i)
            w.wait_stream(f)
            with torch.cuda.stream(w):
                loop.step()
                loop.keep(i)
    for loop in loops:
        loop.same_as(paused)


def test_as_a_graph_that_forks(paused):
    import torch
    loop, capture, side = Loop(*paused.shape), torch.cuda.Stream(), torch.cuda.Stream()
    at = torch.zeros(1, dtype=torch.long, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=capture):
        loop.err.zero_()
        side.wait_stream(capture)
        with torch.cuda.stream(side):
            loop.x.copy_(loop.inputs.index_select(0, at)[0])
        loop.u.copy_(loop.us.index_select(0, at)[0])
        capture.wait_stream(side)
        loop.step()
        loop.got[0].index_copy_(0, at, loop.out[None])
        loop.got[1].index_copy_(0, at, loop.tok[None])
        at.add_(1)
    with torch.cuda.stream(capture):
        for _ in range(STEPS):
            graph.replay()
    loop.same_as(paused)
