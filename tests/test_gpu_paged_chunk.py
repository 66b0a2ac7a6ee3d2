"""Attention of new tokens over a paged cache (lf_attn_paged_chunk) on the GPU
against a plain 64-bit form.

Tolerances as for the decode attention (test_gpu_paged.py): a score is off by
ds = 2^-23 (dim / 16 + 4) * scale sum |q k|, a weight by that and 2^-21 of itself
in numerator and denominator and by eps / 2 through its own rounding in the
numerator; the second sum by 2^-23 per 16 keys, joins by 2^-18; fp16 weights
below 2^-14 lose up to 2^-25 each, 2^-25 keys / (sum of exp) * max |v| in all."""
import math

import numpy as np
import pytest

import paged_reference as ref

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


class Case:
    """Sequences with `new` tokens behind `ctx` cached positions (a negative one: a
    chunk longer than its sequence).  Slots that no new token sees are NaN."""

    def __init__(self, new, ctx, nq, nkv, dim, page, dtype, window=0, seed=0, pad=0, lead=0, stride_extra=0, far=0):
        import torch
        import decode_persistent_sm_gb300 as lf
        g = np.random.default_rng(seed + dim + page)
        gen = torch.Generator(device="cuda").manual_seed(seed + dim + page)
        self.new, self.ctx, self.nq, self.nkv, self.dim, self.page = new, ctx, nq, nkv, dim, page
        self.dtype, self.window, self.lead = dtype, window, lead
        self.lens = [a + b for a, b in zip(new, ctx)]
        n, dt = len(new), ref.torch_dtype(dtype)
        max_pages = max(1, -(-max(self.lens) // page)) + 1
        self.table, n_pages = ref.page_tables(g, n, max_pages, 0)
        if far:
            self.table = np.concatenate([self.table, np.full((n, far // page), -1, dtype=np.int32)], 1)
        per = nkv * page * dim
        pool = torch.full((n_pages, 2 * per + stride_extra), float("nan"), dtype=dt, device="cuda")
        self.k = pool[:, :per].unflatten(1, (nkv, page, dim))
        self.v = pool[:, per:2 * per].unflatten(1, (nkv, page, dim))
        for b in range(n):
            lo = max(0, ctx[b] - window + 1) if window else 0
            if new[b] == 0 or self.lens[b] <= lo:
                continue
            j = np.arange(lo, self.lens[b])
            at = (torch.from_numpy(self.table[b][j // page]).cuda().long(), slice(None), torch.from_numpy(j % page).cuda())
            for c in (self.k, self.v):
                c[at] = torch.randn(len(j), nkv, dim, device="cuda", generator=gen).to(dt)
        self.tokens = lead + sum(new)
        self.rows = self.tokens + pad
        self.q = (1.5 * torch.randn(self.rows, nq, dim, device="cuda", generator=gen)).to(dt)
        self.starts = torch.from_numpy(lead + np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).int().cuda()
        self.ln = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.tb = torch.from_numpy(self.table).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scale = dim ** -0.5
        self.kv = lf.paged_kv(self.k.data_ptr(), self.v.data_ptr(), self.tb.data_ptr(), n_pages=n_pages, n_kv_heads=nkv,
                              page_size=page, head_dim=dim, n_seqs=n, max_pages=self.table.shape[1], dtype=dtype,
                              page_stride=pool.shape[1])

    def workspace(self, tokens=None):
        import torch
        import decode_persistent_sm_gb300 as lf
        n = lf.attn_paged_chunk_workspace(self.kv, self.nq, tokens or self.rows)
        assert n > 0
        return torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere: nothing in it is trusted

    def run(self, out=None, ld=None, ws=None, stream=None, lse=True, max_len=None, q=None):
        import torch
        import decode_persistent_sm_gb300 as lf
        d = self.nq * self.dim
        q = self.q if q is None else q
        out = torch.full((self.rows, d), 9.0, dtype=self.q.dtype, device="cuda") if out is None else out
        ls = torch.full((self.rows, self.nq), 9.0, dtype=torch.float32, device="cuda") if lse else None
        ws = self.workspace() if ws is None else ws
        lf.attn_paged_chunk(self.kv, q.data_ptr(), d, out.data_ptr(), ld or d, ls.data_ptr() if lse else None, self.nq,
                            self.starts.data_ptr(), self.rows, self.ln.data_ptr(),
                            self.table.shape[1] * self.page if max_len is None else max_len, self.window, self.scale,
                            ws.data_ptr(), ws.numel(), self.err.data_ptr(), stream)
        return out, ls

    def want(self):
        """out, lse and the bounds' magnitudes, in 64 bits; a value that a token
        does not see takes no part."""
        import torch
        nq, nkv, d, g = self.nq, self.nkv, self.dim, self.nq // self.nkv
        new = lambda *sh: torch.zeros(*sh, dtype=torch.float64, device="cuda")  # noqa: E731
        t = self.tokens
        out, mag, lse = new(t, nq, d), new(t, nq, d), new(t, nq) - np.inf
        qk, vmax, cond, keys = new(t, nq, 1), new(t, nq, 1), new(t, nq, 1) + 1, new(t, 1, 1)
        at = self.lead
        for b, (c, x) in enumerate(zip(self.new, self.ctx)):
            j = np.arange(max(0, self.lens[b]))
            if c and len(j):
                pg = torch.from_numpy(self.table[b][j // self.page]).cuda().long()
                row = torch.from_numpy(j % self.page).cuda()
                k, v = self.k[pg, :, row].double().transpose(0, 1), self.v[pg, :, row].double().transpose(0, 1)
                jj = torch.from_numpy(j).cuda()
                for i0 in range(0, c, 128):
                    i = torch.arange(i0, min(c, i0 + 128), device="cuda")
                    p = (x + i)[:, None]
                    sees = (jj <= p) & ((jj > p - self.window) if self.window else True)  # [i][j]
                    qb = self.q[at + i].double().view(-1, nkv, g, d).permute(1, 2, 0, 3)  # [kv][g][i][d]
                    kk = torch.where(sees.any(0)[:, None], k, 0.0)
                    sc = (self.scale * (qb @ kk[:, None].transpose(2, 3))).masked_fill(~sees, -math.inf)
                    m = sc.amax(-1, keepdim=True)
                    m = m.masked_fill(m == -math.inf, 0.0)
                    e = (sc - m).exp()
                    total = e.sum(-1, keepdim=True)
                    fin = v.isfinite()
                    vf = torch.where(fin, v, 0.0)[:, None]
                    o = (e @ vf) / total.clamp(min=1e-300)
                    # what is not finite reaches those who see it
                    for h, jx, dx in (~fin & sees.any(0)[:, None]).nonzero().tolist():
                        o[h, :, :, dx] += torch.where(sees[:, jx], v[h, jx, dx], 0.0)
                    rows = lambda y: y.permute(2, 0, 1, 3).reshape(len(i), nq, -1)  # noqa: E731
                    out[at + i], lse[at + i] = rows(o), rows(m + total.log())[..., 0]
                    mag[at + i] = rows((e @ vf.abs()) / total.clamp(min=1e-300))
                    aq = self.scale * (qb.abs() @ kk[:, None].abs().transpose(2, 3))
                    qk[at + i] = rows(aq.masked_fill(~sees, 0.0).amax(-1, keepdim=True))
                    vmax[at + i] = vf.abs().amax()
                    keys[at + i] = sees.sum(-1).double()[:, None, None]
                    cond[at + i] = rows(sees.sum(-1).double()[:, None] / total.clamp(min=1e-300)).clamp(max=1e9)
            at += c
        return [f64(y) for y in (out, lse, mag, qk, vmax, cond, keys)]

    def check(self, out, lse, err=0):
        import torch
        torch.cuda.synchronize()
        assert self.err.item() == err
        nq, d, t, lead = self.nq, self.dim, self.tokens, self.lead
        want, wl, mag, qk, vmax, cond, keys = self.want()
        eps = ref.EPS[self.dtype]
        ds = 2.0 ** -23 * (d / 16 + 4) * qk
        rel = eps / 2 + 2 * ds + 2.0 ** -18 + keys * 2.0 ** -27
        tol = rel * mag + ref.TINY_HALF[self.dtype] * (cond * vmax + 1)
        tol = tol + eps / 2 * (np.abs(want) + tol)
        got = f64(out)[:, :nq * d].reshape(-1, nq, d)
        assert (got[:lead] == 9.0).all() and (got[t:] == 9.0).all()  # rows that are nobody's
        got, want, tol, fin = got[lead:t], want[lead:], tol[lead:], np.isfinite(want[lead:])
        assert np.array_equal(got[~fin], want[~fin], equal_nan=True)
        bad = ~(np.abs(got - want) <= tol) & fin
        assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])
        if lse is not None:
            gl, wl = f64(lse), wl[lead:]
            assert (gl[:lead] == 9.0).all() and (gl[t:] == 9.0).all()
            gl = gl[lead:t]
            assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
            fin = np.isfinite(wl)
            tl = (2 * ds[..., 0] + 2.0 ** -18 + keys[..., 0] * 2.0 ** -24)[lead:] + 2.0 ** -22 * np.abs(np.where(fin, wl, 0))
            assert (np.abs(gl[fin] - wl[fin]) <= tl[fin]).all()


CASES = [
    # new, ctx, nq, nkv, dim, page, dtype, window
    ([5] * 8, [500 + 17 * i for i in range(8)], 32, 16, 128, 64, "f16", 0),
    ([1], [0], 1, 1, 128, 1, "f16", 0),
    ([1, 1], [0, 3], 2, 1, 64, 1, "bf16", 0),
    ([3, 0, 1, 2], [0, 5, 100, 63], 8, 4, 32, 16, "f16", 0),           # one without new tokens
    ([64], [0], 4, 2, 64, 16, "f16", 0),                               # a prompt from nothing
    ([65, 63, 128], [0, 1, 64], 4, 2, 128, 32, "bf16", 0),
    ([200], [300], 6, 2, 64, 8, "bf16", 0),
    ([300, 1, 1, 1, 17], [200, 1000, 77, 0, 5], 8, 2, 64, 16, "f16", 0),   # a prompt beside single tokens
    ([40, 90], [700, 30], 4, 2, 32, 4, "f16", 100),                    # windows
    ([150], [150], 3, 1, 128, 16, "f16", 1),                           # a window of one key
    ([129], [5], 16, 1, 64, 128, "bf16", 64),
    ([7, 70], [-3, -70], 4, 2, 64, 16, "f16", 0),                      # chunks longer than their sequences
    ([90], [-30], 4, 2, 128, 16, "bf16", 20),
    ([33, 20], [100, 2000], 7, 1, 128, 64, "f16", 0),                  # seven heads to a row tile's token
    ([21, 100], [10, 600], 5, 1, 32, 1024, "bf16", 0),
    ([1] * 40, [31 * i for i in range(40)], 8, 8, 64, 32, "f16", 0),   # plain decode
    ([1] * 5, [3000, 100, 0, 64, 1], 16, 1, 128, 64, "bf16", 1000),
    ([513], [0], 2, 2, 64, 2, "f16", 0),
    ([1000], [1500], 8, 4, 128, 64, "f16", 0),
    ([700, 400], [0, 3000], 16, 2, 64, 16, "bf16", 900),
    ([256, 257, 255], [128, 127, 129], 8, 8, 128, 128, "bf16", 0),
    ([600, 33], [0, 0], 12, 4, 128, 16, "f16", 0),
    ([480], [31], 16, 1, 128, 32, "bf16", 0),
    ([0, 0], [5, 9], 4, 4, 32, 8, "f16", 0),                           # nobody has a token
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_chunks(case):
    new, ctx, nq, nkv, dim, page, dtype, window = CASES[case]
    c = Case(new, ctx, nq, nkv, dim, page, dtype, window, seed=case, pad=2)
    c.check(*c.run())


@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 6, 8, 11, 16])
@pytest.mark.parametrize("new", [1, 6, 150])
def test_heads_to_a_kv_head(dim, group, new):
    c = Case([new, 2], [130, 61], 2 * group, 2, dim, 16, "bf16" if group % 2 else "f16", seed=group + new)
    c.check(*c.run())


@pytest.mark.parametrize("new,window", [(8, 0), (8, 50), (300, 0), (300, 200)])
@pytest.mark.parametrize("dim", [64, 128])
def test_strides_padding_and_no_lse(new, window, dim):
    import torch
    c = Case([new, 3], [333, 90], 8, 4, dim, 16, "f16", window, pad=5, lead=3, stride_extra=24, far=1 << 14)
    ld = 8 * dim + 40
    out = torch.full((c.rows, ld), 9.0, dtype=torch.float16, device="cuda")
    c.run(out=out, ld=ld, lse=False)
    torch.cuda.synchronize()
    assert (out[:, 8 * dim:] == 9.0).all()
    c.check(out, None)


@pytest.mark.parametrize("new", [6, 400])
def test_in_place_equals_out_of_place(new):
    import torch
    c = Case([new, 1, new], [100, 900, 0], 8, 2, 128, 32, "bf16")
    out, _ = c.run()
    q = c.q.clone().view(c.rows, -1)
    got, _ = c.run(out=q, q=q)
    torch.cuda.synchronize()
    assert torch.equal(out, got)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new,dim", [(5, 32), (5, 128), (40, 64), (300, 64), (300, 128)])
def test_values_that_are_not_finite_reach_those_who_see_them_alone(new, dim, dtype):
    # an infinite value in the middle of the chunk, a NaN in the last token's
    import torch
    c = Case([new, 2], [77, 200], 4, 2, dim, 16, dtype, seed=7)
    j = 77 + new // 2
    at = lambda b, j: (int(c.table[b][j // 16]), 1, j % 16)  # noqa: E731
    c.v[at(0, j)][3] = math.inf
    c.v[at(0, j + 1)][5] = -math.inf
    c.v[at(0, 77 + new - 1)][0] = math.nan
    c.v[at(1, 201)] = math.inf
    c.v[at(1, 201)][dim - 1] = -math.inf
    out, lse = c.run()
    c.check(out, lse)
    assert torch.isfinite(out[:new // 2]).all() and not torch.isfinite(out[new // 2]).all()


@pytest.mark.parametrize("new", [4, 300])
def test_keys_that_are_not_finite(new):
    # a NaN key makes the rows that see it NaN and no others
    import torch
    c = Case([new], [64], 4, 2, 64, 16, "f16", seed=8)
    j = 64 + new - 2
    c.k[int(c.table[0][j // 16]), 0, j % 16, 9] = math.nan
    out, lse = c.run()
    torch.cuda.synchronize()
    o = out.view(new, 4, 64)
    assert torch.isnan(o[-2:, :2]).all() and torch.isnan(lse[-2:, :2]).all()
    assert torch.isfinite(o[:-2]).all() and torch.isfinite(o[:, 2:]).all() and torch.isfinite(lse[:-2]).all()


@pytest.mark.parametrize("new,ctx", [([4] * 3, [100, 40, 0]), ([500, 1], [100, 900])])
def test_a_captured_call_follows_lengths_and_chunks(new, ctx):
    import torch
    c = Case(new, ctx, 8, 2, 64, 16, "bf16", pad=4, far=1 << 12)
    ws, out = c.workspace(), torch.full((c.rows, 8 * 64), 9.0, dtype=torch.bfloat16, device="cuda")
    c.run(ws=ws)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        _, lse = c.run(out=out, ws=ws, stream=torch.cuda.current_stream().cuda_stream)
    out.fill_(9.0)
    gr.replay()
    c.check(out, lse)
    # other chunks over the same cache: the first sequence's grows into the second's rows
    c.new = [new[0] + 1, new[1] - 1] + list(new[2:])
    c.ctx = [c.lens[b] - c.new[b] for b in range(len(new))]
    if c.new[1] == 0:
        c.ctx[1] = c.lens[1]
    c.starts.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(c.new)]).astype(np.int32)))
    out.fill_(9.0)
    lse.fill_(9.0)
    gr.replay()
    c.check(out, lse)


@pytest.mark.parametrize("new", [2, 200])
@pytest.mark.parametrize("what", ["len", "negative", "start", "order", "behind", "page"])
def test_what_only_the_device_sees_is_checked(new, what):
    import torch
    c = Case([new, new], [50, 60], 4, 2, 64, 16, "f16")
    good, _ = c.run()
    if what == "len":
        c.ln[1] = 1 << 30
    elif what == "negative":
        c.ln[1] = -5
    elif what == "start":
        c.starts[2] = c.rows + 1
    elif what == "order":
        c.starts[2] = new - 1
    elif what == "behind":
        c.starts[1:] = -7
        c.starts[2] = -6
    else:
        c.tb[1, 2] = c.k.shape[0]
    out, lse = c.run()
    torch.cuda.synchronize()
    assert c.err.item() == 1
    if what != "behind":
        assert torch.equal(out[:new], good[:new])  # the other sequence has its result
    if what in ("len", "negative"):  # taken as empty
        assert (out[new:] == 0).all() and torch.isneginf(lse[new:]).all()
    if what in ("start", "order"):
        assert (out[new:] == 9.0).all()


@pytest.mark.parametrize("new,ctx", [([3] * 5, [400, 10, 70, 1000, 0]), ([600, 20], [2000, 40])])
def test_two_calls_at_once_and_again(new, ctx):
    # two streams with workspaces of their own; the result does not depend on timing
    import torch
    c = Case(new, ctx, 16, 4, 128, 32, "f16", seed=3)
    first, _ = c.run()
    torch.cuda.synchronize()
    streams, spaces = [torch.cuda.Stream() for _ in range(2)], [c.workspace() for _ in range(2)]
    outs = [[], []]
    for _ in range(5):
        for s in range(2):
            with torch.cuda.stream(streams[s]):
                outs[s].append(c.run(ws=spaces[s], stream=streams[s].cuda_stream)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for os in outs for o in os)


def test_many_sequences():
    n = 1024
    c = Case([1 + (i % 3 == 0) for i in range(n)], [i % 41 for i in range(n)], 4, 2, 32, 16, "f16")
    c.check(*c.run())


def test_a_workspace_for_more_tokens_serves_fewer():
    import torch
    c = Case([5, 1], [100, 7], 8, 4, 64, 16, "f16")
    ws = c.workspace(5000)
    assert ws.numel() >= c.workspace().numel()
    a, b = c.run(ws=ws)[0], c.run()[0]
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_offsets_past_32_bits():
    # a cache of over 2^32 values: the pages of the sequence lie at both ends
    import torch
    import decode_persistent_sm_gb300 as lf
    nkv, page, dim, n = 2, 64, 128, 300
    n_pages = (1 << 32) // (nkv * page * dim) + 3
    k = torch.empty(n_pages, nkv, page, dim, dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    ids = [n_pages - 1, 0, n_pages - 2, 1, n_pages - 3, 2]
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2, 6, nkv, page, dim, device="cuda", generator=g).half()
    for i, p in enumerate(ids):
        k[p], v[p] = x[0, i], x[1, i]
    for q_rows in (3, 200):
        q = torch.randn(q_rows, 4, dim, device="cuda", generator=g).half()
        outs = []
        for kk, vv, t in ((k, v, ids), (x[0], x[1], list(range(6)))):
            tb = torch.tensor([t], dtype=torch.int32, device="cuda")
            kv = lf.paged_kv(kk.data_ptr(), vv.data_ptr(), tb.data_ptr(), n_pages=kk.shape[0], n_kv_heads=nkv,
                             page_size=page, head_dim=dim, n_seqs=1, max_pages=6, dtype="f16")
            ws = torch.empty(lf.attn_paged_chunk_workspace(kv, 4, q_rows), dtype=torch.uint8, device="cuda")
            st, ln = (torch.tensor(y, dtype=torch.int32, device="cuda") for y in ([0, q_rows], [n]))
            err, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty_like(q)
            lf.attn_paged_chunk(kv, q.data_ptr(), 4 * dim, out.data_ptr(), 4 * dim, None, 4, st.data_ptr(), q_rows,
                                ln.data_ptr(), n, 0, 0.1, ws.data_ptr(), ws.numel(), err.data_ptr())
            torch.cuda.synchronize()
            assert err.item() == 0
            outs.append(out)
        assert torch.equal(*outs)


def drawn(seed):
    """A batch of any kind: few or many sequences, chunks short, long, mixed and
    missing, windows, padding."""
    g = np.random.default_rng(seed)
    log = lambda a, b: int(round(math.exp(g.uniform(math.log(a), math.log(b)))))  # noqa: E731
    n, most, ctx = log(1, 30), log(1, 400), log(1, 1500)
    new = [int(g.integers(0, most + 1)) for _ in range(n)]
    if g.random() < 0.3:  # one chunk beside single tokens
        new = [most] + [1] * (n - 1)
    if g.random() < 0.3:  # drafted tokens
        new = [int(g.integers(1, 9)) for _ in range(n)]
    before = [int(g.integers(0, ctx + 1)) for _ in range(n)]
    if g.random() < 0.1:
        before[0] = -int(g.integers(0, new[0] + 1))
    nkv = int(g.choice([1, 2, 4, 8]))
    group = int(g.choice([1, 2, 3, 4, 5, 8, 16]))
    return Case(new, before, nkv * group, nkv, int(g.choice([32, 64, 128])), int(g.choice([2, 8, 16, 64, 256])),
                str(g.choice(["f16", "bf16"])), int(g.choice([0, 0, 0, 1, 60, 500])), seed=seed, pad=int(g.integers(0, 4)),
                lead=int(g.integers(0, 3)), stride_extra=int(g.choice([0, 16])))


@pytest.mark.parametrize("seed", range(60))
def test_drawn_batches(seed):
    import torch
    c = drawn(seed)
    if c.rows == 0:
        pytest.skip("nobody has a token")
    ws = c.workspace()
    for bound in (max(0, max(c.lens)), c.table.shape[1] * c.page):  # a tight bound and a loose one take other ways
        c.check(*c.run(ws=ws, max_len=bound))
    again, _ = c.run(ws=ws, max_len=max(0, max(c.lens)))
    first, _ = c.run(max_len=max(0, max(c.lens)))
    torch.cuda.synchronize()
    assert torch.equal(first, again)


@pytest.mark.parametrize("new,ctx,nq,nkv,dim", [([1], [300], 2, 2, 128), ([4], [1500], 8, 4, 128), ([20], [700], 8, 4, 64),
                                                ([30] * 2, [500, 900], 16, 4, 32), ([5] * 8, [400] * 8, 32, 16, 128),
                                                ([3] * 5, [60] * 5, 64, 4, 64), ([8] * 30, [700] * 30, 16, 8, 128),
                                                ([2] * 70, [90] * 70, 8, 8, 64), ([64] * 20, [20] * 20, 16, 8, 128),
                                                ([40] * 12, [2000] * 12, 8, 8, 64)])
def test_clusters_of_every_size(new, ctx, nq, nkv, dim):
    # few keys by 1, 2, 4 or 8 CTAs to an item, the list, and both sides of where the tensor cores begin
    c = Case(new, ctx, nq, nkv, dim, 16, "f16", seed=sum(new))
    c.check(*c.run(max_len=max(c.lens)))


def test_a_row_tile_longer_than_a_warps_prefix_sum():
    # more than 32 row tiles to a sequence, on warp-level MMAs (head_dim 32) and on the tensor cores
    c = Case([1500], [100], 4, 1, 32, 16, "f16", seed=1)
    c.check(*c.run())
    c = Case([2300, 3], [50, 9], 16, 1, 64, 32, "bf16", seed=2)
    c.check(*c.run())


@pytest.mark.parametrize("dim", [64, 128])
def test_values_that_are_not_finite_and_come_late_reach_every_row(dim):
    # one masked tile to an item of two row tiles, its scores ready before its values: these alone come from far memory
    import torch
    c = Case([100 + i % 28 for i in range(60)], [0] * 60, 8, 4, dim, 64, "f16", seed=3)
    page = torch.from_numpy(c.table[:, 0]).cuda().long()
    c.v[page, :, 3, 7] = float("inf")
    want, lse = c.run()
    c.check(want, lse)
    far = torch.empty(1 << 26, dtype=torch.float32, device="cuda")
    for _ in range(20):
        far.zero_()
        c.k.sum(), c.q.sum()
        out, again = c.run()
        assert torch.equal(out, want) and torch.equal(again, lse)


@pytest.mark.parametrize("tokens", [1 << 14, 1 << 18])
def test_starts_that_claim_all_rows_many_times_over(tokens):
    # every second sequence claims every row, 2^32 key tiles in all: refused on the device, no row touched
    import torch
    import decode_persistent_sm_gb300 as lf
    n, page, pages, dim = 1024, 1024, 1024, 64
    e = lambda *s, dt=torch.float16, v=0: torch.full(s, v, dtype=dt, device="cuda")  # noqa: E731
    k, v, table = e(1, 1, page, dim), e(1, 1, page, dim), e(n, pages, dt=torch.int32)
    q, out, err = e(tokens, dim), e(tokens, dim, v=9.0), e(1, dt=torch.int32)
    starts = (torch.arange(n + 1, device="cuda") % 2 * tokens).int()
    lens = e(n, dt=torch.int32, v=page * pages)
    kv = lf.paged_kv(k.data_ptr(), v.data_ptr(), table.data_ptr(), n_pages=1, n_kv_heads=1, page_size=page, head_dim=dim,
                     n_seqs=n, max_pages=pages, dtype="f16")
    ws = e(lf.attn_paged_chunk_workspace(kv, 1, tokens), dt=torch.uint8, v=255)
    lf.attn_paged_chunk(kv, q.data_ptr(), dim, out.data_ptr(), dim, None, 1, starts.data_ptr(), tokens, lens.data_ptr(),
                        page * pages, 0, 0.125, ws.data_ptr(), ws.numel(), err.data_ptr())
    torch.cuda.synchronize()
    assert err.item() == 1 and (out == 9.0).all()


@pytest.mark.parametrize("far", [0, 640, 4096])
@pytest.mark.parametrize("new,ctx,nq,nkv,dim,window", [
    ([120], [30], 4, 2, 64, 0), ([130, 70], [300, 0], 8, 2, 128, 0), ([100, 1, 60], [900, 5, 0], 4, 1, 64, 0),
    ([90], [700], 6, 2, 128, 300), ([300], [-20], 3, 1, 128, 0), ([257, 0, 128], [1000, 0, 1], 16, 4, 64, 0),
])
def test_a_cluster_to_an_item_on_tensor_cores(new, ctx, nq, nkv, dim, window, far):
    # far: a bound far above the lengths, so that clusters are larger than their items and some CTAs have no keys
    c = Case(new, ctx, nq, nkv, dim, 64, "bf16" if dim == 64 else "f16", window, seed=far, pad=1, far=far)
    c.check(*c.run())


def test_a_chunk_alone_and_among_sequences_without_new_tokens():
    # a chunk alone, and beside so many sequences without new tokens that there is no cluster for an item
    a = Case([200], [500], 8, 2, 128, 64, "f16", seed=4)
    b = Case([200] + [0] * 200, [500] + [0] * 200, 8, 2, 128, 64, "f16", seed=4)
    for c in (a, b):
        c.check(*c.run())
