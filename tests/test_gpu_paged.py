"""The paged-cache operators (lf_kv_append_paged, lf_attn_paged_shared) on the
GPU against plain 64-bit forms.

Tolerances, derived from the arithmetic (eps = step of the output's type at 1,
a rounding is off by at most eps / 2 of the value):
 - append: the rotation is two products and a sum in fp32, each within 2^-24 of
   the terms' magnitude: 3 * 2^-24 (|x cos| + |y sin|) before the one rounding.
 - attention: a score is a product sum in fp32 whose steps the tensor core may
   truncate (2^-23 of the magnitude per 16 products, two more for the scale):
   ds = 2^-23 (dim / 16 + 4) * scale sum |q k|, and the exponential adds 2^-21;
   a weight p_j is then off by ds + 2^-21 of itself in both numerator and
   denominator, by eps / 2 through its own rounding in the numerator, and the
   second sum by 2^-23 per 16 keys: out is off by at most
   (eps / 2 + 2 ds + 2^-20 + keys 2^-27 + 2^-22) sum p |v| before its own
   rounding; fp16 weights below 2^-14 lose up to 2^-25 each besides, which is
   2^-25 keys / (sum of exp) * max |v|.  The rescaling of partial results adds
   2^-21 per join, covered by 2^-18."""
import numpy as np
import pytest

import paged_reference as ref

pytestmark = pytest.mark.gpu


def make_cache(k, v, table, page, dtype, stride=0):
    import decode_persistent_sm_gb300 as lf
    return lf.paged_kv(k.data_ptr(), v.data_ptr(), table.data_ptr(), n_pages=k.shape[0], n_kv_heads=k.shape[1],
                       page_size=page, head_dim=k.shape[-1], n_seqs=table.shape[0], max_pages=table.shape[1],
                       dtype=dtype, page_stride=stride)


def f64(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("src,dtype", [("f32", "f16"), ("f16", "f16"), ("bf16", "bf16"), ("f32", "bf16"), ("f16", "bf16"),
                                       ("bf16", "f16")])
@pytest.mark.parametrize("nq,nkv,dim,page", [(32, 16, 128, 64), (8, 4, 32, 1), (3, 1, 48, 16), (5, 5, 256, 8), (2, 2, 16, 128)])
def test_append(src, dtype, nq, nkv, dim, page):
    import torch
    import decode_persistent_sm_gb300 as lf
    g = np.random.default_rng(nq * dim + page)
    n_seqs, max_len, pad = 3, 150, 32
    table, n_pages = ref.page_tables(g, n_seqs, -(-max_len // page), 0)
    # ragged: 70 positions of sequence 2, 1 of sequence 0, padding among them
    seq = np.array([2] * 70 + [0] + [-1, -1] + [1] * 7, dtype=np.int32)
    pos = np.array(list(range(70)) + [149] + [5, -9] + list(range(33, 40)), dtype=np.int32)
    t = len(seq)
    x = torch.from_numpy(g.standard_normal((t, (nq + 2 * nkv) * dim + pad))).cuda().to(ref.torch_dtype(src))
    rope = torch.from_numpy(ref.rope_table(max_len, dim)).cuda()
    k = torch.full((n_pages, nkv, page, dim), 7.0, dtype=ref.torch_dtype(dtype), device="cuda")
    v, qo = k.clone(), torch.full((t, nq * dim + 16), 7.0, dtype=ref.torch_dtype(dtype), device="cuda")
    tb, sq, ps = (torch.from_numpy(a).cuda() for a in (table, seq, pos))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = make_cache(k, v, tb, page, dtype)
    e = x.element_size()
    at, ld = x.data_ptr(), x.shape[1]
    lf.kv_append_paged(kv, at, at + nq * dim * e, at + (nq + nkv) * dim * e, src, ld, ld, ld, nq, qo.data_ptr(),
                       nq * dim + 16, sq.data_ptr(), ps.data_ptr(), t, rope.data_ptr(), max_len, err.data_ptr())
    torch.cuda.synchronize()
    assert err.item() == 0
    xs = f64(x)[:, :(nq + 2 * nkv) * dim].reshape(t, nq + 2 * nkv, dim)
    y, mag = ref.rotate(xs[:, :nq + nkv], f64(rope)[np.maximum(pos, 0)])
    tol = ref.EPS[dtype] / 2 * np.abs(y) + 3 * 2.0 ** -24 * mag + ref.TINY_HALF[dtype]
    tol *= 1 + ref.EPS[dtype]
    want_k, want_v, tol_k = np.full(k.shape, 7.0), np.full(v.shape, 7.0), np.zeros(k.shape)
    got_q = f64(qo)
    for i in range(t):
        if seq[i] < 0:
            assert (got_q[i] == 7.0).all()
            continue
        assert (np.abs(got_q[i, :nq * dim].reshape(nq, dim) - y[i, :nq]) <= tol[i, :nq]).all()
        p, r = table[seq[i]][pos[i] // page], pos[i] % page
        want_k[p, :, r], tol_k[p, :, r] = y[i, nq:], tol[i, nq:]
        want_v[p, :, r] = f64(torch.from_numpy(xs[i, nq + nkv:]).to(ref.torch_dtype(dtype)))
    assert (got_q[:, nq * dim:] == 7.0).all()
    assert (np.abs(f64(k) - want_k) <= tol_k).all()
    assert np.array_equal(f64(v), want_v)  # values are rounded only; every other slot is as it was


def test_append_without_rotation_without_queries_and_in_place():
    import torch
    import decode_persistent_sm_gb300 as lf
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.zeros(6, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.tensor([[0, 3], [5, 1]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([6, 1], dtype=torch.int32, device="cuda")
    x = torch.randn(2, 2, 2, 64, device="cuda", generator=g).bfloat16()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = make_cache(k, v, table, 4, "bf16")
    # sequence t for token t, no rotation, no queries
    lf.kv_append_paged(kv, None, x.data_ptr(), x.data_ptr() + 2 * 128, "bf16", 0, 256, 256, 0, None, 0, None,
                       pos.data_ptr(), 2, None, 0, err.data_ptr())
    torch.cuda.synchronize()
    assert torch.equal(k[3, :, 2], x[0, 0]) and torch.equal(k[5, :, 1], x[1, 0])
    assert torch.equal(v[3, :, 2], x[0, 1]) and torch.equal(v[5, :, 1], x[1, 1])
    assert k.count_nonzero() == x[:, 0].count_nonzero() and err.item() == 0
    # queries rotated in place equal the ones rotated into another array
    q = torch.randn(2, 4, 64, device="cuda", generator=g).bfloat16()
    out, rope = torch.empty_like(q), torch.from_numpy(ref.rope_table(8, 64)).cuda()
    for dst in (out, q):
        lf.kv_append_paged(kv, q.data_ptr(), x.data_ptr(), x.data_ptr() + 2 * 128, "bf16", 256, 256, 256, 4,
                           dst.data_ptr(), 256, None, pos.data_ptr(), 2, rope.data_ptr(), 8, err.data_ptr())
    torch.cuda.synchronize()
    assert torch.equal(out, q) and err.item() == 0


@pytest.mark.parametrize("seq,pos,page", [(2, 0, 0), (0, 8, 0), (0, -1, 0), (0, 7, 0), (0, 0, 6), (0, 0, -1), (0, 0, 1 << 30)])
def test_append_checks_what_it_reads_on_the_device(seq, pos, page):
    # sequence, position (past the table, below 0, past the rotation's rows) and page out of range: skipped and flagged
    import torch
    import decode_persistent_sm_gb300 as lf
    k = torch.zeros(6, 2, 4, 64, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.tensor([[page, 3], [5, 1]], dtype=torch.int32, device="cuda")
    sq, ps = torch.tensor([1, seq], dtype=torch.int32, device="cuda"), torch.tensor([2, pos], dtype=torch.int32, device="cuda")
    x = torch.ones(2, 5, 64, dtype=torch.float16, device="cuda")
    q = torch.zeros(2, 1, 64, dtype=torch.float16, device="cuda")
    rope = torch.from_numpy(ref.rope_table(7, 64)).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lf.kv_append_paged(make_cache(k, v, table, 4, "f16"), x.data_ptr(), x.data_ptr() + 128, x.data_ptr() + 384, "f16",
                       320, 320, 320, 1, q.data_ptr(), 64, sq.data_ptr(), ps.data_ptr(), 2, rope.data_ptr(), 7,
                       err.data_ptr())
    torch.cuda.synchronize()
    assert err.item() == 1
    assert v.sum() == 128 and (v[5, :, 2] == 1).all() and not q[1].any() and q[0].any()


# ------------------------------------------------------------- attention

class Case:
    """A batch over a paged cache in which only the positions that some
    sequence sees hold numbers; everything else is NaN."""

    def __init__(self, lens, shared, nq, nkv, dim, page, dtype, window=0, seed=0, stride_extra=0, spare=2, wide=False):
        import torch
        g = np.random.default_rng(seed + dim + page + shared)
        gen = torch.Generator(device="cuda").manual_seed(seed + dim + page + shared)
        n = len(lens)
        self.lens, self.shared, self.window, self.page, self.dtype, self.nq = lens, shared, window, page, dtype, nq
        max_pages = max(1, -(-(max(max(lens), shared)) // page)) + spare
        self.table, n_pages = ref.page_tables(g, n, max_pages, shared // page)
        if wide:  # room for 2^17 positions that no sequence reaches: the bound of the lengths is far above them
            self.table = np.concatenate([self.table, np.full((n, (1 << 17) // page - max_pages), -1, dtype=np.int32)], 1)
        dt = ref.torch_dtype(dtype)
        per = nkv * page * dim
        # K and V interleaved page by page in one pool when stride_extra is set
        pool = torch.full((n_pages, per * (2 if stride_extra else 1) + stride_extra), float("nan"), dtype=dt, device="cuda")
        pool2 = pool if stride_extra else torch.full_like(pool, float("nan"))
        self.stride = pool.shape[1] if stride_extra else 0
        self.k = pool[:, :per].unflatten(1, (nkv, page, dim))
        self.v = (pool[:, per:2 * per] if stride_extra else pool2[:, :per]).unflatten(1, (nkv, page, dim))
        for b in range(n):
            j = ref.visible(lens[b], window)
            pg = np.where(j < shared, self.table[0][j // page], self.table[b][j // page])
            for c in (self.k, self.v):
                c[torch.from_numpy(pg).cuda().long(), :, torch.from_numpy(j % page).cuda()] = torch.randn(
                    len(j), nkv, dim, device="cuda", generator=gen).to(dt)
        self.q = torch.from_numpy(1.5 * g.standard_normal((n, nq, dim))).cuda().to(dt)
        self.scale = dim ** -0.5
        self.tb = torch.from_numpy(self.table).cuda()
        self.ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.kv = make_cache(self.k, self.v, self.tb, page, dtype, self.stride)

    def workspace(self):
        import torch
        import decode_persistent_sm_gb300 as lf
        n = lf.attn_paged_shared_workspace(self.kv, self.nq)
        assert n > 0
        return torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere: nothing in it is trusted

    def run(self, out=None, lse=True, ld=None, stream=None, ws=None, max_len=None):
        import torch
        import decode_persistent_sm_gb300 as lf
        n, nq, d = self.q.shape
        if out is None:
            out = torch.full((n, nq * d), 9.0, dtype=self.q.dtype, device="cuda")
        ls = torch.full((n, nq), 9.0, dtype=torch.float32, device="cuda") if lse else None
        ws = self.workspace() if ws is None else ws
        lf.attn_paged_shared(self.kv, self.q.data_ptr(), nq * d, out.data_ptr(), ld or nq * d,
                             ls.data_ptr() if lse else None, nq, self.ln.data_ptr(),
                             self.table.shape[1] * self.page if max_len is None else max_len, self.shared, self.window,
                             self.scale, ws.data_ptr(), ws.numel(), self.err.data_ptr(), stream)
        return out, ls

    def check(self, out, lse):
        import torch
        torch.cuda.synchronize()
        assert self.err.item() == 0
        n, nq, d = self.q.shape
        want, wl, mag, qk, vmax, cond = (x.cpu().numpy() for x in ref.attention(
            self.q, self.k, self.v, self.table, self.page, self.lens, self.shared, self.window, self.scale))
        eps = ref.EPS[self.dtype]
        keys = np.array([len(ref.visible(x, self.window)) for x in self.lens])[:, None, None]
        ds = 2.0 ** -23 * (d / 16 + 4) * qk
        rel = eps / 2 + 2 * ds + 2.0 ** -18 + keys * 2.0 ** -27
        tol = rel * mag + ref.TINY_HALF[self.dtype] * (cond * vmax + 1)
        tol = tol + eps / 2 * (np.abs(want) + tol)
        got = f64(out)[:, :nq * d].reshape(n, nq, d)
        assert np.isfinite(got).all()
        bad = np.abs(got - want) > tol
        assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - want).max(), tol[bad][:5])
        if lse is not None:
            gl = f64(lse)
            assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
            fin = np.isfinite(wl)
            tl = (2 * ds[..., 0] + 2.0 ** -18 + keys[..., 0] * 2.0 ** -24) + 2.0 ** -22 * np.abs(np.where(fin, wl, 0))
            assert (np.abs(gl[fin] - wl[fin]) <= tl[fin]).all()


def lens_of(shared, own):
    return [shared + x for x in own]


CASES = [
    # lens, shared, nq, nkv, dim, page, dtype, window
    (lens_of(37, [1, 23]), 37, 8, 4, 32, 16, "f16", 0),
    (lens_of(200, [1, 63, 64, 65, 128, 300]), 200, 4, 2, 64, 16, "bf16", 0),
    (lens_of(500, [40, 130, 77]), 500, 32, 16, 128, 64, "f16", 0),
    ([1], 0, 1, 1, 128, 1, "f16", 0),
    ([1], 1, 2, 1, 64, 1, "bf16", 0),
    ([64], 64, 1, 1, 128, 64, "bf16", 0),
    ([0, 5, 0, 130], 0, 6, 2, 64, 32, "f16", 0),          # empty rows, plain paged attention
    ([0, 0], 10, 4, 4, 32, 8, "f16", 0),                  # nobody sees anything
    ([100, 400, 0, 90, 101], 100, 4, 2, 128, 16, "f16", 0),  # one sequence ends inside the common prefix
    ([50, 20, 99], 100, 4, 2, 32, 16, "bf16", 0),         # every sequence does
    (lens_of(1000, [3, 70, 200, 1]), 1000, 6, 2, 64, 16, "bf16", 256),  # windows start inside the prefix
    (lens_of(300, [5, 400, 64]), 300, 4, 2, 128, 32, "f16", 100),       # some windows start behind it
    (lens_of(300, [1, 2, 3]), 300, 4, 2, 64, 4, "f16", 1),              # a window of one key
    (lens_of(129, [7] * 9), 129, 5, 1, 128, 64, "bf16", 0),   # 45 rows
    (lens_of(190, [1 + i % 5 for i in range(23)]), 190, 3, 1, 64, 16, "f16", 0),   # 69 rows: two row tiles
    (lens_of(70, [1 + 3 * i for i in range(40)]), 70, 16, 1, 32, 16, "bf16", 0),   # 640 rows, 16 to a KV head
    (lens_of(64, [33] * 16), 64, 4, 4, 128, 64, "f16", 0),    # 16 rows of one query head
    (lens_of(64, [33] * 17), 64, 8, 8, 64, 32, "f16", 0),     # 17 rows
    (lens_of(4000, [1, 500]), 4000, 14, 2, 128, 128, "bf16", 0),
    (lens_of(33, [1000, 1, 2000]), 33, 8, 8, 64, 1024, "f16", 0),
]

# batches with many rows over a long common range (the tensor-core kernel): rows of one KV head 33, 64, 128, 129, 256,
# 257, 640; pages smaller than, equal to and larger than a tile; the common range cut inside pages at both ends
MANY = [
    # lens, shared, nq, nkv, dim, page, dtype, window
    (lens_of(23040, [1 + i for i in range(11)]), 23040, 24, 8, 128, 16, "f16", 0),
    (lens_of(11500, [5 * i + 1 for i in range(64)]), 11500, 16, 8, 64, 8, "bf16", 0),
    (lens_of(7001, [1] * 64), 7001, 32, 16, 128, 64, "bf16", 0),
    (lens_of(5801, [3] * 43), 5801, 24, 8, 128, 32, "f16", 0),
    (lens_of(6000, [70] * 64), 6000, 32, 8, 64, 128, "f16", 0),
    (lens_of(2901, [2] * 257), 2901, 8, 8, 128, 16, "bf16", 0),
    (lens_of(4700, [1 + i % 7 for i in range(80)]), 4700, 64, 8, 64, 512, "bf16", 0),
    (lens_of(9000, [1 + 3 * i for i in range(50)]), 9000, 48, 16, 128, 1024, "f16", 0),
    (lens_of(6000, [1 + 11 * i for i in range(64)]), 6000, 16, 8, 128, 16, "f16", 6200),    # windows from inside the prefix
    (lens_of(6100, [6200 if i % 16 == 5 else i for i in range(64)]), 6100, 32, 8, 64, 32, "bf16", 6000),   # some start behind it
    ([0, 500, 5990, 7] + lens_of(6000, [9] * 124), 6000, 8, 8, 128, 16, "bf16", 0),  # some end inside it, one is empty
    (lens_of(5700, [5610, 5000] + [1] * 63), 5700, 16, 16, 128, 64, "f16", 5640),  # 30 positions in common: no page
]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_attention_of_many_rows(case):
    lens, shared, nq, nkv, dim, page, dtype, window = MANY[case]
    c = Case(lens, shared, nq, nkv, dim, page, dtype, window, seed=100 + case)
    c.check(*c.run())


def test_attention_of_many_rows_strided_flagged_and_replayed():
    import torch
    c = Case(lens_of(9400, [1 + i for i in range(40)]), 9400, 64, 16, 64, 16, "bf16", stride_extra=24)
    ws, out = c.workspace(), torch.full((40, 64 * 64 + 40), 9.0, dtype=torch.bfloat16, device="cuda")
    c.run(ws=ws)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        _, lse = c.run(out=out, ld=64 * 64 + 40, ws=ws, stream=torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        gr.replay()
    torch.cuda.synchronize()
    assert (out[:, 64 * 64:] == 9.0).all()
    c.check(out, lse)
    c.tb[0, 3] = c.k.shape[0]  # a page of the common range that does not exist
    c.run(ws=ws)
    torch.cuda.synchronize()
    assert c.err.item() == 1


# with a tight bound of the lengths a short batch takes the direct kernel, with a far one the list and the join
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, wide):
    lens, shared, nq, nkv, dim, page, dtype, window = CASES[case]
    c = Case(lens, shared, nq, nkv, dim, page, dtype, window, seed=case, wide=wide)
    c.check(*c.run())


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 16])
def test_attention_groups(dim, group, wide):
    c = Case(lens_of(77, [1, 9, 150]), 77, 2 * group, 2, dim, 8, "f16" if group % 2 else "bf16", wide=wide)
    c.check(*c.run())


@pytest.mark.parametrize("n_seqs,nkv,keys", [(1, 1, 64), (1, 1, 65), (1, 1, 513), (1, 2, 4096), (5, 8, 2000), (3, 21, 300),
                                             (10, 16, 700), (38, 8, 500), (80, 8, 190), (100, 8, 129)])
def test_attention_direct_cluster_sizes(n_seqs, nkv, keys):
    # 1, 2, 4 and 8 CTAs to a sequence and head; some sequences so short that CTAs of the cluster have nothing
    g = np.random.default_rng(keys)
    lens = [keys] + [int(x) for x in g.integers(0, keys + 1, n_seqs - 1)]
    c = Case(lens, min(lens) // 2, 2 * nkv, nkv, 128, 16, "f16", spare=0)
    c.check(*c.run(max_len=keys))
    c = Case(lens, keys // 3, 3 * nkv, nkv, 64, 32, "bf16", window=keys // 2 + 1, spare=0)
    c.check(*c.run(max_len=keys))


def test_attention_of_1024_sequences():
    g = np.random.default_rng(1)
    c = Case([int(x) for x in g.integers(0, 40, 1024)], 0, 2, 1, 32, 16, "f16", spare=0)
    c.check(*c.run())


@pytest.mark.parametrize("wide", [False, True])
def test_attention_strides_interleaved_pool_and_no_lse(wide):
    import torch
    c = Case(lens_of(100, [1, 50, 90]), 100, 4, 2, 64, 16, "bf16", stride_extra=24, wide=wide)
    out = torch.full((3, 4 * 64 + 40), 9.0, dtype=torch.bfloat16, device="cuda")
    got, _ = c.run(out=out, lse=False, ld=4 * 64 + 40)
    c.check(got, None)
    assert (out[:, 4 * 64:] == 9.0).all()


def test_attention_is_repeatable_and_independent_of_the_workspace():
    import torch
    c = Case(lens_of(900, [3 * i + 1 for i in range(12)]), 900, 16, 4, 128, 16, "f16")
    a, la = c.run()
    b, lb = c.run(ws=torch.zeros_like(c.workspace()))
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)
    c.check(a, la)


@pytest.mark.parametrize("wide", [False, True])
def test_attention_captured_and_replayed_as_it_grows(wide):
    # one graph, the lengths changed between replays; another graph with its own workspace on another stream
    import torch
    full = lens_of(120, [40, 64, 1])
    c = Case(full, 120, 8, 4, 64, 16, "f16", wide=wide)
    n, nq, d = c.q.shape
    graphs = []
    for _ in range(2):
        ws, out = c.workspace(), torch.zeros(n, nq * d, dtype=c.q.dtype, device="cuda")
        lse = torch.zeros(n, nq, device="cuda")
        s = torch.cuda.Stream()
        gr = torch.cuda.CUDAGraph()
        import decode_persistent_sm_gb300 as lf
        with torch.cuda.graph(gr, stream=s):
            lf.attn_paged_shared(c.kv, c.q.data_ptr(), nq * d, out.data_ptr(), nq * d, lse.data_ptr(), nq,
                                 c.ln.data_ptr(), c.table.shape[1] * c.page, c.shared, 0, c.scale, ws.data_ptr(),
                                 ws.numel(), c.err.data_ptr(), torch.cuda.current_stream().cuda_stream)
        graphs.append((gr, out, lse, ws, s))
    for lens in ([121, 130, 121], [160, 184, 121], [0, 120, 60]):
        c.lens = lens
        c.ln.copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        for gr, out, lse, _, s in graphs:
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for _, out, lse, _, _ in graphs:
            c.check(out, lse)


@pytest.mark.parametrize("wide", [False, True])
def test_attention_and_append_on_another_stream(wide):
    import torch
    c = Case(lens_of(60, [5, 9]), 60, 4, 2, 64, 16, "f16", wide=wide)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    ws = c.workspace()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = c.run(stream=s.cuda_stream, ws=ws)
    s.synchronize()
    c.check(*got)


@pytest.mark.parametrize("most", [96, 30000])
@pytest.mark.parametrize("bad_len", [-1, 30001, 1 << 30])
def test_attention_flags_a_length_out_of_range(bad_len, most):
    import torch
    c = Case([40, 60], 20, 4, 2, 64, 16, "f16", wide=True)
    c.ln.copy_(torch.tensor([bad_len, 60], dtype=torch.int32))
    c.lens = [0, 60]
    out, lse = c.run(max_len=most)
    torch.cuda.synchronize()
    assert c.err.item() == 1
    c.err.zero_()
    c.check(out, lse)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("bad_page", [-1, 1 << 30, 1000])
def test_attention_flags_a_page_out_of_range(bad_page, wide):
    import torch
    c = Case([40, 60], 0, 4, 2, 64, 16, "f16", wide=wide)
    c.tb[0, 1] = bad_page
    out, _ = c.run()
    torch.cuda.synchronize()
    assert c.err.item() == 1
    assert torch.isfinite(out[1]).all()  # the other sequence is not touched by it


def test_offsets_past_32_bits():
    # pages 2^31 elements into the pool and beyond
    import torch
    import decode_persistent_sm_gb300 as lf
    nkv, page, dim, stride = 2, 16, 64, 1 << 28
    pool = torch.empty(18 * stride, dtype=torch.float16, device="cuda")  # 9.7 GB
    table = torch.tensor([[17, 9], [17, 16]], dtype=torch.int32, device="cuda")
    pages = pool.view(18, stride)[:, :2 * nkv * page * dim]
    kv = lf.paged_kv(pool.data_ptr(), pool.data_ptr() + 2 * nkv * page * dim, table.data_ptr(), n_pages=18, n_kv_heads=nkv,
                     page_size=page, head_dim=dim, n_seqs=2, max_pages=2, dtype="f16", page_stride=stride)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(44, 2 * nkv, dim, device="cuda", generator=g).half()
    seq = torch.tensor([0] * 28 + [1] * 16, dtype=torch.int32, device="cuda")
    pos = torch.tensor(list(range(28)) + list(range(16, 32)), dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lf.kv_append_paged(kv, None, x.data_ptr(), x.data_ptr() + 2 * nkv * dim, "f16", 0, 2 * nkv * dim, 2 * nkv * dim, 0, None, 0,
                       seq.data_ptr(), pos.data_ptr(), 44, None, 0, err.data_ptr())
    assert torch.equal(pages[9].view(2, nkv, page, dim)[0, :, 11], x[27, :nkv])
    assert torch.equal(pages[16].view(2, nkv, page, dim)[1, :, 15], x[43, nkv:])
    q = torch.randn(2, 4, dim, device="cuda", generator=g).half()
    lens = torch.tensor([28, 32], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(lf.attn_paged_shared_workspace(kv, 4), dtype=torch.uint8, device="cuda")
    lf.attn_paged_shared(kv, q.data_ptr(), 4 * dim, out.data_ptr(), 4 * dim, None, 4, lens.data_ptr(), 32, 16, 0, 0.125,
                         ws.data_ptr(), ws.numel(), err.data_ptr())
    torch.cuda.synchronize()
    assert err.item() == 0
    for b, rows in enumerate((list(range(28)), list(range(16)) + list(range(28, 44)))):
        kk, vv = f64(x)[rows, :nkv], f64(x)[rows, nkv:]
        for h in range(4):
            s = 0.125 * kk[:, h // 2] @ f64(q)[b, h]
            e = np.exp(s - s.max())
            want = e @ vv[:, h // 2] / e.sum()
            # at most 32 keys: two roundings of 2^-11 and fp32 sums
            assert np.abs(f64(out)[b, h] - want).max() <= 2.0 ** -10 * np.abs(vv[:, h // 2]).max()
