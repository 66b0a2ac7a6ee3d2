"""The filtered draw (lf_sample_filtered) on the GPU against its definition in
64 bits.  The token is a whole number and has to be the definition's: the
kernel's masses are exact to about 2^-40, so a draw could differ only where u
lies within about 1e-12 of a border, which none of these inputs does.  The log
share is (z - max) / T - log1p(mass - 1) in fp32, two terms of one sign: a
difference and a quotient (2^-24 each), a conversion (2^-24 of the mass - 1, at
most 2^-24 of its log1p), the logarithm (two units, 2^-22) and the last
difference (2^-24) make at most 2^-21 of the result; the mass itself is good to 2^-40."""
import numpy as np
import pytest

import paged_reference as ref

pytestmark = pytest.mark.gpu


def gpu_draw(z, dtype, t=None, k=None, p=None, mp=None, u=None, ld=None, offset=0, logprob=True, stream=None):
    """z: float32 numpy [rows][vocab]; returns (tokens, log shares, the logits
    as the kernel reads them in float64)."""
    import torch
    import decode_persistent_sm_gb300 as lf
    rows, vocab = z.shape
    ld = ld or vocab
    store = torch.full((offset + rows * ld,), float("nan"), dtype=ref.torch_dtype(dtype), device="cuda")
    view = store[offset:].view(rows, ld)[:, :vocab]
    view.copy_(torch.from_numpy(z))
    dev = lambda a, dt: None if a is None else torch.from_numpy(np.broadcast_to(np.asarray(a, dtype=dt), (rows,)).copy()).cuda()  # noqa: E731
    tt, kk, pp, mm, uu = dev(t, np.float32), dev(k, np.int32), dev(p, np.float32), dev(mp, np.float32), dev(u, np.float32)
    tok = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((rows,), 7.0, dtype=torch.float32, device="cuda") if logprob else None
    ptr = lambda x: None if x is None else x.data_ptr()  # noqa: E731
    lf.sample_filtered(view.data_ptr(), dtype, rows, vocab, ld, ptr(tt), ptr(kk), ptr(pp), ptr(mm), ptr(uu), ptr(tok),
                       ptr(lp), stream)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), None if lp is None else lp.cpu().numpy(), view.double().cpu().numpy()


def check(z, dtype, t=None, k=None, p=None, mp=None, u=None, **kw):
    rows = z.shape[0]
    tok, lp, z64 = gpu_draw(z, dtype, t, k, p, mp, u, **kw)
    at = lambda a, i, d, dt: d if a is None else np.broadcast_to(np.asarray(a, dtype=dt), (rows,))[i].item()  # noqa: E731
    for i in range(rows):
        args = (at(t, i, 1.0, np.float32), at(k, i, 0, np.int32), at(p, i, 1.0, np.float32), at(mp, i, 0.0, np.float32),
                at(u, i, 0.0, np.float32))
        want, share = ref.draw(z64[i], *args)
        assert tok[i] == want, (i, tok[i], want, args)
        if lp is not None:
            if np.isnan(share):
                assert np.isnan(lp[i])
            else:
                assert abs(lp[i] - share) <= 2.0 ** -21 * abs(share) + 2.0 ** -40, (i, lp[i], share)
    return tok


def params(g, rows):
    pick = lambda *v: g.choice(v, rows)  # noqa: E731
    return dict(t=pick(0.0, 0.3, 0.7, 1.0, 1.5, 30.0), k=pick(0, 1, 2, 17, 50, 5000), p=pick(1.0, 0.2, 0.8, 0.95, 0.999),
                mp=pick(0.0, 0.0, 1e-4, 0.05, 0.5), u=g.random(rows, dtype=np.float32))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 32000), (7, 1024), (40, 1000), (3, 50257), (16, 32000), (200, 37), (90, 2500)])
def test_draws(dtype, rows, vocab):
    g = np.random.default_rng(rows + vocab)
    z = (2.5 * g.standard_normal((rows, vocab))).astype(np.float32)
    check(z, dtype, **params(g, rows))


@pytest.mark.parametrize("rows,vocab,dtype", [(2, 262144, "f32"), (3, 262143, "bf16"), (160, 100001, "f32"),
                                              (300, 60000, "f16")])
def test_large_vocabularies(rows, vocab, dtype):
    g = np.random.default_rng(vocab)
    z = (2.0 * g.standard_normal((rows, vocab))).astype(np.float32)
    check(z, dtype, **params(g, rows))


def test_each_filter_alone_and_none():
    g = np.random.default_rng(11)
    rows = 64
    z = (3.0 * g.standard_normal((rows, 5003))).astype(np.float32)
    u = g.random(rows, dtype=np.float32)
    check(z, "f32", u=u)  # every parameter NULL
    check(z, "f32", t=np.linspace(0.05, 4, rows), u=u)
    check(z, "f32", k=np.arange(rows) - 3, u=u)
    check(z, "f32", k=5002 + np.arange(rows) % 3, u=u)  # one short of the vocabulary, equal to it, above it
    check(z, "f32", p=np.linspace(1e-6, 1, rows), u=u)
    check(z, "f32", mp=np.linspace(0, 1, rows), u=u)


@pytest.mark.parametrize("vocab", [1, 2, 31, 33, 512, 513, 4096, 16385])
def test_odd_vocabularies(vocab):
    g = np.random.default_rng(vocab)
    z = (2.0 * g.standard_normal((50, vocab))).astype(np.float32)
    check(z, "f32", **params(g, 50))


def test_edges_of_u():
    z = np.log(np.array([[0.25, 0.25, 0.25, 0.25]], dtype=np.float32)).repeat(6, 0)
    tok = check(z, "f32", u=[0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 0.24999])
    assert list(tok) == [0, 1, 2, 3, 3, 0]
    assert list(check(z, "f32", t=[-0.0, 1, 1, 1, 1, 1], mp=-0.0, u=[-0.0, -0.0, 1e-45, 1e-38, 2.0 ** -149, 1e-20])) == [0] * 6


def test_equal_logits():
    # ties at the k-th value and at the nucleus border are all kept; greedy takes the lowest index
    z = np.zeros((8, 3001), dtype=np.float32)
    z[:, 1000:] = -1.0
    u = np.linspace(0, 0.999, 8)
    check(z, "f32", k=10, u=u)
    check(z, "f32", p=0.01, u=u)
    check(z, "f32", k=1005, p=0.9, u=u)
    assert (check(z, "bf16", t=0.0, u=u) == 0).all()
    z[:, :1000] = 0.0
    z[:, 5:1000:2] = -0.0  # -0 and +0 are equal
    check(z, "f32", k=3, u=u)
    check(np.full((4, 40000), 3.25, dtype=np.float32), "f16", k=7, p=0.5, mp=0.9, u=[0.0, 0.4, 0.6, 0.99])


def test_many_ties_in_16_bits():
    g = np.random.default_rng(8)
    z = np.round(4 * g.standard_normal((30, 30000))).astype(np.float32) / 4
    check(z, "bf16", **params(g, 30))


def test_masked_logits():
    g = np.random.default_rng(5)
    z = (2.0 * g.standard_normal((40, 9000))).astype(np.float32)
    z[g.random(z.shape) < 0.95] = -np.inf
    z[:, 4321] = 0.5
    check(z, "f32", **params(g, 40))
    few = np.full((24, 40000), -np.inf, dtype=np.float32)  # fewer tokens than top_k, all in one part of the row or spread
    few[:12, 39000:39030] = g.standard_normal((12, 30))
    few[12:, ::1300] = g.standard_normal((12, 31))
    check(few, "f32", t=0.8, k=np.tile([5, 30, 31, 50, 400, 39999], 4), p=np.tile([1.0, 0.9, 0.6], 8), u=g.random(24, dtype=np.float32))
    only = np.full((3, 20000), -np.inf, dtype=np.float32)
    only[0, 0] = only[1, 19999] = only[2, 777] = -5.0
    assert list(check(only, "f32", t=[1.0, 0.0, 0.7], k=[50, 0, 2], p=0.9, u=0.999)) == [0, 19999, 777]
    low = np.full((2, 3000), np.finfo(np.float32).min, dtype=np.float32)  # the type's lowest value as the mask
    low[:, 7] = 1.0
    assert (check(low, "f32", t=[1.0, 5.0], k=[3, 0], p=[0.99, 1.0], u=0.99999) == 7).all()


def test_rows_without_a_draw():
    z = np.zeros((12, 100), dtype=np.float32)
    z[0] = -np.inf
    z[1, 50] = np.nan
    t, p, mp, u = np.ones(12), np.ones(12), np.zeros(12), np.full(12, 0.5)
    t[2], t[3], t[4], p[5], p[6], p[7], mp[8], mp[9], u[10], u[11] = -1, np.inf, np.nan, 0, 1.5, np.nan, -0.1, 1.1, 1.0, -0.5
    tok = check(z, "f32", t=t, p=p, mp=mp, u=u)
    assert (tok == -1).all()


def test_infinite_logits():
    z = np.zeros((6, 3000), dtype=np.float32)
    z[:, [5, 900, 2999]] = np.inf
    z[:, 100] = -np.inf
    tok = check(z, "f32", t=[1.0, 0.0, 2.0, 0.5, 1.0, 1.0], k=[0, 0, 2, 1, 10, 0], p=[1, 1, 1, 0.5, 0.9, 1],
                mp=[0, 0, 0, 0, 0, 0.3], u=[0.0, 0.9, 0.5, 0.5, 0.99, 0.34])
    assert list(tok) == [5, 5, 900, 900, 2999, 900]


def test_extreme_temperatures():
    g = np.random.default_rng(13)
    z = g.standard_normal((8, 2000)).astype(np.float32)
    tok = check(z, "f32", t=[1e-38, 1e-30, 1e-5, 1e5, 1e30, 3e38, 1e-42, 1.0], p=0.9, u=0.7)
    assert (tok[[0, 5, 6]] == -1).all() and (tok[[1, 2, 3, 4, 7]] >= 0).all()
    big = z / np.abs(z).max() * np.float32(3.4e38)  # differences above the type's largest value
    check(big, "f32", t=[1.0, 1e30, 1e29, 0.5, 1e-30, 1e20, 2.0, 1e30], k=[0, 0, 9, 3, 0, 0, 0, 100], u=0.7)


def test_strides_and_alignment():
    g = np.random.default_rng(17)
    z = (2.0 * g.standard_normal((9, 4097))).astype(np.float32)
    for dtype in ("f32", "f16", "bf16"):
        for ld, off in [(4097, 1), (4100, 3), (5003, 0), (4104, 8)]:
            check(z, dtype, ld=ld, offset=off, **params(np.random.default_rng(ld), 9))
    check(z, "f32", u=0.3, logprob=False)


def test_the_draw_is_repeatable_and_follows_u():
    g = np.random.default_rng(19)
    z = np.repeat((1.0 * g.standard_normal((1, 8000))).astype(np.float32), 512, 0)
    u = (np.arange(512) / 512).astype(np.float32)
    a, la, _ = gpu_draw(z, "f32", t=1.0, p=0.97, k=4000, u=u)
    b, lb, _ = gpu_draw(z, "f32", t=1.0, p=0.97, k=4000, u=u)
    assert np.array_equal(a, b) and np.array_equal(la, lb)
    assert (np.diff(a) >= 0).all() and len(set(a)) > 300


def test_same_draw_as_the_framework_sampler():
    # lf_sample draws its u from Philox; given that u, the filtered draw is the same token
    import torch
    import decode_persistent_sm_gb300 as lf
    import oracle
    g = np.random.default_rng(23)
    z = (3.0 * g.standard_normal(32000)).astype(np.float32)
    zd, out = torch.from_numpy(z).cuda(), torch.zeros(50, dtype=torch.int32, device="cuda")
    u = []
    for i in range(50):
        lf.sample_token(zd.data_ptr(), 32000, 0.8, 0.9, 99, i, 2, out[i:].data_ptr())
        u.append(oracle.sample(z.astype(np.float64), 0.8, 0.9, 99, i, 2)[1])
    torch.cuda.synchronize()
    tok, _, _ = gpu_draw(np.repeat(z[None], 50, 0), "f32", t=0.8, p=np.float32(0.9), u=np.array(u, dtype=np.float32))
    # (lf_sample sums in fp32: a border case may differ, as its own test allows)
    assert (tok == out.cpu().numpy()).sum() >= 49


def test_captured_draw():
    import torch
    import decode_persistent_sm_gb300 as lf
    g = np.random.default_rng(29)
    z = torch.from_numpy((2.0 * g.standard_normal((5, 6000))).astype(np.float32)).cuda()
    u = torch.zeros(5, device="cuda")
    tok = torch.zeros(5, dtype=torch.int32, device="cuda")
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        lf.sample_filtered(z.data_ptr(), "f32", 5, 6000, 6000, None, None, None, None, u.data_ptr(), tok.data_ptr(), None,
                           torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        uu = g.random(5, dtype=np.float32)
        u.copy_(torch.from_numpy(uu))
        gr.replay()
        torch.cuda.synchronize()
        want = [ref.draw(z[i].double().cpu().numpy(), 1.0, 0, 1.0, 0.0, float(uu[i]))[0] for i in range(5)]
        assert list(tok.cpu().numpy()) == want
