"""Argument checks of the paged-cache operators and the filtered draw (no GPU
needed: every refusal here comes before the first CUDA call)."""
import ctypes

import numpy as np
import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 7
A = 1 << 20  # an aligned non-null address that is never followed


@pytest.fixture(scope="module")
def lib():
    from decode_persistent_sm_gb300 import build
    build.build()
    import decode_persistent_sm_gb300 as lfp
    return lfp.load_library()


def cache(**kw):
    import decode_persistent_sm_gb300 as lf
    d = dict(n_pages=10, n_kv_heads=4, page_size=16, head_dim=64, n_seqs=3, max_pages=5, dtype="f16", page_stride=0)
    ptr = {k: kw.pop(k) for k in ("k", "v", "table") if k in kw}
    d.update(kw)
    return lf.paged_kv(ptr.get("k", A), ptr.get("v", A), ptr.get("table", A), **d)


def append(lib, kv=None, **kw):
    d = dict(q=A, k=A, v=A, dt=0, ldq=512, ldk=256, ldv=256, nq=8, qo=2 * A, ldqo=512, seq=A, pos=A, n=3, rope=A, rlen=9,
             err=A)
    d.update(kw)
    return lib.lf_kv_append_paged(ctypes.byref(kv or cache()), d["q"], d["k"], d["v"], d["dt"], d["ldq"], d["ldk"],
                                  d["ldv"], d["nq"], d["qo"], d["ldqo"], d["seq"], d["pos"], d["n"], d["rope"],
                                  d["rlen"], d["err"], None)


def attend(lib, kv=None, **kw):
    d = dict(q=A, ldq=512, out=A, ldo=512, lse=A, nq=8, lens=A, max_len=80, shared=16, window=0, scale=0.1, ws=A,
             nws=0, err=A)
    d.update(kw)
    return lib.lf_attn_paged_shared(ctypes.byref(kv or cache()), d["q"], d["ldq"], d["out"], d["ldo"], d["lse"],
                                    d["nq"], d["lens"], d["max_len"], d["shared"], d["window"], d["scale"], d["ws"],
                                    d["nws"], d["err"], None)


def sample(lib, **kw):
    d = dict(z=A, dt=0, rows=2, vocab=100, ld=100, t=A, k=A, p=A, mp=A, u=A, tok=A, lp=A)
    d.update(kw)
    return lib.lf_sample_filtered(d["z"], d["dt"], d["rows"], d["vocab"], d["ld"], d["t"], d["k"], d["p"], d["mp"],
                                  d["u"], d["tok"], d["lp"], None)


BAD_CACHES = [dict(n_pages=0), dict(n_kv_heads=0), dict(page_size=0), dict(page_size=24), dict(page_size=2048),
              dict(head_dim=0), dict(head_dim=24), dict(head_dim=272), dict(n_seqs=0), dict(max_pages=0),
              dict(dtype="f32"), dict(page_stride=4 * 16 * 64 - 8), dict(page_stride=4 * 16 * 64 + 4), dict(k=0),
              dict(v=A + 8), dict(table=A + 2), dict(max_pages=1 << 28)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_cache_descriptions_are_refused(lib, bad):
    kv = cache(**bad)
    assert append(lib, kv) == INVALID
    assert attend(lib, kv) == INVALID
    assert lib.lf_attn_paged_shared_workspace(ctypes.byref(kv), 8) == 0


def test_positions_that_a_last_tile_would_carry_past_32_bits_are_refused(lib):
    most = (1 << 31) - (1 << 16)
    assert append(lib, cache(page_size=1, max_pages=most), n=0) == OK
    assert append(lib, cache(page_size=1, max_pages=most + 1), n=0) == INVALID
    assert append(lib, cache(page_size=1024, max_pages=most // 1024), n=0) == OK
    assert append(lib, cache(page_size=1024, max_pages=most // 1024 + 1), n=0) == INVALID
    assert attend(lib, cache(page_size=1024, max_pages=most // 1024 + 1)) == INVALID


def test_no_cache_is_refused(lib):
    assert lib.lf_attn_paged_shared_workspace(None, 8) == 0
    assert lib.lf_kv_append_paged(None, A, A, A, 0, 512, 256, 256, 8, A, 512, A, A, 1, A, 9, A, None) == INVALID
    assert lib.lf_attn_paged_shared(None, A, 512, A, 512, A, 8, A, 1, 0, 0, 1.0, A, 1, A, None) == INVALID


@pytest.mark.parametrize("bad", [dict(dt=3), dict(dt=-1), dict(n=-1), dict(nq=-1), dict(k=0), dict(v=0), dict(pos=0),
                                 dict(err=0), dict(q=0), dict(qo=0), dict(q=A + 4), dict(k=A + 8), dict(v=A + 2),
                                 dict(qo=A + 8), dict(ldq=511), dict(ldk=255), dict(ldv=100), dict(ldq=514),
                                 dict(ldk=258, dt=1), dict(ldqo=508), dict(ldqo=516), dict(rope=A + 8), dict(rlen=0),
                                 dict(seq=None, n=4), dict(seq=A + 1), dict(pos=A + 2), dict(qo=A),
                                 dict(qo=A, dt=2), dict(qo=A, dt=1, ldqo=520)])
def test_append_refusals(lib, bad):
    assert append(lib, **bad) == INVALID


def test_append_of_nothing_is_accepted(lib):
    assert append(lib, n=0) == OK
    assert append(lib, n=0, nq=0, q=None, qo=None) == OK
    assert append(lib, n=0, rope=None, rlen=0) == OK


@pytest.mark.parametrize("bad", [dict(nq=0), dict(nq=6), dict(q=0), dict(out=0), dict(lens=0), dict(ws=0), dict(err=0),
                                 dict(q=A + 8), dict(out=A + 4), dict(lse=A + 2), dict(lens=A + 1), dict(ws=A + 128),
                                 dict(ldq=504), dict(ldo=504), dict(ldq=516), dict(ldo=516), dict(max_len=-1),
                                 dict(max_len=81), dict(shared=-1), dict(shared=81), dict(max_len=10), dict(window=-1),
                                 dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
                                 dict(scale=3e38)])
def test_attention_refusals(lib, bad):
    assert attend(lib, **bad) == INVALID


def test_the_calls_above_are_refused_for_their_fault_alone(lib):
    # the unchanged call passes every check of the arguments: without a GPU it
    # fails at the first CUDA call, with one at the workspace of 0 bytes
    import torch
    assert attend(lib) == (INVALID if torch.cuda.is_available() else 3)


@pytest.mark.parametrize("kw,nq", [(dict(head_dim=48), 8), (dict(head_dim=256), 8), (dict(n_kv_heads=1), 17),
                                   (dict(n_seqs=1025), 8)])
def test_attention_shapes_without_a_kernel(lib, kw, nq):
    kv = cache(**kw)
    assert attend(lib, kv, nq=nq, ldq=8192, ldo=8192) == UNSUPPORTED
    assert lib.lf_attn_paged_shared_workspace(ctypes.byref(kv), nq) == 0


@pytest.mark.parametrize("bad", [dict(z=0), dict(dt=3), dict(rows=-1), dict(vocab=0), dict(ld=99), dict(u=None),
                                 dict(tok=0), dict(z=A + 2), dict(z=A + 1, dt=1), dict(t=A + 1), dict(k=A + 2),
                                 dict(p=A + 3), dict(mp=A + 1), dict(u=A + 2), dict(tok=A + 1), dict(lp=A + 2)])
def test_draw_refusals(lib, bad):
    assert sample(lib, **bad) == INVALID


def test_draw_limits(lib):
    assert sample(lib, vocab=262145, ld=262145) == UNSUPPORTED
    assert sample(lib, rows=0) == OK


def test_reference_draw_against_enumeration():
    # four tokens, every filter: the plain form against sets worked out by hand
    import paged_reference as ref
    z = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    keeps = {(0, 1.0, 0.0): [0, 1, 2, 3], (2, 1.0, 0.0): [1, 3], (0, 0.6, 0.0): [1, 3], (0, 0.71, 0.0): [1, 2, 3],
             (0, 1.0, 0.5): [1, 2, 3], (3, 0.8, 0.0): [1, 2, 3], (3, 0.75, 0.6): [1, 3]}
    prob = np.exp(z)
    for (k, p, mp), kept in keeps.items():
        c = np.cumsum(prob[kept]) / prob[kept].sum()
        for u in (0.0, 0.3, 0.55, 0.97):
            want = kept[int(np.searchsorted(c, u, side="right"))]
            tok, lp = ref.draw(z, 1.0, k, p, mp, u)
            assert tok == want
            assert abs(lp - np.log(prob[want] / prob[kept].sum())) < 1e-12


def test_reference_attention_against_dense_softmax():
    import paged_reference as ref
    import torch
    g = np.random.default_rng(2)
    table, n = ref.page_tables(g, 2, 4, 1)
    k, v = g.standard_normal((2, n, 1, 4, 8))
    q = g.standard_normal((2, 2, 8))
    t = torch.from_numpy
    out, lse, *_ = (x.numpy() for x in ref.attention(t(q), t(k), t(v), table, 4, [9, 0], 3, 5, 0.5))
    rows = [(table[0][j // 4], j % 4) for j in range(4, 9)]
    kk, vv = np.array([k[p, 0, r] for p, r in rows]), np.array([v[p, 0, r] for p, r in rows])
    for h in range(2):
        e = np.exp(0.5 * kk @ q[0, h])
        assert np.allclose(out[0, h], e @ vv / e.sum(), atol=1e-12)
        assert np.isclose(lse[0, h], np.log(e.sum()))
    assert not out[1].any() and np.isneginf(lse[1]).all()
