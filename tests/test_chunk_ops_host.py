"""Argument checks of the operators of a pass over several new tokens (no GPU
needed: every refusal here comes before the first CUDA call)."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 7
A = 1 << 20  # an aligned non-null address that is never followed
F32, F16, BF16, E4M3 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from decode_persistent_sm_gb300 import build
    build.build()
    import decode_persistent_sm_gb300 as lfp
    return lfp.load_library()



def norm(lib, **kw):
    d = dict(x=A, dx=F32, ldx=64, res=2 * A, sum=3 * A, dr=F32, ldr=64, lds=64, gain=4 * A, dg=F16, rows=2, cols=64,
             eps=1e-5, out=5 * A, do=F16, ldo=64, scale=None)
    d.update(kw)
    return lib.lf_add_rmsnorm(d["x"], d["dx"], d["ldx"], d["res"], d["sum"], d["dr"], d["ldr"], d["lds"], d["gain"],
                              d["dg"], d["rows"], d["cols"], d["eps"], d["out"], d["do"], d["ldo"], d["scale"], None)


@pytest.mark.parametrize("bad", [dict(dx=3), dict(dx=-1), dict(dr=3), dict(dg=3), dict(do=4), dict(do=-1), dict(rows=-1),
                                 dict(cols=0), dict(x=0), dict(out=0), dict(ldx=63), dict(ldr=63), dict(lds=63),
                                 dict(ldo=63), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                                 dict(eps=float("inf")), dict(do=E4M3), dict(do=E4M3, scale=A + 2), dict(x=A + 2),
                                 dict(res=A + 1), dict(sum=A + 2), dict(gain=A + 1), dict(out=A + 1), dict(sum=5 * A),
                                 dict(sum=A, dr=F16), dict(sum=A, lds=72), dict(sum=2 * A, lds=72), dict(out=A),
                                 dict(out=A, do=F32, ldo=72), dict(out=2 * A), dict(out=2 * A, do=F32, ldo=72)])
def test_norm_refusals(lib, bad):
    assert norm(lib, **bad) == INVALID


def test_norm_limits(lib):
    wide = dict(ldx=1 << 16, ldr=1 << 16, lds=1 << 16, ldo=1 << 16)
    assert norm(lib, cols=32769, **wide) == UNSUPPORTED
    assert norm(lib, cols=32768, rows=0, **wide) == OK
    assert norm(lib, rows=0, res=None, sum=None, gain=None, dr=9, dg=9) == OK
    assert norm(lib, rows=0, do=E4M3, scale=A) == OK


def matmul(lib, **kw):
    d = dict(a=A, sa=2 * A, b=3 * A, sb=4 * A, c=5 * A, dt=F16, m=5, n=7, k=32, err=A)
    d.update(kw)
    return lib.lf_matmul_f8(d["a"], d["sa"], d["b"], d["sb"], d["c"], d["dt"], d["m"], d["n"], d["k"], d["err"], None)


@pytest.mark.parametrize("bad", [dict(a=0), dict(b=0), dict(c=0), dict(err=0), dict(dt=3), dict(dt=-1), dict(m=-1),
                                 dict(n=-1), dict(k=0), dict(k=8), dict(k=40), dict(k=-16), dict(a=A + 8), dict(b=A + 4),
                                 dict(c=A + 1), dict(c=A + 2, dt=F32), dict(sa=A + 2), dict(sb=A + 1), dict(err=A + 2)])
def test_matmul_refusals(lib, bad):
    assert matmul(lib, **bad) == INVALID


def test_matmul_limits(lib):
    big = (1 << 31) - 1
    assert matmul(lib, m=big) == UNSUPPORTED
    assert matmul(lib, n=big) == UNSUPPORTED
    assert matmul(lib, m=1 << 24, n=1 << 24) == UNSUPPORTED
    assert matmul(lib, m=0) == OK and matmul(lib, n=0) == OK and matmul(lib, m=0, sa=None, sb=None) == OK


def cache(**kw):
    import decode_persistent_sm_gb300 as lf
    d = dict(n_pages=10, n_kv_heads=4, page_size=16, head_dim=64, n_seqs=3, max_pages=5, dtype="f16", page_stride=0)
    ptr = {k: kw.pop(k) for k in ("k", "v", "table") if k in kw}
    d.update(kw)
    return lf.paged_kv(ptr.get("k", A), ptr.get("v", A), ptr.get("table", A), **d)


def chunk(lib, kv=None, **kw):
    d = dict(q=A, ldq=512, out=2 * A, ldo=512, lse=A, nq=8, starts=A, n=9, lens=A, max_len=80, window=0, scale=0.1, ws=A,
             nws=1 << 40, err=A)
    d.update(kw)
    return lib.lf_attn_paged_chunk(ctypes.byref(kv or cache()), d["q"], d["ldq"], d["out"], d["ldo"], d["lse"], d["nq"],
                                   d["starts"], d["n"], d["lens"], d["max_len"], d["window"], d["scale"], d["ws"],
                                   d["nws"], d["err"], None)


@pytest.mark.parametrize("bad", [dict(n_pages=0), dict(page_size=24), dict(head_dim=24), dict(n_seqs=0), dict(dtype="f32"),
                                 dict(page_stride=4 * 16 * 64 - 8), dict(k=0), dict(v=A + 8), dict(table=A + 2),
                                 dict(max_pages=1 << 28)])
def test_bad_cache_descriptions_are_refused(lib, bad):
    kv = cache(**bad)
    assert chunk(lib, kv) == INVALID
    assert lib.lf_attn_paged_chunk_workspace(ctypes.byref(kv), 8, 9) == 0


def test_no_cache_is_refused(lib):
    assert lib.lf_attn_paged_chunk_workspace(None, 8, 9) == 0
    assert lib.lf_attn_paged_chunk(None, A, 512, A, 512, A, 8, A, 1, A, 1, 0, 1.0, A, 1 << 40, A, None) == INVALID


@pytest.mark.parametrize("bad", [dict(nq=0), dict(nq=6), dict(q=0), dict(out=0), dict(starts=0), dict(lens=0), dict(ws=0),
                                 dict(err=0), dict(q=A + 8), dict(out=A + 4), dict(lse=A + 2), dict(lens=A + 1),
                                 dict(starts=A + 2), dict(ws=A + 128), dict(err=A + 1), dict(ldq=504), dict(ldo=504),
                                 dict(ldq=516), dict(ldo=516), dict(out=A, ldo=520), dict(n=-1), dict(max_len=-1),
                                 dict(max_len=81), dict(window=-1), dict(scale=0.0), dict(scale=-1.0),
                                 dict(scale=float("inf")), dict(scale=float("nan")), dict(scale=3e38)])
def test_chunk_refusals(lib, bad):
    assert chunk(lib, **bad) == INVALID


def test_the_calls_above_are_refused_for_their_fault_alone(lib):
    import torch
    assert norm(lib, rows=0) == OK and matmul(lib, m=0) == OK and logprobs(lib, rows=0) == OK
    if not torch.cuda.is_available():
        assert norm(lib) == 3 and matmul(lib) == 3 and logprobs(lib) == 3 and chunk(lib) == 3
        assert chunk(lib, out=A) == 3  # in place


@pytest.mark.parametrize("kw,nq,n", [(dict(head_dim=48), 8, 9), (dict(head_dim=256), 8, 9), (dict(n_kv_heads=1), 17, 9),
                                     (dict(n_seqs=1025), 8, 9), (dict(), 8, (1 << 26) + 1)])
def test_chunk_shapes_without_a_kernel(lib, kw, nq, n):
    kv = cache(**kw)
    assert chunk(lib, kv, nq=nq, ldq=8192, ldo=8192, n=n) == UNSUPPORTED
    assert lib.lf_attn_paged_chunk_workspace(ctypes.byref(kv), nq, n) == 0


def logprobs(lib, **kw):
    d = dict(z=A, dt=F32, rows=2, vocab=100, ld=100, t=A, tok=A, top=5, lp=A, rank=A, ent=A, tt=A, tl=A)
    d.update(kw)
    return lib.lf_token_logprobs(d["z"], d["dt"], d["rows"], d["vocab"], d["ld"], d["t"], d["tok"], d["top"], d["lp"],
                                 d["rank"], d["ent"], d["tt"], d["tl"], None)


@pytest.mark.parametrize("bad", [dict(z=0), dict(dt=3), dict(dt=-1), dict(rows=-1), dict(vocab=0), dict(ld=99),
                                 dict(z=A + 2), dict(z=A + 1, dt=F16), dict(t=A + 2), dict(tok=A + 1), dict(lp=A + 2),
                                 dict(rank=A + 2), dict(ent=A + 1), dict(tt=A + 2), dict(tl=A + 3), dict(top=-1),
                                 dict(top=33), dict(top=5, vocab=4), dict(tok=None), dict(tok=None, lp=None),
                                 dict(tok=None, rank=None)])
def test_logprobs_refusals(lib, bad):
    assert logprobs(lib, **bad) == INVALID


def test_logprobs_limits(lib):
    assert logprobs(lib, vocab=262145, ld=262145) == UNSUPPORTED
    assert logprobs(lib, rows=0, tok=None, lp=None, rank=None) == OK
    assert logprobs(lib, rows=0, vocab=262144, ld=262144, t=None, ent=None, tt=None, tl=None, top=0) == OK


def test_the_binding_passes_types_by_name():
    import decode_persistent_sm_gb300 as lf
    with pytest.raises(KeyError):
        lf.matmul_f8(A, None, A, None, A, "f64", 0, 1, 16, A)
    with pytest.raises(lf.LaneformerError):
        lf.matmul_f8(A, None, A, None, A, "f16", 0, 1, 17, A)
    lf.matmul_f8(A, None, A, None, A, "f16", 0, 1, 16, A)
