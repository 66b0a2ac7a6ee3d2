"""Where lf_attn_paged_chunk begins to refuse sizes for the number of their key tiles:
what counts are the items that the new tokens can have, not the sequences without any."""
import pytest

pytestmark = pytest.mark.gpu
UNSUPPORTED = 7


def attend(n_tokens, n_seqs, max_len, nkv=16, nq=32, dim=128, page=1024):
    """One new token (of the last sequence, at position 99) among rows of padding; its output and the definition's."""
    import torch
    import decode_persistent_sm_gb300 as lf
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).half()  # noqa: E731
    k, v, q = r(1, nkv, page, dim), r(1, nkv, page, dim), r(n_tokens, nq, dim)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    table, starts, lens, err = i32(n_seqs, max_len // page), i32(n_seqs + 1), i32(n_seqs), i32(1)
    starts[-1], lens[-1] = 1, 100
    out = torch.full_like(q, 9.0)
    kv = lf.paged_kv(k.data_ptr(), v.data_ptr(), table.data_ptr(), n_pages=1, n_kv_heads=nkv, page_size=page, head_dim=dim,
                     n_seqs=n_seqs, max_pages=max_len // page, dtype="f16")
    ws = torch.empty(lf.attn_paged_chunk_workspace(kv, nq, n_tokens), dtype=torch.uint8, device="cuda")
    lf.attn_paged_chunk(kv, q.data_ptr(), nq * dim, out.data_ptr(), nq * dim, None, nq, starts.data_ptr(), n_tokens,
                        lens.data_ptr(), max_len, 0, dim ** -0.5, ws.data_ptr(), ws.numel(), err.data_ptr())
    torch.cuda.synchronize()
    assert err.item() == 0 and (out[1:] == 9.0).all()
    s = torch.einsum("hgd,hjd->hgj", q[0].view(nkv, -1, dim).double(), k[0, :, :100].double()) * dim ** -0.5
    return out[0].double(), torch.einsum("hgj,hjd->hgd", s.softmax(-1), v[0, :, :100].double()).reshape(nq, dim)


@pytest.mark.parametrize("n_tokens,n_seqs,max_len", [(1, 1024, 1 << 23), (5, 900, 1 << 24), (40, 1024, 1 << 23),
                                                        (300, 1000, 1 << 24), (1, 1, 1 << 30)])
def test_sequences_without_new_tokens_do_not_count(n_tokens, n_seqs, max_len):
    assert n_tokens * (max_len + 128) * 16 < 1 << 37  # what the header says is never refused
    got, want = attend(n_tokens, n_seqs, max_len)
    # P and the result rounded to 11 bits, |v| < 6: 2^-11 (sum p |v| + |o|) and fp32 sums of 100 terms
    assert ((got - want).abs() <= 2.0 ** -11 * (6 + want.abs()) + 2.0 ** -16).all()


def test_more_key_tiles_than_32_bits_hold():
    import decode_persistent_sm_gb300 as lf
    with pytest.raises(lf.LaneformerError) as e:
        attend(1024, 1024, 1 << 23)
    assert e.value.code == UNSUPPORTED
