"""The operators of a pass over several new tokens one behind the other, as a
caller runs them: norm (8 bits) -> 8-bit product -> append -> chunk attention ->
product -> norm with the residual -> LM head -> log probabilities, over several
steps on one cache (a prompt in chunks, then drafted tokens to check)."""
import numpy as np
import pytest

import paged_reference as ref

pytestmark = pytest.mark.gpu

D, NQ, NKV, DH, V, PAGE, PAGES = 512, 8, 4, 64, 2000, 16, 24
STEPS = [[100, 70, 1], [90, 1, 130], [4, 4, 4], [1, 0, 5], [3, 2, 1]]  # new tokens of each sequence


class Model:
    def __init__(self, seed=0):
        import torch
        import decode_persistent_sm_gb300 as lf
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        n = (NQ + 2 * NKV) * DH
        w = r(n, D)
        self.w_scale = (w.abs().amax(-1) / 448).contiguous()
        self.w = (w / self.w_scale[:, None]).to(torch.float8_e4m3fn)
        self.w_scale *= D ** -0.5
        self.wo = (r(D, NQ * DH) * (NQ * DH) ** -0.5).half()
        self.head = (r(V, D) * D ** -0.5 * 2).half()
        self.gains = (1 + 0.1 * r(2, D)).half()
        self.rope = torch.from_numpy(ref.rope_table(PAGES * PAGE, DH)).cuda()
        self.emb = r(V, D)
        self.g = g
        self.table = torch.randperm(3 * PAGES, device="cuda", generator=g).view(3, PAGES).int()
        self.k = torch.zeros(3 * PAGES, NKV, PAGE, DH, dtype=torch.float16, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.kv = lf.paged_kv(self.k.data_ptr(), self.v.data_ptr(), self.table.data_ptr(), n_pages=3 * PAGES, n_kv_heads=NKV,
                              page_size=PAGE, head_dim=DH, n_seqs=3, max_pages=PAGES, dtype="f16")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        most = max(sum(s) for s in STEPS)
        self.ws = torch.full((lf.attn_paged_chunk_workspace(self.kv, NQ, most),), 255, dtype=torch.uint8, device="cuda")

    def inputs(self):
        import torch
        lens, out = np.zeros(3, dtype=np.int64), []
        for new in STEPS:
            pos = np.concatenate([lens[b] + np.arange(c) for b, c in enumerate(new)])
            lens = lens + new
            seq = np.repeat(np.arange(3), new)
            t = len(seq)
            tok = torch.randint(V, (t,), device="cuda", generator=self.g).int()
            i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
            out.append(dict(tok=tok, x=self.emb[tok.long()].contiguous(), pos=i32(pos), seq=i32(seq), lens=i32(lens),
                            starts=i32(np.concatenate([[0], np.cumsum(new)])), want=torch.roll(tok, -1).contiguous()))
        return out

    def buffers(self, t):
        import torch
        e = lambda *s, dt=torch.float16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        n = (NQ + 2 * NKV) * DH
        return dict(y8=e(t, D, dt=torch.float8_e4m3fn), s8=e(t, dt=torch.float32), qkv=e(t, n), q=e(t, NQ * DH),
                    att=e(t, NQ * DH), lse=e(t, NQ, dt=torch.float32), proj=e(t, D, dt=torch.float32),
                    res=e(t, D, dt=torch.float32), y=e(t, D), logits=e(t, V, dt=torch.float32), lp=e(t, dt=torch.float32),
                    ent=e(t, dt=torch.float32), rank=e(t, dt=torch.int32), top=e(t, 4, dt=torch.int32),
                    tlp=e(t, 4, dt=torch.float32))

    def step(self, s, b, stream, pause=None):
        import decode_persistent_sm_gb300 as lf
        p = lambda t: t.data_ptr()  # noqa: E731
        t, n = s["x"].shape[0], (NQ + 2 * NKV) * DH
        err = p(self.err)
        calls = [
            lambda: lf.add_rmsnorm(p(s["x"]), "f32", D, None, None, "f32", D, D, p(self.gains), "f16", t, D, 1e-5, p(b["y8"]),
                                   "e4m3", D, p(b["s8"]), stream),
            lambda: lf.matmul_f8(p(b["y8"]), p(b["s8"]), p(self.w), p(self.w_scale), p(b["qkv"]), "f16", t, n, D, err, stream),
            lambda: lf.kv_append_paged(self.kv, p(b["qkv"]), p(b["qkv"]) + 2 * NQ * DH, p(b["qkv"]) + 2 * (NQ + NKV) * DH,
                                       "f16", n, n, n, NQ, p(b["q"]), NQ * DH, p(s["seq"]), p(s["pos"]), t, p(self.rope),
                                       PAGES * PAGE, err, stream),
            lambda: lf.attn_paged_chunk(self.kv, p(b["q"]), NQ * DH, p(b["att"]), NQ * DH, p(b["lse"]), NQ, p(s["starts"]), t,
                                        p(s["lens"]), PAGES * PAGE, 0, DH ** -0.5, p(self.ws), self.ws.numel(), err, stream),
            lambda: lf.matmul_f16_async(p(b["att"]), p(self.wo), p(b["proj"]), t, D, NQ * DH, err, stream),
            lambda: lf.add_rmsnorm(p(b["proj"]), "f32", D, p(s["x"]), p(b["res"]), "f32", D, D, p(self.gains) + 2 * D, "f16", t,
                                   D, 1e-5, p(b["y"]), "f16", D, None, stream),
            lambda: lf.matmul_f16_async(p(b["y"]), p(self.head), p(b["logits"]), t, V, D, err, stream),
            lambda: lf.token_logprobs(p(b["logits"]), "f32", t, V, V, None, p(s["want"]), 4, p(b["lp"]), p(b["rank"]),
                                      p(b["ent"]), p(b["top"]), p(b["tlp"]), stream),
        ]
        for c in calls:
            c()
            if pause:
                pause()


def same(a, b):
    import torch
    for x, y in zip(a, b):
        for k in x:
            u, v = (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in (x[k], y[k]))
            assert torch.equal(u, v), k


def test_steps_against_plain_torch():
    import torch
    m = Model()
    steps = m.inputs()
    bufs = [m.buffers(s["x"].shape[0]) for s in steps]
    for s, b in zip(steps, bufs):
        m.step(s, b, None)
    torch.cuda.synchronize()
    assert m.err.item() == 0
    # The same pass from the library's 8-bit rows on, in 64 bits with its roundings.  The tolerances:
    #   y8    half a step of 4 bits, 2^-4 of the value (1 % for the fp32 before it), or of the subnormals, 2^-10 of the scale
    #   qkv   the rounding to 11 bits, and fp32 sums of 512 terms
    #   att   P and o rounded to 11 bits: 2^-11 (sum p |v| + |o|), with sum p |v| below 7 times the largest |o| of all rows
    #   res   fp32 sums of 512 products (their expected error is sqrt(512) 2^-24 = 1.3e-6 of the terms' size)
    #   y     the rounding to 11 bits, and res's 1e-5 of the largest value, which is below 10 times the rms
    #   lp    fp32: differences and logarithms below 16, each to 2^-21, a handful of them
    ks = [torch.zeros(0, NKV, DH, dtype=torch.float64, device="cuda") for _ in range(3)]
    vs = [k.clone() for k in ks]
    for s, b in zip(steps, bufs):
        t = s["x"].shape[0]
        x = s["x"].double()
        y = x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt() * m.gains[0].double()
        got = b["y8"].double() * b["s8"].double()[:, None]
        assert ((got - y).abs() <= y.abs().amax(-1, keepdim=True) / 448 * 2 ** -10 + y.abs() * 2 ** -4 * 1.01).all()
        qkv = (b["y8"].double() * b["s8"].double()[:, None]) @ (m.w.double() * m.w_scale.double()[:, None]).t()
        assert ((b["qkv"].double() - qkv).abs() <= qkv.abs() * 2 ** -11 + 2e-5 * qkv.abs().amax()).all()
        h = b["qkv"].double().view(t, NQ + 2 * NKV, DH)
        cs = m.rope.double()[s["pos"].long()]
        a, bb, c, sn = h[..., :DH // 2], h[..., DH // 2:], cs[:, None, :, 0], cs[:, None, :, 1]
        rot = torch.cat([a * c - bb * sn, a * sn + bb * c], -1).half().double()
        st = s["starts"].tolist()
        out = torch.zeros(t, NQ, DH, dtype=torch.float64, device="cuda")
        for i in range(3):
            r = slice(st[i], st[i + 1])
            ks[i], vs[i] = torch.cat([ks[i], rot[r, NQ:NQ + NKV]]), torch.cat([vs[i], h[r, NQ + NKV:]])
            n, new = len(ks[i]), st[i + 1] - st[i]
            q = rot[r, :NQ].view(new, NKV, NQ // NKV, DH)
            sc = torch.einsum("ihgd,jhd->hgij", q, ks[i]) * DH ** -0.5
            gone = torch.arange(n, device="cuda") > (n - new + torch.arange(new, device="cuda"))[:, None]
            p = sc.masked_fill(gone, -np.inf).softmax(-1)
            out[r] = torch.einsum("hgij,jhd->ihgd", p, vs[i]).reshape(new, NQ, DH)
        att = b["att"].double().view(t, NQ, DH)
        assert ((att - out).abs() <= 4e-3 * out.abs().amax()).all()
        res = b["att"].double() @ m.wo.double().t() + x
        assert ((b["res"].double() - res).abs() <= 1e-5 * res.abs().amax()).all()
        y = res / (res.square().mean(-1, keepdim=True) + 1e-5).sqrt() * m.gains[1].double()
        assert ((b["y"].double() - y).abs() <= y.abs() * 2 ** -11 + 1e-4).all()
        lp = torch.log_softmax(b["logits"].double(), -1)
        assert ((b["lp"].double() - lp.gather(1, s["want"].long()[:, None])[:, 0]).abs() <= 1e-5).all()
        top = b["logits"].double().sort(dim=-1, descending=True, stable=True).indices[:, :4]
        assert torch.equal(top.int(), b["top"])


def test_back_to_back_on_a_stream_and_as_graphs():
    import torch
    a, b, c = Model(), Model(), Model()
    ins = [m.inputs() for m in (a, b, c)]
    outs = [[m.buffers(s["x"].shape[0]) for s in i] for m, i in zip((a, b, c), ins)]
    for s, o in zip(ins[0], outs[0]):  # a pause behind each call
        a.step(s, o, None, torch.cuda.synchronize)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for s, o in zip(ins[1], outs[1]):
        b.step(s, o, st.cuda_stream)
    graphs = []
    for s, o in zip(ins[2], outs[2]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.step(s, o, torch.cuda.current_stream().cuda_stream)
        graphs.append(g)
    for _ in range(2):  # replayed twice: the same cache again
        c.k.zero_()
        c.v.zero_()
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert [m.err.item() for m in (a, b, c)] == [0, 0, 0]
    same(outs[0], outs[1])
    same(outs[0], outs[2])
    assert torch.equal(a.k, b.k) and torch.equal(a.k, c.k) and torch.equal(a.v, c.v)
