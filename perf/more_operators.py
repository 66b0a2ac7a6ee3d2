"""Timed cases of the operators of a pass over several new tokens per sequence:
the norm with the residual's addition (16 and 8 bits out), the product of 8-bit
operands with scales, the attention of a chunk of new tokens over a paged cache,
and the log probabilities of given tokens.

``run`` computes an operator in its plain form (elementary torch operations)
while ``own`` is false, and through the framework's calls while it is true.
Outputs are whole: the updated residual stream, scales and statistics among
them."""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}


def listed():
    return [
        # Five drafted tokens to check in each of 8 samples that are early in their generation: the smallest chunk.
        dict(name="chunk 8 x 5 at 512", op="chunk", seqs=8, new_lo=5, new_hi=5, ctx_lo=500, ctx_hi=640, q_heads=32,
             kv_heads=16, dim=128, page=64, window=0, cache="f16"),
        # One step of a mixed batch in a sliding-window layer: a chunk of a prompt beside single tokens, 64-wide heads.
        dict(name="chunk mixed windowed bf16", op="chunk", seqs=13, new_lo=1, new_hi=500, mixed=True, ctx_lo=1,
             ctx_hi=2500, q_heads=24, kv_heads=8, dim=64, page=16, window=1024, cache="bf16"),
        # The last 512 positions of a prompt that fills the 4096-token context, in one chunk.
        dict(name="chunk 512 at 3584", op="chunk", seqs=1, new_lo=512, new_hi=512, ctx_lo=3584, ctx_hi=3584, q_heads=32,
             kv_heads=16, dim=128, page=64, window=0, cache="f16"),
        # Two long documents read in chunks of 2048, eight query heads to a KV head.
        dict(name="chunk 2 x 2048 at 14336 bf16", op="chunk", seqs=2, new_lo=1777, new_hi=2048, ctx_lo=9001,
             ctx_hi=14336, q_heads=64, kv_heads=8, dim=128, page=32, window=0, cache="bf16"),
        # One row of the framework's vocabulary: what a single decoded token was worth.
        dict(name="logprobs 1 x 32000", op="logprobs", rows=1, vocab=32000, top=5, spread=2.5, masked=0.0, src="f32"),
        # A chunk of a prompt scored, an odd vocabulary under a grammar that forbids two thirds of it.
        dict(name="logprobs 300 x 50257 masked", op="logprobs", rows=300, vocab=50257, top=20, spread=3.0, masked=0.66,
             src="f32"),
        # Many tokens scored over a large vocabulary in 16 bits.
        dict(name="logprobs 2048 x 131072 bf16", op="logprobs", rows=2048, vocab=131072, top=8, spread=2.0, masked=0.0,
             src="bf16"),
        # One decode step of 16 samples, fp32 rows as the product leaves them, 8 bits out.
        dict(name="norm 16 x 4096 e4m3", op="norm", rows=16, cols=4096, src="f32", res="f32", out="e4m3"),
        # A 3584-position prompt, 8 bits out.
        dict(name="norm 3584 x 4096 e4m3", op="norm", rows=3584, cols=4096, src="f32", res="f32", out="e4m3"),
        # Everything in 16 bits, an odd number of wide rows.
        dict(name="norm 8191 x 7168 bf16", op="norm", rows=8191, cols=7168, src="bf16", res="bf16", out="bf16"),
        # The 16 samples' fused QKV projection.
        dict(name="matmul 16 x 8192 x 4096", op="matmul", m=16, n=8192, k=4096, out="f16"),
        # The same projection of a 3584-position prompt.
        dict(name="matmul 3584 x 8192 x 4096", op="matmul", m=3584, n=8192, k=4096, out="f16"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "logprobs", "norm", "matmul"])
    if op == "chunk":
        while True:
            kv, new, ctx = rng.choice([1, 2, 4, 8, 16]), _log(rng, 1, 2048), _log(rng, 1, 14336)
            c = dict(op=op, seqs=_log(rng, 1, 64), new_lo=rng.randint(1, new), new_hi=new, mixed=rng.random() < 0.3,
                     ctx_lo=rng.randint(0, ctx), ctx_hi=ctx, q_heads=kv * rng.choice([1, 2, 3, 4, 5, 8]), kv_heads=kv,
                     dim=rng.choice([32, 64, 128]), page=rng.choice([8, 16, 32, 64, 128]),
                     window=rng.choice([0, 0, 0, 64, 1000, 4096]), cache=rng.choice(["f16", "bf16"]))
            if c["seqs"] * c["q_heads"] * new * (new + ctx) < 4e9 and work(c)["flops"] < 9e11:
                return c
    if op == "logprobs":
        vocab = _log(rng, 100, 131072)
        return dict(op=op, rows=_log(rng, 1, min(8192, 2 ** 28 // vocab // 2)), vocab=vocab,
                    top=rng.choice([0, 1, 5, 20, 32]), spread=round(rng.uniform(1.0, 4.0), 2),
                    masked=rng.choice([0.0, 0.0, 0.3, 0.9]), src=rng.choice(["f32", "f16", "bf16"]))
    if op == "norm":
        cols = 8 * _log(rng, 8, 2048)
        return dict(op=op, rows=_log(rng, 1, min(16384, 50_000_000 // cols)), cols=cols,
                    src=rng.choice(["f32", "f16", "bf16"]), res=rng.choice(["f32", "f16", "bf16"]),
                    out=rng.choice(["f16", "bf16", "e4m3", "e4m3"]))
    return dict(op=op, m=_log(rng, 1, 3500), n=_log(rng, 64, 8192), k=16 * _log(rng, 4, 256),
                out=rng.choice(["f16", "bf16"]))


def _uneven(n, lo, hi, step):
    """n numbers from lo to hi, the same for every seed."""
    return [hi if n == 1 else lo + (hi - lo) * ((step * i + 3) % n) // max(1, n - 1) for i in range(n)]


def _split(case):
    """Every sequence's new tokens and its positions before them."""
    n = case["seqs"]
    new = _uneven(n, case["new_lo"], case["new_hi"], 5)
    if case.get("mixed"):  # one chunk, the others decode
        new = [case["new_hi"]] + [1] * (n - 1)
    return new, _uneven(n, case["ctx_lo"], case["ctx_hi"], 7)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = dict(device="cuda", generator=g)
    s = dict(case)
    if case["op"] == "chunk":
        new, ctx = _split(case)
        nkv, d, ps, n = case["kv_heads"], case["dim"], case["page"], case["seqs"]
        per = -(-max(a + b for a, b in zip(new, ctx)) // ps)
        pages = n * per
        s["table"] = torch.randperm(pages, **dev).view(n, per).int()
        s["starts"] = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).int().cuda()
        s["lens"] = torch.tensor([a + b for a, b in zip(new, ctx)], dtype=torch.int32, device="cuda")
        s["max_len"], s["tokens"], s["most"] = max(a + b for a, b in zip(new, ctx)), sum(new), max(new)
        s["k"] = torch.randn(pages, nkv, ps, d, **dev).to(DT[case["cache"]])
        s["v"] = torch.randn(pages, nkv, ps, d, **dev).to(DT[case["cache"]])
        s["q"] = (1.5 * torch.randn(sum(new), case["q_heads"], d, **dev)).to(DT[case["cache"]])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(sum(new), case["q_heads"], dtype=torch.float32, device="cuda")
        s["scale"] = d ** -0.5
        return s
    if case["op"] == "logprobs":
        rows, v, top = case["rows"], case["vocab"], case["top"]
        z = torch.empty(rows, v, device="cuda").normal_(0.0, case["spread"], generator=g)
        likely = torch.randint(v, (rows,), **dev)[:, None] + torch.arange(12, device="cuda") * (v // 12 + 1)
        z.scatter_(1, likely % v, 3.0 * case["spread"] + 3.0 * torch.rand(rows, 12, **dev))  # a model's few likely tokens
        if case["masked"]:
            z.masked_fill_(torch.rand(rows, v, **dev) < case["masked"], -math.inf)
            z[:, 0] = 0.0
        s["logits"] = z.to(DT[case["src"]])
        # text is mostly likely tokens: every other row asks for one of them
        s["token"] = torch.where(torch.rand(rows, **dev) < 0.5, likely[:, 0] % v, torch.randint(v, (rows,), **dev)).int()
        t = torch.tensor([0.6, 0.8, 1.0, 1.0], device="cuda")
        s["temperature"] = t[torch.randint(4, (rows,), **dev)]
        s["logprob"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        s["entropy"] = torch.empty_like(s["logprob"])
        s["rank"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        s["top_token"] = torch.empty(rows, top, dtype=torch.int32, device="cuda")
        s["top_logprob"] = torch.empty(rows, top, dtype=torch.float32, device="cuda")
        return s
    if case["op"] == "norm":
        rows, cols, s["res_type"] = case["rows"], case["cols"], case["res"]
        s["x"] = (0.5 * torch.randn(rows, cols, **dev)).to(DT[case["src"]])
        s["res"] = (2.0 * torch.randn(rows, cols, **dev) * (0.5 + torch.rand(rows, 1, **dev))).to(DT[case["res"]])
        s["gain"] = (1.0 + 0.1 * torch.randn(cols, **dev)).half()
        s["sum"] = torch.empty_like(s["res"])
        s["y"] = torch.empty(rows, cols, dtype=DT[case["out"]], device="cuda")
        s["scale"] = torch.empty(rows, dtype=torch.float32, device="cuda") if case["out"] == "e4m3" else None
        s["eps"] = 1e-5
        return s
    m, n, k = case["m"], case["n"], case["k"]
    s["a"] = (100.0 * torch.randn(m, k, **dev)).clamp(-448, 448).to(torch.float8_e4m3fn)
    s["b"] = (100.0 * torch.randn(n, k, **dev)).clamp(-448, 448).to(torch.float8_e4m3fn)
    s["sa"] = (0.5 + torch.rand(m, **dev)) / 100.0
    s["sb"] = (0.5 + torch.rand(n, **dev)) * (k ** -0.5 / 100.0)
    s["c"] = torch.empty(m, n, dtype=DT[case["out"]], device="cuda")
    return s


# ---- the framework's calls

def _own(s):
    import decode_persistent_sm_gb300 as lf
    if "err" not in s:
        s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if s["op"] == "chunk":
        if "kv" not in s:  # the cache's description and the workspace, made once
            t = s["table"]
            s["kv"] = lf.paged_kv(s["k"].data_ptr(), s["v"].data_ptr(), t.data_ptr(), n_pages=s["k"].shape[0],
                                  n_kv_heads=s["kv_heads"], page_size=s["page"], head_dim=s["dim"], n_seqs=t.shape[0],
                                  max_pages=t.shape[1], dtype=s["cache"])
            size = lf.attn_paged_chunk_workspace(s["kv"], s["q_heads"], s["tokens"])
            s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        ld = s["q_heads"] * s["dim"]
        lf.attn_paged_chunk(s["kv"], s["q"].data_ptr(), ld, s["out"].data_ptr(), ld, s["lse"].data_ptr(), s["q_heads"],
                            s["starts"].data_ptr(), s["tokens"], s["lens"].data_ptr(), s["max_len"], s["window"],
                            s["scale"], s["ws"].data_ptr(), s["ws"].numel(), s["err"].data_ptr())
        return s["out"], s["lse"]
    if s["op"] == "logprobs":
        z, top = s["logits"], s["top"]
        lf.token_logprobs(z.data_ptr(), s["src"], z.shape[0], z.shape[1], z.shape[1], s["temperature"].data_ptr(),
                          s["token"].data_ptr(), top, s["logprob"].data_ptr(), s["rank"].data_ptr(),
                          s["entropy"].data_ptr(), s["top_token"].data_ptr() if top else None,
                          s["top_logprob"].data_ptr() if top else None)
        return s["logprob"], s["rank"], s["entropy"], s["top_token"], s["top_logprob"]
    if s["op"] == "norm":
        cols = s["cols"]
        lf.add_rmsnorm(s["x"].data_ptr(), s["src"], cols, s["res"].data_ptr(), s["sum"].data_ptr(),
                       s["res_type"], cols, cols, s["gain"].data_ptr(), "f16", s["rows"], cols, s["eps"],
                       s["y"].data_ptr(), s["out"], cols, None if s["scale"] is None else s["scale"].data_ptr())
        return (s["sum"], s["y"]) if s["scale"] is None else (s["sum"], s["y"], s["scale"])
    lf.matmul_f8(s["a"].data_ptr(), s["sa"].data_ptr(), s["b"].data_ptr(), s["sb"].data_ptr(), s["c"].data_ptr(),
                 s["out"], s["m"], s["n"], s["k"], s["err"].data_ptr())
    return s["c"]


# ---- the plain forms

def _chunk(s):
    nq, nkv, d, w, n, most = s["q_heads"], s["kv_heads"], s["dim"], s["window"], s["seqs"], s["most"]
    g, dev = nq // nkv, s["q"].device
    first, lens = s["starts"][:-1].long(), s["lens"].long()
    new = s["starts"][1:].long() - first
    i = torch.arange(most, device=dev)
    row = torch.where(i < new[:, None], first[:, None] + i, s["tokens"])  # short chunks are padded with a row behind the last
    pos = (lens - new)[:, None] + i
    q = s["q"][row.clamp(max=s["tokens"] - 1)].float() * s["scale"]  # [sequences, most, nq, d]
    q = q.view(n, most, nkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, nkv, g * most, d)
    k, v = (s[c][s["table"].long()].float().transpose(1, 2).reshape(n, nkv, -1, d) for c in "kv")
    j = torch.arange(k.shape[2], device=dev)
    sees = (j <= pos[..., None]) & (j < lens[:, None, None])
    if w:
        sees &= j > pos[..., None] - w
    p = (q @ k.transpose(2, 3)).view(n, nkv, g, most, -1)
    p.masked_fill_(~sees[:, None, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0.0)
    p.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(n, nkv, g * most, -1) @ v).view(n, nkv, g, most, d) / total.clamp(min=1e-30)
    lse = (m + total.log())[..., 0]
    out = torch.empty(s["tokens"] + 1, nq, d, dtype=s["q"].dtype, device=dev)
    out[row] = o.permute(0, 3, 1, 2, 4).reshape(n, most, nq, d).to(s["q"].dtype)
    all_lse = torch.empty(s["tokens"] + 1, nq, device=dev)
    all_lse[row] = lse.permute(0, 3, 1, 2).reshape(n, most, nq)
    return out[:-1], all_lse[:-1]


def _logprobs(s):
    raw, v, top = s["logits"].float() + 0.0, s["vocab"], s["top"]  # (no -0 among them)
    t = s["temperature"][:, None]
    m = raw.amax(-1, keepdim=True)
    a = (raw - m) / t
    e = a.exp()
    total = e.sum(-1, keepdim=True)
    norm = total.log()
    token = s["token"].long()[:, None]
    zt = raw.gather(1, token)
    j = torch.arange(v, device=raw.device)
    rank = ((raw > zt) | ((raw == zt) & (j < token))).sum(-1)
    entropy = norm - torch.where(e > 0, a * e, 0.0).sum(-1, keepdim=True) / total
    bits = raw.view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7fffffff)).long() * v + (v - 1 - j)  # by value, then by index
    at = v - 1 - key.topk(top, -1).values % v
    lp = a.gather(1, at) - norm
    at = torch.where(lp > -math.inf, at, -1)
    return (a.gather(1, token) - norm)[:, 0], rank.int(), entropy[:, 0], at.int(), lp


def _norm(s):
    x = s["x"].float() + s["res"].float()
    y = x * (x.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * s["gain"].float()
    if s["scale"] is None:
        return x.to(s["res"].dtype), y.to(s["y"].dtype)
    scale = y.abs().amax(-1) / 448.0
    scale = torch.where(scale > 0, scale, 1.0)
    return x.to(s["res"].dtype), (y / scale[:, None]).to(s["y"].dtype), scale


def _matmul(s):
    c = (s["a"].float() @ s["b"].float().t()) * s["sa"][:, None] * s["sb"]
    return c.to(s["c"].dtype)


def run(state):
    if own:
        return _own(state)
    return {"chunk": _chunk, "logprobs": _logprobs, "norm": _norm, "matmul": _matmul}[state["op"]](state)


def work(case):
    if case["op"] == "chunk":
        nq, nkv, d, w = case["q_heads"], case["kv_heads"], case["dim"], case["window"]
        new, ctx = _split(case)
        read = sum(c + t - (max(0, c - w + 1) if w else 0) for t, c in zip(new, ctx))
        # (token, position) pairs: all before the token and itself, or the window's
        full = lambda x: x * (x + 1) // 2  # noqa: E731
        seen = sum(full(c + t) - full(c) - (full(max(0, c + t - w)) - full(max(0, c - w)) if w else 0)
                   for t, c in zip(new, ctx))
        return {"bytes": 4 * read * nkv * d + sum(new) * nq * (4 * d + 4), "flops": 4 * seen * nq * d}
    if case["op"] == "logprobs":
        rows, v = case["rows"], case["vocab"]
        return {"bytes": rows * (v * SIZE[case["src"]] + 20 + 8 * case["top"]), "flops": 5 * rows * v}
    if case["op"] == "norm":
        size = SIZE[case["src"]] + 2 * SIZE[case["res"]] + SIZE[case["out"]]
        return {"bytes": case["rows"] * (case["cols"] * size + 4) + 2 * case["cols"],
                "flops": 5 * case["rows"] * case["cols"]}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": (m + n) * (k + 4) + 2 * m * n, "flops": 2 * m * n * k}


# ---- the definitions in 64 bits, one sequence or block of rows at a time

def exact(case, seed):
    if work(case)["flops"] > 4e11 and case["op"] == "chunk":
        return None  # (several seconds of 64-bit products)
    s = prepare(case, seed)
    if case["op"] == "chunk":
        nq, nkv, d, ps, w = (case[k] for k in ("q_heads", "kv_heads", "dim", "page", "window"))
        out, lse = [], []
        new, ctx = _split(case)
        at = 0
        for b, (t, c) in enumerate(zip(new, ctx)):
            j = torch.arange(c + t, device="cuda")
            page = s["table"][b, j // ps].long()
            k, v = s["k"][page, :, j % ps].double(), s["v"][page, :, j % ps].double()  # [keys, heads, d]
            for i0 in range(0, t, 256):
                i = torch.arange(i0, min(t, i0 + 256), device="cuda")
                q = s["q"][at + i].double().view(len(i), nkv, nq // nkv, d)
                a = torch.einsum("ihgd,jhd->ihgj", q, k) * s["scale"]
                gone = (j > c + i[:, None]) | ((j <= c + i[:, None] - w) if w else False)
                a.masked_fill_(gone[:, None, None], -math.inf)
                lse.append(a.logsumexp(-1).reshape(len(i), nq))
                out.append(torch.einsum("ihgj,jhd->ihgd", a.softmax(-1), v).reshape(len(i), nq, d))
            at += t
        return torch.cat(out), torch.cat(lse)
    if case["op"] == "logprobs":
        got = []
        for r in range(0, case["rows"], 64):
            z = s["logits"][r:r + 64].double()
            lp = torch.log_softmax(z / s["temperature"][r:r + 64].double()[:, None], -1)
            t = s["token"][r:r + 64].long()[:, None]
            order = z.sort(stable=True, dim=-1, descending=True).indices
            rank = (order == t).int().argmax(-1)
            best = order[:, :case["top"]]
            blp = lp.gather(1, best)
            got.append((lp.gather(1, t)[:, 0], rank.int(), -torch.special.xlogy(lp.exp(), lp.exp()).sum(-1),
                        best.masked_fill(blp == -math.inf, -1).int(), blp))
        return tuple(torch.cat(x) for x in zip(*got))
    if case["op"] == "norm":
        x = s["x"].double() + s["res"].double()
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[1] + s["eps"]) * s["gain"].double()
        if s["scale"] is None:
            return x, y
        amax = y.abs().max(-1).values
        scale = torch.where(amax == 0, 1.0, amax / 448.0)
        q = y / scale[:, None]
        step = 2.0 ** (torch.frexp(q).exponent.double() - 4).clamp(min=-9)  # e4m3: four bits of mantissa, at least 2^-9
        return x, (q / step).round() * step, scale
    b = s["b"].double().t() * s["sb"].double()
    return torch.cat([(s["a"][i:i + 512].double() * s["sa"][i:i + 512, None].double()) @ b
                      for i in range(0, case["m"], 512)])
