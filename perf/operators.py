"""Timed cases of the serving operators: the append to a paged KV cache with
RoPE, the decode attention over that cache with a prefix that all sequences
share, and the filtered draw of a token per row.

``run`` computes an operator in its plain form (elementary torch operations)
while ``own`` is false, and through the framework's calls while it is true.
Both write the outputs, the caches among them, whole."""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # One decode step of 16 samples (the batched decode's most), fp32 rows as the QKV product leaves them.
        dict(name="append 16 samples", op="append", seqs=16, tokens=16, q_heads=32, kv_heads=16, dim=128, page=64,
             ctx=4096, src="f32", cache="f16"),
        # A 3584-position prompt written in one pass, rows of one fused FP16 projection.
        dict(name="append prompt 3584", op="append", seqs=1, tokens=3584, q_heads=32, kv_heads=16, dim=128, page=64,
             ctx=4096, src="f16", cache="f16"),
        # Several prompts of odd lengths at once, small heads and small pages.
        dict(name="append ragged 8191 bf16", op="append", seqs=7, tokens=8191, q_heads=24, kv_heads=8, dim=64,
             page=16, ctx=4096, src="bf16", cache="bf16"),
        # The smallest call: the tiny model's heads, two samples of a short prompt.
        dict(name="attend tiny", op="attend", seqs=2, q_heads=8, kv_heads=4, dim=32, page=16, shared=37, lo=1, hi=23,
             window=0, cache="f16"),
        # pass@8 early in its generation: the timed step of the decode (512 positions) as the common prompt.
        dict(name="attend 8 x 512", op="attend", seqs=8, q_heads=32, kv_heads=16, dim=128, page=64, shared=512, lo=40,
             hi=130, window=0, cache="f16"),
        # 16 samples of the long workload: 3584 positions of prompt, up to 512 of their own.
        dict(name="attend 16 x 3584", op="attend", seqs=16, q_heads=32, kv_heads=16, dim=128, page=64, shared=3584,
             lo=100, hi=512, window=0, cache="f16"),
        # A sliding-window layer whose window starts inside the prompt, 64-wide heads, ragged lengths.
        dict(name="attend 24 windowed bf16", op="attend", seqs=24, q_heads=24, kv_heads=8, dim=64, page=16, shared=1999,
             lo=1, hi=700, window=1024, cache="bf16"),
        # A large group of continuations of one long document, eight query heads to a KV head.
        dict(name="attend 64 x 16384 bf16", op="attend", seqs=64, q_heads=64, kv_heads=8, dim=128, page=32,
             shared=16384, lo=1, hi=1024, window=0, cache="bf16"),
        # One row of the framework's vocabulary, every filter on: the latency of a single draw.
        dict(name="sample 1 x 32000", op="sample", rows=1, vocab=32000, spread=2.5, masked=0.0, src="f32"),
        # The batched decode's 16 rows.
        dict(name="sample 16 x 32000", op="sample", rows=16, vocab=32000, spread=2.5, masked=0.0, src="f32"),
        # An odd vocabulary under a grammar that forbids two thirds of it, many rows.
        dict(name="sample 100 x 50257 masked", op="sample", rows=100, vocab=50257, spread=3.0, masked=0.66, src="f32"),
        # A large vocabulary in 16 bits (many equal logits), a large group of rows.
        dict(name="sample 256 x 131072 bf16", op="sample", rows=256, vocab=131072, spread=2.0, masked=0.0, src="bf16"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "sample"])
    if op == "append":
        kv = rng.choice([1, 2, 4, 8, 16])
        seqs = _log(rng, 1, 64)
        return dict(op=op, seqs=seqs, tokens=max(seqs, _log(rng, 1, 8191)), q_heads=kv * rng.choice([1, 2, 3, 4]),
                    kv_heads=kv, dim=rng.choice([32, 64, 128]), page=rng.choice([1, 8, 16, 32, 64, 128]),
                    ctx=min(8192, 32768 // seqs),
                    src=rng.choice(["f32", "f16", "bf16"]), cache=rng.choice(["f16", "bf16"]))
    if op == "attend":
        kv = rng.choice([1, 2, 4, 8])
        hi = _log(rng, 1, 1024)
        return dict(op=op, seqs=_log(rng, 1, 64), q_heads=kv * rng.choice([1, 2, 3, 4, 5, 8]), kv_heads=kv,
                    dim=rng.choice([32, 64, 128]), page=rng.choice([16, 32, 64, 128]), shared=_log(rng, 1, 16384) - 1,
                    lo=rng.randint(1, hi), hi=hi, window=rng.choice([0, 0, 0, 64, 1000, 4096]),
                    cache=rng.choice(["f16", "bf16"]))
    vocab = _log(rng, 100, 131072)
    return dict(op=op, rows=_log(rng, 1, 256), vocab=vocab, spread=round(rng.uniform(1.0, 4.0), 2),
                masked=rng.choice([0.0, 0.0, 0.3, 0.9]), src=rng.choice(["f32", "f16", "bf16"]))


def _own_lens(case):
    """The sequences' own lengths: from lo to hi, uneven, the same for every seed."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    return [hi if n == 1 else lo + (hi - lo) * ((7 * i + 3) % n) // max(1, n - 1) for i in range(n)]


def _token_split(case):
    """Tokens per sequence of an append: uneven, adding up to the case's tokens."""
    n, t = case["seqs"], case["tokens"]
    cut = [t * (i * (i + 1)) // (n * (n + 1)) for i in range(n + 1)]
    got = [cut[i + 1] - cut[i] for i in range(n)]
    return got if t > n else [1] * n


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = dict(device="cuda", generator=g)
    s = dict(case)
    if case["op"] == "append":
        nq, nkv, d, ps, n = case["q_heads"], case["kv_heads"], case["dim"], case["page"], case["seqs"]
        split = _token_split(case)
        per = -(-case["ctx"] // ps)
        start = [0 if t > 1 else (997 * (i + 1)) % case["ctx"] for i, t in enumerate(split)]
        seq = [i for i, t in enumerate(split) for _ in range(t)]
        pos = [start[i] + j for i, t in enumerate(split) for j in range(t)]
        pages = n * per
        half = torch.arange(d // 2, dtype=torch.float64, device="cuda")
        ang = torch.arange(per * ps, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2.0 * half / d)
        s["rope"] = torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()
        s["qkv"] = torch.randn(len(seq), (nq + 2 * nkv) * d, **dev).to(DT[case["src"]])
        s["q_out"] = torch.zeros(len(seq), nq, d, dtype=DT[case["cache"]], device="cuda")
        s["k"] = torch.zeros(pages, nkv, ps, d, dtype=DT[case["cache"]], device="cuda")
        s["v"] = torch.zeros_like(s["k"])
        s["table"] = torch.randperm(pages, **dev).view(n, per).int()
        s["seq"] = torch.tensor(seq, dtype=torch.int32, device="cuda")
        s["pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
        return s
    if case["op"] == "attend":
        nkv, d, ps, n, sh = case["kv_heads"], case["dim"], case["page"], case["seqs"], case["shared"]
        ahead, per = sh // ps, -(-(sh + case["hi"]) // ps)
        pages = per + (n - 1) * (per - ahead)
        order = torch.randperm(pages, **dev).int()
        table = order[:per].repeat(n, 1)
        table[1:, ahead:] = order[per:].view(n - 1, per - ahead)
        s["table"] = table.contiguous()
        s["lens"] = torch.tensor([sh + t for t in _own_lens(case)], dtype=torch.int32, device="cuda")
        s["max_len"] = sh + case["hi"]
        s["k"] = torch.randn(pages, nkv, ps, d, **dev).to(DT[case["cache"]])
        s["v"] = torch.randn(pages, nkv, ps, d, **dev).to(DT[case["cache"]])
        s["q"] = (1.5 * torch.randn(n, case["q_heads"], d, **dev)).to(DT[case["cache"]])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(n, case["q_heads"], dtype=torch.float32, device="cuda")
        s["scale"] = d ** -0.5
        return s
    rows, v = case["rows"], case["vocab"]
    z = case["spread"] * torch.randn(rows, v, **dev)
    top = torch.randint(v, (rows, 12), **dev)  # a model's few likely tokens
    z.scatter_(1, top, 3.0 * case["spread"] + 3.0 * torch.rand(rows, 12, **dev))
    if case["masked"]:
        z.masked_fill_(torch.rand(rows, v, **dev) < case["masked"], -math.inf)
        z[:, 0] = 0.0
    pick = lambda vals, dt: torch.tensor(vals, dtype=dt, device="cuda")[torch.randint(len(vals), (rows,), **dev)]  # noqa: E731
    s["logits"] = z.to(DT[case["src"]])
    s["temperature"] = pick([0.0, 0.6, 0.8, 1.0, 1.2], torch.float32)
    s["top_k"] = pick([0, 0, 1, 20, 50, 400], torch.int32)
    s["top_p"] = pick([1.0, 0.8, 0.95, 0.99], torch.float32)
    s["min_p"] = pick([0.0, 0.0, 0.001, 0.05], torch.float32)
    s["u"] = torch.rand(rows, **dev)
    s["token"] = torch.empty(rows, dtype=torch.int32, device="cuda")
    s["logprob"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    return s


# ---- the framework's calls

def _cache(s):
    """The cache's description and the attention's workspace, made once per state."""
    import decode_persistent_sm_gb300 as lf
    if "kv" not in s:
        t = s["table"]
        s["kv"] = lf.paged_kv(s["k"].data_ptr(), s["v"].data_ptr(), t.data_ptr(), n_pages=s["k"].shape[0],
                              n_kv_heads=s["kv_heads"], page_size=s["page"], head_dim=s["dim"], n_seqs=t.shape[0],
                              max_pages=t.shape[1], dtype=s["cache"])
        s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if s["op"] == "attend":
            s["ws"] = torch.empty(lf.attn_paged_shared_workspace(s["kv"], s["q_heads"]), dtype=torch.uint8, device="cuda")
    return lf, s["kv"]


def _own(s):
    if s["op"] == "append":
        lf, kv = _cache(s)
        nq, nkv, d, x = s["q_heads"], s["kv_heads"], s["dim"], s["qkv"]
        at, ld = x.data_ptr(), x.shape[1]
        e = x.element_size()
        lf.kv_append_paged(kv, at, at + nq * d * e, at + (nq + nkv) * d * e, s["src"], ld, ld, ld, nq,
                           s["q_out"].data_ptr(), nq * d, s["seq"].data_ptr(), s["pos"].data_ptr(), x.shape[0],
                           s["rope"].data_ptr(), s["rope"].shape[0], s["err"].data_ptr())
        return s["q_out"], s["k"], s["v"]
    if s["op"] == "attend":
        lf, kv = _cache(s)
        ld = s["q_heads"] * s["dim"]
        lf.attn_paged_shared(kv, s["q"].data_ptr(), ld, s["out"].data_ptr(), ld, s["lse"].data_ptr(), s["q_heads"],
                             s["lens"].data_ptr(), s["max_len"], s["shared"], s["window"], s["scale"],
                             s["ws"].data_ptr(), s["ws"].numel(), s["err"].data_ptr())
        return s["out"], s["lse"]
    import decode_persistent_sm_gb300 as lf
    z = s["logits"]
    lf.sample_filtered(z.data_ptr(), s["src"], z.shape[0], z.shape[1], z.shape[1], s["temperature"].data_ptr(),
                       s["top_k"].data_ptr(), s["top_p"].data_ptr(), s["min_p"].data_ptr(), s["u"].data_ptr(),
                       s["token"].data_ptr(), s["logprob"].data_ptr())
    return s["token"], s["logprob"]


# ---- the plain forms

def _append(s):
    nq, nkv, d, ps = s["q_heads"], s["kv_heads"], s["dim"], s["page"]
    pos, t = s["pos"].long(), s["qkv"].shape[0]
    x = s["qkv"].float().view(t, nq + 2 * nkv, d)
    c, n = s["rope"][pos].unbind(-1)
    c, n = c[:, None], n[:, None]
    a, b = x[:, :nq + nkv, :d // 2], x[:, :nq + nkv, d // 2:]
    y = torch.cat([a * c - b * n, a * n + b * c], -1).to(s["k"].dtype)
    page, slot = s["table"][s["seq"].long(), pos // ps].long(), pos % ps
    s["k"][page, :, slot] = y[:, nq:]
    s["v"][page, :, slot] = x[:, nq + nkv:].to(s["v"].dtype)
    s["q_out"].copy_(y[:, :nq])
    return s["q_out"], s["k"], s["v"]


def _attend(s):
    n, nq, nkv, d, ps, sh, w = s["lens"].shape[0], s["q_heads"], s["kv_heads"], s["dim"], s["page"], s["shared"], s["window"]
    gl, ahead, dev = nq // nkv, sh // ps, s["q"].device
    lens = s["lens"].long()
    first = (lens - w).clamp(min=0) if w else torch.zeros_like(lens)
    q = s["q"].float().view(n, nkv, gl, d) * s["scale"]
    head = s["table"][0, :-(-sh // ps)].long()

    def common(c):  # [heads, shared, d]
        return c[head].float().transpose(0, 1).reshape(nkv, -1, d)[:, :sh]

    def each(c):  # [sequences, heads, positions from ahead * ps on, d]
        return c[s["table"][:, ahead:].long()].float().transpose(1, 2).reshape(n, nkv, -1, d)

    sp = (q.transpose(0, 1).reshape(nkv, n * gl, d) @ common(s["k"]).transpose(1, 2)).view(nkv, n, gl, sh).transpose(0, 1)
    so = q @ each(s["k"]).transpose(2, 3)
    j = torch.arange(sh, device=dev)
    sees = (j < lens[:, None]) & (j >= first[:, None])
    sp = sp.masked_fill(~sees[:, None, None], -math.inf)
    j = ahead * ps + torch.arange(so.shape[-1], device=dev)
    sees = (j >= sh) & (j < lens[:, None]) & (j >= first[:, None])
    so = so.masked_fill(~sees[:, None, None], -math.inf)
    m = so.amax(-1, keepdim=True) if sh == 0 else torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
    safe = m.masked_fill(m == -math.inf, 0.0)
    pp, po = (sp - safe).exp(), (so - safe).exp()
    total = pp.sum(-1, keepdim=True) + po.sum(-1, keepdim=True)
    o = (pp.transpose(0, 1).reshape(nkv, n * gl, sh) @ common(s["v"])).view(nkv, n, gl, d).transpose(0, 1)
    o = (o + po @ each(s["v"])) / total.clamp(min=1e-30)
    return o.reshape(n, nq, d).to(s["q"].dtype), (safe + total.log()).view(n, nq)


def _sample(s):
    z = s["logits"].double()
    rows, v = z.shape
    t = s["temperature"].double()[:, None]
    warm = torch.where(t > 0, t, 1.0)
    m = z.amax(-1, keepdim=True)
    zs = z.sort(-1, descending=True).values
    k = s["top_k"].long()[:, None]
    tau_k = torch.where(k > 0, zs.gather(1, (k - 1).clamp(0, v - 1)), -math.inf)
    c = torch.where(zs >= tau_k, ((zs - m) / warm).exp(), 0.0).cumsum(-1)
    top_p = s["top_p"].double()[:, None]
    at = (c < top_p * c[:, -1:]).sum(-1, keepdim=True).clamp(max=v - 1)
    tau_p = torch.where(top_p < 1, zs.gather(1, at), -math.inf)
    tau_m = m + warm * s["min_p"].double()[:, None].log()
    kept = torch.where(z >= torch.maximum(torch.maximum(tau_k, tau_p), tau_m), ((z - m) / warm).exp(), 0.0)
    run_ = kept.cumsum(-1)
    token = (run_ <= s["u"].double()[:, None] * run_[:, -1:]).sum(-1, keepdim=True).clamp(max=v - 1)
    logprob = (kept.gather(1, token) / run_[:, -1:]).log()
    greedy = (z < m).int().argmin(-1, keepdim=True)
    token, logprob = torch.where(t > 0, token, greedy), torch.where(t > 0, logprob, 0.0)
    return token[:, 0].int(), logprob[:, 0].float()


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "attend": _attend, "sample": _sample}[state["op"]](state)


def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if case["op"] == "append":
        nq, nkv, d, t = case["q_heads"], case["kv_heads"], case["dim"], max(case["tokens"], case["seqs"])
        vals = t * (nq + 2 * nkv) * d
        return {"bytes": vals * (size[case["src"]] + size[case["cache"]]) + t * (8 + 4 * d), "flops": 3 * t * (nq + nkv) * d}
    if case["op"] == "attend":
        nq, nkv, d, n, sh, w = (case[k] for k in ("q_heads", "kv_heads", "dim", "seqs", "shared", "window"))
        lens = [sh + t for t in _own_lens(case)]
        first = [max(0, t - w) if w else 0 for t in lens]
        read = max(0, sh - min(first)) + sum(t - max(f, sh) for t, f in zip(lens, first))
        seen = sum(t - f for t, f in zip(lens, first))
        return {"bytes": 4 * read * nkv * d + 4 * n * nq * d + 4 * n * nq, "flops": 4 * seen * nq * d}
    return {"bytes": case["rows"] * (case["vocab"] * size[case["src"]] + 28), "flops": 4 * case["rows"] * case["vocab"]}


# ---- the definitions in 64 bits, one sequence, token or row at a time

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        nq, nkv, d, ps = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
        seq, pos = s["seq"].long(), s["pos"].long()
        x = s["qkv"].double().view(-1, nq + 2 * nkv, d)
        r = torch.view_as_complex(s["rope"].double())[pos][:, None]
        z = torch.complex(x[:, :nq + nkv, :d // 2].contiguous(), x[:, :nq + nkv, d // 2:].contiguous()) * r
        y = torch.cat([z.real, z.imag], -1)
        k, v = s["k"].double(), s["v"].double()
        row = (s["table"][seq, pos // ps].long() * nkv)[:, None] + torch.arange(nkv, device="cuda")
        row = row * ps + (pos % ps)[:, None]
        k.view(-1, d)[row] = y[:, nq:]
        v.view(-1, d)[row] = x[:, nq + nkv:]
        return y[:, :nq], k, v
    if case["op"] == "attend":
        nq, nkv, d, ps, sh, w = (case[k] for k in ("q_heads", "kv_heads", "dim", "page", "shared", "window"))
        out, lse = [], []
        for b, n in enumerate(s["lens"].tolist()):
            j = torch.arange(max(0, n - w) if w else 0, n, device="cuda")
            page = torch.where(j < sh, s["table"][0, j // ps], s["table"][b, j // ps]).long()
            k, v = s["k"][page, :, j % ps].double(), s["v"][page, :, j % ps].double()  # [keys, heads, d]
            q = s["q"][b].double().view(nkv, nq // nkv, d)
            a = torch.einsum("hgd,jhd->hgj", q, k) * s["scale"]
            lse.append(a.logsumexp(-1).reshape(nq))
            out.append(torch.einsum("hgj,jhd->hgd", a.softmax(-1), v).reshape(nq, d))
        return torch.stack(out), torch.stack(lse)
    if case["rows"] * case["vocab"] > 40_000_000:
        return None
    tokens, logprobs = [], []
    f = lambda k: s[k].double().cpu().numpy()  # noqa: E731
    for z, t, k, p, mp, u in zip(f("logits"), f("temperature"), f("top_k"), f("top_p"), f("min_p"), f("u")):
        best = z.max()
        if t == 0:
            tokens.append(int(np.flatnonzero(z == best)[0]))
            logprobs.append(0.0)
            continue
        ids = np.argsort(-z, kind="stable")
        w = np.exp((z[ids] - best) / t)
        if k > 0:
            w = w[z[ids] >= z[ids][min(int(k), len(ids)) - 1]]
        if p < 1:
            c = np.cumsum(w)
            last = z[ids][np.searchsorted(c, p * c[-1])]
            w = w[z[ids][:len(w)] >= last]
        w = w[w >= mp]
        at = np.sort(ids[:len(w)])
        w = np.exp((z[at] - best) / t)
        c = np.cumsum(w)
        i = min(int(np.searchsorted(c, u * c[-1], side="right")), len(at) - 1)
        tokens.append(int(at[i]))
        logprobs.append(float(np.log(w[i] / c[-1])))
    return np.array(tokens, dtype=np.int32), np.array(logprobs)
