"""Plain 64-bit forms of the paged-cache operators and of the filtered draw,
and the inputs their tests share."""
import numpy as np

EPS = {"f32": 2.0 ** -23, "f16": 2.0 ** -10, "bf16": 2.0 ** -7}
TINY_HALF = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}  # half of the smallest step, where it matters


def torch_dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def rope_table(n, dim, theta=10000.0):
    ang = np.arange(n)[:, None] * theta ** (-2.0 * np.arange(dim // 2) / dim)
    return np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)


def rotate(x, cs):
    """x [tokens][heads][dim], cs [tokens][dim / 2][2]; also the sum of the
    magnitudes of the two terms, for error bounds."""
    h = x.shape[-1] // 2
    a, b, c, s = x[..., :h], x[..., h:], cs[:, None, :, 0], cs[:, None, :, 1]
    y = np.concatenate([a * c - b * s, a * s + b * c], -1)
    mag = np.concatenate([np.abs(a * c) + np.abs(b * s), np.abs(a * s) + np.abs(b * c)], -1)
    return y, mag


def visible(length, window):
    return np.arange(max(0, length - window) if window else 0, length)


def attention(q, k, v, table, page, lens, shared, window, scale):
    """q [seqs][heads][dim], k and v [pages][kv heads][page][dim], torch tensors,
    computed in float64 where they are; table and lens: numpy, list.  Returns out,
    lse and, for error bounds, the per-value magnitude sum_j p_j |v_j| and per
    row the largest sum of |q k|, the largest |v| and keys / sum of exp."""
    import torch
    n, nq, d = q.shape
    nkv = k.shape[1]
    g = nq // nkv
    new = lambda *sh: torch.zeros(*sh, dtype=torch.float64, device=q.device)  # noqa: E731
    out, mag, lse = new(n, nq, d), new(n, nq, d), new(n, nq) - np.inf
    qk, vmax, cond = new(n, nq, 1), new(n, nq, 1), new(n, nq, 1) + 1
    for b in range(n):
        j = visible(int(lens[b]), window)
        if not len(j):
            continue
        pages = torch.from_numpy(np.where(j < shared, table[0][j // page], table[b][j // page])).to(q.device).long()
        row = torch.from_numpy(j % page).to(q.device)
        kb, vb = k[pages, :, row].double().transpose(0, 1), v[pages, :, row].double().transpose(0, 1)  # [kv heads][keys][dim]
        qb = q[b].double().view(nkv, g, d)
        sc = scale * (qb @ kb.transpose(1, 2))
        m = sc.amax(-1, keepdim=True)
        e = (sc - m).exp()
        total = e.sum(-1, keepdim=True)
        out[b] = ((e @ vb) / total).view(nq, d)
        mag[b] = ((e @ vb.abs()) / total).view(nq, d)
        lse[b] = (m + total.log()).view(nq)
        qk[b, :, 0] = scale * (qb.abs() @ kb.abs().transpose(1, 2)).amax(-1).view(nq)
        vmax[b, :, 0] = vb.abs().amax((1, 2)).repeat_interleave(g)
        cond[b, :, 0] = (len(j) / total).view(nq)
    return out, lse, mag, qk, vmax, cond


def draw(z, t, k, p, mp, u):
    """Token and log share of one row; (-1, nan) for a row that has no draw."""
    z = np.asarray(z, dtype=np.float64)
    best = z.max() if not np.isnan(z).any() else np.nan
    if not (best > -np.inf) or not (t == 0 or np.float32(1e-30) <= t <= np.float32(1e30)) or not (0 < p <= 1) or not (0 <= mp <= 1) or not (0 <= u < 1):
        return -1, np.nan
    if t == 0:
        return int(np.flatnonzero(z == best)[0]), 0.0
    if best == np.inf:
        w = (z == np.inf).astype(np.float64)
    else:
        w = np.exp((z - best) / t)
    kept = np.ones(len(z), dtype=bool)
    if 0 < k < len(z):
        kept &= z >= np.sort(z)[-k]
    if p < 1:
        order = np.argsort(-z, kind="stable")
        c = np.cumsum(np.where(kept, w, 0.0)[order])
        kept &= z >= z[order[np.searchsorted(c, p * c[-1])]]
    if mp > 0:
        kept &= w >= mp
    c = np.cumsum(np.where(kept, w, 0.0))
    i = int(np.searchsorted(c, u * c[-1], side="right"))
    return i, float(np.log(w[i] / c[-1]))


def page_tables(g, n_seqs, max_pages, shared_pages, n_extra=3):
    """Random pages: the first shared_pages entries common, the others each
    sequence's own; returns (table, number of pages)."""
    own = max_pages - shared_pages
    n = shared_pages + n_seqs * own + n_extra
    order = g.permutation(n).astype(np.int32)
    table = np.empty((n_seqs, max_pages), dtype=np.int32)
    table[:, :shared_pages] = order[:shared_pages]
    table[:, shared_pages:] = order[shared_pages:shared_pages + n_seqs * own].reshape(n_seqs, own)
    return table, n
