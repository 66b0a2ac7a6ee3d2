"""Token log probabilities (lf_token_logprobs) on the GPU against the definition
in 64 bits.

Tolerances: a scaled difference (z - m) / T is off by 2^-23 of itself (a subtraction,
a product and 1 / T rounded); an exponential by that and 2^-21, so a sum of positive
terms, each off by at most 2^-23 |a| + 2^-21 of itself, plus 2^-24 per step of a
thread's sum and of the joins, is within 2^-18 of itself for the shares that have
weight (a > -30; what lies below holds less than vocab e^-30).  ln S adds its own
rounding 2^-23 |ln S|, so |logprob| is off by 2^-17 + 2^-22 (|a_t| + |ln S|) at most
and the entropy, ln S - E / S with E / S within 2^-17 of itself, likewise."""
import math

import numpy as np
import pytest

import paged_reference as ref

pytestmark = pytest.mark.gpu


def call(z, dtype, token, temp=None, top=0, ld=None, stream=None, want=("logprob", "rank", "entropy", "top_token",
                                                                      "top_logprob")):
    import torch
    import decode_persistent_sm_gb300 as lf
    rows, vocab = z.shape
    new = lambda *s, dt=torch.float32: torch.full(s, 77, dtype=dt, device="cuda")  # noqa: E731
    r = dict(logprob=new(rows), rank=new(rows, dt=torch.int32), entropy=new(rows),
             top_token=new(rows, top, dt=torch.int32), top_logprob=new(rows, top))
    p = {k: r[k].data_ptr() if k in want and r[k].numel() else None for k in r}
    lf.token_logprobs(z.data_ptr(), dtype, rows, vocab, z.stride(0) if ld is None else ld,
                      None if temp is None else temp.data_ptr(), None if token is None else token.data_ptr(), top,
                      p["logprob"], p["rank"], p["entropy"], p["top_token"], p["top_logprob"], stream)
    return r


def definition(z, token, t, top):
    """One row: logprob, rank, entropy, tokens, their log probabilities."""
    z = np.asarray(z, dtype=np.float64)
    m = z.max() if not np.isnan(z).any() else np.nan
    if not m > -np.inf or not (np.float32(1e-30) <= t <= np.float32(1e30)):
        return np.nan, -1, np.nan, np.full(top, -1), np.full(top, np.nan)
    with np.errstate(invalid="ignore", over="ignore"):
        a = np.where(z == np.inf, 0.0, -np.inf) if m == np.inf else (z - m) / np.float64(t)
    e = np.exp(a)
    norm = np.log(e.sum())
    lp = a - norm
    ent = -(e[e > 0] / e.sum() * lp[e > 0]).sum()
    order = np.argsort(-z, kind="stable")
    tok, tl = order[:top].copy(), lp[order[:top]]
    tok[z[tok] == -np.inf] = -1
    if not 0 <= token < len(z):
        return np.nan, -1, ent, tok, tl
    return lp[token], int(np.flatnonzero(order == token)[0]), ent, tok, tl


def check(z, token, temp, top, r, rows=None):
    import torch
    torch.cuda.synchronize()
    zs = z.double().cpu().numpy()
    n = len(zs)
    token = [-1] * n if token is None else token.tolist()
    temp = [1.0] * n if temp is None else temp.tolist()
    got = {k: v.cpu().numpy() for k, v in r.items()}
    for i in (range(n) if rows is None else rows):
        lp, rank, ent, tok, tl = definition(zs[i], token[i], np.float32(temp[i]), top)

        def near(x, y):
            if not np.isfinite(y):
                return np.array_equal(np.float64(x), y, equal_nan=True)
            return abs(x - y) <= 2.0 ** -17 + 2.0 ** -21 * abs(y) + 2.0 ** -22 * math.log(len(zs[i]))

        assert got["rank"][i] == rank, (i, got["rank"][i], rank)
        assert near(got["logprob"][i], lp), (i, got["logprob"][i], lp)
        assert near(got["entropy"][i], ent), (i, got["entropy"][i], ent)
        assert np.array_equal(got["top_token"][i], tok), (i, got["top_token"][i], tok)
        assert all(near(x, y) for x, y in zip(got["top_logprob"][i], tl)), (i, got["top_logprob"][i], tl)


def logits(rows, vocab, dtype, seed, spread=2.5, ld=None, masked=0.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = spread * torch.randn(rows, ld or vocab, device="cuda", generator=g)
    if masked:
        z.masked_fill_(torch.rand(z.shape, device="cuda", generator=g) < masked, -math.inf)
    z = z.to(ref.torch_dtype(dtype))[:, :vocab]
    token = torch.randint(vocab, (rows,), device="cuda", generator=g).int()
    return z, token


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (3, 2, 2), (5, 7, 5), (2, 33, 32), (4, 255, 20), (3, 1000, 0),
                                            (2, 4099, 7), (1, 32000, 5), (16, 32000, 32), (3, 50257, 1), (2, 131072, 20),
                                            (1, 262144, 32), (700, 5003, 3)])
def test_rows(dtype, rows, vocab, top):
    import torch
    z, token = logits(rows, vocab, dtype, vocab + top)
    temp = torch.tensor([0.5 + 0.3 * (i % 5) for i in range(rows)], device="cuda")
    r = call(z, dtype, token, temp, top)
    check(z, token, temp, top, r, rows=range(0, rows, max(1, rows // 40)))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("off", [1, 2, 3, 5])
def test_rows_that_begin_anywhere(dtype, off):
    # strides and starts that are no multiple of 16 bytes: single logits before and behind the 16-byte pieces
    z, _ = logits(6, 9001, dtype, off, ld=9001 + 2 * off + 1)
    z = z[:, off:off + 9000 - off]
    import torch
    token = torch.tensor([0, z.shape[1] - 1, 1, 7, 4000, 2], dtype=torch.int32, device="cuda")
    check(z, token, None, 9, call(z, dtype, token, None, 9))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [40, 6000, 32000, 131072])
def test_equal_logits_go_by_index(dtype, vocab):
    import torch
    z, _ = logits(6, vocab, dtype, 5)
    z[0] = 0.0                                     # all equal
    z[1] = (z[1] > 0).to(z.dtype)                  # two values
    z[2] = torch.round(z[2])                       # a few
    z[3] = 0.0
    z[3, 1::2] = -0.0                              # the two zeros are equal
    z[4] = torch.arange(vocab, device="cuda").flip(0).clamp(max=900).to(z.dtype)  # a long run of the largest
    z[5] = -math.inf
    z[5, vocab // 3:vocab // 3 + 3] = 1.0          # three tokens allowed
    token = torch.tensor([vocab - 1, vocab // 2, 17, 12, 30, vocab // 3 + 1], dtype=torch.int32, device="cuda")
    check(z, token, None, 32, call(z, dtype, token, None, 32))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("vocab", [50, 32000])
def test_many_candidates_in_one_threads_share(dtype, vocab):
    # every large logit lies where one thread of a row's CTA walks
    import torch
    z = torch.full((2, vocab), -3.0, device="cuda")
    step = 4 * 256 if dtype == "f32" else 8 * 256
    for i in range(4):
        z[0, i::step] = 5.0 - 0.01 * torch.arange(len(z[0, i::step]), device="cuda") % 3
    z[1, ::3] = torch.linspace(0, 30, len(z[1, ::3]), device="cuda")
    z = z.to(ref.torch_dtype(dtype))
    token = torch.tensor([0, vocab - 1], dtype=torch.int32, device="cuda")
    check(z, token, None, 32, call(z, dtype, token, None, 32))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [100, 32000, 100000])
def test_infinities_nans_and_masks(dtype, vocab):
    import torch
    z, token = logits(10, vocab, dtype, 9, masked=0.7)
    z[0] = -math.inf                      # nothing allowed
    z[1] = -math.inf
    z[1, vocab - 1] = -2.0                # one token
    z[2, 5] = math.inf
    z[2, vocab // 2] = math.inf
    z[3, vocab - 2] = math.nan
    z[4] = torch.finfo(z.dtype).min       # a mask of the type's lowest value
    z[4, 3] = 1.0
    z[5, 3] = -math.inf
    z[6] = -math.inf
    z[6, 1] = math.nan
    z[7, :] = math.inf
    z[8] = math.nan
    z[9, 0], z[9, 1] = math.inf, math.nan
    token[1], token[2], token[4], token[5], token[7] = vocab - 1, 5, 4, 3, 9
    check(z, token, None, 6, call(z, dtype, token, None, 6))
    token[2] = 6                          # not one of the infinite
    check(z, token, None, 6, call(z, dtype, token, None, 6))


def test_temperatures_and_tokens_outside_their_range():
    import torch
    z, token = logits(9, 3000, "f32", 4)
    z[0] *= 1000.0
    temp = torch.tensor([1e-30, 1e30, 0.0, -1.0, math.nan, math.inf, 1e-31, 1.0, 0.3], device="cuda")
    token[7], token[8] = -1, 3000
    check(z, token, temp, 4, call(z, "f32", token, temp, 4))


def test_results_that_are_not_wanted():
    import torch
    z, token = logits(5, 7000, "f16", 2)
    full = call(z, "f16", token, None, 3)
    for want in (("logprob",), ("rank",), ("entropy",), ("top_token",), ("top_logprob",), ()):
        r = call(z, "f16", token, None, 3, want=want)
        torch.cuda.synchronize()
        for k in r:
            assert torch.equal(r[k], full[k]) if k in want else (r[k] == 77).all()
    r = call(z, "f16", None, None, 3, want=("entropy", "top_token"))
    torch.cuda.synchronize()
    assert torch.equal(r["entropy"], full["entropy"]) and torch.equal(r["top_token"], full["top_token"])


def test_a_likely_token_keeps_its_small_log_probability():
    # p = 1 - 1e-5: fp32 sums hold 1 + x to 2^-24
    import torch
    z = torch.full((1, 1000), -20.0, device="cuda")
    z[0, 3] = 0.0
    token = torch.tensor([3], dtype=torch.int32, device="cuda")
    r = call(z, "f32", token)
    torch.cuda.synchronize()
    want = -math.log1p(999 * math.exp(-20.0))
    assert abs(r["logprob"].item() - want) <= 2.0 ** -22


def test_on_another_stream_captured_and_twice_the_same():
    import torch
    z, token = logits(40, 20011, "bf16", 8)
    first = call(z, "bf16", token, None, 10)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = call(z, "bf16", token, None, 10, stream=s.cuda_stream)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        third = call(z, "bf16", token, None, 10, stream=torch.cuda.current_stream().cuda_stream)
    gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first[k], again[k]) and torch.equal(first[k], third[k]) for k in first)


def test_rows_past_32_bits():
    import torch
    rows, vocab = 17000, 262144
    z = torch.zeros(rows, vocab, dtype=torch.float16, device="cuda")
    z[-1, 5:9] = torch.tensor([3.0, 9.0, 9.0, 4.0]).half()
    token = torch.full((rows,), 8, dtype=torch.int32, device="cuda")
    r = call(z, "f16", token, None, 0)
    torch.cuda.synchronize()
    lp, rank, ent, _, _ = definition(z[-1].double().cpu().numpy(), 8, np.float32(1), 0)
    assert abs(r["logprob"][-1].item() - lp) < 1e-4 and r["rank"][-1] == rank and abs(r["entropy"][-1].item() - ent) < 1e-4
    assert (r["rank"][:-1] == 8).all()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("rows,vocab", [(1, 8001), (19, 32003), (20, 64000), (38, 20000), (40, 16001), (76, 9000), (77, 33000),
                                        (152, 8000), (153, 8000)])
def test_rows_of_1_2_4_and_8_ctas(dtype, rows, vocab):
    z, token = logits(rows, vocab, dtype, rows, masked=0.3)
    z[0, ::7] = -math.inf
    z[rows // 2, :] = -math.inf
    z[rows // 2, vocab - 1] = 0.5
    check(z, token, None, 32, call(z, dtype, token, None, 32), rows=range(0, rows, max(1, rows // 8)))


def test_a_masked_value_after_clean_ones_and_before():
    # a thread goes over to the masked way in the middle of its walk
    import torch
    z, token = logits(4, 40000, "f32", 3)
    z[0, 39000:] = -math.inf
    z[1, :1000] = -math.inf
    z[2, 20000] = torch.finfo(torch.float32).min
    z[3, 20000] = math.nan
    check(z, token, None, 5, call(z, "f32", token, None, 5))
