"""The attention's tensor-core kernel: batches with many rows over a long common
range, large enough for the rule that chooses it (products of common positions of
at least 9.5e8, three key tiles of 128 a CTA), against the 64-bit form with the
tolerances of the paged attention's other tests."""
import pytest

from test_gpu_paged import Case, lens_of

pytestmark = pytest.mark.gpu

# rows of one KV head 33, 64, 65, 128, 129, 150, 256, 257, 640; pages smaller than, equal to and larger than a tile; the
# common range cut inside pages at both ends
CASES = [
    # lens, shared, nq, nkv, dim, page, dtype, window
    (lens_of(29700, [1 + i for i in range(11)]), 29700, 24, 8, 128, 16, "f16", 0),
    (lens_of(15400, [5 * i + 1 for i in range(64)]), 15400, 16, 8, 64, 8, "bf16", 0),
    (lens_of(8001, [1] * 64), 8001, 16, 16, 128, 64, "bf16", 0),
    (lens_of(3901, [1 + i % 3 for i in range(64)]), 3901, 32, 16, 128, 64, "f16", 0),
    (lens_of(7801, [3] * 43), 7801, 24, 8, 128, 32, "f16", 0),
    (lens_of(8000, [70] * 64), 8000, 32, 8, 64, 128, "f16", 0),
    (lens_of(3901, [2] * 257), 3901, 8, 8, 128, 16, "bf16", 0),
    (lens_of(4700, [1 + i % 7 for i in range(80)]), 4700, 64, 8, 64, 512, "bf16", 0),
    (lens_of(9000, [1 + 3 * i for i in range(50)]), 9000, 48, 16, 128, 1024, "f16", 0),
    (lens_of(8000, [1 + 11 * i for i in range(64)]), 8000, 16, 8, 128, 16, "f16", 8200),    # windows from inside the prefix
    (lens_of(8100, [8200 if i % 16 == 5 else i for i in range(64)]), 8100, 32, 8, 64, 32, "bf16", 8000),   # some start behind it
    ([0, 500, 7990, 7] + lens_of(8000, [9] * 124), 8000, 8, 8, 128, 16, "bf16", 0),  # some end inside it, one is empty
    (lens_of(7700, [7610, 7000] + [1] * 63), 7700, 16, 16, 128, 64, "f16", 7650),  # 40 positions in common: no page
]


def chosen(lens, shared, nq, nkv, dim, window, n_sm=152):
    rows, keys = len(lens) * nq // nkv, min(window, shared) if window else shared
    return rows * keys * nkv * dim >= 9.5e8 and keys // 128 * -(-rows // 256) * nkv >= 3 * n_sm


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_of_many_rows(case):
    lens, shared, nq, nkv, dim, page, dtype, window = CASES[case]
    assert chosen(lens, shared, nq, nkv, dim, window)
    c = Case(lens, shared, nq, nkv, dim, page, dtype, window, seed=200 + case)
    c.check(*c.run())


@pytest.mark.parametrize("bad_page", [-1, 1 << 30])
def test_page_of_the_common_range_out_of_range(bad_page):
    import torch
    c = Case(lens_of(8100, [1 + i for i in range(64)]), 8100, 16, 8, 128, 16, "f16")
    c.tb[0, 3] = bad_page
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == 1


def test_repeatable_and_independent_of_the_workspace():
    import torch
    c = Case(lens_of(8100, [1 + i for i in range(64)]), 8100, 16, 8, 128, 16, "bf16")
    a, la = c.run()
    b, lb = c.run(ws=torch.zeros_like(c.workspace()))
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)
    c.check(a, la)


@pytest.mark.parametrize("lens", [[50, 20, 99], [0, 7, 8], [300, 299, 1]])
def test_tight_bound_where_every_sequence_ends_inside_the_prefix(lens):
    # the bound as the number of common positions: the same positions through the same row of the table
    shared = max(lens) + 30
    c = Case(lens, shared, 4, 2, 64, 16, "f16", seed=3)
    want, wl = c.run()
    c.shared = max(lens)
    got, gl = c.run(max_len=max(lens))
    c.shared = shared
    c.check(got, gl)
    c.check(want, wl)
