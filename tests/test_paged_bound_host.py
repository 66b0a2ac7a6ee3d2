"""The bound of the lengths and the common positions of lf_attn_paged_shared (no GPU
needed): up to the bound they are accepted, above it refused, as the header says."""
import os
import re

import pytest

from test_paged_host import INVALID, attend, lib  # noqa: F401  (lib: the fixture)


@pytest.mark.parametrize("max_len", [0, 1, 10, 63, 80])
def test_common_positions_up_to_the_bound(lib, max_len):  # noqa: F811
    # (an accepted call is stopped at the first CUDA call, or at the workspace of 0 bytes where there is a GPU)
    import torch
    passed = INVALID if torch.cuda.is_available() else 3
    assert attend(lib, max_len=max_len, shared=max_len) == passed
    assert attend(lib, max_len=max_len, shared=max_len + 1) == INVALID


def test_the_header_names_the_limit():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"\s*\*\s*", " ", open(os.path.join(root, "include", "laneformer.h")).read())
    assert "shared_len above max_len" in text
