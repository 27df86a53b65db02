"""The workspace of gdn_verify_tokens: what serves a batch serves every smaller one, with fewer
drafts and a smaller vocabulary too (a server allocates once).  No GPU."""
import pytest
import torch

import gated_deltanet_linear_13_gb300 as gdn
from gated_deltanet_linear_13_gb300 import build_lib


@pytest.fixture(scope="module")
def size():
    build_lib.build()
    gdn.load_library()
    return gdn.gdn_verify_tokens_workspace_size


TYPES = [(dtype, draft) for dtype in (torch.bfloat16, torch.float32) for draft in (False, True)]


@pytest.mark.parametrize("dtype,draft", TYPES)
@pytest.mark.parametrize("t", [0, 1, 4, 64])
@pytest.mark.parametrize("v", [1, 600, 4096, 4097, 8193, 151936, 248320])
def test_never_less_for_more_sequences(size, v, t, dtype, draft):
    sizes = [size(b, t, v, dtype, draft) for b in range(1, 1100)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("dtype,draft", TYPES)
@pytest.mark.parametrize("b", [1, 7, 64, 152, 300, 457])
def test_never_less_for_more_drafts_or_logits(size, b, dtype, draft):
    for v in (1, 4096, 5000, 151936):
        sizes = [size(b, t, v, dtype, draft) for t in range(65)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    for t in (0, 1, 3, 64):
        sizes = [size(b, t, v, dtype, draft) for v in (*range(1, 20000, 37), *range(20000, 300000, 997))]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("b,t,v", [(1, 1, 100), (64, 4, 248320), (300, 7, 5000)])
def test_never_less_with_draft_logits(size, b, t, v):
    for dtype in (torch.bfloat16, torch.float32):
        assert size(b, t, v, dtype, False) <= size(b, t, v, dtype, True)
