"""A caller's workspace for the full-attention layers' operators: only one piece of memory on the
tensors' device is taken, as a whole and no more."""
import pytest
import torch

import gated_deltanet_linear_13_gb300 as gdn
from gated_deltanet_linear_13_gb300 import build_lib


def test_workspace_checks():
    cpu = torch.device("cpu")
    assert gdn._workspace_bytes(torch.empty(5, 3), cpu) == 60
    with pytest.raises(ValueError, match="contiguous"):
        gdn._workspace_bytes(torch.empty(64, dtype=torch.uint8)[::2], cpu)
    with pytest.raises(ValueError, match="expected cuda:0"):
        gdn._workspace_bytes(torch.empty(64), torch.device("cuda:0"))


@pytest.mark.gpu
def test_host_and_strided_workspaces_are_refused():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_lib.build()
    gdn.load_library()
    q = torch.zeros(1, 1, 2, 128, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(1, 1, 16, 128, dtype=torch.bfloat16, device="cuda")
    one = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    x, ent = torch.zeros(2, 5000, device="cuda"), torch.empty(2, device="cuda")
    need = max(gdn.gdn_prefix_attention_workspace_size(1, 1, 2, 1, 128),
               gdn.gdn_token_logprobs_workspace_size(2, 5000, 0, torch.float32))
    for ws in (torch.empty(need, dtype=torch.uint8),
               torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            gdn.gdn_prefix_attention(q, kv, kv, torch.empty_like(q), pages=one, kv_len=one[0],
                                     workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            gdn.gdn_token_logprobs(x, None, None, ent, workspace=ws)
    assert gdn.gdn_get_device_error() == 0
