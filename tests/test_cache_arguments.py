"""A cache given in part is refused with what is missing, in either format."""
import pytest
import torch

import gated_deltanet_linear_13_gb300 as gdn

DEVICES = ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)]


@pytest.mark.parametrize("device", DEVICES)
@pytest.mark.parametrize("f8", [False, True])
def test_a_cache_without_values(f8, device):
    if device == "cuda" and not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    k = torch.zeros(1, 2, 16, 128, dtype=torch.uint8 if f8 else torch.bfloat16, device=device)
    exps = [torch.zeros(1, 2, 16, dtype=torch.uint8, device=device)] * 2 if f8 else [None, None]
    k = k.view(torch.float8_e4m3fn) if f8 else k
    with pytest.raises(ValueError, match="v_cache is required" if device == "cuda" else "CUDA"):
        gdn._kv_cache(k, None, *exps)


@pytest.mark.gpu
def test_rotation_into_a_cache_without_values():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    q = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    at = torch.zeros(2, dtype=torch.int32, device="cuda")
    cache = torch.zeros(1, 2, 16, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="v_cache is required"):
        gdn.gdn_qk_norm_rope(q, q, None, None, q, v=q, k_cache=cache, slots=at)
