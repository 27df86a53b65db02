"""gdn_verify_tokens where its numbers are far apart: log probabilities of accepted drafts whose
logits lie further below the row's largest than fp32 reaches."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as m
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    m.load_library()
    return m


def _run(gdn, target, **kw):
    b, t1, _ = target.shape
    tokens = torch.full((b, t1), -9, device="cuda", dtype=torch.int32)
    accepted = torch.full((b,), -9, device="cuda", dtype=torch.int32)
    logprobs = torch.full((b, t1), 9.0, device="cuda")
    gdn.gdn_verify_tokens(target, tokens, accepted, logprobs=logprobs, **kw)
    assert gdn.gdn_get_device_error() == 0
    return tokens, accepted, logprobs


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [2.0 ** -64, 2.0 ** -40, 2.0 ** -2])
def test_log_probabilities_of_far_drafts(gdn, scale, dtype):
    """p / q = 1 for a draft 6e38 below its row's largest logit: accepted, with its log probability."""
    v = 50
    x = torch.zeros(1, 2, v, device="cuda", dtype=dtype)
    x[..., 0], x[..., 1] = 3e38, -3e38
    tokens, accepted, logprobs = _run(
        gdn, x, clocks=torch.ones(1, v, device="cuda"), draft_logits=x[:, :1].contiguous(),
        draft_ids=torch.ones(1, 1, device="cuda", dtype=torch.int32),
        accept_u=torch.full((1, 1), 0.25, device="cuda"), scale=torch.full((1,), scale, device="cuda"))
    assert int(accepted) == 1 and tokens.tolist() == [[1, 0]]
    want = (float(x[0, 0, 1]) - float(x[0, 0, 0])) * scale   # (z is 1)
    assert abs(float(logprobs[0, 0]) - want) <= 2.0 ** -22 * abs(want)
    assert abs(float(logprobs[0, 1])) <= 4e-6
