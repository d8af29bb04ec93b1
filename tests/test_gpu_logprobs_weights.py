"""The gradient of token log probabilities and entropies where its weights are large, zero or absent."""
import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_logprobs import _backward, _forward, _host, _i

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("weight", [1e6, 1e9, 1e30, -1e30])
def test_large_entropy_weights(kl, weight, dtype):
    """Classes without any probability get zeros whatever the entropy's weight is (a loss scale, say); the others its multiple."""
    rng = np.random.default_rng(2)
    z = torch.as_tensor(rng.standard_normal((5, 3001)) * 2, dtype=torch.float32).to(dtype)
    z[:, 1::2] = float("-inf")
    z[1, 4::8] = -3.3e38
    tok = np.array([0, 2, -1, 6, 8])
    zd, td = z.cuda(), _i(tok)
    _, ent, norm, _, _ = _forward(kl, zd, td, 0)
    b = torch.full((5,), weight, device="cuda")
    got = _host(_backward(kl, zd, td, norm, ent, None, b, torch.float32))
    assert kl.kl_device_status() == 0
    p = torch.softmax(z.double(), 1).numpy()
    assert (got[p == 0] == 0).all()
    want = O.token_logprobs_bwd(_host(z), tok, np.zeros(5), np.full(5, weight))
    # the bound of test_backward_matches_oracle, whose weights are below 5, for this weight
    tol = 2.0 ** -24 * np.abs(want) + abs(weight) * 1e-4 * p * (1 + np.abs(np.log(np.maximum(p, 1e-300))) + np.log(3001)) + 1e-30
    assert (np.abs(got - want) <= tol).all()
