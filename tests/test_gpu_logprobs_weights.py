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


@pytest.mark.parametrize("dtype,dz_dtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("V", [700, 40001])
def test_rows_without_weight(kl, V, dtype, dz_dtype):
    """Rows without a token, or with weights of zero, get zeros whatever they hold (padding may be NaN); the others keep theirs."""
    rng = np.random.default_rng(3)
    z = torch.as_tensor(rng.standard_normal((8, V)) * 2, dtype=torch.float32).to(dtype)
    z[1], z[2, V // 2], z[4, 3], z[6] = float("nan"), float("inf"), float("nan"), float("nan")
    tok = np.array([5, -1, -1, 7, 9, -1, 3, 2])
    zd, td = z.cuda(), _i(tok)
    _, ent, norm, _, _ = _forward(kl, zd, td, 0)
    a = torch.as_tensor(rng.standard_normal(8).astype(np.float32)).cuda()
    a[1], a[2], a[4], a[7] = float("nan"), 2.0, 0.0, 0.0      # what a row without a token has here is not read
    zero = torch.zeros(8, device="cuda")
    only_a = _backward(kl, zd, td, norm, None, a, None, dz_dtype)
    assert (only_a[[1, 2, 4, 5, 7]] == 0).all() and torch.isnan(only_a[6]).all() and (only_a[[0, 3]] != 0).any()
    assert torch.equal(_backward(kl, zd, td, norm, ent, a, zero, dz_dtype)[[0, 1, 2, 3, 4, 5, 7]], only_a[[0, 1, 2, 3, 4, 5, 7]])
    assert (_backward(kl, zd, td, norm, ent, None, zero, dz_dtype) == 0).all() and (_backward(kl, zd, td, norm, None, None, None, dz_dtype) == 0).all()
    # an entropy's weight counts without a token
    b = zero.clone()
    b[[1, 5]] = 1.0
    both = _backward(kl, zd, td, norm, ent, a, b, dz_dtype)
    assert torch.isnan(both[1]).all() and (both[5] != 0).any() and torch.equal(both[[0, 2, 3, 4, 7]], only_a[[0, 2, 3, 4, 7]])
    if dtype == dz_dtype:
        assert torch.equal(_backward(kl, zd, td, norm, None, a, None, dz_dtype, inplace=True)[[0, 1, 2, 3, 4, 5, 7]], only_a[[0, 1, 2, 3, 4, 5, 7]])
    assert kl.kl_device_status() == 0
