"""oracle/rows.py against torch and closed forms."""
import numpy as np
import torch

from oracle import rows as O


def test_logprobs_against_torch():
    x = torch.randn(5, 301, generator=torch.Generator().manual_seed(0), dtype=torch.float64) * 3
    x[1, 40:80] = -torch.inf
    for t in (1.0, 0.5, 3.0):
        lp, h = O.logprobs(x.numpy(), t)
        want = torch.log_softmax(x / t, -1)
        assert np.allclose(lp, want.numpy(), rtol=1e-13, atol=1e-13)
        for r in range(5):
            some = x[r] > -torch.inf
            want_h = torch.distributions.Categorical(logits=x[r][some] / t).entropy()
            assert abs(h[r] - float(want_h)) < 1e-12
        assert abs(np.exp(lp).sum(-1) - 1).max() < 1e-12


def test_uniform_and_undefined_rows():
    lp, h = O.logprobs(np.array([[-np.inf] * 8, [2.0] * 8, [np.nan] + [0.0] * 7, [np.inf] + [0.0] * 7]))
    assert np.allclose(lp[:2], -np.log(8)) and np.allclose(h[:2], np.log(8)) and np.isnan(lp[2:]).all() and np.isnan(h[2:]).all()


def test_order():
    assert O.order([1.0, np.nan, 3.0, 3.0, -np.inf, np.inf, np.nan]).tolist() == [1, 6, 5, 2, 3, 0, 4]
    assert O.order([0.0, -0.0, 0.0]).tolist() == [0, 1, 2]
