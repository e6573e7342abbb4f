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


def test_project_against_torch():
    g = torch.Generator().manual_seed(2)
    x, w, a, b = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((6, 10), (7, 10), (3, 2, 10), (3, 7, 2)))
    s, bias = torch.rand(3, generator=g).double(), torch.randn(7, generator=g).double()
    ids = torch.tensor([0, 2, -1, 1, 2, 5])
    y, size, low, ranks = O.project(x, w, a, b, s, ids, bias)
    full = torch.stack([w + s[k] * b[k] @ a[k] if 0 <= k < 3 else w for k in ids.tolist()])
    want = torch.einsum("nok,nk->no", full, x) + bias
    assert np.allclose(y, want.numpy(), rtol=1e-12, atol=1e-12)
    assert (size + low >= np.abs(y - bias.numpy()) - 1e-12).all() and (ranks[2] == 0).all() and (ranks[0] > 0).all()
