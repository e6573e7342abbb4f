"""Pins of oracle/paged.py: its attention equals torch's scaled dot product
attention under the same explicit mask (f64), its visible sets a brute-force
statement, its rotation a complex product."""
import numpy as np
import pytest
import torch

from oracle import paged as O


def pool(rng, pages, nkv, P, D):
    return rng.standard_normal((pages, nkv, P, D)), rng.standard_normal((pages, nkv, P, D))


@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 0), (5, 3), (1, 0), (64, 40)])
def test_attention_equals_torch_under_the_same_mask(window, sinks):
    rng = np.random.default_rng(1)
    NH, NKV, D, P, n, length = 6, 2, 16, 16, 7, 53
    k, v = pool(rng, 9, NKV, P, D)
    table = np.array([7, 2, 5, 0, -1])
    q = rng.standard_normal((n, NH, D))
    pos = np.arange(length - n, length)
    out, lse, mean, big = O.attend(q, k, v, table, length, pos, window, sinks)
    rows = np.arange(length)
    kk = torch.from_numpy(O.gather(k, table, rows)).transpose(0, 1).repeat_interleave(NH // NKV, 0)
    vv = torch.from_numpy(O.gather(v, table, rows)).transpose(0, 1).repeat_interleave(NH // NKV, 0)
    mask = torch.zeros(n, length, dtype=torch.bool)
    for i, p in enumerate(pos):
        for j in range(length):
            mask[i, j] = bool(j <= p and (window == 0 or p - j < window or j < sinks))
    qq = torch.from_numpy(q).transpose(0, 1)
    want = torch.nn.functional.scaled_dot_product_attention(qq, kk, vv, attn_mask=mask)
    s = (qq @ kk.transpose(1, 2) / D ** 0.5).masked_fill(~mask, -np.inf)
    # the oracle rounds the scale to f32 as the C ABI does
    np.testing.assert_allclose(out, want.transpose(0, 1).numpy(), rtol=0, atol=1e-6)
    np.testing.assert_allclose(lse, torch.logsumexp(s, -1).T.numpy(), rtol=0, atol=1e-6)
    assert (mean >= np.abs(out) - 1e-12).all() and big >= np.abs(s[s > -np.inf]).max().item() - 1e-6


def test_rows_that_see_nothing_and_scores_of_minus_infinity():
    rng = np.random.default_rng(2)
    k, v = pool(rng, 2, 1, 16, 8)
    q = np.abs(rng.standard_normal((3, 2, 8))) + 0.1
    out, lse, _, _ = O.attend(q, k, v, np.array([0]), 2, [-1, 0, 1])
    assert (out[0] == 0).all() and (lse[0] == -np.inf).all()
    np.testing.assert_array_equal(out[1], np.broadcast_to(v[0, 0, 0], (2, 8)))
    k[0, 0, 1] = -np.inf                      # the second key's score is -inf
    out, lse, _, _ = O.attend(q, k, v, np.array([0]), 2, [1, 1, 1])
    np.testing.assert_array_equal(out, np.broadcast_to(v[0, 0, 0], (3, 2, 8)))


def test_norm_and_rotation():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 3, 10))
    ang = rng.standard_normal((4, 5)) * 3
    y = O.norm_rope(x, None, 0.0, np.cos(ang), np.sin(ang))
    z = (x[..., :5] + 1j * x[..., 5:]) * np.exp(1j * ang)[:, None]
    np.testing.assert_allclose(y, np.concatenate((z.real, z.imag), -1), atol=1e-12)
    w = rng.standard_normal(10)
    y = O.norm_rope(x, w, 1e-6, np.ones((4, 5)), np.zeros((4, 5)))
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (10,), torch.from_numpy(w), 1e-6)
    np.testing.assert_allclose(y, want.numpy(), atol=1e-12)


@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 3), (1, 0), (20, 60)])
def test_all_rows_at_once_equals_row_by_row(window, sinks):
    rng = np.random.default_rng(5)
    NH, NKV, D, P, length = 6, 2, 16, 16, 50
    k, v = pool(rng, 9, NKV, P, D)
    table = np.array([7, 2, 5, 0, -1])
    k[2, 0, 3] = -np.inf                      # scores of -inf and +inf from head 0's keys
    q = rng.standard_normal((9, NH, D))
    q[:, :3] = np.abs(q[:, :3])
    pos = np.arange(-2, length, 6)
    want = O.attend(q, k, v, table, length, pos, window, sinks)
    kk, vv = (torch.from_numpy(O.gather(x, table, np.arange(length))) for x in (k, v))
    got = O.attend_all(torch.from_numpy(q), kk, vv, torch.from_numpy(pos), window, sinks)
    for a, b in zip(got[:3], want[:3]):
        np.testing.assert_allclose(a.numpy(), b, rtol=0, atol=1e-12)
    assert abs(got[3].max().item() - want[3]) < 1e-12 and (got[3][:1] == 0).all()
    empty = O.attend_all(torch.from_numpy(q), kk[:0], vv[:0], torch.from_numpy(pos))
    assert (empty[0] == 0).all() and torch.isneginf(empty[1]).all()
