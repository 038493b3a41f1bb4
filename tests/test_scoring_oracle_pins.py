"""The scoring oracle against torch's fp64 operations, its own definitions and
differences (CPU)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import scoring_oracle as o


def test_e4m3_rounding_is_torchs_over_the_whole_range():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    grid = np.unique(codes[torch.isfinite(codes)].double().numpy())
    assert np.array_equal(o.e4m3_round(grid), grid)
    mid = (grid[1:] + grid[:-1]) / 2  # ties
    x = np.concatenate([mid, np.random.RandomState(0).uniform(-448, 448, 20000),
                        np.random.RandomState(1).normal(0, 0.01, 20000)])
    x = x.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(o.e4m3_round(x), want)
    assert o.e4m3_round(1e9) == 448 and o.e4m3_round(-460.0) == -448


def test_bf16_rounding_is_torchs():
    x = np.random.RandomState(0).normal(0, 3, 10000).astype(np.float32)
    assert np.array_equal(o.bf16_round(x), torch.from_numpy(x).bfloat16().double().numpy())


def test_norm_gradient_against_autograd_and_differences():
    rs = np.random.RandomState(0)
    x, res, w, dy, dh = (rs.normal(size=s) for s in ((3, 24), (3, 24), (24,), (3, 24), (3, 24)))
    h = torch.tensor(x + res, requires_grad=True)
    wt = torch.tensor(w, requires_grad=True)
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * wt
    ((y * torch.tensor(dy)).sum() + (h * torch.tensor(dh)).sum()).backward()
    dx, dw = o.add_rms_norm_backward(dy, dh, x + res, w, 1e-6)
    assert np.allclose(dx, h.grad.numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(dw, wt.grad.numpy(), rtol=1e-12, atol=1e-12)
    f = lambda v: (v / np.sqrt((v * v).mean(-1, keepdims=True) + 1e-6) * w * dy).sum() + (v * dh).sum()
    e = np.zeros_like(x)
    e[1, 5] = 1e-6
    assert abs((f(x + res + e) - f(x + res - e)) / 2e-6 - dx[1, 5]) < 1e-7


def test_block_matmul_is_the_product_of_decoded_matrices():
    rs = np.random.RandomState(0)
    x, w = rs.normal(size=(5, 300)), rs.normal(size=(140, 300))
    sx, sw = o.block_scales(x, 1), o.block_scales(w, 128)
    assert sx.shape == (5, 3) and sw.shape == (2, 3)
    qx = o.e4m3_round(x / o.spread(sx, 5, 300, 1))
    qw = o.e4m3_round(w / o.spread(sw, 140, 300, 128))
    d, mag = o.block_matmul(qx, sx, qw, sw)
    # each factor is off by at most half a step (2^-4) of its value, or of the
    # smallest step (2^-10 of its scale)
    ax = np.abs(x) * 2.0 ** -4 + o.spread(sx, 5, 300, 1) * 2.0 ** -10
    aw = np.abs(w) * 2.0 ** -4 + o.spread(sw, 140, 300, 128) * 2.0 ** -10
    bound = ax @ np.abs(w).T + np.abs(x) @ aw.T + ax @ aw.T
    assert (np.abs(d - x @ w.T) <= bound).all()


@pytest.mark.parametrize("T", [1.0, 0.7])
def test_token_logprobs_against_torch(T):
    torch.manual_seed(0)
    z = torch.randn(6, 50, dtype=torch.float64) * 3
    z[2, ::3] = -np.inf
    z[3, 7] = z[3, 9] = z[3].max() + 1  # a tie
    t = torch.tensor([3, 49, 1, 9, -100, 70])
    zt = z.clone().requires_grad_(True)
    lsm = torch.log_softmax(zt / T, -1)
    p = lsm.exp()
    ent = -torch.where(p > 0, p * torch.where(p > 0, lsm, 0.0), 0.0).sum(-1)
    got = o.token_logprobs(z.numpy(), t.numpy(), -100, T, 4)
    kept = [0, 1, 2, 3]
    assert np.allclose(got["logp"][kept], lsm[kept, t[kept]].detach(), atol=1e-12)
    assert np.allclose(got["entropy"][kept], ent[kept].detach(), atol=1e-12)
    assert got["logp"][4] == got["entropy"][4] == 0 and (got["top_ids"][4] == -1).all()
    assert got["logp"][5] == 0 and got["entropy"][5] > 0
    assert list(got["top_ids"][3][:2]) == [7, 9]
    gl, ge, gt = torch.randn(6).double(), torch.randn(6).double(), torch.randn(6, 4).double()
    loss = sum(gl[r] * lsm[r, t[r]] + ge[r] * ent[r] for r in kept) + ge[5] * ent[5]
    for r in kept + [5]:
        loss = loss + (gt[r] * lsm[r, torch.from_numpy(got["top_ids"][r])]).sum()
    loss.backward()
    dz, _ = o.token_logprobs_backward(z.numpy(), t.numpy(), got, gl.numpy(), ge.numpy(),
                                      gt.numpy(), -100, T)
    want = torch.nan_to_num(zt.grad, nan=0.0).numpy()
    assert np.allclose(dz, want, atol=1e-12)


def test_token_logprobs_gradient_against_differences():
    rs = np.random.RandomState(3)
    z, t = rs.normal(size=(2, 9)), np.array([4, 0])
    gl, ge, gt = rs.normal(size=2), rs.normal(size=2), rs.normal(size=(2, 3))
    base = o.token_logprobs(z, t, -100, 1.3, 3)

    def f(v):
        r = o.token_logprobs(v, t, -100, 1.3, 3)
        return (gl * r["logp"]).sum() + (ge * r["entropy"]).sum() + (gt * r["top_logp"]).sum()

    dz, _ = o.token_logprobs_backward(z, t, base, gl, ge, gt, -100, 1.3)
    for r in range(2):
        for c in range(9):
            e = np.zeros_like(z)
            e[r, c] = 1e-6
            assert abs((f(z + e) - f(z - e)) / 2e-6 - dz[r, c]) < 1e-8


def test_rows_that_hold_nothing():
    z = np.full((2, 5), -np.inf)
    z[1] = np.finfo(np.float32).min
    got = o.token_logprobs(z, np.array([1, 1]), -100, 1.0, 2)
    assert got["logp"][0] == -np.inf and got["entropy"][0] == 0 and got["lse"][0] == -np.inf
    assert list(got["top_ids"][0]) == [0, 1] and (got["top_logp"][0] == -np.inf).all()
    assert np.isclose(got["logp"][1], -np.log(5)) and np.isclose(got["entropy"][1], np.log(5))
