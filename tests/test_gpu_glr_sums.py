"""Sums over tokens in the gradients of a gate's parameters, where tiles take the sequence: what the waves of a tile
hand in cancels, and what is left has to stay."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("beta", [False, True])
def test_a_tiles_sum_keeps_what_cancels(beta):
    """One token in 16 passes its gradient on (elsewhere the gate closes, e^g is zero and so is dg), so a wave's sum is
    one number and exact, and ddt_bias is the sum of the dg that are returned. Tokens come as V, small, -V, small: a
    tile's sum is small, and only its rounding to a row of 32 bits and the result's count."""
    T, D, gen = 8192, 64, torch.Generator().manual_seed(1)
    hot = torch.arange(7, T, 16)
    g = torch.full((1, T, D), 1e4)
    g[0, hot] = 0.25
    d_y = torch.zeros(1, T, D)
    v = torch.randn(len(hot), D, generator=gen)
    v[0::4] = v[0::4] * 1e5
    v[2::4] = -v[0::4]
    d_y[0, hot] = v
    y = torch.ones(1, T, D)
    more = dict(beta=torch.ones(1, T, D, device=DEV)) if beta else {}
    x = torch.ones(1, T, D, device=DEV) if beta else None
    dx, dg, _, _, dA, db = kda.glr_bwd(x, g.to(DEV), y.to(DEV), d_y.to(DEV), gate="softplus", want_dh0=False,
                                       A_log=torch.zeros(D, device=DEV), dt_bias=torch.zeros(D, device=DEV), **more)
    torch.cuda.synchronize()
    dg = dg.double().cpu()[0]
    cold = torch.ones(T, dtype=torch.bool)
    cold[hot] = False
    assert (dg[cold] == 0).all() and (dg[hot] != 0).all()
    want = dg.sum(0)
    rows = dg.reshape(T // (64 if beta else 128), -1, D).sum(1).abs().sum(0)
    assert ((db.double().cpu() - want).abs() <= 2.0 ** -24 * (rows + want.abs()) * (1 + 2.0 ** -20)).all()
    # every hot token has the same decay, so dA_log is the same sum times act / (-ea sigmoid(u)), each term rounded thrice
    u = torch.tensor(0.25, dtype=torch.float64)
    ratio = torch.nn.functional.softplus(u) / torch.sigmoid(u)
    assert ((dA.double().cpu() - want * ratio).abs() <= 2.0 ** -20 * dg.abs().sum(0)).all()
