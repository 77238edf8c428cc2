"""bf16 gradients of the gated delta rule where the tokens of one chunk differ by many orders of magnitude, and
the bars that the kept 16-bit values are held to.

Every row (token and head) is compared for itself. A row's final rounding to bf16 is off by at most 2^-8 of each
value; what is kept with 11 bits before it enters with 2^-11 of its terms, which may exceed their sum a few
times: 2^-6 of the row's norm."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda
from errlog import report_named
from gdn_cases import make, to
from oracle.gdn import gdn_gradients, gdn_recurrent
from test_gpu_gdn_backward import LEAVES, OUTS, cotangents

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def gradients(a, d_o, dh):
    got = dict(zip(OUTS, kda.gdn_bwd(**to(a, DEV), d_o=d_o.to(DEV), dht=None if dh is None else dh.to(DEV))))
    leaves = {n: a[n] for n in LEAVES if a.get(n) is not None}
    return got, gdn_gradients(leaves, d_o, dh, **{n: x for n, x in a.items() if n not in LEAVES})


def rows_agree(got, want, tol, what):
    x, y = got.double().cpu(), want.double()
    assert torch.isfinite(x).all(), what
    err, size = (x - y).norm(dim=-1), y.norm(dim=-1)
    bad = err > tol * size
    assert not bad.any(), f"{what}: {int(bad.sum())} rows, worst {float((err / size.clamp_min(1e-300)).max()):.2e}"


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_gradients_of_o_of_many_sizes(K, V):
    a = make(T=150, H=2, K=K, V=V, h0=True, seed=21)
    d_o, _ = cotangents(a)
    gen = torch.Generator().manual_seed(2)
    d_o *= torch.exp2(-torch.randint(0, 61, (1, 150, 2, 1), generator=gen)).to(BF)     # exact
    got, want = gradients(a, d_o, None)
    rows_agree(got["q"], want["q"], 2.0 ** -6, "dq")


@pytest.mark.parametrize("raw", [False, True])
def test_betas_of_many_sizes(raw):
    # a token's dv is in proportion to its beta
    a = make(T=200, H=2, G=2, K=64, V=64, h0=True, raw=raw, seed=22)
    gen = torch.Generator().manual_seed(3)
    n = torch.randint(0, 41, a["beta"].shape, generator=gen)
    a["beta"] = (-n * 0.6931).to(BF) if raw else (a["beta"].float() * torch.exp2(-n)).to(BF)
    got, want = gradients(a, *cotangents(a))
    rows_agree(got["v"], want["v"], 2.0 ** -6, "dv")


@pytest.mark.parametrize("T", [64, 100])
def test_values_of_many_sizes(T):
    # v grows from token to token, and so does what a token adds: its dbeta is in proportion to that (all heads
    # of a token as one row, as one dot product may cancel)
    a = make(T=T, H=16, K=64, V=64, seed=23)
    a["v"] = (a["v"].float() * torch.exp2((torch.arange(T) - T) * 0.7)[None, :, None, None]).to(BF)
    got, want = gradients(a, *cotangents(a))
    rows_agree(got["beta"], want["beta"], 2.0 ** -5, "dbeta")


@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
def test_gradients_err_by_their_own_rounding(K, V):
    # Rounding a value to bf16 errs by at most 2^-8, on the mean by at most 2^-8 / sqrt(3) = 2.26e-3; what is kept
    # with 11 bits adds at most 2^-11 / sqrt(3) a matrix, four of them, enlarged up to four times where sums
    # cancel (dg): sqrt(2.26^2 + (2 x 4 x 0.28)^2) 1e-3 = 3.2e-3. (Kept as bf16 they gave 5.5e-3 of dg.)
    a = make(T=300, H=4, K=K, V=V, h0=True, seed=24)
    got, want = gradients(a, *cotangents(a))
    errs = {n: float((got[n].double().cpu() - want[n]).norm() / want[n].norm()) for n in ("q", "k", "v", "g", "beta")}
    report_named(**errs)
    assert max(errs.values()) <= 3.2e-3, errs


@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
def test_states_of_two_parts(K, V):
    # A part pair holds x to 2^-17 and a product leaves out the low-by-low term, 2^-16: on the mean (2^-16 / sqrt(3))
    # of the terms, five products behind each other, both errors: 2^-16 / sqrt(3) x sqrt(10) = 2.8e-5
    a = make(T=300, H=4, K=K, V=V, h0=True, seed=25)
    _, fin = kda.gdn_fwd(**to(a, DEV))
    ref, rfin = gdn_recurrent(**a)
    d_o, dh = cotangents(a)
    got, want = gradients(a, d_o, dh)
    for x, y in ((fin, rfin), (got["initial_state"], want["initial_state"])):
        err = (x.double().cpu() - y).flatten(2).norm(dim=2) / y.flatten(2).norm(dim=2)
        assert err.max() <= 2.8e-5, float(err.max())
