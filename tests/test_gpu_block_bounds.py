"""fp32 layer norm and recurrence (ordinary gates) against 64 bits, held to the roundings
they have.

Tolerances (relative Frobenius error), fixed from the arithmetic. Norm: a row's sums are
added in a tree of a few tens of 2^-24 roundings, of values that average out, then rsqrt
(one ulp) and three products: four roundings in quadrature, 2.4e-7; 1e-6 allowed. The
weights' gradients add up to 2100 rows: 2^-24 sqrt(2100 / 3) = 1.6e-6 if every rounding
counted in full; 2e-6. Recurrence: e^-g is off by |g| 2^-24 of itself, 1.2e-7 to 6e-7 for gates
of mean 2 and deviation 2, and a result's roundings fall off with its tokens': 1e-6."""
from __future__ import annotations

import pytest
import torch

import block_reference as ref
from chunked_weight_mlp_amd import block as K
from parity_check import rel_fro, report

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    K.load()


def rand(shape, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g) * std + mean


def close(got, want, tol, label):
    e = rel_fro(got.double().cpu().numpy(), want.numpy())
    report(f"[fp32 bounds] {label}: rel_fro {e:.2e} (tol {tol:.0e})")
    assert e <= tol, (label, e)


@pytest.mark.parametrize("n,d", [(2100, 1030), (64, 2560), (9, 8192), (5, 16384), (700, 63)])
def test_norm_fp32(n, d):
    x, r, dy, dh = (rand((n, d), k) for k in (1, 2, 5, 6))
    gamma, beta = rand((d,), 3, 0.2, 1.0), rand((d,), 4)
    op = K.Norm(gamma.to(DEV), beta.to(DEV))
    y, h, mean, rstd = op.forward(x.to(DEV), r.to(DEV))
    want = ref.norm_forward(x, r, gamma, beta, 1e-5)
    close(y, want[0], 1e-6, f"norm {n}x{d} y")
    close(rstd, want[3], 1e-6, f"norm {n}x{d} rstd")
    got = op.backward(h, mean, rstd, dy.to(DEV), dh.to(DEV))
    dx, dgamma, dbeta = ref.norm_backward(h.cpu(), mean.cpu(), rstd.cpu(), gamma, dy, dh)
    close(got["dx"], dx, 1e-6, f"norm {n}x{d} dx")
    close(got["dgamma"], dgamma, 2e-6, f"norm {n}x{d} dgamma")
    close(got["dbeta"], dbeta, 2e-6, f"norm {n}x{d} dbeta")


@pytest.mark.parametrize("n,length,d", [(2, 1500, 64), (3, 700, 130), (4, 16, 33), (5, 1, 300), (1, 4097, 65)])
def test_recurrence_fp32(n, length, d):
    g, v, dh = rand((n, length, d), 1, 2.0, 2.0), rand((n, length, d), 2), rand((n, length, d), 3)
    h0, dl = rand((n, d), 4), rand((n, d), 5)
    st = (rand((n, length), 6) > 2.5).to(torch.uint8)
    h, last = K.recurrence_forward(g.to(DEV), v.to(DEV), h0=h0.to(DEV), starts=st.to(DEV))
    want, wlast = ref.recurrence(g, v, h0, st, None)
    got = K.recurrence_backward(g.to(DEV), v.to(DEV), h, dh.to(DEV), h0=h0.to(DEV), dh_last=dl.to(DEV),
                                starts=st.to(DEV))
    dg, dv, dh0 = ref.recurrence_backward(g, v, h.cpu(), dh, h0, dl, st, None)
    for name, a, b in (("h", h, want), ("last", last, wlast), ("dg", got["dg"], dg), ("dv", got["dv"], dv),
                       ("dh0", got["dh0"], dh0)):
        close(a, b, 1e-6, f"recurrence {n}x{length}x{d} {name}")
