"""The gated feed-forward block's products, held to what their arithmetic gives: large
tiles in every product, whole and with edges, forward and backward, and bounds that a
result of fewer bits or of fewer plane products would miss.

References are products in 64 bits on the GPU. Tolerances (relative Frobenius error over
4096 values or more), fixed from the arithmetic:
  bf16 results: an operand rounded to bf16 (z, dA or dU; rounding is 1.7e-3 in the mean
    square) and the result's own rounding add in quadrature, 2.4e-3: 3e-3 (with
    pre-activations rounded to bf16 too they are off by 3.5e-3);
  a, u: fp32 sums of exact products, 2^-24 times the root of at most 3584 terms is 4e-6:
    1e-5 (rounded to bf16 they would be off by 1.7e-3);
  fp32 results: sums of up to 6 x 12288 / 32 partial sums, 2^-24 sqrt(2304) = 2.9e-6 if
    every rounding counted in full: 3e-6 (one of the six plane pairs left out of a
    product is 9.7e-6)."""
from __future__ import annotations

import pytest
import torch

from chunked_weight_mlp_amd import block as K
from parity_check import report

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
RESULT = {"bf16": 3e-3, "f32": 3e-6}
PRE = {"bf16": 1e-5, "f32": 3e-6}


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    K.load()


def rand(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def close(got, want, tol, label):
    assert got.shape == want.shape and want.numel() >= 4096, label
    err = float((got.double() - want).norm() / want.norm())
    report(f"[ff products] {label}: rel_fro {err:.2e} (tol {tol:.0e})")
    assert err <= tol, (label, err)


def check(n, d, f, dtype, backward=True, pad=0):
    t = TYPES[dtype]
    g = torch.Generator(device=DEV).manual_seed(n + d + f)
    wg, wu, wd = (rand(g, s, t, s[1] ** -0.5) for s in ((f, d), (f, d), (d, f)))
    x, dy = rand(g, (n, d + pad), t)[:, :d], rand(g, (n, d + pad), t)[:, :d]
    op = K.FeedForward(wg, wu, wd)
    tag = f"{dtype} {n}x{d}x{f}"
    y, a, u = op.forward(x, save=True)
    assert torch.equal(op.forward(x), y)   # saving changes nothing
    X, WG, WU, WD, DY = (v.double() for v in (x, wg, wu, wd, dy))
    A, U = X.mm(WG.t()), X.mm(WU.t())
    S = torch.sigmoid(A)
    Z = A * S * U
    close(a, A, PRE[dtype], tag + " a")
    close(u, U, PRE[dtype], tag + " u")
    close(y, Z.mm(WD.t()), RESULT[dtype], tag + " y")
    if not backward:
        return
    got = op.backward(x, a, u, dy)
    DZ = DY.mm(WD)
    DA, DU = DZ * U * (S + A * S * (1 - S)), DZ * A * S
    del S, DZ
    for name, want in (("dx", lambda: DA.mm(WG) + DU.mm(WU)), ("dw_gate", lambda: DA.t().mm(X)),
                       ("dw_up", lambda: DU.t().mm(X)), ("dw_down", lambda: DY.t().mm(Z))):
        close(got[name], want(), RESULT[dtype], f"{tag} {name}")


def pad64(k):
    return -(-k // 64) * 64


def tiles(rows, cols, edge_r, edge_c):
    return -(-rows // edge_r) * -(-cols // edge_c)


def operands_only(n, d, f, planes):
    """The backward's workspace without partial sums of split products: its operands."""
    dp, fp, tp = pad64(d), pad64(f), pad64(n)
    rows = [(n, dp), (f, dp), (n, 2 * fp), (n if planes > 1 else 0, fp), (d, 2 * fp), (d, tp), (d, tp),
            (2 * fp, tp), (fp, tp)]
    return sum(-(-2 * planes * r * c // 256) * 256 for r, c in rows)


# 256 x 256 tiles, which three quarters of 256 CUs filled select, in the dz product and the
# three products after it, none of those split. 4100 x 2100 x 4200: edges everywhere, d_ff
# no multiple of 64 and, padded, no multiple of the tile's 256, so that the boundary
# between dW_gate and dW_up falls inside a tile; 4096 x 2048 x 4096 and 2304 x 2048 x 6144: whole tiles alone.
LARGE = [("bf16", 4100, 2100, 4200), ("bf16", 4096, 2048, 4096), ("bf16", 4161, 2056, 4104),
         ("f32", 2900, 2100, 4200), ("f32", 2304, 2048, 6144)]


@pytest.mark.parametrize("dtype,n,d,f", LARGE)
def test_large_tiles_in_every_product_of_the_backward(dtype, n, d, f):
    desc = K.FFDesc(d=d, d_ff=f, dtype=K._DT[TYPES[dtype]])
    planes = 1 if dtype == "bf16" else 3
    assert K.ipttt_ff_backward_workspace_bytes(desc, n) == operands_only(n, d, f, planes)
    assert tiles(f, n, 256, 256) >= 192
    fp = pad64(f)
    assert tiles(d, n, 256, 256) + tiles(d, 2 * fp, 256, 256) + tiles(f, d, 256, 256) >= 192
    check(n, d, f, dtype)


# the forward's second product in large tiles (the first, 128 rows of two matrices a tile,
# has them above)
@pytest.mark.parametrize("dtype,n,d,f", [("bf16", 4100, 3500, 1100), ("bf16", 4096, 3584, 1024),
                                         ("f32", 4100, 3500, 700)])
def test_large_tiles_in_the_down_product(dtype, n, d, f):
    assert tiles(d, n, 256, 256) >= 192
    check(n, d, f, dtype, backward=False)


# the other kernels and tile sizes: single tokens, few tokens, small tiles, split products
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,f,pad", [
    (8, 1024, 2048, 0), (30, 512, 600, 0), (64, 256, 640, 1), (130, 200, 72, 5), (257, 320, 513, 8),
    (300, 128, 2000, 0), (513, 1024, 576, 0), (600, 901, 1100, 1), (1100, 1001, 2003, 3),
    (2048, 1024, 2048, 0)])
def test_bounds_of_the_arithmetic(dtype, n, d, f, pad):
    check(n, d, f, dtype, pad=pad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [200, 320, 321])
def test_both_sides_of_the_few_token_limit(n, dtype):
    """A backward of up to 320 tokens takes the weights as they lie, beyond them a copy."""
    check(n, 2048, 8192, dtype)
