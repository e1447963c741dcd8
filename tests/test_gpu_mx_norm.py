"""Precision of the norm and of its 8-bit outputs, against float64.

Bounds from the kernel's operations (u = 2^-24).  The squares go through a chain of
at most 8 fused multiply-adds a column, 3 additions across a thread's columns and 5
across a warp, each off by at most u of a sum of positive terms; across warps the
rounding errors are kept.  So the sum is off by at most 16 u, its root by 8 u.  The
root itself is held in two floats and h * root * w is rounded once: u more, and less
than u / 10 for all that is of second order (the Newton step's residual, the low
parts' own roundings).  9.1 u in all, and 1.1 u where the sum of squares is exact.

An 8-bit code is then the correctly rounded one of a value that far from y / scale;
with a float32 scale the quotient 1 / scale and the product add u each."""
import numpy as np
import pytest
import torch

import mx_reference as R
from test_gpu_mx import DTYPES, HALF, TINY, U, f64, gen, raw

pytestmark = pytest.mark.gpu

SUM_U = 8 * U    # of the root, from the sum of squares
ROUND_U = 1.1 * U


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_ffn_gb300 import build, moe as m

    build.build()
    return m


def check(moe, o, h, w, eps, quant, tol, dtype):
    T, H = h.shape
    y = R.rms_norm(f64(h), f64(w), eps)
    # in float32 the output's rounding is the one that tol counts
    more = 0.0 if dtype == torch.float32 else HALF[dtype]
    assert (np.abs(f64(o["out"]) - y) <= (tol + more) * np.abs(y) + TINY[dtype]).all()
    yp = np.zeros((T, R.padded(H)))
    yp[:, :H] = y
    if quant == moe.MOE_QUANT_MX_E4M3:
        e = raw(o["scales"]).astype(int) - 127
        amax = np.abs(yp).reshape(T, -1, 32).max(2)
        assert (R.scale_exponents(amax * (1 - tol), "e4m3") <= e).all()
        assert (e <= R.scale_exponents(amax * (1 + tol), "e4m3")).all()
        z = yp / np.repeat(np.ldexp(1.0, e), 32, 1)
    else:
        s = f64(o["scales"])
        amax = np.abs(yp).reshape(T, -1, 128).max(2)
        assert (np.abs(s - np.maximum(amax / 448, 2.0 ** -126)) <= (tol + U) * s).all()
        z = yp / np.repeat(s, 128, 1)
        tol = tol + 2 * U
    codes = raw(o["codes"]).astype(int)
    lo, hi = R.nearest(z * (1 - tol), R.E4M3), R.nearest(z * (1 + tol), R.E4M3)
    mag = codes & 127
    assert ((lo <= mag) & (mag <= hi)).all()
    assert ((codes >> 7)[mag > 0] == np.signbit(z)[mag > 0]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("quant", [1, 2])
@pytest.mark.parametrize("T,H", [(1, 7168), (700, 64), (513, 1000), (511, 2880), (160, 8200),
                                 (2, 65536)])
def test_norm_within_its_roundings(moe, T, H, quant, dtype):
    g = gen(T + H + quant)
    strong = 1.0 + 20.0 * (torch.rand(H, generator=g, device="cuda") < 0.004)
    x = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    r = (torch.randn((T, H), generator=g, device="cuda") * strong).to(dtype)
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(dtype)
    o = moe.moe_add_rms_norm(x, w, residual=r, quant=quant)
    check(moe, o, o["residual"], w, 1e-6, quant, SUM_U + ROUND_U, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("quant", [1, 2])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.3])
@pytest.mark.parametrize("T,H", [(1, 31), (3, 7168), (400, 320), (513, 1000), (300, 2880), (2, 40000)])
def test_norm_of_rows_with_an_exact_sum_is_rounded_once(moe, T, H, eps, quant, dtype):
    """Powers of two from 1/2 to 4: every sum of their squares is exact in float32, so only the root
    and the products round."""
    g = gen(H + quant)
    x = torch.exp2(torch.randint(-1, 3, (T, H), generator=g, device="cuda").float())
    x = (x * (1 - 2 * torch.randint(0, 2, (T, H), generator=g, device="cuda"))).to(dtype)
    w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(dtype)
    o = moe.moe_add_rms_norm(x, w, eps=eps, quant=quant)
    # the call's eps is a float32
    check(moe, o, x, w, float(np.float32(eps)), quant, ROUND_U, dtype)
