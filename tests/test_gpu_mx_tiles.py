"""The grouped product of microscaled rows over many tiles a CTA: every tile
form with at least three tiles for each CTA (or pair of CTAs), so that the
accumulators, the operand ring and the scale ring are handed from tile to tile,
with K above the ring's depth and both a multiple of four stages of 128 columns
and not (the scales travel four stages at a time, skewed where a row's scales do
not fill 16-byte chunks), ragged experts and empty ones.

The reference is float64 on the values that the operands stand for (which
moe_mx_dequantize gives exactly in float32); the bounds are those that
test_gpu_mx.py derives."""
import numpy as np
import pytest
import torch

from test_gpu_mx import ACTS, HALF, TINY, U, gen, mx_weights, rows_of, segments

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_ffn_gb300 import build, moe as m

    build.build()
    return m


# form: (tokens a tile, CTAs a tile), and the counts that choose it
COUNTS = {
    "16": (16, 1, [i % 9 for i in range(96)]),              # up to 8 rows an expert
    "64": (64, 1, [(i * 37) % 80 for i in range(64)]),      # up to 48
    "96 pair": (96, 2, [(i * 71) % 220 for i in range(40)]),   # up to 160, or a short K
    "224 pair": (224, 2, [(i * 131) % 640 for i in range(16)]),
}


def check(moe, counts, a, w, bias, act, lim, N, out, dtype, mx_out):
    seg = np.cumsum([0] + counts)
    av = moe.moe_mx_dequantize(*a, a[0].shape[1], dtype=torch.float32).double()
    for e, n in enumerate(counts):
        if n == 0:
            continue
        lo, hi = int(seg[e]), int(seg[e + 1])
        wv = moe.moe_mx_dequantize(w[0][e], w[1][e], w[0].shape[2] * 2, dtype=torch.float32).double()
        p, mag = av[lo:hi] @ wv.t(), av[lo:hi].abs() @ wv.abs().t()
        if bias is not None:
            p, mag = p + bias[e].double(), mag + bias[e].double().abs()
        d = (av.shape[1] / 32 + 4) * 2 * U * mag
        if act == "none":
            v, dv = p, d
        else:
            inter = act == "swiglu"
            g, u = (p[:, 0::2], p[:, 1::2]) if inter else (p[:, :N], p[:, N:])
            dg, du = (d[:, 0::2], d[:, 1::2]) if inter else (d[:, :N], d[:, N:])
            limit, alpha, beta = lim if inter else (0.0, 1.0, 0.0)
            dv = 1.13 * max(1.0, alpha) * (u.abs() + abs(beta)) * dg + (g.abs() + dg) * du
            if inter:
                g, u = g.clamp(max=limit), u.clamp(-limit, limit)
            v = g * torch.sigmoid(alpha * g) * (u + beta)
            dv = dv + 2.0 ** -16 * v.abs()
        if not mx_out:
            err = (out[lo:hi].double() - v).abs()
            assert (err <= dv + HALF[dtype] * (v.abs() + dv) + TINY[dtype]).all(), (e, err.max().item())
            continue
        Np = moe.moe_mx_columns(N)
        vp, dp = (torch.nn.functional.pad(t, (0, Np - N)) for t in (v, dv))
        s = out[1][lo:hi].float().double()
        amax, more = vp.abs().view(n, -1, 32).amax(2), dp.view(n, -1, 32).amax(2)
        # the smallest power of two (at least 2^-127) with amax / s <= 448
        assert (amax - more <= 448 * s).all() and ((amax + more > 224 * s) | (s == 2.0 ** -127)).all()
        got = moe.moe_mx_dequantize(out[0][lo:hi].clone(), out[1][lo:hi].clone(), Np,
                                    dtype=torch.float32).double()
        err = (got - vp).abs()
        assert (err <= dp + 2.0 ** -4 * (vp.abs() + dp) +
                2.0 ** -10 * s.repeat_interleave(32, 1)).all(), (e, err.max().item())


@pytest.mark.parametrize("form,N,K,act,dtype,mx_out", [
    ("16", 700, 1280, "silu_and_mul", torch.bfloat16, False),
    ("16", 700, 1024, "swiglu", torch.bfloat16, True),
    ("16", 1400, 1280, "none", torch.float32, False),
    ("64", 900, 1280, "swiglu", torch.float16, False),
    ("64", 900, 1024, "silu_and_mul", torch.bfloat16, True),
    ("64", 1800, 1408, "none", torch.bfloat16, False),
    ("96 pair", 1100, 1280, "swiglu", torch.bfloat16, False),
    ("96 pair", 1100, 1024, "silu_and_mul", torch.bfloat16, True),
    ("96 pair", 1100, 2944, "swiglu", torch.bfloat16, True),
    ("96 pair", 2200, 1408, "none", torch.float32, False),
    ("224 pair", 2100, 1920, "silu_and_mul", torch.bfloat16, False),
    ("224 pair", 2100, 2048, "swiglu", torch.float16, False),
    ("224 pair", 2100, 3712, "swiglu", torch.bfloat16, True),
    ("224 pair", 2100, 4096, "silu_and_mul", torch.bfloat16, True),
    ("224 pair", 4200, 1920, "none", torch.float32, False),
])
def test_many_tiles_a_cta(moe, form, N, K, act, dtype, mx_out):
    nmax, ctas, counts = COUNTS[form]
    M, E = sum(counts), len(counts)
    gated = act != "none"
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = sum(-(-n // nmax) for n in counts) * -(-N // ((128 if gated else 256) * ctas))
    assert tiles >= 3 * (sms // ctas), "three tiles a CTA"
    g = gen(N + K)
    a = moe.moe_mx_quantize(rows_of(g, M, K, torch.float32) * 0.01)
    w = mx_weights(moe, g, E, 2 * N if gated else N, K)
    bias = (torch.randn((E, w[0].shape[1]), generator=g, device="cuda") * 0.3).to(dtype)
    lim = (7.0, 1.702, 1.0)
    ap = moe.act_params(ACTS[act], swiglu_fusion=1, limit=lim[0], alpha=lim[1], beta=lim[2]) \
        if gated else None
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kw = dict(act=ap, bias=bias, dtype=dtype, mx_out=mx_out, ws=ws)
    out = moe.moe_grouped_gemm_mx(*a, *w, segments(counts), N, **kw)
    assert moe.moe_sync_status(ws) == moe.MOE_OK
    check(moe, counts, a, w, bias, act, lim, N, out, dtype, mx_out)
    # the same rows through an index list, in another order in memory, bit for bit, twice
    order = torch.randperm(M, generator=g, device="cuda")
    shuffled = tuple(t.view(torch.uint8)[order].contiguous() for t in a)
    back = torch.empty(M, dtype=torch.int32, device="cuda")
    back[order] = torch.arange(M, device="cuda", dtype=torch.int32)
    for _ in range(2):
        again = moe.moe_grouped_gemm_mx(*shuffled, *w, segments(counts), N, row_to_route=back, **kw)
        for x, y in zip(out if mx_out else (out,), again if mx_out else (again,)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
