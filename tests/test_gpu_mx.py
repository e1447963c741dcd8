"""Microscaled quantisation, the RMS norm with 8-bit outputs and the grouped
GEMM over microscaled operands, against float64 (mx_reference.py).

Tolerances, from the operations (u = 2^-24; ut, half a step of the output type
relative to the value: bf16 2^-8, f16 2^-11, f32 2^-24, e4m3 2^-4):
* quantisation: scales and codes are exact functions of the input, equal bit
  for bit; dequantisation in bf16 / f32 likewise, f16 is one rounding.
* h = x + r: one float32 addition and one rounding: (u + ut) |x + r|.
* y: the squares are summed in chains of at most 64 additions a thread and 10
  across threads, so mean(h^2) is off by at most 76 u; its root halves that;
  rsqrtf adds 2 ulp = 4 u, the division and eps 1 u each before the root, the
  two products 2 u: 46 u in all, plus ut where y is written.
* codes of y: half an e4m3 step, 2^-4 |y| (or half of the smallest step,
  2^-10 scales), plus y's own 46 u; with a float32 scale also the quotient's and
  the scale's roundings, 3 u.
* products: operand values and their products are exact in float32; the sum
  of K terms goes through K / 32 accumulations, each off by at most 2 u of the
  terms' magnitude, four more for the sum inside a step and the bias:
  d = (K / 32 + 4) 2 u sum |a w|.
* activations: |act'| <= 1.13 max(1, alpha) per unit of the gate, times
  |up| + beta; the up half passes |act(g)| <= |g|; the fast exponential and quotient
  are within 2^-16 of the value over the arguments used here.  erf is within
  2 ulp of its result, which the factor covers.
"""
import numpy as np
import pytest
import torch

import mx_reference as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_ffn_gb300 import build, moe as m

    build.build()
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def f64(t):
    return t.double().cpu().numpy()


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


def rows_of(g, R_, K, dtype):
    """Rows of very different sizes."""
    x = torch.randn((R_, K), generator=g, device="cuda")
    return (x * torch.exp2(torch.randint(-12, 12, (R_, 1), generator=g, device="cuda"))).to(dtype)


def fmt_of(moe, fmt):
    return moe.MOE_MX_E2M1 if fmt == "e2m1" else moe.MOE_MX_E4M3


def check_quant(moe, x, fmt, got):
    codes, scales = got
    rc, rs = R.quantize(f64(x), fmt)
    assert np.array_equal(raw(scales), rs)
    assert np.array_equal(raw(codes), R.pack(rc) if fmt == "e2m1" else rc)


# ------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 32), (3, 33), (7, 128), (5, 129), (2, 1000),
                                    (67, 2880), (300, 255)])
def test_quantize_equals_the_definition(moe, rows, K, dtype, fmt):
    x = rows_of(gen(rows * K), rows, K, dtype)
    check_quant(moe, x, fmt, moe.moe_mx_quantize(x, fmt_of(moe, fmt)))


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("K,wide,shift", [(64, 80, 0), (64, 80, 1), (100, 101, 0), (256, 264, 8)])
def test_quantize_strided_rows(moe, K, wide, shift, fmt):
    big = rows_of(gen(wide), 9, wide + shift, torch.bfloat16)
    x = big[:, shift:shift + K]
    check_quant(moe, x.contiguous(), fmt, moe.moe_mx_quantize(x, fmt_of(moe, fmt)))


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_special_values(moe, dtype, fmt):
    """Zero blocks, signed zeros, the smallest and largest values, every tie and table value,
    infinities and NaNs."""
    fi = torch.finfo(dtype)
    big = fi.max
    table = R.E4M3 if fmt == "e4m3" else R.E2M1
    mids = (table[1:] + table[:-1]) / 2
    x = torch.zeros((12, 160), dtype=torch.float64)
    x[1, 0], x[1, 40] = -0.0, fi.tiny
    x[2, :8] = torch.tensor([big, -big, fi.tiny, 1.0, -1.0, 0.5, big / 2, fi.smallest_normal])
    x[3, 3] = float(fi.smallest_normal) * fi.eps  # the smallest subnormal
    x[4, 5] = float("inf")
    x[5, 100] = float("nan")
    x[6, 0], x[6, 31], x[6, 32] = float("-inf"), float("nan"), 3.0
    pts = np.concatenate([table, mids])
    pts = pts[pts <= table[-1]]
    for r in range(4):  # blocks led by the largest value, so the points meet scale 1
        take = np.random.RandomState(r).choice(pts, 31)
        x[7 + r, 0] = float(table[-1])
        x[7 + r, 1:32] = torch.from_numpy(take * np.random.RandomState(r).choice([-1, 1], 31))
    x[11, :5] = torch.tensor([7.0, -6.5, 6.0, 5.0, 7.9])  # e2m1 saturates above 6
    x = x.to(dtype).cuda()
    got = moe.moe_mx_quantize(x, fmt_of(moe, fmt))
    check_quant(moe, x, fmt, got)
    v = moe.moe_mx_dequantize(*got, 160, dtype=torch.float32)
    assert torch.isnan(v[4, :32]).all() and torch.isfinite(v[4, 32:]).all()
    assert torch.isnan(v[5, 96:128]).all() and torch.isnan(v[6, :32]).all()
    assert torch.isfinite(v[6, 32:]).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("rows,K", [(1, 1), (5, 129), (33, 256), (67, 2880)])
def test_dequantize(moe, rows, K, out, fmt):
    codes, scales = moe.moe_mx_quantize(rows_of(gen(K), rows, K, torch.float32), fmt_of(moe, fmt))
    v = moe.moe_mx_dequantize(codes, scales, K, dtype=out)
    c = R.unpack(raw(codes)) if fmt == "e2m1" else raw(codes)
    ref = torch.from_numpy(R.values(c, raw(scales), fmt)[:, :K])
    assert torch.equal(v.cpu(), ref.to(out))


def test_quantize_past_32_bit_offsets(moe):
    """More than 2^31 elements: the first and the last rows."""
    K, rows = 7168, 300_001
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    for at in (slice(0, 3), slice(rows - 3, rows)):
        x[at] = rows_of(gen(3), 3, K, torch.bfloat16)
    for fmt in ("e4m3", "e2m1"):
        codes, scales = moe.moe_mx_quantize(x, fmt_of(moe, fmt))
        for at in (slice(0, 3), slice(rows - 3, rows)):
            check_quant(moe, x[at], fmt, (codes[at], scales[at]))
        v = moe.moe_mx_dequantize(codes, scales, K)
        assert torch.equal(v[-3:], moe.moe_mx_dequantize(codes[-3:], scales[-3:], K))


# ------------------------------------------------------------------ norm
NORM_U = 46 * U


def check_norm(moe, x, w, r, eps, quant, o):
    dt = x.dtype
    h = x if r is None else o["residual"]
    if r is not None:
        s = f64(x) + f64(r)
        assert (np.abs(f64(h) - s) <= (U + HALF[dt]) * np.abs(s) + TINY[dt]).all()
    y = R.rms_norm(f64(h), f64(w), eps)
    if o["out"] is not None:
        assert (np.abs(f64(o["out"]) - y) <= (NORM_U + HALF[dt]) * np.abs(y) + TINY[dt]).all()
    if quant == moe.MOE_QUANT_NONE:
        return
    T, H = x.shape
    Hp = R.padded(H)
    yp = np.zeros((T, Hp))
    yp[:, :H] = y
    if quant == moe.MOE_QUANT_MX_E4M3:
        got = R.values(raw(o["codes"]), raw(o["scales"]), "e4m3")
        s = np.ldexp(1.0, raw(o["scales"]).astype(int) - 127)
        amax = np.abs(yp).reshape(T, -1, 32).max(2)
        lo = R.scale_exponents(amax * (1 - NORM_U), "e4m3")
        hi = R.scale_exponents(amax * (1 + NORM_U), "e4m3")
        e = raw(o["scales"]).astype(int) - 127
        assert ((lo <= e) & (e <= hi)).all()
        step, more = np.repeat(s, 32, 1), NORM_U
    else:
        s = f64(o["scales"])
        amax = np.abs(yp).reshape(T, -1, 128).max(2)
        assert (np.abs(s - np.maximum(amax / 448, 2.0 ** -126)) <= (NORM_U + U) * s).all()
        step, more = np.repeat(s, 128, 1), NORM_U + 3 * U
        got = R.values(raw(o["codes"]), np.full((T, Hp // 32), 127, np.uint8), "e4m3") * step
    assert (np.abs(got - yp) <= (2.0 ** -4 + more) * np.abs(yp) + 2.0 ** -10 * step * (1 + more)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("quant", [0, 1, 2])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 7168), (3, 31), (5, 129), (2, 1000), (700, 64),
                                 (513, 1024), (400, 2880), (160, 8200), (2, 65536)])
def test_add_rms_norm(moe, T, H, quant, dtype):
    g = gen(T * H + quant)
    x, r = (torch.randn((T, H), generator=g, device="cuda").to(dtype) for _ in range(2))
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(dtype)
    check_norm(moe, x, w, r, 1e-6, quant, moe.moe_add_rms_norm(x, w, residual=r, quant=quant))
    o = moe.moe_add_rms_norm(x, w, eps=1e-3, quant=quant, out=quant == 0)
    assert o["residual"] is None
    check_norm(moe, x, w, None, 1e-3, quant, o)


def test_add_rms_norm_in_place_and_unaligned(moe):
    g = gen(5)
    flat = torch.randn(3 * 9 * 264 + 3, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.ones(264, dtype=torch.bfloat16, device="cuda")
    for off in (0, 1):  # one element off a 16-byte boundary: the element-wise loads
        x = flat[off:off + 9 * 264].view(9, 264)
        r = flat[9 * 264 + off + 1:2 * 9 * 264 + off + 1].view(9, 264)
        apart = moe.moe_add_rms_norm(x, w, residual=r, quant=1)
        mine = r.clone()
        same = moe.moe_add_rms_norm(x, w, residual=mine, residual_out=mine, quant=1)
        assert same["residual"].data_ptr() == mine.data_ptr()
        for k in ("residual", "out", "codes", "scales"):
            assert torch.equal(apart[k].view(torch.uint8), same[k].view(torch.uint8)), k
        check_norm(moe, x, w, r, 1e-6, 1, apart)


@pytest.mark.parametrize("quant", [1, 2])
def test_add_rms_norm_rows_of_zeros_and_non_finite(moe, quant):
    H = 320
    x = torch.randn((5, H), generator=gen(1), device="cuda")
    x[1] = 0
    x[2, 7] = float("inf")
    x[3, 300] = float("nan")
    w = torch.ones(H, device="cuda")
    w[40] = float("inf")
    o = moe.moe_add_rms_norm(x, w, quant=quant)
    s = o["scales"].float()
    block = 32 if quant == 1 else 128
    hit = 40 // block
    # one column's infinite weight spoils its block alone; the row of zeros gives 0 * inf there
    for t in (0, 4):
        assert torch.isnan(s[t, hit]) and not torch.isnan(s[t, hit + 1:]).any()
        assert (o["codes"].float()[t, hit * block:(hit + 1) * block] == 0).all()
    assert torch.isnan(s[1, hit]) and (o["out"][1, 64:] == 0).all()
    # an infinite element makes the row's mean square infinite: inf * 0 in its place, 0 elsewhere
    assert torch.isnan(o["out"][2, 7]) and torch.isnan(s[2, 7 // block])
    assert torch.isnan(o["out"][3]).all() and torch.isnan(s[3, :H // block]).all()


def test_norm_feeds_the_fp8_grouped_gemm(moe):
    """The block-128 rows are the operand of moe_grouped_gemm_fp8_masked: its result is the
    product of the values that codes and scales stand for."""
    g = gen(8)
    T, H, N = 40, 256, 128
    x = torch.randn((T, H), generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    o = moe.moe_add_rms_norm(x, w, quant=moe.MOE_QUANT_E4M3_BLOCK128)
    b = torch.randn((1, N, H), generator=g, device="cuda").to(torch.float8_e4m3fn)
    bs = torch.ones((1, N // 128, H // 128), device="cuda")
    out = moe.moe_grouped_gemm_fp8_masked(o["codes"][None], o["scales"][None], b, bs,
                                          torch.tensor([T], dtype=torch.int32, device="cuda"))
    a = f64(o["codes"].float()) * np.repeat(f64(o["scales"]), 128, 1)
    bv = f64(b[0].float())
    ref, mag = a @ bv.T, np.abs(a) @ np.abs(bv).T
    # K / 32 steps, and a scale product and one addition per 128 columns
    assert (np.abs(f64(out[0]) - ref) <= 2.0 ** -8 * np.abs(ref) + (H / 32 + H / 128 + 6) * 2 * U * mag).all()


# ------------------------------------------------------------------ grouped GEMM
ACTS = {"none": None, "silu_and_mul": 0, "swiglu": 1, "gelu_and_mul": 3, "relu": 4, "gelu": 5,
        "silu": 6, "identity": 2}
GATED = ("silu_and_mul", "swiglu", "gelu_and_mul")


def mx_weights(moe, g, E, N, K):
    w = torch.randn((E, N, K), generator=g, device="cuda") * K ** -0.5
    return moe.moe_mx_quantize(w, moe.MOE_MX_E2M1)


def segments(counts):
    return torch.tensor(np.cumsum(counts), dtype=torch.int32, device="cuda")


def reference(a, w, bias, seg, act, N, inter, lim):
    """act(p) in float64 and how far the kernel's float32 value may be from it."""
    av = R.values(raw(a[0]), raw(a[1]), "e4m3")
    wv = R.values(R.unpack(raw(w[0])), raw(w[1]), "e2m1")
    p, mag = R.grouped(av, wv, None if bias is None else f64(bias), seg.cpu().numpy())
    d = (av.shape[1] / 32 + 4) * 2 * U * mag
    v = R.activation(p, act, N, inter, *lim)
    if act in GATED:
        limit, alpha, beta = lim
        g, u = (p[:, 0::2], p[:, 1::2]) if inter else (p[:, :N], p[:, N:])
        dg, du = (d[:, 0::2], d[:, 1::2]) if inter else (d[:, :N], d[:, N:])
        if act != "swiglu":
            alpha, beta = 1.0, 0.0
        dv = 1.13 * max(1.0, alpha) * (np.abs(u) + abs(beta)) * dg + (np.abs(g) + dg) * du
        return v, dv + 2.0 ** -16 * np.abs(v)
    return v, 1.13 * d + (2.0 ** -16 * np.abs(v) if act in ("gelu", "silu") else 0.0)


def run_gemm(moe, counts, N, K, act="none", bias=False, dtype=torch.bfloat16, inter=False,
             lim=(0.0, 1.0, 0.0), mx_out=False, seed=0, extra_rows=0):
    g = gen(seed + N + K)
    E, M = len(counts), int(np.sum(counts))
    a = moe.moe_mx_quantize(rows_of(g, M + extra_rows, K, torch.float32) * 0.01)
    N1 = 2 * N if act in GATED else N
    w = mx_weights(moe, g, E, N1, K)
    b = (torch.randn((E, N1), generator=g, device="cuda") * 0.3).to(dtype) if bias else None
    seg = segments(counts)
    kind = ACTS[act]
    ap = None if kind is None else moe.act_params(kind, swiglu_fusion=1 if inter else 2,
                                                  limit=lim[0], alpha=lim[1], beta=lim[2])
    ws = torch.zeros(moe.moe_grouped_gemm_mx_workspace_size(M + extra_rows, N, K, E),
                     dtype=torch.uint8, device="cuda")
    Np = moe.moe_mx_columns(N)
    rows = M + extra_rows
    if mx_out:  # guarded outputs: rows past the last segment and bytes past the end stay
        flat = torch.full(((rows + 1) * Np,), 0x5A, dtype=torch.uint8, device="cuda")
        sflat = torch.full(((rows + 1) * Np // 32,), 0x5A, dtype=torch.uint8, device="cuda")
        out = (flat[:rows * Np].view(rows, Np), sflat[:rows * (Np // 32)].view(rows, Np // 32))
        got = moe.moe_grouped_gemm_mx(*a, *w, seg, N, act=ap, bias=b, dtype=dtype, mx_out=True,
                                      out=out[0], out_scale=out[1], ws=ws)
        tail = [flat[M * Np:], sflat[M * (Np // 32):]]
    else:
        flat = torch.full(((rows + 1) * N,), 123.0, dtype=dtype, device="cuda")
        got = moe.moe_grouped_gemm_mx(*a, *w, seg, N, act=ap, bias=b, dtype=dtype,
                                      out=flat[:rows * N].view(rows, N), ws=ws)
        tail = [flat[M * N:]]
    assert moe.moe_sync_status(ws) == moe.MOE_OK
    for t in tail:
        assert (t == (0x5A if mx_out else 123.0)).all(), "wrote outside its rows"
    v, d = reference((a[0][:M], a[1][:M]), w, b, seg, act, N, inter, lim)
    if not mx_out:
        err = np.abs(f64(got[:M]) - v)
        ok = err <= d + HALF[dtype] * (np.abs(v) + d) + TINY[dtype]
        assert ok.all(), (int((~ok).sum()), float(err[~ok].max()))
        return
    codes, scales = raw(got[0])[:M], raw(got[1])[:M]
    vp, dp = np.zeros((M, Np)), np.zeros((M, Np))
    vp[:, :N], dp[:, :N] = v, d
    top = np.abs(vp).reshape(M, Np // 32, 32)
    more = dp.reshape(M, Np // 32, 32).max(2)
    lo = R.scale_exponents(np.maximum(top.max(2) - more, 0), "e4m3")
    hi = R.scale_exponents(top.max(2) + more, "e4m3")
    e = scales.astype(int) - 127
    assert ((lo <= e) & (e <= hi)).all()
    s = np.repeat(np.ldexp(1.0, e), 32, 1)
    err = np.abs(R.values(codes, scales, "e4m3") - vp)
    assert (err <= dp + 2.0 ** -4 * (np.abs(vp) + dp) + 2.0 ** -10 * s).all()
    assert (codes[:, N:] & 127 == 0).all()  # padding columns


@pytest.mark.parametrize("N,K", [(1, 1), (5, 32), (130, 129), (256, 384), (300, 2880), (1000, 640)])
@pytest.mark.parametrize("counts", [[1], [3, 0, 1], [0, 17, 5, 0], [40, 0, 100], [113, 1, 300],
                                    [450]])
def test_gemm_mx_plain(moe, counts, N, K):
    run_gemm(moe, counts, N, K, bias=len(counts) > 1, extra_rows=2)


@pytest.mark.parametrize("act", ["silu_and_mul", "gelu_and_mul", "relu", "gelu", "silu", "identity"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mx_out", [False, True])
def test_gemm_mx_activations(moe, act, dtype, mx_out):
    run_gemm(moe, [20, 0, 9, 60], 144, 256, act=act, bias=True, dtype=dtype, mx_out=mx_out)
    run_gemm(moe, [2, 1], 72, 160, act=act, dtype=dtype, mx_out=mx_out)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("mx_out", [False, True])
@pytest.mark.parametrize("counts", [[3, 0, 4], [70, 33, 0, 1], [260, 500]])
def test_gemm_mx_swiglu(moe, counts, inter, mx_out):
    run_gemm(moe, counts, 200, 416, act="swiglu", bias=True, inter=inter, lim=(7.0, 1.702, 1.0),
             mx_out=mx_out, extra_rows=1)
    run_gemm(moe, counts, 45, 96, act="swiglu", inter=inter, lim=(0.0, 1.0, 0.0), mx_out=mx_out)


@pytest.mark.parametrize("mx_out", [False, True])
def test_gemm_mx_no_rows(moe, mx_out):
    run_gemm(moe, [0, 0, 0], 64, 128, extra_rows=3, mx_out=mx_out)
    g = gen(1)
    w = mx_weights(moe, g, 2, 64, 128)
    a = moe.moe_mx_quantize(torch.zeros((0, 128), device="cuda"))
    out = moe.moe_grouped_gemm_mx(*a, *w, segments([0, 0]), 64)
    assert out.shape == (0, 64)


@pytest.mark.parametrize("rows", [6, 200, 1500])
def test_gemm_mx_gathered_rows(moe, rows):
    """Rows through row_to_route equal the product of the gathered copy, bit for bit; entries
    out of range give rows of zeros."""
    g = gen(rows)
    E, N, K, T, k = 5, 272, 544, max(3, rows // 3), 3
    a = moe.moe_mx_quantize(rows_of(g, T, K, torch.float32))
    w = mx_weights(moe, g, E, N, K)
    r2r = torch.randint(0, T * k, (rows,), generator=g, device="cuda").to(torch.int32)
    cuts = torch.sort(torch.randint(0, rows + 1, (E - 1,), generator=g, device="cuda")).values
    seg = torch.cat([cuts, torch.tensor([rows], device="cuda")]).to(torch.int32)
    got = moe.moe_grouped_gemm_mx(*a, *w, seg, N, row_to_route=r2r, top_k=k)
    at = (r2r // k).long()
    copy = (a[0].view(torch.uint8)[at], a[1].view(torch.uint8)[at])
    assert torch.equal(got, moe.moe_grouped_gemm_mx(*copy, *w, seg, N))
    bad = r2r.clone()
    bad[0], bad[-1] = -1, T * k
    got2 = moe.moe_grouped_gemm_mx(*a, *w, seg, N, row_to_route=bad, top_k=k)
    assert (got2[0] == 0).all() and (got2[-1] == 0).all() and torch.equal(got2[1:-1], got[1:-1])


def test_gemm_mx_nan_scale_and_zero_rows(moe):
    g = gen(3)
    x = rows_of(g, 6, 192, torch.float32)
    x[2, 70] = float("inf")
    x[4] = 0
    a = moe.moe_mx_quantize(x)
    w = mx_weights(moe, g, 1, 96, 192)
    out = moe.moe_grouped_gemm_mx(*a, *w, segments([6]), 96)
    assert torch.isnan(out[2]).all() and (out[4] == 0).all()
    assert torch.isfinite(out[[0, 1, 3, 5]]).all()
    q = moe.moe_grouped_gemm_mx(*a, *w, segments([6]), 96, mx_out=True)
    assert torch.isnan(q[1].float()[2, :3]).all() and torch.isfinite(q[1].float()[[0, 1, 3, 5]]).all()


def test_gemm_mx_past_32_bit_offsets(moe):
    """Weights of more than 4 GB and rows of more than 2^31 bytes: the last expert's rows."""
    g = gen(4)
    E, N, K, M = 330, 4096, 7168, 300_100
    one = mx_weights(moe, g, 1, N, K)
    w = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.zeros((E, N, K // 32), dtype=torch.uint8, device="cuda")
    w[-1], ws[-1] = one[0][0], one[1].view(torch.uint8)[0]
    few = moe.moe_mx_quantize(rows_of(g, 100, K, torch.float32))
    a = torch.zeros((M, K), dtype=torch.uint8, device="cuda")
    s = torch.zeros((M, K // 32), dtype=torch.uint8, device="cuda")
    a[-100:], s[-100:] = few[0].view(torch.uint8), few[1].view(torch.uint8)
    r2r = torch.arange(M - 100, M, device="cuda", dtype=torch.int32)
    seg = torch.zeros(E, dtype=torch.int32, device="cuda")
    seg[-1] = 100
    got = moe.moe_grouped_gemm_mx(a, s, w, ws, seg, N, row_to_route=r2r, top_k=1)
    assert torch.equal(got, moe.moe_grouped_gemm_mx(*few, *one, segments([100]), N))


@pytest.mark.parametrize("mx_out", [False, True])
@pytest.mark.parametrize("ends", [[70, 20, 40, 300], [-5, 10, 5, 64], [500, 900, -3, 2], [0, 0, 0, -1]])
def test_gemm_mx_clamps_segment_ends(moe, ends, mx_out):
    """Segment ends outside [0, M] or below the one before are clamped: an expert owns the rows
    from the end before it to its own, none if that is behind it; nothing else is written."""
    M, N, K = 64, 144, 256
    g = gen(M)
    a = moe.moe_mx_quantize(torch.randn((M, K), generator=g, device="cuda"))
    w = mx_weights(moe, g, 4, 2 * N, K)
    seg = torch.tensor(ends, dtype=torch.int32, device="cuda")
    act = moe.act_params()
    Np = moe.moe_mx_columns(N)
    fill = 0x5A
    out = torch.full((M + 2, Np if mx_out else 2 * N), fill, dtype=torch.uint8, device="cuda")
    sc = torch.full((M + 2, Np // 32), fill, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    if mx_out:
        moe.moe_grouped_gemm_mx(*a, *w, seg, N, act=act, mx_out=True, out=out[:M], out_scale=sc[:M],
                                ws=ws)
    else:
        moe.moe_grouped_gemm_mx(*a, *w, seg, N, act=act, out=out[:M].view(torch.bfloat16), ws=ws)
    assert moe.moe_sync_status(ws) == moe.MOE_OK
    start = [0] + [min(max(e, 0), M) for e in ends]
    want = torch.full_like(out, fill)
    for e in range(4):  # an expert that several ranges reach: each on its own, in expert order
        lo, hi = start[e], start[e + 1]
        if hi > lo:
            one = torch.tensor([hi - lo], dtype=torch.int32, device="cuda")
            part = (a[0][lo:hi].clone(), a[1][lo:hi].clone())  # aligned copies
            r = moe.moe_grouped_gemm_mx(*part, w[0][e:e + 1], w[1][e:e + 1], one, N, act=act,
                                        mx_out=mx_out)
            if mx_out:
                want[lo:hi] = r[0].view(torch.uint8)
            else:
                want[lo:hi] = r.view(torch.uint8)
    seen = torch.zeros(M + 2, dtype=torch.int32)
    for e in range(4):
        seen[start[e]:max(start[e + 1], start[e])] += 1
    once = (seen <= 1).cuda()  # rows that two ranges share hold either's result
    assert torch.equal(out[once], want[once])
    assert (out[M:] == fill).all() and (sc[M:] == fill).all()


def test_gemm_mx_most_experts(moe):
    counts = [i % 3 for i in range(1024)]
    run_gemm(moe, counts, 40, 128)


def test_gemm_mx_repeats_itself_on_streams_and_in_a_graph(moe):
    g = gen(12)
    a = moe.moe_mx_quantize(rows_of(g, 300, 512, torch.float32))
    w = mx_weights(moe, g, 4, 320, 512)
    seg = segments([10, 0, 250, 40])
    ws = [torch.zeros(moe.moe_grouped_gemm_mx_workspace_size(300, 320, 512, 4), dtype=torch.uint8,
                      device="cuda") for _ in range(3)]
    first = moe.moe_grouped_gemm_mx(*a, *w, seg, 320, ws=ws[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = moe.moe_grouped_gemm_mx(*a, *w, seg, 320, ws=ws[1])
    again = moe.moe_grouped_gemm_mx(*a, *w, seg, 320, ws=ws[0])
    torch.cuda.current_stream().wait_stream(side)
    x = torch.randn((300, 512), generator=g, device="cuda").to(torch.bfloat16)
    wt = torch.ones(512, dtype=torch.bfloat16, device="cuda")

    def step():
        n = moe.moe_add_rms_norm(x, wt, quant=moe.MOE_QUANT_MX_E4M3, out=False)
        return moe.moe_grouped_gemm_mx(n["codes"], n["scales"], *w, seg, 320, ws=ws[2])

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    out.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, other) and torch.equal(first, again) and torch.equal(out, want)


# ------------------------------------------------------------------ the layer
def layer_inputs(moe, T, H, F, E, k, act, dtype, seed=0):
    g = gen(seed + T)
    gated = act in GATED
    N1 = 2 * F if gated else F
    hidden = moe.moe_mx_quantize(torch.randn((T, H), generator=g, device="cuda"))
    logits = torch.randn((T, E), generator=g, device="cuda")
    w1, w2 = mx_weights(moe, g, E, N1, H), mx_weights(moe, g, E, H, F)
    b1 = (torch.randn((E, N1), generator=g, device="cuda") * 0.1).to(dtype)
    b2 = (torch.randn((E, H), generator=g, device="cuda") * 0.1).to(dtype)
    return hidden, logits, w1, w2, b1, b2


@pytest.mark.parametrize("T,H,F,E,k,act,dtype,scoring", [
    (1, 256, 128, 8, 2, "swiglu", torch.bfloat16, "softmax"),
    (37, 200, 96, 6, 3, "silu_and_mul", torch.float16, "sigmoid"),
    (300, 384, 260, 16, 4, "swiglu", torch.bfloat16, "softmax"),
    (64, 128, 72, 600, 2, "gelu", torch.bfloat16, "sqrt_softplus"),  # separate route and permute
    (33, 130, 64, 5, 5, "silu_and_mul", torch.bfloat16, "softmax"),  # columns not a multiple of 4
    (20, 256, 96, 12, 9, "gelu_and_mul", torch.float32, "softmax"),
])
def test_layer_equals_its_stages(moe, T, H, F, E, k, act, dtype, scoring):
    """Bit for bit the staged calls', and the down product's float64 value from the kernels'
    own activation codes, combined."""
    hidden, logits, w1, w2, b1, b2 = layer_inputs(moe, T, H, F, E, k, act, dtype)
    p = moe.route_params(k, scoring, True)
    ap = moe.act_params(ACTS[act], swiglu_fusion=1, limit=7.0, alpha=1.702, beta=1.0)
    ti = torch.empty((T, k), dtype=torch.int32, device="cuda")
    ws = torch.zeros(moe.moe_workspace_size_mx(T, H, F, E, k), dtype=torch.uint8, device="cuda")
    out = moe.moe_ffn_forward_mx(*hidden, logits, *w1, *w2, H, F, p, ap, b_gate_up=b1, b_down=b2,
                                 dtype=dtype, topk_ids_out=ti, ws=ws)
    assert moe.moe_sync_status(ws) == moe.MOE_OK
    tw, ids, _, _ = moe.moe_route(logits, p)
    assert torch.equal(ids, ti)
    m = moe.moe_permute(ids, E)
    mid = moe.moe_grouped_gemm_mx(*hidden, *w1, m["seg_end"], F, act=ap, bias=b1, dtype=dtype,
                                  row_to_route=m["row_to_route"], top_k=k, mx_out=True)
    y = moe.moe_grouped_gemm_mx(*mid, *w2, m["seg_end"], H, bias=b2.float(), dtype=torch.float32)
    assert torch.equal(out, moe.moe_combine(y, tw, m["route_to_row"]).to(dtype))
    v, d = reference(mid, w2, b2, m["seg_end"], "none", H, False, (0, 1, 0))
    at = m["route_to_row"].long().cpu().numpy().reshape(T, k)
    wt = f64(tw)
    ref = sum(wt[:, j:j + 1] * v[at[:, j]] for j in range(k))
    tol = sum(np.abs(wt[:, j:j + 1]) * (d[at[:, j]] + (4 + k) * U * np.abs(v[at[:, j]]))
              for j in range(k))
    assert (np.abs(f64(out) - ref) <= tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(ref) + TINY[dtype]).all()


def test_layer_after_the_norm_with_fixed_experts(moe):
    """norm -> layer as a program runs them, with fixed expert ids and a correction bias's
    scoring; an empty batch is a no-op."""
    T, H, F, E, k = 12, 320, 160, 10, 2
    g = gen(9)
    _, logits, w1, w2, _, _ = layer_inputs(moe, T, H, F, E, k, "silu_and_mul", torch.bfloat16)
    x, r = (torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    wt = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    n = moe.moe_add_rms_norm(x, wt, residual=r, quant=moe.MOE_QUANT_MX_E4M3)
    ids = torch.stack([torch.randperm(E)[:k] for _ in range(T)]).to(torch.int32).cuda()
    p, ap = moe.route_params(k, "sigmoid", True, routed_scaling_factor=2.5), moe.act_params()
    bias = torch.randn(E, generator=g, device="cuda")
    out = moe.moe_ffn_forward_mx(n["codes"], n["scales"], logits, *w1, *w2, H, F, p, ap,
                                 correction_bias=bias, expert_ids=ids)
    tw, got, _, _ = moe.moe_route(logits, p, correction_bias=bias, expert_ids=ids)
    m = moe.moe_permute(got, E)
    mid = moe.moe_grouped_gemm_mx(n["codes"], n["scales"], *w1, m["seg_end"], F, act=ap,
                                  row_to_route=m["row_to_route"], top_k=k, mx_out=True)
    y = moe.moe_grouped_gemm_mx(*mid, *w2, m["seg_end"], H, dtype=torch.float32)
    assert torch.equal(out, moe.moe_combine(y, tw, m["route_to_row"]).to(torch.bfloat16))
    empty = moe.moe_ffn_forward_mx(n["codes"][:0], n["scales"][:0], logits[:0], *w1, *w2, H, F, p, ap)
    assert empty.shape == (0, H)


# ------------------------------------------------------------------ the binding's refusals
def test_binding_refuses_mismatched_tensors(moe):
    g = gen(2)
    x = torch.randn((8, 256), generator=g, device="cuda").to(torch.bfloat16)
    one = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    a = moe.moe_mx_quantize(x)
    w = mx_weights(moe, g, 2, 64, 256)
    seg = segments([3, 5])
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    bad = [
        lambda: moe.moe_mx_quantize(x, codes=small),
        lambda: moe.moe_mx_quantize(x, scales=small),
        lambda: moe.moe_mx_quantize(x.t()),
        lambda: moe.moe_mx_dequantize(*a, 300),
        lambda: moe.moe_mx_dequantize(*a, 256, out=small),
        lambda: moe.moe_add_rms_norm(x, one, out=small),
        lambda: moe.moe_add_rms_norm(x, one, quant=1, codes=small),
        lambda: moe.moe_add_rms_norm(x, one, quant=2, scales=small),
        lambda: moe.moe_add_rms_norm(x, one.float()),
        lambda: moe.moe_add_rms_norm(x, one[:128]),
        lambda: moe.moe_add_rms_norm(x, one, residual=x[:4]),
        lambda: moe.moe_add_rms_norm(x, one, residual=x, residual_out=small),
        lambda: moe.moe_grouped_gemm_mx(*a, *w, seg, 65),
        lambda: moe.moe_grouped_gemm_mx(*a, *w, seg, 64, act=moe.act_params()),
        lambda: moe.moe_grouped_gemm_mx(*a, *w, seg[:1], 64),
        lambda: moe.moe_grouped_gemm_mx(*a, *w, seg.long(), 64),
        lambda: moe.moe_grouped_gemm_mx(x, a[1], *w, seg, 64),
        lambda: moe.moe_grouped_gemm_mx(*a, *w, seg, 64, out=small),
        lambda: moe.moe_grouped_gemm_mx(*a, *w, seg, 64, mx_out=True, out=small),
        lambda: moe.moe_grouped_gemm_mx(*a, *w, seg, 64, bias=torch.zeros((2, 64), device="cuda")),
        lambda: moe.moe_ffn_forward_mx(*a, torch.zeros((8, 2), device="cuda"), *w, *w, 256, 64,
                                       moe.route_params(1), moe.act_params()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            raise AssertionError(f"call {i} was accepted")
    with pytest.raises(moe.MoEError) as e:  # scales off a 16-byte boundary
        moe.moe_grouped_gemm_mx(a[0][1:], a[1].view(torch.uint8)[1:], *w, segments([3, 4]), 64)
    assert e.value.status == moe.MOE_ERR_UNSUPPORTED
