"""Gradients of the routed layer's stages on the GPU against float64 definitions
(grad_reference.py), with the bounds that file derives: sizes from one token, odd ones,
empty experts, dropped routes, rows behind the last segment, NaN next door, graphs and
streams."""
import numpy as np
import pytest
import torch

import grad_reference as R
import mx_reference

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
KINDS = {"silu": 0, "swiglu": 1, "identity": 2, "gelu": 3, "relu": 4, "gelu1": 5, "silu1": 6}
GATED = ("silu", "swiglu", "gelu")


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_ffn_gb300 import build, moe as m

    build.build()
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def segments(counts):
    return torch.tensor(np.cumsum(counts), dtype=torch.int32, device="cuda")


def shuffled(g, M):
    return torch.randperm(M, generator=g, device="cuda").to(torch.int32)


# ------------------------------------------------------------------ tokens and routes
SIZES = [(1, 1, 1), (1, 8, 7168), (3, 2, 100), (7, 3, 33), (37, 8, 264), (130, 5, 2880), (64, 64, 24)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K,H", SIZES)
def test_combine_backward(moe, T, K, H, dtype):
    g = gen(T * K + H)
    M = T * K
    d, y = randn(g, T, H, dtype=dtype), randn(g, M, H, dtype=dtype)
    w, r2r = torch.rand((T, K), generator=g, device="cuda"), shuffled(g, M)
    dy, dw = moe.moe_combine_backward(d, y, w, r2r, scale=1.75)
    ry, rw, sy, sw = R.combine_backward(d, y, w, r2r, 1.75)
    R.close(dy, ry, sy, "d_expert_out")
    R.close(dw, rw, sw, "d_topk_weights")
    # each output on its own is the same
    only_y, none = moe.moe_combine_backward(d, None, w, r2r, scale=1.75, d_topk_weights=False)
    assert none is None and torch.equal(only_y, dy)
    none, only_w = moe.moe_combine_backward(d, y, w, r2r, scale=1.75, d_expert_out=False)
    assert none is None and torch.equal(only_w, dw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K,H", SIZES)
def test_permute_backward(moe, T, K, H, dtype):
    g = gen(T * K * H)
    x, r2r = randn(g, T * K, H, dtype=dtype), shuffled(g, T * K)
    out = moe.moe_permute_backward(x, r2r, K)
    ref, slack = R.permute_backward(x, r2r, K)
    R.close(out, ref, slack, "d_hidden")


@pytest.mark.parametrize("H", [64, 77, 7168])
def test_unaligned_rows(moe, H):
    """Tensors that start one element into an allocation."""
    g = gen(H)
    T, K = 5, 3
    M = T * K
    flat = lambda n, dt: randn(g, n + 1, dtype=dt)[1:]  # noqa: E731
    for dt in DTYPES:
        d, y = flat(T * H, dt).view(T, H), flat(M * H, dt).view(M, H)
        w, r2r = torch.rand((T, K), generator=g, device="cuda"), shuffled(g, M)
        dy = flat(M * H, dt).view(M, H)
        moe.moe_combine_backward(d, y, w, r2r, d_expert_out=dy)
        ry, _, sy, _ = R.combine_backward(d, y, w, r2r, 1.0)
        R.close(dy, ry, sy)
        ref, slack = R.permute_backward(y, r2r, K)
        R.close(moe.moe_permute_backward(y, r2r, K), ref, slack)


@pytest.mark.parametrize("H", [40, 7168])
def test_routes_without_a_row(moe, H):
    """Entries outside [0, T * K): a zero weight gradient, no row written, nothing added; NaN in
    the rows that nothing names stays out."""
    g = gen(2)
    T, K = 9, 4
    M = T * K
    d, y = randn(g, T, H, dtype=torch.bfloat16), randn(g, M, H, dtype=torch.bfloat16)
    w, r2r = torch.rand((T, K), generator=g, device="cuda"), shuffled(g, M)
    gone = [0, 5, 17, M - 1, 20, 21, 22, 23]  # a whole token among them
    free = r2r[gone].long()
    r2r[gone] = torch.tensor([-1, M, 2 ** 31 - 1, -2 ** 31, -1, -1, M + 7, -5], dtype=torch.int32,
                             device="cuda")
    y[free] = float("nan")
    dy = torch.full((M, H), 7.0, dtype=torch.bfloat16, device="cuda")
    _, dw = moe.moe_combine_backward(d, y, w, r2r, d_expert_out=dy)
    assert (dy[free] == 7).all() and (dw.flatten()[gone] == 0).all()
    ry, rw, sy, sw = R.combine_backward(d, y, w, r2r, 1.0)
    ry[free], sy[free] = 7.0, 0.0
    R.close(dy, ry, sy)
    R.close(dw, rw, sw)
    out = moe.moe_permute_backward(y, r2r, K)
    ref, slack = R.permute_backward(y, r2r, K)
    R.close(out, ref, slack)
    assert (out[5] == 0).all()


def test_combine_backward_non_finite(moe):
    """A NaN or an infinity stays in its route (weights) and its token (rows)."""
    g = gen(3)
    T, K, H = 6, 2, 512
    d, y = randn(g, T, H), randn(g, T * K, H)
    w, r2r = torch.rand((T, K), generator=g, device="cuda"), shuffled(g, T * K)
    y[int(r2r[3]), 100] = float("nan")
    d[4, 7] = float("inf")
    w[0, 0] = 0.0
    dy, dw = moe.moe_combine_backward(d, y, w, r2r)
    nan = torch.isnan(dw).flatten()
    assert nan[3] and int(nan.sum()) == 1
    assert torch.isinf(dw[4]).all() and (dy[r2r[8:10].long(), 7] == float("inf")).all()
    assert (dy[int(r2r[0])] == 0).all()


def test_no_tokens(moe):
    e = torch.empty
    i32 = dict(dtype=torch.int32, device="cuda")
    dy, dw = moe.moe_combine_backward(e((0, 8), device="cuda"), e((0, 8), device="cuda"),
                                      e((0, 2), device="cuda"), e(0, **i32))
    assert dy.shape == (0, 8) and dw.shape == (0, 2)
    assert moe.moe_permute_backward(e((0, 8), device="cuda"), e(0, **i32), 2).shape == (0, 8)
    assert moe.moe_act_checkpoint(e((0, 8), device="cuda"), moe.act_params())[0].shape == (0, 4)
    assert moe.moe_act_backward(e((0, 8), device="cuda"), e((0, 4), device="cuda"),
                                moe.act_params())[0].shape == (0, 8)
    assert moe.moe_route_backward(e((0, 8), device="cuda"), e((0, 2), **i32),
                                  e((0, 2), device="cuda"), moe.route_params(2)).shape == (0, 8)


def test_rows_past_32_bits(moe):
    """More than 2^32 bytes and 2^31 elements of rows."""
    T, K, H = 37500, 8, 7176
    M = T * K
    assert M * H > 2 ** 31
    d = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    d[0], d[T - 1] = 2.0, 3.0
    y = torch.ones((M, H), dtype=torch.bfloat16, device="cuda")
    w = torch.full((T, K), 0.5, device="cuda")
    r2r = torch.arange(M - 1, -1, -1, dtype=torch.int32, device="cuda")
    dy, dw = moe.moe_combine_backward(d, y, w, r2r)
    assert (dw[0] == 2 * H).all() and (dw[T - 1] == 3 * H).all() and (dw[1:-1] == 0).all()
    assert (dy[M - K:] == 1).all() and (dy[:K] == 1.5).all() and (dy[K:M - K] == 0).all()
    y[M - 1], y[0] = 5.0, 7.0
    out = moe.moe_permute_backward(y, r2r, K)
    assert (out[0] == 12).all() and (out[T - 1] == 14).all() and (out[1:-1] == 8).all()


# ------------------------------------------------------------------ activation
def act_params(moe, kind, inter):
    return moe.act_params(KINDS[kind], swiglu_fusion=1 if inter else 2,
                          limit=7.0 if kind == "swiglu" else 0.0, alpha=1.702, beta=1.0)


ACTS = [("silu", False), ("gelu", False), ("swiglu", False), ("swiglu", True), ("relu", False),
        ("gelu1", False), ("silu1", False), ("identity", False)]
REF = dict(limit=7.0, alpha=1.702, beta=1.0)


def argument(g, M, F, kind, dtype):
    """Rows with values past the clamps, at them, at zero and tiny."""
    N1 = 2 * F if kind in GATED else F
    p = torch.randn((M, N1), generator=g, device="cuda") * 3
    p[:, ::7] *= 4
    p.view(-1)[::11] = 7.0
    p.view(-1)[5::13] = -7.0
    p.view(-1)[3::17] = 0.0
    p.view(-1)[4::19] *= 1e-6
    return p.to(dtype)


ROWS = [(1, 1), (1, 8), (3, 20), (5, 33), (9, 32), (17, 96), (2, 2880), (40, 768), (3, 104), (300, 64)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind,inter", ACTS)
@pytest.mark.parametrize("M,F", ROWS)
def test_act_checkpoint(moe, M, F, kind, inter, dtype):
    p = argument(gen(M + F), M, F, kind, dtype)
    ap = act_params(moe, kind, inter)
    out, codes, scales = moe.moe_act_checkpoint(p, ap)
    rc, rs = mx_reference.quantize(p.double().cpu().numpy(), "e4m3")
    assert np.array_equal(scales.view(torch.uint8).cpu().numpy(), rs)
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), rc)
    a, slack, _, _ = R.act_backward(p, torch.zeros((M, F), device="cuda"), kind, inter,
                                    fast=dtype != torch.float32, **REF)
    R.close(out, a, slack, "out")
    again = moe.moe_act_checkpoint(p, ap, out=False)
    assert again[0] is None and torch.equal(again[1].view(torch.uint8), codes.view(torch.uint8))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind,inter", ACTS)
@pytest.mark.parametrize("M,F", ROWS)
def test_act_backward(moe, M, F, kind, inter, dtype):
    g = gen(M * F)
    p, d = argument(g, M, F, kind, dtype), randn(g, M, F, dtype=dtype)
    ap = act_params(moe, kind, inter)
    _, codes, scales = moe.moe_act_checkpoint(p, ap, out=False)
    saved = moe.moe_mx_dequantize(codes, scales, p.shape[1], dtype=torch.float32)
    fast = dtype != torch.float32
    for arg, sc, val in ((codes, scales, saved), (p, None, p)):
        dp, out = moe.moe_act_backward(arg, d, ap, scales=sc)
        a, s_a, r, s_r = R.act_backward(val, d, kind, inter, fast=fast, **REF)
        R.close(out, a, s_a, "out")
        R.close(dp, r, s_r, "d_p")
        dp2, none = moe.moe_act_backward(arg, d, ap, scales=sc, out=False)
        assert none is None and torch.equal(dp2, dp)


@pytest.mark.parametrize("kind,inter", ACTS)
def test_act_against_differences(moe, kind, inter):
    """The float64 definition's central differences, away from the clamps' edges."""
    g = gen(11)
    M, F = 6, 32
    p = torch.randn((M, 2 * F if kind in GATED else F), generator=g, device="cuda") * 2 + 0.01
    d = randn(g, M, F)
    dp, _ = moe.moe_act_backward(p, d, act_params(moe, kind, inter))
    h = 1e-5
    num = torch.empty(p.shape, dtype=torch.float64, device="cuda")
    for c in range(p.shape[1]):
        q = p.double()
        q[:, c] += h
        up = R.act_forward(q, kind, inter, **REF)
        q[:, c] -= 2 * h
        num[:, c] = ((up - R.act_forward(q, kind, inter, **REF)) * d.double()).sum(1) / (2 * h)
    # float32 arithmetic, and a central difference's h^2 / 6 of a third derivative below 100
    assert (dp.double() - num).abs().max() < 1e-4 * (1 + num.abs().max())


@pytest.mark.parametrize("kind,inter", ACTS)
@pytest.mark.parametrize("F", [31, 64])
@pytest.mark.parametrize("dtype", DTYPES)
def test_act_keeps_nan_in_its_block(moe, kind, inter, F, dtype):
    """A NaN or infinity makes its 32 columns NaN in the checkpoint, no others."""
    g = gen(5)
    p, d = randn(g, 4, 2 * F if kind in GATED else F, dtype=dtype), randn(g, 4, F, dtype=dtype)
    p[1, 3], p[2, 0] = float("nan"), float("-inf")
    ap = act_params(moe, kind, inter)
    out, codes, scales = moe.moe_act_checkpoint(p, ap)
    s = scales.view(torch.uint8)
    assert s[1, 0] == 255 and s[2, 0] == 255 and int((s == 255).sum()) == 2
    assert (codes.view(torch.uint8)[1:3, :32] == 0).all()
    hit = 1 if inter else 3
    want = torch.zeros((4, F), dtype=torch.bool, device="cuda")
    want[1, hit] = True
    if kind not in ("relu", "identity"):
        want[2, 0] = True  # -inf * 0
    assert torch.equal(torch.isnan(out), want)
    dp, act = moe.moe_act_backward(codes, d, ap, scales=scales)
    n = 16 if inter else min(32, F)
    want = torch.zeros((4, F), dtype=torch.bool, device="cuda")
    want[1:3, :n] = True
    if kind in GATED and not inter and F < 32:  # the block reaches into the up half
        want[1:3] |= torch.arange(F, device="cuda") < 32 - F
    assert torch.equal(torch.isnan(act), want)
    if kind != "identity":
        assert torch.isnan(dp[1:3, 0]).all()
    assert torch.isfinite(dp[0]).all() and torch.isfinite(dp[3]).all()


@pytest.mark.parametrize("kind,inter", ACTS)
@pytest.mark.parametrize("F", [31, 64])
@pytest.mark.parametrize("dtype", DTYPES)
def test_act_nan_of_the_argument(moe, kind, inter, F, dtype):
    """Without a checkpoint a NaN reaches what the formula takes it for: the activation always,
    the gradients of a gate or a single value but identity's, of a NaN up value the gate's alone
    and not past the gate's clamp."""
    g = gen(15)
    gated = kind in GATED
    p, d = randn(g, 4, 2 * F if gated else F, dtype=dtype), randn(g, 4, F, dtype=dtype)
    at, up = (2 * 5, 2 * 5 + 1) if inter else (5, F + 5)
    nan = float("nan")
    p[1, at] = nan
    if gated:
        p[2, up], p[3, up] = nan, nan
        p[3, at] = 9.0  # past SwiGLU's clamp of 7
    dp, out = moe.moe_act_backward(p, d, act_params(moe, kind, inter))
    want_out = torch.zeros((4, F), dtype=torch.bool, device="cuda")
    want = torch.zeros(p.shape, dtype=torch.bool, device="cuda")
    want_out[1, 5], want[1, at] = True, kind != "identity"
    if gated:
        want_out[2:, 5], want[1, up], want[2, at] = True, True, True
        want[3, at] = kind != "swiglu"
        if kind == "swiglu":
            assert dp[3, at] == 0
    assert torch.equal(torch.isnan(out), want_out)
    assert torch.equal(torch.isnan(dp), want)


@pytest.mark.parametrize("F", [20, 64])
@pytest.mark.parametrize("end,live", [(3, 3), (0, 0), (-4, 0), (99, 8)])
def test_act_rows_behind_the_last_segment(moe, F, end, live):
    g = gen(6)
    M = 8
    p, d = randn(g, M, 2 * F, dtype=torch.bfloat16), randn(g, M, F, dtype=torch.bfloat16)
    seg = torch.tensor([1, 2, end], dtype=torch.int32, device="cuda")
    ap = moe.act_params()
    Np = moe.moe_mx_columns(2 * F)
    out = torch.full((M, F), 9.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((M, Np), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((M, Np // 32), 78, dtype=torch.uint8, device="cuda")
    moe.moe_act_checkpoint(p, ap, seg_end=seg, out=out, codes=codes, scales=scales)
    ref = moe.moe_act_checkpoint(p, ap)
    assert (out[live:] == 9).all() and (codes[live:] == 77).all() and (scales[live:] == 78).all()
    assert torch.equal(out[:live], ref[0][:live])
    assert torch.equal(codes[:live], ref[1].view(torch.uint8)[:live])
    dp = torch.full((M, 2 * F), 9.0, dtype=torch.bfloat16, device="cuda")
    act = out.clone().fill_(9.0)
    moe.moe_act_backward(ref[1], d, ap, scales=ref[2], seg_end=seg, d_p=dp, out=act)
    rp, ra = moe.moe_act_backward(ref[1], d, ap, scales=ref[2])
    assert (dp[live:] == 9).all() and (act[live:] == 9).all()
    assert torch.equal(dp[:live], rp[:live]) and torch.equal(act[:live], ra[:live])


def test_act_unaligned(moe):
    g = gen(7)
    M, F = 5, 64
    ap = moe.act_params()
    for dt in DTYPES:
        p = randn(g, M * 2 * F + 1, dtype=dt)[1:].view(M, 2 * F)
        d = randn(g, M * F + 1, dtype=dt)[1:].view(M, F)
        got, ref = moe.moe_act_checkpoint(p, ap), moe.moe_act_checkpoint(p.clone(), ap)
        assert torch.equal(got[0], ref[0])
        assert torch.equal(got[1].view(torch.uint8), ref[1].view(torch.uint8))
        a = moe.moe_act_backward(got[1], d, ap, scales=got[2])
        b = moe.moe_act_backward(got[1], d.clone(), ap, scales=got[2])
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        a, b = moe.moe_act_backward(p, d, ap), moe.moe_act_backward(p.clone(), d.clone(), ap)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_act_past_32_bits(moe):
    """More than 2^32 bytes of argument."""
    M, F = 540000, 2048
    p = torch.full((M, 2 * F), 2.0, dtype=torch.bfloat16, device="cuda")
    p[M - 1] = 3.0
    ap = moe.act_params()
    out, codes, scales = moe.moe_act_checkpoint(p, ap)
    small = moe.moe_act_checkpoint(p[M - 2:], ap)
    del p
    assert (out[:M - 1] == small[0][0]).all() and (out[M - 1] == small[0][1]).all()
    assert (codes.view(torch.uint8)[:M - 1] == small[1].view(torch.uint8)[0]).all()
    assert torch.equal(codes.view(torch.uint8)[M - 1], small[1].view(torch.uint8)[1])
    dp, act = moe.moe_act_backward(codes, out, ap, scales=scales)
    a, b = moe.moe_act_backward(small[1], small[0], ap, scales=small[2])
    assert (dp[:M - 1] == a[0]).all() and torch.equal(dp[M - 1], a[1])
    assert (act[:M - 1] == b[0]).all() and torch.equal(act[M - 1], b[1])


# ------------------------------------------------------------------ grouped products
SEGS = [[1], [0, 1, 0], [3, 0, 5], [64], [16, 48, 0, 64], [17, 130, 1, 0, 63, 65], [300, 2],
        [0, 0, 700]]
WIDTHS = [(8, 8), (64, 64), (256, 128), (72, 200), (136, 520), (512, 768), (33, 50), (1, 1), (7, 264)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts", SEGS)
@pytest.mark.parametrize("N,K", WIDTHS)
def test_dgrad(moe, counts, N, K, dtype):
    g = gen(sum(counts) + N + K)
    M, E = sum(counts), len(counts)
    d, w = randn(g, M, N, dtype=dtype), randn(g, E, N, K, dtype=dtype, std=0.1)
    ws = torch.zeros(moe.MOE_STATUS_BYTES, dtype=torch.uint8, device="cuda")
    out = moe.moe_grouped_gemm_dgrad(d, w, segments(counts), ws=ws)
    ref, slack = R.dgrad(d, w, segments(counts))
    R.close(out, ref, slack, "d_a")
    assert moe.moe_sync_status(ws) == moe.MOE_OK
    assert torch.equal(out, moe.moe_grouped_gemm_dgrad(d, w, segments(counts), ws=ws))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts", SEGS)
@pytest.mark.parametrize("N,K", WIDTHS)
def test_wgrad(moe, counts, N, K, dtype):
    g = gen(sum(counts) * N + K)
    M, E = sum(counts), len(counts)
    d, a = randn(g, M, N, dtype=dtype, std=0.1), randn(g, M, K, dtype=dtype)
    ws = torch.zeros(moe.moe_grouped_gemm_wgrad_workspace_size(M, N, K, E), dtype=torch.uint8,
                     device="cuda")
    dw = torch.full((E, N, K), float("nan"), dtype=dtype, device="cuda")
    db = torch.full((E, N), float("nan"), dtype=dtype, device="cuda")
    moe.moe_grouped_gemm_wgrad(d, a, segments(counts), bias=db, d_w=dw, ws=ws)
    rw, sw, rb, sb = R.wgrad(d, a, segments(counts))
    R.close(dw, rw, sw, "d_w")
    R.close(db, rb, sb, "d_bias")
    assert moe.moe_sync_status(ws) == moe.MOE_OK
    again, none = moe.moe_grouped_gemm_wgrad(d, a, segments(counts), ws=ws)
    assert none is None and torch.equal(again, dw)


@pytest.mark.parametrize("dtype", DTYPES[:2])
@pytest.mark.parametrize("counts", [[1], [16, 48, 0, 64], [300, 2], [0, 7] * 20])
@pytest.mark.parametrize("N,K", [(1032, 8), (1032, 520), (2056, 1032)])
def test_dgrad_long_sums(moe, counts, N, K, dtype):
    g = gen(sum(counts) + N + K)
    M, E = sum(counts), len(counts)
    d, w = randn(g, M, N, dtype=dtype), randn(g, E, N, K, dtype=dtype, std=0.03)
    ref, slack = R.dgrad(d, w, segments(counts))
    R.close(moe.moe_grouped_gemm_dgrad(d, w, segments(counts)), ref, slack, "d_a")


@pytest.mark.parametrize("dtype", DTYPES[:2])
@pytest.mark.parametrize("counts", [[33, 0, 5] * 14, [0] * 500 + [3, 0, 64] * 8 + [0] * 500,
                                    [1] * 1024, [130] * 40])
@pytest.mark.parametrize("N,K", [(520, 776), (264, 136)])
def test_wgrad_many_tiles(moe, counts, N, K, dtype):
    """Several tiles a CTA, up to 1024 experts, most of them empty or none: the same workspace
    twice, the second time with its counters as the first left them."""
    g = gen(len(counts) + N)
    M, E = sum(counts), len(counts)
    d, a = randn(g, M, N, dtype=dtype, std=0.1), randn(g, M, K, dtype=dtype)
    ws = torch.zeros(moe.moe_grouped_gemm_wgrad_workspace_size(M, N, K, E), dtype=torch.uint8,
                     device="cuda")
    rw, sw, rb, sb = R.wgrad(d, a, segments(counts))
    for _ in range(2):
        dw, db = moe.moe_grouped_gemm_wgrad(d, a, segments(counts), bias=True, ws=ws)
        R.close(dw, rw, sw, "d_w")
        R.close(db, rb, sb, "d_bias")
    assert moe.moe_sync_status(ws) == moe.MOE_OK and (ws[:256] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES[:2])
@pytest.mark.parametrize("counts", [[2600], [7000, 0, 901], [5000, 3], [0, 1, 9000, 0],
                                    [4097, 2047]])
@pytest.mark.parametrize("N,K", [(8, 8), (72, 200), (256, 264), (264, 136), (520, 40)])
def test_wgrad_in_parts(moe, counts, N, K, dtype):
    """Few tiles and many rows: the rows in parts, added up in order.  Experts without rows, with
    fewer than a part, and with NaN next door; every element written."""
    g = gen(sum(counts) + N * K)
    M, E = sum(counts) + 5, len(counts)
    seg = segments(counts)
    need = moe.moe_grouped_gemm_wgrad_workspace_size(M, N, K, E)
    assert need > moe.MOE_STATUS_BYTES
    d, a = randn(g, M, N, dtype=dtype, std=0.1), randn(g, M, K, dtype=dtype)
    d[M - 5:], a[M - 5:] = float("nan"), float("inf")
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    ws[moe.MOE_STATUS_BYTES:] = 255  # partial sums that no part writes are NaN
    dw = torch.full((E, N, K), float("nan"), dtype=dtype, device="cuda")
    db = torch.full((E, N), float("nan"), dtype=dtype, device="cuda")
    moe.moe_grouped_gemm_wgrad(d, a, seg, bias=db, d_w=dw, ws=ws)
    rw, sw, rb, sb = R.wgrad(d, a, seg)
    R.close(dw, rw, sw, "d_w")
    R.close(db, rb, sb, "d_bias")
    assert moe.moe_sync_status(ws) == moe.MOE_OK and (ws[:moe.MOE_STATUS_BYTES] == 0).all()
    assert torch.equal(moe.moe_grouped_gemm_wgrad(d, a, seg, ws=ws)[0], dw)
    with pytest.raises(moe.MoEError):
        moe.moe_grouped_gemm_wgrad(d, a, seg, ws=ws[:need - 256])


def test_wgrad_of_one_among_many(moe):
    """All of more than 2^26 rows on one of 100 experts: cut by the rows themselves, where the
    average would not be.  Whole numbers whose sums float32 holds: exact but for the rounding."""
    M, N, K, E = (1 << 26) + 12345, 8, 8, 100
    g = gen(23)
    d, a = (torch.randint(-1, 2, (M, N), generator=g, device="cuda", dtype=torch.int8
                          ).to(torch.bfloat16) for _ in range(2))
    counts = [0] * E
    counts[41], counts[77] = M - 3, 3
    dw, _ = moe.moe_grouped_gemm_wgrad(d, a, segments(counts))
    ref = torch.zeros((E, N, K), dtype=torch.float64, device="cuda")
    for lo in range(0, M - 3, 1 << 22):
        x, y = (t[lo:min(lo + (1 << 22), M - 3)].float() for t in (d, a))
        ref[41] += (x.t() @ y).double()  # partial sums below 2^22: exact
    ref[77] = d[-3:].double().t() @ a[-3:].double()
    assert ref.abs().max() < 2 ** 24
    assert torch.equal(dw, ref.to(torch.bfloat16))


@pytest.mark.parametrize("dtype,N,K,off", [(torch.float32, 40, 64, 0), (torch.float32, 7, 33, 0),
                                           (torch.bfloat16, 42, 64, 0), (torch.float16, 40, 64, 1)])
def test_wgrad_in_the_status_bytes(moe, dtype, N, K, off):
    """Sums in float32 FMA over an expert of many rows take a workspace of the status alone."""
    g = gen(17)
    M, seg = 5000, segments([5000])
    d = randn(g, M * N + off, dtype=dtype)[off:].view(M, N)
    a = randn(g, M, K, dtype=dtype)
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    ws[moe.MOE_STATUS_BYTES:] = 77
    dw, db = moe.moe_grouped_gemm_wgrad(d, a, seg, bias=True, ws=ws[:moe.MOE_STATUS_BYTES])
    rw, sw, rb, sb = R.wgrad(d, a, seg)
    R.close(dw, rw, sw)
    R.close(db, rb, sb)
    assert (ws[moe.MOE_STATUS_BYTES:] == 77).all()
    with pytest.raises(moe.MoEError):
        moe.moe_grouped_gemm_wgrad(randn(g, M, 40, dtype=torch.bfloat16),
                                   randn(g, M, 64, dtype=torch.bfloat16), seg,
                                   ws=ws[:moe.MOE_STATUS_BYTES])


def test_wgrad_on_two_streams(moe):
    """Calls that run at the same time, with workspaces of their own."""
    g = gen(20)
    counts = [200, 0, 77, 300, 1]
    M, N, K = sum(counts), 1024, 768
    seg = segments(counts)
    sets = [(randn(g, M, N, dtype=torch.bfloat16, std=0.1), randn(g, M, K, dtype=torch.bfloat16),
             torch.zeros(4096, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    want = [moe.moe_grouped_gemm_wgrad(d, a, seg, bias=True, ws=ws) for d, a, ws in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (d, a, ws) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i].append(moe.moe_grouped_gemm_wgrad(d, a, seg, bias=True, ws=ws))
    torch.cuda.synchronize()
    for i in range(2):
        for dw, db in got[i]:
            assert torch.equal(dw, want[i][0]) and torch.equal(db, want[i][1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", [(1, 8), (5000, 40), (70000, 72), (333, 33)])
def test_bias_of_long_columns(moe, M, N, dtype):
    """Column sums over many rows, also into a bias that starts between 16-byte lines."""
    g = gen(M)
    d, a = randn(g, M, N, dtype=dtype), randn(g, M, 8, dtype=dtype)
    seg = segments([M - M // 3, 0, M // 3])
    _, _, rb, sb = R.wgrad(d, a, seg)
    # a chain of at most M / 8 + 64 additions and a tree: the bound's M terms hold
    R.close(moe.moe_grouped_gemm_wgrad(d, a, seg, bias=True)[1], rb, sb)
    odd = torch.empty(3 * N + 1, dtype=dtype, device="cuda")[1:].view(3, N)
    moe.moe_grouped_gemm_wgrad(d, a, seg, bias=odd)
    R.close(odd, rb, sb)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,K", [(64, 64), (264, 328), (45, 30)])
def test_products_keep_to_their_rows(moe, N, K, dtype):
    """NaN in a neighbour's rows, and behind the last segment, does not get in; rows behind it are
    left as they were."""
    g = gen(N)
    counts, M = [5, 37, 0, 81], 150  # 123 live rows
    seg = segments(counts)
    d, a = randn(g, M, N, dtype=dtype, std=0.1), randn(g, M, K, dtype=dtype)
    w = randn(g, 4, N, K, dtype=dtype, std=0.1)
    nan = float("nan")
    d[5:42], a[5:42] = nan, nan
    d[123:], a[123:] = nan, float("inf")
    dw, db = moe.moe_grouped_gemm_wgrad(d, a, seg, bias=True)
    assert torch.isnan(dw[1]).all() and torch.isnan(db[1]).all()
    rw, sw, rb, sb = R.wgrad(d, a, seg)
    for e in (0, 2, 3):
        R.close(dw[e], rw[e], sw[e], "d_w")
        R.close(db[e], rb[e], sb[e], "d_bias")
    da = torch.full((M, K), 3.0, dtype=dtype, device="cuda")
    moe.moe_grouped_gemm_dgrad(d, w, seg, d_a=da)
    assert (da[123:] == 3).all() and torch.isnan(da[5:42]).all()
    ref, slack = R.dgrad(d, w, seg)
    for lo, hi in ((0, 5), (42, 123)):
        R.close(da[lo:hi], ref[lo:hi], slack[lo:hi], "d_a")


@pytest.mark.parametrize("dtype", DTYPES)
def test_products_without_rows(moe, dtype):
    """Zero weight gradients where no row is; segment ends out of order or of range stay inside."""
    g = gen(1)
    N, K = 64, 72
    e = lambda *s: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    dw = torch.full((3, N, K), 5.0, dtype=dtype, device="cuda")
    _, db = moe.moe_grouped_gemm_wgrad(e(0, N), e(0, K), segments([0, 0, 0]), bias=True, d_w=dw)
    assert (dw == 0).all() and (db == 0).all()
    assert moe.moe_grouped_gemm_dgrad(e(0, N), e(3, N, K), segments([0, 0, 0])).shape == (0, K)
    d, a, w = randn(g, 20, N, dtype=dtype), randn(g, 20, K, dtype=dtype), randn(g, 4, N, K,
                                                                               dtype=dtype)
    seg = torch.tensor([-3, 8, 4, 99], dtype=torch.int32, device="cuda")
    dw, db = moe.moe_grouped_gemm_wgrad(d, a, seg, bias=True)
    rw, sw, rb, sb = R.wgrad(d, a, seg)
    R.close(dw, rw, sw)
    R.close(db, rb, sb)
    moe.moe_grouped_gemm_dgrad(d, w, seg)  # overlapping segments: any of the two, inside the buffer
    torch.cuda.synchronize()


def test_products_unaligned(moe):
    """16-bit tensors that do not start on 16 bytes take the other kernel."""
    g = gen(4)
    N = K = 64
    seg = segments([9, 0, 31])
    for dt in (torch.bfloat16, torch.float16):
        d = randn(g, 40 * N + 1, dtype=dt)[1:].view(40, N)
        a, w = randn(g, 40, K, dtype=dt), randn(g, 3, N, K, dtype=dt)
        ref, slack = R.dgrad(d, w, seg)
        R.close(moe.moe_grouped_gemm_dgrad(d, w, seg), ref, slack)
        rw, sw, _, _ = R.wgrad(d, a, seg)
        R.close(moe.moe_grouped_gemm_wgrad(d, a, seg)[0], rw, sw)


# ------------------------------------------------------------------ router
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (3, 8, 2), (65, 128, 8), (9, 37, 5), (5, 1000, 64),
                                   (700, 256, 8)])
def test_route_backward(moe, T, E, K, scoring, renorm, dtype):
    g = gen(T + E + K)
    z = randn(g, T, E, dtype=dtype, std=2.0)
    p = moe.route_params(K, scoring, renorm, routed_scaling_factor=2.5)
    ids = moe.moe_route(z, p)[1]
    dw = randn(g, T, K)
    out = moe.moe_route_backward(z, ids, dw, p)
    ref, slack = R.route_backward(z, ids, dw, scoring, renorm, 2.5)
    R.close(out, ref, slack, "d_logits")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_given_ids(moe, scoring, renorm):
    """Hash routing: the same id twice adds up, an id out of range takes no part."""
    g = gen(8)
    T, E, K = 40, 24, 6
    z = randn(g, T, E)
    ids = torch.randint(0, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    ids[0] = 5
    ids[1, 2], ids[2, 0], ids[3] = -1, E, torch.tensor([7, 7, 9, 2 ** 31 - 1, -2 ** 31, 7])
    dw = randn(g, T, K)
    dw[1, 2] = float("nan")  # the gradient of a route that is none
    p = moe.route_params(K, scoring, renorm)
    out = moe.moe_route_backward(z, ids, dw, p)
    dw[1, 2] = 0
    ref, slack = R.route_backward(z, ids, dw, scoring, renorm, 1.0)
    R.close(out, ref, slack)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_masked_and_far_logits(moe, scoring, renorm):
    """Experts masked with -inf or the type's lowest value, logits far out: no NaN, zeros for the
    masked."""
    g = gen(9)
    T, E, K = 16, 16, 4
    z = randn(g, T, E)
    z[:, 3], z[:, 7] = float("-inf"), torch.finfo(torch.float32).min
    z[:, 0], z[:, 1] = 60.0, -70.0
    ids = torch.tensor([[0, 1, 3, 7]], dtype=torch.int32, device="cuda").repeat(T, 1)
    ids[8:] = torch.tensor([0, 3, 4, 5], dtype=torch.int32)
    dw = randn(g, T, K)
    out = moe.moe_route_backward(z, ids, dw, moe.route_params(K, scoring, renorm))
    assert torch.isfinite(out).all() and (out[:, [3, 7]] == 0).all()
    zr = z.clamp(min=-700)  # float64 has exp(-700)
    ref, slack = R.route_backward(zr, ids, dw, scoring, renorm, 1.0)
    R.close(out, ref, slack + 1e-40)
    # a NaN logit stays in its token
    z[2, 0] = float("nan")
    out2 = moe.moe_route_backward(z, ids, dw, moe.route_params(K, scoring, renorm))
    assert torch.isnan(out2[2, 0]) and torch.equal(out2[3:], out[3:]) and torch.equal(out2[:2], out[:2])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid", "sqrt_softplus"])
def test_route_backward_far_choices(moe, scoring, dtype):
    """Every chosen logit so low that its float32 score is zero: the weights' ratios remain.
    Chosen experts masked with -inf weigh nothing, and a choice of these alone has no gradient."""
    g = gen(13)
    E, K, low, inf = 16, 4, torch.finfo(dtype).min, float("-inf")
    rows = [(-100, -100, -100, -100), (-100, -120, -95, -110), (low,) * 4, (low, low, inf, inf),
            (inf,) * 4, (inf, -96, inf, inf)]
    T = len(rows)
    z = randn(g, T, E, dtype=dtype)
    z[:, :K] = torch.tensor(rows, device="cuda")
    ids = torch.arange(K, dtype=torch.int32, device="cuda").repeat(T, 1)
    dw = randn(g, T, K)
    p = moe.route_params(K, scoring, True, routed_scaling_factor=2.5)
    out = moe.moe_route_backward(z, ids, dw, p)
    ref, slack = R.route_backward(z[:2], ids[:2], dw[:2], scoring, True, 2.5)
    R.close(out[:2], ref, slack, "far")
    # equal scores: weights of 1/4 and 1/2, exact; dlog score / dz is 1, of sqrt_softplus 1/2
    l = 0.5 if scoring == "sqrt_softplus" else 1.0
    for t, n in ((2, 4), (3, 2)):
        h = dw[t, :n].double()
        want = torch.zeros(E, dtype=torch.float64, device="cuda")
        want[:n] = 2.5 / n * l * (h - h.mean())
        mag = torch.zeros_like(want)
        mag[:n] = 2.5 / n * l * (h.abs() + h.abs().mean())
        # three additions of the sum, the difference and three products, of R.U each
        R.close(out[t], want, 8 * R.U * mag, ("lowest", n))
    assert (out[4:] == 0).all()
    # a NaN among the masks is kept
    z[4, 1] = float("nan")
    assert torch.isnan(moe.moe_route_backward(z, ids, dw, p)[4, :K]).all()


@pytest.mark.parametrize("z", [0.5, -30.0, -100.0, -1e30, float("-inf")])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid", "sqrt_softplus"])
def test_route_backward_single_weight(moe, scoring, z):
    """One renormalised weight is 1 whatever its logit."""
    logits = torch.full((3, 8), z, device="cuda")
    ids = torch.tensor([[0], [7], [3]], dtype=torch.int32, device="cuda")
    out = moe.moe_route_backward(logits, ids, torch.full((3, 1), 1.7, device="cuda"),
                                 moe.route_params(1, scoring, True))
    assert (out == 0).all()


@pytest.mark.parametrize("E", [5, 200, 600, 1000])
@pytest.mark.parametrize("dtype", DTYPES)
def test_route_backward_softmax_without_a_logit(moe, E, dtype):
    """Softmax weights as they are: a row whose mask leaves no expert has a zero gradient, its
    neighbours theirs; a NaN makes its row NaN."""
    g = gen(E)
    K = 3
    z, dw = randn(g, 4, E, dtype=dtype), randn(g, 4, K)
    ids = torch.arange(K, dtype=torch.int32, device="cuda").repeat(4, 1)
    p = moe.route_params(K, "softmax", False)
    ref = moe.moe_route_backward(z, ids, dw, p)
    z[1], z[2] = float("-inf"), float("-inf")
    z[2, E - 1] = float("nan")
    out = moe.moe_route_backward(z, ids, dw, p)
    assert (out[1] == 0).all() and torch.isnan(out[2]).all()
    assert torch.equal(out[::3], ref[::3])


def test_route_against_differences(moe):
    g = gen(10)
    T, E, K = 4, 9, 3
    for scoring in ("softmax", "sigmoid", "sqrt_softplus"):
        for renorm in (True, False):
            z, dw = randn(g, T, E), randn(g, T, K)
            p = moe.route_params(K, scoring, renorm)
            ids = moe.moe_route(z, p)[1]
            out = moe.moe_route_backward(z, ids, dw, p)
            num = torch.empty((T, E), dtype=torch.float64, device="cuda")
            for i in range(E):
                q = z.double()
                q[:, i] += 1e-5
                up = R.route_weights(q, ids, scoring, renorm, 1.0)
                q[:, i] -= 2e-5
                num[:, i] = ((up - R.route_weights(q, ids, scoring, renorm, 1.0)) *
                             dw.double()).sum(1) / 2e-5
            # float32 arithmetic, and h^2 / 6 of a third derivative below 10
            assert (out.double() - num).abs().max() < 1e-5


# ------------------------------------------------------------------ together
def layer(moe, T, H, F, E, K, dtype, kind="swiglu", inter=True, seed=0, drop=False):
    g = gen(seed)
    s = dict(x=randn(g, T, H, dtype=dtype), logits=randn(g, T, E), d_out=randn(g, T, H, dtype=dtype),
             w1=randn(g, E, 2 * F, H, dtype=dtype, std=H ** -0.5),
             w2=randn(g, E, H, F, dtype=dtype, std=F ** -0.5),
             b1=randn(g, E, 2 * F, dtype=dtype, std=0.1), b2=randn(g, E, H, dtype=dtype, std=0.1),
             route=moe.route_params(K, "softmax", True, routed_scaling_factor=1.5),
             act=act_params(moe, kind, inter), kind=kind, inter=inter)
    return s


def train_step(moe, s, ws=None):
    """Forward and backward as a training program runs them."""
    E, N1, H = s["w1"].shape
    F = s["w2"].shape[2]
    T, K = s["x"].shape[0], s["route"].top_k
    ws1, ws2, ws3 = ws or (None, None, None)
    tw, ti, _, _, maps = moe.moe_route_permute(s["logits"], s["route"], ws=ws1)
    seg, rows = maps["seg_end"], maps["route_to_row"]
    x = moe.moe_permute_gather(s["x"], seg, maps["row_to_route"], K, ws=ws2)
    p = moe.moe_grouped_gemm(x, s["w1"], moe.MOE_LAYOUT_PSUM, seg, N1, bias=s["b1"], ws=ws2)
    a, codes, scales = moe.moe_act_checkpoint(p, s["act"], seg_end=seg)
    y = moe.moe_grouped_gemm_down(a, s["w2"], seg, s["b2"], ws=ws2)
    out = moe.moe_combine(y, tw, rows)
    del p, a
    d_y, d_tw = moe.moe_combine_backward(s["d_out"], y, tw, rows)
    d_a = moe.moe_grouped_gemm_dgrad(d_y, s["w2"], seg, ws=ws2)
    d_p, a = moe.moe_act_backward(codes, d_a, s["act"], scales=scales, seg_end=seg)
    d_w2, d_b2 = moe.moe_grouped_gemm_wgrad(d_y, a, seg, bias=True, ws=ws3)
    d_w1, d_b1 = moe.moe_grouped_gemm_wgrad(d_p, x, seg, bias=True, ws=ws3)
    d_x = moe.moe_grouped_gemm_dgrad(d_p, s["w1"], seg, ws=ws2)
    d_hidden = moe.moe_permute_backward(d_x, rows, K)
    d_logits = moe.moe_route_backward(s["logits"], ti, d_tw, s["route"])
    return dict(out=out, d_hidden=d_hidden, d_logits=d_logits, d_w1=d_w1, d_w2=d_w2, d_b1=d_b1,
                d_b2=d_b2), dict(ids=ti, codes=codes, scales=scales, maps=maps)


class Checkpointed(torch.autograd.Function):
    """act(p) forward; backward with the checkpoint's p, and act of it for what follows."""

    @staticmethod
    def forward(ctx, p, saved, s):
        ctx.save_for_backward(saved)
        ctx.s = s
        return R.act_forward(p, s["kind"], s["inter"], **REF)

    @staticmethod
    def backward(ctx, d):
        return R.act_backward(ctx.saved_tensors[0], d, ctx.s["kind"], ctx.s["inter"], **REF)[2], \
            None, None


class Down(torch.autograd.Function):
    """a w^T, the weights' gradient from the recomputed activation."""

    @staticmethod
    def forward(ctx, a, w, again):
        ctx.save_for_backward(w, again)
        return a @ w.t()

    @staticmethod
    def backward(ctx, d):
        w, again = ctx.saved_tensors
        return d @ w, d.t() @ again, None


def reference_step(moe, s, kept):
    leaf = {k: s[k].double().requires_grad_() for k in ("x", "logits", "w1", "w2", "b1", "b2")}
    T, H = s["x"].shape
    E, N1, _ = s["w1"].shape
    K = s["route"].top_k
    ids = kept["ids"]
    w = R.route_weights(leaf["logits"], ids, "softmax", True, 1.5)
    saved = moe.moe_mx_dequantize(kept["codes"], kept["scales"], N1, dtype=torch.float32).double()
    rows = kept["maps"]["route_to_row"].view(T, K)
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for k in range(K):
        for e in range(E):
            t = (ids[:, k] == e).nonzero().flatten()
            if not t.numel():
                continue
            p = leaf["x"][t] @ leaf["w1"][e].t() + leaf["b1"][e]
            ph = saved[rows[t, k].long()]
            a = Checkpointed.apply(p, ph, s)
            again = R.act_forward(ph, s["kind"], s["inter"], **REF)
            y = Down.apply(a, leaf["w2"][e], again) + leaf["b2"][e]
            out = out.index_add(0, t, y * w[t, k:k + 1])
    names = ("x", "logits", "w1", "w2", "b1", "b2")
    grads = torch.autograd.grad(out, [leaf[n] for n in names], s["d_out"].double())
    keys = ("d_hidden", "d_logits", "d_w1", "d_w2", "d_b1", "d_b2")
    return dict(zip(keys, grads), out=out.detach())


@pytest.mark.parametrize("T,H,F,E,K,kind,inter",
                         [(33, 64, 96, 6, 2, "swiglu", True), (50, 72, 40, 8, 3, "silu", False),
                          (7, 30, 21, 4, 1, "gelu", False)])
def test_training_step(moe, T, H, F, E, K, kind, inter):
    """The whole step in float32 against float64 differentiation of the layer: every gradient
    within 1e-4 of its norm (sums of at most 200 terms through eight stages, 1600 u)."""
    s = layer(moe, T, H, F, E, K, torch.float32, kind, inter, seed=T)
    got, kept = train_step(moe, s)
    ref = reference_step(moe, s, kept)
    if K == 1:  # a single renormalised weight is 1: no gradient, and float64's is its rounding
        assert (got["d_logits"] == 0).all() and ref.pop("d_logits").abs().max() < 1e-14
    for k, r in ref.items():
        err = (got[k].double() - r).norm() / r.norm()
        assert err < 1e-4, (k, float(err))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_training_step_16_bits(moe, dtype):
    """On the tensor cores: six roundings of 16-bit intermediates in a row (p, a, y or d_y, d_a,
    d_p, d_x and the result), each half a step, and as much again for what they carry along."""
    s = layer(moe, 300, 256, 192, 8, 2, dtype, seed=3)
    got, kept = train_step(moe, s)
    ref = reference_step(moe, s, kept)
    for k, r in ref.items():
        err = (got[k].double() - r).norm() / r.norm()
        assert err < 14 * torch.finfo(dtype).eps / 2, (k, float(err))


def test_training_step_in_a_graph(moe):
    """Captured once and replayed on new values, next to the same step on another stream with
    workspaces of its own: bit for bit the plain calls'."""
    dt = torch.bfloat16
    a, b = (layer(moe, 100, 128, 64, 8, 2, dt, seed=i) for i in (1, 2))
    want = [train_step(moe, s)[0] for s in (a, b)]

    def spaces():
        M, E = 200, 8
        n = max(moe.moe_permute_workspace_size(M, E),
                moe.moe_grouped_gemm_wgrad_workspace_size(M, 256, 256, E))
        return [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(3)]

    live = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in a.items()}
    ws, other_ws = spaces(), spaces()
    train_step(moe, live, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = train_step(moe, live, ws)[0]
    side = torch.cuda.Stream()
    for s, ref in ((b, want[1]), (a, want[0])):
        for k, v in s.items():
            if isinstance(v, torch.Tensor):
                live[k].copy_(v)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            beside = train_step(moe, b, other_ws)[0]
        torch.cuda.synchronize()
        for k, r in ref.items():
            assert torch.equal(got[k], r), k
        for k, r in want[1].items():
            assert torch.equal(beside[k], r), k


def test_training_step_without_some_routes(moe):
    """Routes that have no row (an id that is no expert): their weights have no gradient, the
    others' are as without them."""
    g = gen(12)
    T, H, F, E, K = 20, 64, 32, 4, 2
    ids = torch.randint(0, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    ids[::3, 1] = -1
    ids[4] = E
    maps = moe.moe_permute(ids, E)
    seg, rows = maps["seg_end"], maps["route_to_row"]
    live = int(seg[-1])
    assert live < T * K
    tw = torch.rand((T, K), generator=g, device="cuda")
    d, y = randn(g, T, H), torch.full((T * K, H), float("nan"), device="cuda")
    y[:live] = randn(g, live, H)
    dy, dw = moe.moe_combine_backward(d, y, tw, rows)
    none = (ids < 0) | (ids >= E)
    assert (dw[none] == 0).all() and torch.isfinite(dw).all()
    p = randn(g, T * K, 2 * F)
    p[live:] = float("nan")
    w2 = randn(g, E, H, F)
    d_a = moe.moe_grouped_gemm_dgrad(dy, w2, seg)
    d_p, a = moe.moe_act_backward(p, d_a, moe.act_params(), seg_end=seg)
    d_w2, d_b2 = moe.moe_grouped_gemm_wgrad(dy, a, seg, bias=True)
    assert torch.isfinite(d_w2).all() and torch.isfinite(d_b2).all()
    assert torch.isfinite(d_p[:live]).all()
    assert torch.isfinite(moe.moe_permute_backward(y, rows, K)).all()
