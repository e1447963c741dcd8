"""Edges of the microscaled operators on the GPU: NaN through the clamped and
rectified activations, infinite weights and mean squares of zero in the norm."""
import pytest
import torch

from test_gpu_mx import ACTS, DTYPES, GATED, gen, layer_inputs, mx_weights, raw, rows_of, segments

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_ffn_gb300 import build, moe as m

    build.build()
    return m


# ------------------------------------------------------------------ NaN through the activations
@pytest.mark.parametrize("act,inter", [("swiglu", True), ("swiglu", False), ("relu", False),
                                       ("silu_and_mul", False), ("gelu_and_mul", False),
                                       ("gelu", False), ("silu", False), ("identity", False)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mx_out", [False, True])
@pytest.mark.parametrize("counts", [[3, 0, 4], [30, 40, 0, 5]])
def test_product_keeps_nan(moe, counts, mx_out, dtype, act, inter):
    """A row with a non-finite block has a NaN scale, every product with it is NaN, and so is every
    activation of a NaN, the clamped and the rectified ones among them."""
    g = gen(len(counts))
    M, N, K, E = sum(counts), 96, 192, len(counts)
    x = rows_of(g, M, K, torch.float32) * 0.01
    bad = [0, M - 2]
    x[bad[0], 7], x[bad[1], K - 1] = float("nan"), float("-inf")
    a = moe.moe_mx_quantize(x)
    w = mx_weights(moe, g, E, 2 * N if act in GATED else N, K)
    ap = moe.act_params(ACTS[act], swiglu_fusion=1 if inter else 2, limit=7.0, alpha=1.702, beta=1.0)
    out = moe.moe_grouped_gemm_mx(*a, *w, segments(counts), N, act=ap, dtype=dtype, mx_out=mx_out)
    good = [i for i in range(M) if i not in bad]
    if mx_out:
        s = out[1].float()[:, :N // 32]
        assert torch.isnan(s[bad]).all() and torch.isfinite(s[good]).all()
        assert (raw(out[0])[bad] == 0).all()
    else:
        assert torch.isnan(out[bad]).all() and torch.isfinite(out[good]).all()


def test_product_keeps_nan_of_the_up_half_and_of_the_bias(moe):
    """Gate and up are clamped apart: a NaN in either is a NaN."""
    g = gen(1)
    N, K = 64, 128
    a = moe.moe_mx_quantize(rows_of(g, 5, K, torch.float32) * 0.01)
    w = mx_weights(moe, g, 1, 2 * N, K)
    ap = moe.act_params(moe.MOE_ACT_SWIGLU, swiglu_fusion=1, limit=7.0, alpha=1.702, beta=1.0)
    b = torch.zeros((1, 2 * N), device="cuda")
    b[0, 2 * 3], b[0, 2 * 9 + 1] = float("nan"), float("nan")
    out = moe.moe_grouped_gemm_mx(*a, *w, segments([5]), N, act=ap, bias=b, dtype=torch.float32)
    hit = torch.zeros(N, dtype=torch.bool, device="cuda")
    hit[[3, 9]] = True
    assert torch.isnan(out[:, hit]).all() and torch.isfinite(out[:, ~hit]).all()


def test_layer_keeps_nan(moe):
    """A token with a NaN in its hidden row is NaN in the whole output row, every other finite."""
    T, H, F, E, k = 21, 256, 128, 8, 2
    hidden, logits, w1, w2, b1, b2 = layer_inputs(moe, T, H, F, E, k, "swiglu", torch.bfloat16)
    x = torch.randn((T, H), generator=gen(7), device="cuda")
    x[4, 100] = float("nan")
    out = moe.moe_ffn_forward_mx(*moe.moe_mx_quantize(x), logits, *w1, *w2, H, F,
                                 moe.route_params(k),
                                 moe.act_params(1, swiglu_fusion=1, limit=7.0, alpha=1.702, beta=1.0),
                                 b_gate_up=b1, b_down=b2)
    assert torch.isnan(out[4]).all()
    assert torch.isfinite(out[[i for i in range(T) if i != 4]]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts", [[3, 0, 4], [60, 75, 0, 5], [600]])
def test_unscaled_products_and_swiglu_keep_nan(moe, counts, dtype):
    """The same activations behind the bf16, f16 and f32 grouped products and on their own."""
    g = gen(2)
    M, F, K, E = sum(counts), 64, 128, len(counts)
    x = torch.randn((M, K), generator=g, device="cuda").to(dtype)
    x[1, 5] = float("nan")
    good = [i for i in range(M) if i != 1]
    seg = segments(counts)
    for act, inter in (("swiglu", 1), ("swiglu", 2), ("relu", 0)):
        n1 = 2 * F if act == "swiglu" else F
        w = (torch.randn((E, n1, K), generator=g, device="cuda") * K ** -0.5).to(dtype)
        ap = moe.act_params(ACTS[act], swiglu_fusion=inter or 2, limit=7.0, alpha=1.702, beta=1.0)
        out = moe.moe_grouped_gemm_act(x, w, seg, F, ap)
        assert torch.isnan(out[1]).all() and torch.isfinite(out[good]).all(), (act, inter)
    both = torch.randn((8, 2 * F), generator=g, device="cuda").to(dtype)
    both[2, 3], both[4, F + 5] = float("nan"), float("nan")
    out = moe.swiglu(both[:, :F].contiguous(), both[:, F:].contiguous(), 2, 7.0, 1.702, 1.0)
    want = torch.zeros((8, F), dtype=torch.bool, device="cuda")
    want[2, 3], want[4, 5] = True, True
    assert torch.equal(torch.isnan(out), want)


# ------------------------------------------------------------------ norm: infinities
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H", [(5, 320), (400, 64), (3, 2880)])
def test_norm_infinite_weight_gives_infinities(moe, T, H, dtype):
    """h * root * inf is an infinity of h's sign (NaN where h is zero); a NaN weight gives NaN; the
    other columns are as without."""
    g = gen(T + H)
    x = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    x[0, 40] = 0
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(dtype)
    plain = moe.moe_add_rms_norm(x, w)["out"]
    w2 = w.clone()
    w2[40], w2[41], w2[H - 1] = float("inf"), float("nan"), float("-inf")
    y = moe.moe_add_rms_norm(x, w2)["out"]
    assert torch.isnan(y[0, 40]) and torch.isnan(y[:, 41]).all()
    assert torch.equal(y[1:, 40], torch.sign(x[1:, 40]) * float("inf"))
    assert torch.equal(y[:, H - 1], torch.sign(x[:, H - 1]) * float("-inf"))
    rest = torch.ones(H, dtype=torch.bool, device="cuda")
    rest[[40, 41, H - 1]] = False
    assert torch.equal(y[:, rest], plain[:, rest])


def test_norm_of_a_mean_square_of_zero(moe):
    """In float32 squares below 2^-149 are zero: without eps the root is infinite, and h times it an
    infinity of h's sign, NaN where h is zero."""
    x = torch.zeros((4, 256), device="cuda")
    x[0], x[1, ::2], x[2, 5] = 1e-30, -1e-30, 1.0
    w = torch.ones(256, device="cuda")
    y = moe.moe_add_rms_norm(x, w, eps=0.0)["out"]
    assert (y[0] == float("inf")).all()
    assert (y[1, ::2] == float("-inf")).all() and torch.isnan(y[1, 1::2]).all()
    assert y[2, 5] == 16.0 and (y[2, 6:] == 0).all()
    assert torch.isnan(y[3]).all()
    # with eps the rows are finite
    assert torch.isfinite(moe.moe_add_rms_norm(x, w, eps=1e-6)["out"]).all()


def test_norm_of_rows_whose_squares_overflow(moe):
    """A mean square past float32 is infinite, its root zero: zeros of h's sign, NaN for an infinite
    h."""
    x = torch.full((2, 160), 1e30, device="cuda")
    x[1, 3] = float("inf")
    y = moe.moe_add_rms_norm(x, torch.ones(160, device="cuda"))["out"]
    assert (y[0] == 0).all() and torch.isnan(y[1, 3]) and (y[1, 4:] == 0).all()
