"""Edges of the microscaled operators on the GPU: NaN through the clamped and
rectified activations."""
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
