"""Host-only checks of the microscaled operators: refusals before any launch
(placeholder addresses that are never dereferenced, so only where no GPU is
visible), workspace sizes, and pins of the float64 reference."""
import ctypes

import numpy as np
import pytest
import torch

import mx_reference as R

nogpu = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: CPU only")
A = lambda i, off=0: ctypes.c_void_p(0x7F0000000000 + i * (1 << 36) + off)  # noqa: E731


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_ffn_gb300 import build, moe as m

    build.build()
    m.load_library()
    return m


# ------------------------------------------------------------------ reference pins
def test_reference_codes_are_torch_casts():
    """Inside one block of scale 1, e4m3 codes are torch's float8 cast."""
    x = np.random.RandomState(0).randn(64, 31) * 60
    x = np.concatenate([np.full((64, 1), 448.0), x], 1)
    x = np.clip(x, -448, 448).astype(np.float32)
    codes, scales = R.quantize(x.astype(np.float64), "e4m3")
    assert (scales[:, 0] == 127).all()
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes[:, :32], ref)


def test_reference_e2m1_by_hand():
    x = np.zeros((1, 32))
    x[0, :12] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5.1, -0.3, 7.9, -0.0]
    codes, scales = R.quantize(x, "e2m1")
    assert scales[0, 0] == 127  # floor(log2 7.9) - 2 = 0
    assert R.values(codes, scales, "e2m1")[0, :12].tolist() == \
        [6, 0, 1, 1, 2, 2, 4, 4, -6, -0.5, 6, 0]
    assert np.array_equal(R.unpack(R.pack(codes)), codes)


@pytest.mark.parametrize("amax,fmt,e", [(448.0, "e4m3", 0), (448.5, "e4m3", 1), (449.0, "e4m3", 1),
                                        (511.0, "e4m3", 1), (512.0, "e4m3", 1), (896.0, "e4m3", 1),
                                        (1.0, "e4m3", -8), (6.0, "e2m1", 0), (7.99, "e2m1", 0),
                                        (8.0, "e2m1", 1), (0.0, "e2m1", -127), (1e-45, "e4m3", -127)])
def test_reference_scales(amax, fmt, e):
    assert R.scale_exponents(np.array([amax]), fmt)[0] == e


# ------------------------------------------------------------------ refusals
@nogpu
def test_quantize_refuses(moe):
    lib = moe.load_library()

    def q(x=A(0), rows=4, K=64, stride=64, dt=moe.MOE_BF16, fmt=0, codes=A(1), scales=A(2)):
        return lib.moe_mx_quantize(x, rows, K, stride, dt, fmt, codes, scales, None)

    inv, uns, ovl = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_OVERLAP
    for kw in (dict(rows=-1), dict(K=0), dict(stride=63), dict(dt=7), dict(fmt=2), dict(fmt=-1),
               dict(x=None), dict(codes=None), dict(scales=None), dict(x=A(0, 1)),
               dict(rows=1 << 31), dict(rows=1 << 28, K=128, stride=128)):
        assert q(**kw) == inv, kw
    assert q(codes=A(1, 8)) == uns and q(scales=A(2, 4)) == uns
    assert q(codes=A(0, 64)) == ovl and q(scales=A(1)) == ovl
    assert q(rows=0, x=None, codes=None, scales=None) == moe.MOE_OK

    def d(codes=A(1), scales=A(2), rows=4, K=64, fmt=1, dt=moe.MOE_F16, out=A(0)):
        return lib.moe_mx_dequantize(codes, scales, rows, K, fmt, dt, out, None)

    for kw in (dict(rows=-1), dict(K=0), dict(fmt=5), dict(dt=-1), dict(codes=None), dict(out=None),
               dict(scales=None), dict(out=A(0, 1))):
        assert d(**kw) == inv, kw
    assert d(codes=A(1, 4)) == uns and d(out=A(2)) == ovl and d(rows=0, out=None) == moe.MOE_OK


@nogpu
def test_norm_refuses(moe):
    lib = moe.load_library()

    def n(x=A(0), r=A(1), w=A(2), T=4, H=64, dt=moe.MOE_BF16, eps=1e-6, q=1, ro=A(3), out=A(4),
          codes=A(5), scales=A(6)):
        return lib.moe_add_rms_norm(x, r, w, T, H, dt, eps, q, ro, out, codes, scales, None)

    inv, uns, ovl = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_OVERLAP
    for kw in (dict(T=-1), dict(H=0), dict(H=65537), dict(dt=3), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(q=3), dict(q=-1), dict(x=None),
               dict(w=None), dict(ro=None), dict(r=None), dict(codes=None), dict(scales=None),
               dict(q=0), dict(x=A(0, 1)), dict(out=A(4, 1))):
        assert n(**kw) == inv, kw
    assert n(codes=A(5, 4)) == uns and n(scales=A(6, 8)) == uns
    assert n(ro=A(0)) == ovl and n(out=A(0, 64)) == ovl and n(out=A(3)) == ovl
    assert n(ro=A(1, 2)) == ovl and n(codes=A(2)) == ovl
    assert n(T=0, x=None, r=None, w=None, ro=None, out=None, codes=None, scales=None) == moe.MOE_OK


@nogpu
def test_gemm_mx_refuses(moe):
    lib = moe.load_library()
    act = moe.act_params(moe.MOE_ACT_SWIGLU, swiglu_fusion=1)

    def g(a=A(0), asc=A(1), rows=64, r2r=None, k=1, w=A(2), wsc=A(3), bias=None, seg=A(4), M=64,
          N=128, K=256, E=8, dt=moe.MOE_BF16, act=None, out=A(5), osc=None, ws=A(6),
          wsb=moe.moe_grouped_gemm_mx_workspace_size(64, 128, 256, 8)):
        return lib.moe_grouped_gemm_mx(a, asc, rows, r2r, k, w, wsc, bias, seg, M, N, K, E, dt,
                                       None if act is None else ctypes.byref(act), out, osc, ws,
                                       wsb, None)

    inv, uns, ovl = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_OVERLAP
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(E=0), dict(E=1025), dict(dt=9), dict(rows=63),
               dict(rows=-1), dict(r2r=A(7), k=0), dict(w=None), dict(wsc=None), dict(seg=None),
               dict(out=None), dict(a=None), dict(asc=None), dict(M=1 << 30, rows=1 << 30),
               dict(act=moe.act_params(9)), dict(act=moe.act_params(1, swiglu_fusion=0))):
        assert g(**kw) == inv, kw
    for kw in (dict(dt=moe.MOE_F32, out=A(5, 2)), dict(bias=A(7, 1)), dict(a=A(0, 8)), dict(asc=A(1, 4)), dict(w=A(2, 16)),
               dict(wsc=A(3, 8)), dict(out=A(5, 1)), dict(out=A(5, 8), osc=A(7)),
               dict(osc=A(7, 8))):
        assert g(**kw) == uns, kw
    assert g(ws=None) == moe.MOE_ERR_WORKSPACE and g(wsb=255) == moe.MOE_ERR_WORKSPACE
    assert g(ws=A(6, 128)) == moe.MOE_ERR_WORKSPACE
    for kw in (dict(out=A(0)), dict(out=A(2, 64)), dict(out=A(4)), dict(osc=A(5)), dict(out=A(6)),
               dict(act=act, out=A(3))):
        assert g(**kw) == ovl, kw
    assert g(M=0, rows=0, a=None, asc=None, out=None) == moe.MOE_OK


@nogpu
def test_layer_mx_refuses(moe):
    lib = moe.load_library()
    need = moe.moe_workspace_size_mx(16, 256, 128, 8, 2)

    def f(h=A(0), hs=A(1), lg=A(2), w1=A(3), s1=A(4), w2=A(5), s2=A(6), cb=None, ids=None, b1=None,
          b2=None, T=16, H=256, F=128, E=8, dt=moe.MOE_BF16, p=moe.route_params(2),
          act=moe.act_params(), out=A(7), tw=None, ti=None, ws=A(8), wsb=need):
        return lib.moe_ffn_forward_mx(h, hs, lg, w1, s1, w2, s2, cb, ids, b1, b2, T, H, F, E, dt,
                                      ctypes.byref(p), ctypes.byref(act), out, tw, ti, ws, wsb, None)

    inv, uns, ovl = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_OVERLAP
    for kw in (dict(T=-1), dict(H=0), dict(F=0), dict(E=0), dict(E=1025), dict(dt=4), dict(h=None),
               dict(hs=None), dict(lg=None), dict(w1=None), dict(s1=None), dict(w2=None),
               dict(s2=None), dict(out=None), dict(p=moe.route_params(9)), dict(cb=A(9)),
               dict(act=moe.act_params(1, swiglu_fusion=0)),
               dict(p=moe.route_params(2, local_expert_count=4))):
        assert f(**kw) == inv, kw
    for kw in (dict(dt=moe.MOE_F32, out=A(7, 2)), dict(b1=A(9, 1)), dict(h=A(0, 4)), dict(hs=A(1, 8)), dict(w1=A(3, 16)),
               dict(w2=A(5, 16)), dict(s1=A(4, 4)), dict(s2=A(6, 8)), dict(out=A(7, 1))):
        assert f(**kw) == uns, kw
    assert f(wsb=need - 1) == moe.MOE_ERR_WORKSPACE and f(ws=None) == moe.MOE_ERR_WORKSPACE
    for kw in (dict(out=A(0)), dict(out=A(8)), dict(ws=A(3)), dict(ti=A(2)), dict(tw=A(7))):
        assert f(**kw) == ovl, kw
    assert f(T=0, h=None, hs=None, out=None) == moe.MOE_OK


def test_workspace_sizes(moe):
    a = moe.moe_workspace_size_mx(2048, 2880, 2880, 128, 4)
    M, Fp = 2048 * 4, 2944
    assert a >= M * (Fp + Fp // 32 + 2880 * 4) and a % 256 == 0
    assert moe.moe_workspace_size_mx(-1, 1, 1, 1, 1) == 0
    assert moe.moe_workspace_size_mx(1 << 29, 8, 8, 8, 2) == 0
    assert moe.moe_grouped_gemm_mx_workspace_size(64, 64, 64, 8) >= 256
    assert moe.moe_grouped_gemm_mx_workspace_size(64, 0, 64, 8) == 0
    assert moe.moe_mx_columns(2880) == 2944 and moe.moe_mx_columns(1) == 128


def test_binding_refuses_host_tensors_and_mismatched_extents(moe):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        moe.moe_mx_quantize(x)
    with pytest.raises(ValueError):
        moe.moe_add_rms_norm(x, torch.zeros(64))
    with pytest.raises(ValueError):
        moe.moe_mx_dequantize(x.to(torch.uint8), x.to(torch.uint8), 64)
