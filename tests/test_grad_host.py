"""Refusals of the gradient entry points on the CPU: the C ABI's before any launch
(placeholder addresses that are never dereferenced, so only where no GPU is visible) and
the Python binding's, in front of a library that records what it is called with."""
import ctypes

import pytest
import torch

nogpu = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: CPU only")
A = lambda i, off=0: ctypes.c_void_p(0x7F0000000000 + i * (1 << 36) + off)  # noqa: E731
BF, F32 = 1, 0
OK, BAD, OVERLAP, UNSUP, _, _, _, SPACE = range(8)


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_ffn_gb300 import build, moe as m

    build.build()
    return m.load_library()


# ------------------------------------------------------------------ the C ABI
@nogpu
def test_combine_backward_refuses(lib):
    def call(d=A(0), y=A(1), w=A(2), r=A(3), T=4, K=2, H=64, dt=BF, dy=A(4), dw=A(5)):
        return lib.moe_combine_backward(d, y, w, r, T, K, H, dt, 1.0, dy, dw, None)

    assert call(T=0) == OK
    for kw in (dict(T=-1), dict(K=0), dict(H=0), dict(dt=3), dict(T=1 << 30, K=4), dict(d=None),
               dict(r=None), dict(y=None), dict(w=None), dict(dy=None, dw=None), dict(d=A(0, 1)),
               dict(y=A(1, 1)), dict(dy=A(4, 1)), dict(d=A(0, 2), dt=F32)):
        assert call(**kw) == BAD, kw
    for kw in (dict(dy=A(0)), dict(dy=A(1, 64)), dict(dw=A(4, 64)), dict(dw=A(2)), dict(dy=A(3))):
        assert call(**kw) == OVERLAP, kw


@nogpu
def test_permute_backward_refuses(lib):
    def call(x=A(0), r=A(1), T=4, K=2, H=64, dt=BF, h=A(2)):
        return lib.moe_permute_backward(x, r, T, K, H, dt, h, None)

    assert call(T=0) == OK
    for kw in (dict(T=-1), dict(K=0), dict(H=0), dict(dt=-1), dict(x=None), dict(r=None),
               dict(h=None), dict(T=1 << 30, K=2), dict(x=A(0, 1)), dict(h=A(2, 1))):
        assert call(**kw) == BAD, kw
    assert call(h=A(0, 512)) == OVERLAP and call(h=A(1)) == OVERLAP


@nogpu
def test_activation_refuses(lib):
    from mixture_experts_ffn_gb300 import moe

    def ckpt(p=A(0), seg=A(1), M=4, F=64, E=2, dt=BF, act=moe.act_params(), out=A(2), c=A(3),
             s=A(4)):
        return lib.moe_act_checkpoint(p, seg, M, F, E, dt, ctypes.byref(act) if act else None, out,
                                      c, s, None)

    def back(p=A(0), s=A(4), d=A(5), seg=A(1), M=4, F=64, E=2, dt=BF, act=moe.act_params(),
             dp=A(6), out=A(2)):
        return lib.moe_act_backward(p, s, d, seg, M, F, E, dt, ctypes.byref(act) if act else None,
                                    dp, out, None)

    split = moe.act_params(moe.MOE_ACT_SWIGLU, swiglu_fusion=0)
    assert ckpt(M=0) == OK and back(M=0) == OK
    both = (dict(M=-1), dict(F=0), dict(F=(1 << 23) + 1), dict(E=0), dict(dt=7), dict(act=None),
            dict(act=split), dict(act=moe.act_params(9)), dict(p=None),
            dict(M=1 << 24, F=1024), dict(out=A(2, 1)))
    for kw in both:
        assert ckpt(**kw) == BAD, kw
        assert back(**kw) == BAD, kw
    for kw in (dict(c=None), dict(s=None), dict(p=A(0, 1))):
        assert ckpt(**kw) == BAD, kw
    for kw in (dict(d=None), dict(dp=None), dict(d=A(5, 1)), dict(dp=A(6, 1)),
               dict(s=None, p=A(0, 1))):
        assert back(**kw) == BAD, kw
    assert ckpt(c=A(3, 8)) == UNSUP and ckpt(s=A(4, 4)) == UNSUP
    assert back(p=A(0, 8)) == UNSUP and back(s=A(4, 4)) == UNSUP
    for kw in (dict(out=A(0)), dict(c=A(0, 16)), dict(s=A(3)), dict(out=A(1))):
        assert ckpt(**kw) == OVERLAP, kw
    for kw in (dict(dp=A(0)), dict(dp=A(5)), dict(out=A(6)), dict(dp=A(4)), dict(out=A(1))):
        assert back(**kw) == OVERLAP, kw


@nogpu
def test_products_refuse(lib):
    def dg(d=A(0), w=A(1), seg=A(2), M=8, N=64, K=32, E=2, dt=BF, da=A(3), ws=A(4), n=256):
        return lib.moe_grouped_gemm_dgrad(d, w, seg, M, N, K, E, dt, da, ws, n, None)

    def wg(d=A(0), a=A(1), seg=A(2), M=8, N=64, K=32, E=2, dt=BF, dw=A(3), db=A(5), ws=A(4),
           n=1 << 20):
        return lib.moe_grouped_gemm_wgrad(d, a, seg, M, N, K, E, dt, dw, db, ws, n, None)

    assert dg(M=0) == OK
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(E=0), dict(E=1025), dict(dt=5), dict(d=None),
               dict(seg=None), dict(d=A(0, 1)), dict(M=1 << 30)):
        assert dg(**kw) == BAD, kw
        assert wg(**kw) == BAD, kw
    for kw in (dict(w=None), dict(da=None), dict(w=A(1, 1)), dict(da=A(3, 1))):
        assert dg(**kw) == BAD, kw
    for kw in (dict(a=None), dict(dw=None), dict(dw=None, M=0), dict(a=A(1, 1)), dict(dw=A(3, 1)),
               dict(db=A(5, 1))):
        assert wg(**kw) == BAD, kw
    for f in (dg, wg):
        for kw in (dict(ws=None), dict(ws=A(4, 8)), dict(n=64)):
            assert f(**kw) == SPACE, kw
    for kw in (dict(da=A(0)), dict(da=A(1, 64)), dict(da=A(2)), dict(ws=A(0))):
        assert dg(**kw) == OVERLAP, kw
    for kw in (dict(dw=A(0)), dict(dw=A(1, 64)), dict(db=A(3, 64)), dict(ws=A(0)), dict(db=A(2))):
        assert wg(**kw) == OVERLAP, kw
    assert lib.moe_grouped_gemm_wgrad_workspace_size(8, 64, 32, 2) >= 256
    assert lib.moe_grouped_gemm_wgrad_workspace_size(-1, 64, 32, 2) == 0


@nogpu
def test_route_backward_refuses(lib):
    from mixture_experts_ffn_gb300 import moe

    def call(z=A(0), ids=A(1), dw=A(2), T=4, E=16, p=moe.route_params(2), dz=A(3)):
        return lib.moe_route_backward(z, ids, dw, T, E, ctypes.byref(p) if p else None, dz, None)

    assert call(T=0) == OK
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(p=None), dict(p=moe.route_params(0)),
               dict(p=moe.route_params(17)), dict(p=moe.route_params(2, 7)), dict(z=None),
               dict(ids=None), dict(dw=None), dict(dz=None), dict(z=A(0, 1)), dict(dz=A(3, 2)),
               dict(p=moe.route_params(2, local_expert_count=4)),
               dict(p=moe.route_params(2, routed_scaling_factor=-1.0))):
        assert call(**kw) == BAD, kw
    for kw in (dict(dz=A(0)), dict(dz=A(1)), dict(dz=A(2))):
        assert call(**kw) == OVERLAP, kw


@nogpu
def test_wgrad_takes_the_space_it_uses(lib):
    """One expert of many rows: the tensor-core kernel sums in parts and needs room for these,
    the float32 FMA one (float32, other widths, unaligned operands) the status alone."""
    M, N, K = 16384, 512, 512
    size = lib.moe_grouped_gemm_wgrad_workspace_size
    need = size(M, N, K, 1)
    assert need > 256 and size(M, N + 1, K, 1) == 256 and size(M, N, K - 4, 1) == 256

    def call(d=A(0), a=A(1), N=N, K=K, dt=BF, n=256, dw=A(3)):  # dw == ws: never launched
        return lib.moe_grouped_gemm_wgrad(d, a, A(2), M, N, K, 1, dt, dw, None, A(3), n, None)

    assert call() == SPACE and call(n=need - 1) == SPACE and call(n=need) == OVERLAP
    for kw in (dict(dt=F32), dict(N=N + 1), dict(K=K - 4), dict(d=A(0, 2)), dict(a=A(1, 8)),
               dict(dw=A(3, 2))):
        assert call(**kw) == OVERLAP, kw
        assert call(**kw, n=255) == SPACE, kw


@nogpu
def test_wgrad_cuts_rows_without_end(lib):
    """An expert may have all of the rows, however many experts there are: past 2^26 rows there
    are parts, one for each 2^26, so that no tile takes as long as the kernel waits for it."""
    def parts(m, n=8, k=8, e=1024):
        return (lib.moe_grouped_gemm_wgrad_workspace_size(m, n, k, e) - 256) // (4 * e * n * k)

    assert parts(1 << 26) == 0
    assert parts((1 << 26) + 1) == 2 and parts(1 << 28) == 4 and parts((1 << 30) - 1) == 16
    assert parts((1 << 30) - 1, e=1) > 16


# ------------------------------------------------------------------ the binding
class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append(name)
            return 4096 if "workspace_size" in name else 0

        return entry


@pytest.fixture
def moe(monkeypatch):
    from mixture_experts_ffn_gb300 import moe as m

    def as_if_on_the_gpu(t):
        if t.is_meta:
            raise ValueError("libmoe takes CUDA tensors only")

    rec = Recorder()
    monkeypatch.setattr(m, "load_library", lambda: rec)
    monkeypatch.setattr(m, "_on_gpu", as_if_on_the_gpu)
    monkeypatch.setattr(m, "_is_current", lambda device: True)
    monkeypatch.setattr(m, "_stream_of", lambda t: 0)
    m.recorder = rec
    yield m
    del m.recorder


T, K, H, E, F, N = 6, 2, 32, 4, 48, 40
M = T * K
z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
f32 = lambda *s: torch.zeros(s)  # noqa: E731
u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731


def calls(moe):
    """Every entry point's right call: (function, arguments, outputs that may be given)."""
    act, rp = moe.act_params(), moe.route_params(K)
    return {
        "combine": (moe.moe_combine_backward,
                    dict(d_out=z(T, H), expert_out=z(M, H), topk_weights=f32(T, K),
                         route_to_row=i32(M)),
                    dict(d_expert_out=z(M, H), d_topk_weights=f32(T, K))),
        "permute": (moe.moe_permute_backward,
                    dict(d_expert_input=z(M, H), route_to_row=i32(M), K=K), dict(d_hidden=z(T, H))),
        "checkpoint": (moe.moe_act_checkpoint, dict(p=z(M, 2 * F), act=act, seg_end=i32(E)),
                       dict(out=z(M, F), codes=u8(M, 128), scales=u8(M, 4))),
        "act": (moe.moe_act_backward,
                dict(p=u8(M, 128), d_out=z(M, F), act=act, scales=u8(M, 4), seg_end=i32(E)),
                dict(d_p=z(M, 2 * F), out=z(M, F))),
        "act_plain": (moe.moe_act_backward, dict(p=z(M, 2 * F), d_out=z(M, F), act=act),
                      dict(d_p=z(M, 2 * F), out=z(M, F))),
        "dgrad": (moe.moe_grouped_gemm_dgrad, dict(d_out=z(M, N), w=z(E, N, H), seg_end=i32(E)),
                  dict(d_a=z(M, H), ws=u8(256))),
        "wgrad": (moe.moe_grouped_gemm_wgrad, dict(d_out=z(M, N), a=z(M, H), seg_end=i32(E)),
                  dict(d_w=z(E, N, H), bias=z(E, N), ws=u8(4096))),
        "route": (moe.moe_route_backward,
                  dict(logits=f32(T, E), topk_ids=i32(T, K), d_topk_weights=f32(T, K), p=rp),
                  dict(d_logits=f32(T, E))),
    }


NAMES = ["combine", "permute", "checkpoint", "act", "act_plain", "dgrad", "wgrad", "route"]


def refused(moe, f, kw, why):
    before = [c for c in moe.recorder.calls if "workspace" not in c]
    with pytest.raises((TypeError, ValueError)):
        f(**kw)
    assert [c for c in moe.recorder.calls if "workspace" not in c] == before, why


@pytest.mark.parametrize("name", NAMES)
def test_right_calls_pass(moe, name):
    f, kw, outs = calls(moe)[name]
    f(**kw)
    f(**kw, **outs)
    assert len([c for c in moe.recorder.calls if "workspace" not in c]) == 2


@pytest.mark.parametrize("name", NAMES)
def test_binding_refuses_every_wrong_tensor(moe, name):
    """Each tensor in turn: another type, another shape, not contiguous, not on the GPU."""
    f, kw, outs = calls(moe)[name]
    every = {**kw, **outs}
    for k, t in every.items():
        if not isinstance(t, torch.Tensor) or k == "ws":
            continue
        refused(moe, f, {**every, k: t.to(torch.float64)}, (k, "type"))
        other = torch.zeros((*t.shape[:-1], t.shape[-1] + 3), dtype=t.dtype)
        if not (k == "seg_end" and name in ("checkpoint", "act")):  # there any number of experts
            refused(moe, f, {**every, k: other}, (k, "shape"))
        refused(moe, f, {**every, k: torch.zeros((*t.shape[:-1], 2 * t.shape[-1]),
                                                 dtype=t.dtype)[..., ::2]}, (k, "strides"))
        refused(moe, f, {**every, k: t.to("meta")}, (k, "device"))


@pytest.mark.parametrize("name", NAMES)
def test_binding_refuses_another_device(moe, name, monkeypatch):
    f, kw, _ = calls(moe)[name]
    monkeypatch.setattr(moe, "_is_current", lambda device: False)
    refused(moe, f, kw, "current device")


@pytest.mark.parametrize("none", [False, None])
def test_outputs_left_out(moe, none):
    """False and None leave an output out; the weights' gradient left out takes no expert_out."""
    c = calls(moe)
    f, kw, _ = c["combine"]
    d_y, d_w = f(**{**kw, "expert_out": None}, d_topk_weights=none)
    assert d_w is None and d_y.shape == (M, H)
    d_y, d_w = f(**kw, d_expert_out=none)
    assert d_y is None and d_w.shape == (T, K)
    f, kw, _ = c["checkpoint"]
    assert f(**kw, out=none)[0] is None
    f, kw, _ = c["act"]
    assert f(**kw, out=none)[1] is None
    f, kw, _ = c["wgrad"]
    assert f(**kw, bias=none)[1] is None


def test_binding_asks_for_parts_where_they_are_used(moe):
    f, kw, _ = calls(moe)["wgrad"]
    f(**{**kw, "d_out": f32(M, N), "a": f32(M, H)})
    assert moe.recorder.calls == ["moe_grouped_gemm_wgrad"]
    f(**kw)
    assert moe.recorder.calls[1:] == ["moe_grouped_gemm_wgrad_workspace_size",
                                      "moe_grouped_gemm_wgrad"]


def test_binding_refuses_other_mistakes(moe):
    c = calls(moe)
    f, kw, _ = c["combine"]
    refused(moe, f, {**kw, "expert_out": None}, "no expert_out")
    f(**{**kw, "expert_out": None}, d_topk_weights=False)
    f, kw, _ = c["permute"]
    refused(moe, f, {**kw, "K": 5}, "K")
    refused(moe, f, {**kw, "K": 0}, "K")
    refused(moe, f, {**kw, "d_hidden": False}, "no output")
    f, kw, _ = c["checkpoint"]
    refused(moe, f, {**kw, "p": z(M, 2 * F + 1)}, "odd gated width")
    refused(moe, f, {**kw, "seg_end": i32(0)}, "no experts")
    f, kw, _ = c["act"]
    refused(moe, f, {**kw, "d_p": False}, "no output")
    refused(moe, f, {**kw, "scales": None}, "codes without scales")
    for name in ("dgrad", "wgrad", "route"):
        f, kw, outs = c[name]
        refused(moe, f, {**kw, next(iter(outs)): False}, "no output")
