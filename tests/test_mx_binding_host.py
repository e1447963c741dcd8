"""The Python binding's checks of the microscaled operators, on the CPU: the
library behind the binding is a stand-in that records the calls it gets, so a
call that must be refused is seen to get no further, and no kernel runs."""
import os
import subprocess
import sys

import pytest
import torch


class Recorder:
    """Stands in for libmoe.so: every entry point returns MOE_OK, a workspace
    size 4096."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, args))
            return 4096 if "workspace_size" in name else 0

        return entry

    def launched(self):
        return [n for n, _ in self.calls if "workspace_size" not in n]


@pytest.fixture
def moe(monkeypatch):
    from mixture_experts_ffn_gb300 import moe as m

    def as_if_on_the_gpu(t):  # the binding's check of the device: a meta tensor fails it
        if t.is_meta:
            raise ValueError("libmoe takes CUDA tensors only")

    rec = Recorder()
    monkeypatch.setattr(m, "load_library", lambda: rec)
    monkeypatch.setattr(m, "_on_gpu", as_if_on_the_gpu)
    monkeypatch.setattr(m, "_stream_of", lambda t: 0)
    m.recorder = rec
    yield m
    del m.recorder


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


E, N, K, M = 2, 64, 384, 8


def product(moe, **kw):
    """A product's call with every argument right but those in kw."""
    args = dict(a=u8(M, K), a_scale=u8(M, K // 32), w=u8(E, N, K // 2), w_scale=u8(E, N, K // 32),
                seg_end=torch.tensor([3, M], dtype=torch.int32), N=N)
    args.update(kw)
    return moe.moe_grouped_gemm_mx(**args)


def refused(moe, call, error=(TypeError, ValueError)):
    before = len(moe.recorder.launched())
    with pytest.raises(error):
        call()
    assert len(moe.recorder.launched()) == before, "the library was called"


def test_the_right_calls_pass(moe):
    for dt in (torch.bfloat16, torch.float16, torch.float32):
        assert product(moe, dtype=dt).dtype == dt
        product(moe, dtype=dt, mx_out=True, bias=torch.zeros((E, N), dtype=dt))
    assert moe.recorder.launched() == ["moe_grouped_gemm_mx"] * 6


@pytest.mark.parametrize("mx_out", [False, True])
@pytest.mark.parametrize("dtype", [torch.uint8, torch.float8_e4m3fn, torch.int16, torch.int32,
                                   torch.float64, torch.complex64])
def test_product_refuses_output_types_it_does_not_write(moe, dtype, mx_out):
    """The kernel writes bf16, f16 or f32 (4 bytes); a buffer of another type holds less, or other
    numbers."""
    refused(moe, lambda: product(moe, dtype=dtype, mx_out=mx_out), TypeError)
    refused(moe, lambda: product(moe, dtype=dtype, out=torch.zeros((M, N), dtype=dtype)), TypeError)


def test_product_refuses_an_output_scale_without_mx_output(moe):
    """The C entry takes a scale buffer as the request for MX rows: it would write [M, Np] codes into
    the [M, N] output (128 bytes a row where N = 1 in bf16 has 2) and scales past a short buffer."""
    for osc in (u8(1), u8(M, 4)):
        refused(moe, lambda: product(moe, out_scale=osc), ValueError)
    product(moe, mx_out=True, out=u8(M, 128), out_scale=u8(M, 4))


T, H = 4, 256


def norm(moe, dtype=torch.bfloat16, residual=False, **kw):
    x = torch.zeros((T, H), dtype=dtype)
    return moe.moe_add_rms_norm(x, torch.ones(H, dtype=dtype),
                                residual=torch.zeros_like(x) if residual else None, **kw)


def test_outputs_of_another_type_of_the_same_size_are_refused(moe):
    """The kernels write the type the call asks for: the bits of one 16-bit type read as another are
    other numbers."""
    h16, i16 = torch.zeros((M, N), dtype=torch.float16), torch.zeros((M, N), dtype=torch.int16)
    i32 = torch.zeros((M, N), dtype=torch.int32)
    product(moe, dtype=torch.float16, out=h16)
    refused(moe, lambda: product(moe, out=h16))
    refused(moe, lambda: product(moe, out=i16))
    refused(moe, lambda: product(moe, dtype=torch.float32, out=i32))
    for dt, other in ((torch.bfloat16, torch.float16), (torch.float16, torch.bfloat16),
                      (torch.float32, torch.int32)):
        right, wrong = torch.zeros((T, H), dtype=dt), torch.zeros((T, H), dtype=other)
        norm(moe, dt, out=right)
        refused(moe, lambda: norm(moe, dt, out=wrong))
        norm(moe, dt, residual=True, residual_out=right)
        refused(moe, lambda: norm(moe, dt, residual=True, residual_out=wrong))
    refused(moe, lambda: norm(moe, quant=moe.MOE_QUANT_E4M3_BLOCK128,
                              scales=torch.zeros((T, H // 128), dtype=torch.int32)))


TOPK, F = 2, 96


def layer(moe, **kw):
    """The layer's call with every argument right but those in kw."""
    fp = moe.moe_mx_columns(F)
    args = dict(hidden=u8(T, H), hidden_scale=u8(T, H // 32), logits=torch.zeros((T, E)),
                w_gate_up=u8(E, 2 * F, H // 2), w_gate_up_scale=u8(E, 2 * F, H // 32),
                w_down=u8(E, H, fp // 2), w_down_scale=u8(E, H, fp // 32), H=H, F=F,
                p=moe.route_params(TOPK), act=moe.act_params())
    args.update(kw)
    return moe.moe_ffn_forward_mx(**args)


def every_other(*shape, dtype=torch.float32):
    """A view of this shape of every other element."""
    return torch.zeros((*shape[:-1], 2 * shape[-1]), dtype=dtype)[..., ::2]


def elsewhere(*shape, dtype=torch.float32):
    """A tensor whose memory the GPU must not be handed (on the CPU: a meta tensor)."""
    return torch.zeros(shape, dtype=dtype, device="meta")


def test_every_buffer_the_library_writes_is_checked(moe):
    """Workspaces and the routing outputs too: a strided view's elements lie apart, and a host
    tensor's address is none of the GPU's."""
    i32 = torch.int32
    layer(moe, ws=u8(4096), topk_weights_out=torch.zeros((T, TOPK)),
          topk_ids_out=torch.zeros((T, TOPK), dtype=i32))
    for make in (every_other, elsewhere):
        refused(moe, lambda: layer(moe, topk_weights_out=make(T, TOPK)))
        refused(moe, lambda: layer(moe, topk_ids_out=make(T, TOPK, dtype=i32)))
        refused(moe, lambda: layer(moe, ws=make(4096, dtype=torch.uint8)))
        refused(moe, lambda: layer(moe, out=make(T, H, dtype=torch.bfloat16)))
        refused(moe, lambda: product(moe, ws=make(4096, dtype=torch.uint8)))
        refused(moe, lambda: product(moe, out=make(M, N, dtype=torch.bfloat16)))
        refused(moe, lambda: norm(moe, out=make(T, H, dtype=torch.bfloat16)))


def test_layer_refuses_routing_tensors_of_another_type(moe):
    f, i = torch.zeros((T, TOPK)), torch.zeros((T, TOPK), dtype=torch.int32)
    layer(moe, expert_ids=i, topk_weights_out=f, topk_ids_out=i, correction_bias=torch.zeros(E))
    refused(moe, lambda: layer(moe, expert_ids=f), TypeError)
    refused(moe, lambda: layer(moe, topk_weights_out=i), TypeError)
    refused(moe, lambda: layer(moe, topk_ids_out=f), TypeError)
    refused(moe, lambda: layer(moe, correction_bias=torch.zeros(E, dtype=torch.int32)), TypeError)


def test_tensors_of_the_right_count_and_the_wrong_shape_are_refused(moe):
    """Axes exchanged, the elements are the right number in the wrong order."""
    i32 = torch.int32
    fp = moe.moe_mx_columns(F)
    for kw in (dict(a_scale=u8(K // 32, M)), dict(w_scale=u8(E, K // 32, N)),
               dict(w_scale=u8(N, E, K // 32)), dict(bias=torch.zeros((N, E), dtype=torch.bfloat16)),
               dict(out=torch.zeros((N, M), dtype=torch.bfloat16)),
               dict(mx_out=True, out=u8(128, M)), dict(mx_out=True, out_scale=u8(4, M))):
        refused(moe, lambda: product(moe, **kw), ValueError)
    for kw in (dict(hidden_scale=u8(H // 32, T)), dict(logits=torch.zeros((E, T))),
               dict(w_gate_up_scale=u8(2 * F, E, H // 32)), dict(w_down=u8(H, E, fp // 2)),
               dict(w_down=u8(E, fp // 2, H)), dict(w_down_scale=u8(E, fp // 32, H)),
               dict(b_gate_up=torch.zeros((2 * F, E), dtype=torch.bfloat16)),
               dict(b_down=torch.zeros((H, E), dtype=torch.bfloat16)),
               dict(expert_ids=torch.zeros((TOPK, T), dtype=i32)),
               dict(topk_ids_out=torch.zeros((TOPK, T), dtype=i32)),
               dict(topk_weights_out=torch.zeros((TOPK, T))),
               dict(out=torch.zeros((H, T), dtype=torch.bfloat16))):
        refused(moe, lambda: layer(moe, **kw), ValueError)
    for kw in (dict(out=torch.zeros((H, T), dtype=torch.bfloat16)),
               dict(residual=True, residual_out=torch.zeros((H, T), dtype=torch.bfloat16)),
               dict(quant=1, codes=u8(H, T)), dict(quant=1, scales=u8(H // 32, T)),
               dict(quant=2, scales=torch.zeros((H // 128, T)))):
        refused(moe, lambda: norm(moe, **kw), ValueError)
    codes, scales = u8(T, H), u8(T, H // 32)
    moe.moe_mx_dequantize(codes, scales, H, out=torch.zeros((T, H)))
    refused(moe, lambda: moe.moe_mx_dequantize(codes, scales, H, out=torch.zeros((H, T))), ValueError)


def test_codes_and_scales_of_another_format_are_refused(moe):
    """Bytes (uint8, int8) or the format's own type: an e5m2 tensor's bytes are not e4m3 codes, nor
    e4m3 values power-of-two scales."""
    e4, e5, e8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
    i8 = torch.int8
    product(moe, a=u8(M, K).view(e4), a_scale=u8(M, K // 32).view(e8), w_scale=u8(E, N, K // 32).view(i8))
    product(moe, mx_out=True, out=u8(M, 128).view(e4), out_scale=u8(M, 4).view(e8))
    for kw in (dict(a=u8(M, K).view(e5)), dict(a=u8(M, K).view(e8)), dict(a=u8(M, K).bool()),
               dict(a_scale=u8(M, K // 32).view(e4)), dict(w=u8(E, N, K // 2).view(e4)),
               dict(w_scale=u8(E, N, K // 32).view(e4)),
               dict(mx_out=True, out=u8(M, 128).view(e5)),
               dict(mx_out=True, out_scale=u8(M, 4).view(e4))):
        refused(moe, lambda: product(moe, **kw), TypeError)
    fp = moe.moe_mx_columns(F)
    for kw in (dict(hidden=u8(T, H).view(e5)), dict(hidden_scale=u8(T, H // 32).view(e4)),
               dict(w_gate_up=u8(E, 2 * F, H // 2).view(e4)),
               dict(w_gate_up_scale=u8(E, 2 * F, H // 32).view(e5)),
               dict(w_down=u8(E, H, fp // 2).view(e4)), dict(w_down_scale=u8(E, H, fp // 32).view(e4))):
        refused(moe, lambda: layer(moe, **kw), TypeError)
    x = torch.zeros((T, H))
    for fmt, wide in ((moe.MOE_MX_E4M3, H), (moe.MOE_MX_E2M1, H // 2)):
        moe.moe_mx_quantize(x, fmt, codes=u8(T, wide), scales=u8(T, H // 32))
        refused(moe, lambda: moe.moe_mx_quantize(x, fmt, codes=u8(T, wide).view(e5)), TypeError)
        refused(moe, lambda: moe.moe_mx_quantize(x, fmt, scales=u8(T, H // 32).view(e4)), TypeError)
        refused(moe, lambda: moe.moe_mx_dequantize(u8(T, wide).view(e5), u8(T, H // 32), H), TypeError)
        refused(moe, lambda: moe.moe_mx_dequantize(u8(T, wide), u8(T, H // 32).view(e4), H), TypeError)
    refused(moe, lambda: moe.moe_mx_quantize(x, moe.MOE_MX_E2M1, codes=u8(T, H // 2).view(e4)), TypeError)
    refused(moe, lambda: norm(moe, quant=1, codes=u8(T, H).view(e5)), TypeError)
    refused(moe, lambda: norm(moe, quant=1, scales=u8(T, H // 32).view(e4)), TypeError)


def test_the_binding_imports_without_a_cuda_build_of_torch():
    """A torch built for the CPU has no stream handles to ask for; the binding is imported there all
    the same (build checks, workspace sizes)."""
    code = ("import torch\n"
            "del torch._C._cuda_getCurrentRawStream\n"
            "from mixture_experts_ffn_gb300 import moe\n"
            "assert moe.moe_mx_columns(2880) == 2944\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root)
    assert r.returncode == 0, r.stderr
