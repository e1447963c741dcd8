"""Cases, plain forms and measurements of the routed layer's gradients.

* ``tokens``  the combine's gradient (rows of every route, routing weights) and the
              permutation's (rows of a token's routes summed)
* ``save``    the activation and an 8-bit checkpoint of its argument (MX e4m3)
* ``act``     the activation's gradient, and the activation again, from the checkpoint
* ``dgrad``   the grouped product's gradient of its rows
* ``wgrad``   the grouped product's gradient of the weights and of the bias
* ``route``   the router's gradient of the logits

Routes are sorted by expert: route r = t * top_k + k sits in row route_to_row[r], and
expert e owns the rows seg_end[e - 1] .. seg_end[e].  An MX row of K values holds e4m3
codes, padded with zeros to a multiple of 128 columns, and one power of two per 32
columns (e8m0: the byte s stands for 2^(s - 127), 255 for NaN).
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
LIMIT, ALPHA, BETA = 7.0, 1.702, 1.0  # the clamped SwiGLU


def padded(k):
    return (k + 127) // 128 * 128


def wide(case):
    """Columns of the activation's argument: gate and up, or one."""
    return case["F"] * (1 if case["act"] == "relu" else 2)


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # the last, nearly empty batch of an epoch: latency alone
        dict(name="tokens 3x2048 top 8", op="tokens", T=3, H=2048, top_k=8, E=128, dtype="bf16"),
        # a training batch of the largest layer
        dict(name="tokens 8192x7168 top 8", op="tokens", T=8192, H=7168, top_k=8, E=256,
             dtype="bf16"),
        # a ragged micro-batch of narrow experts, float16
        dict(name="save 1021x768 silu", op="save", M=1021, F=768, act="silu", dtype="f16"),
        # all routes of 8192 tokens on 8 experts each
        dict(name="save 65536x2048 silu", op="save", M=65536, F=2048, act="silu", dtype="bf16"),
        # a few rows of a float32 run, interleaved gate and up
        dict(name="act 37x2880 swiglu", op="act", M=37, F=2880, act="swiglu", dtype="f32"),
        # routes of 8192 tokens on 4 experts each, clamped and interleaved
        dict(name="act 32768x2880 swiglu", op="act", M=32768, F=2880, act="swiglu", dtype="bf16"),
        # gate_up of 333 tokens on 8 of 128 narrow experts, float16, an odd number of rows
        dict(name="dgrad 2661 rows 1536 2048", op="dgrad", M=2661, E=128, N=1536, K=2048,
             dtype="f16"),
        # gate_up of 8192 tokens on 8 of 64 experts: bound by the products
        dict(name="dgrad 65536 rows 4096 7168", op="dgrad", M=65536, E=64, N=4096, K=7168,
             dtype="bf16"),
        # down product of a small batch with bias: the experts' gradients are what is written
        dict(name="wgrad 999 rows 2880 2880", op="wgrad", M=999, E=32, N=2880, K=2880,
             dtype="bf16", bias=True),
        # down product of 8192 tokens on 8 of 64 experts
        dict(name="wgrad 65536 rows 7168 2048", op="wgrad", M=65536, E=64, N=7168, K=2048,
             dtype="bf16", bias=False),
        # a small batch, softmax over all experts, bfloat16 logits
        dict(name="route 61x128 softmax", op="route", T=61, E=128, top_k=4, scoring="softmax",
             renormalize=False, scale=1.0, dtype="bf16"),
        # a training batch with sigmoid scores
        dict(name="route 8192x256 sigmoid", op="route", T=8192, E=256, top_k=8, scoring="sigmoid",
             renormalize=True, scale=2.5, dtype="f32"),
    ]


def draw(rng):
    def size(lo, hi, of=1):
        return of * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("tokens", "save", "act", "dgrad", "wgrad", "dgrad", "wgrad", "route"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "tokens":
        e = size(4, 256)
        return dict(op=op, T=size(1, 8192), H=size(8, 896, rng.choice((8, 8, 7))),
                    top_k=rng.randint(1, min(8, e)), E=e, dtype=dtype)
    if op in ("save", "act"):
        return dict(op=op, M=size(1, 65536), F=rng.choice((size(1, 64, 32), size(8, 2048))),
                    act=rng.choice(("silu", "swiglu", "gelu", "relu")),
                    dtype=rng.choice((dtype, "bf16")))
    if op == "route":
        e = size(4, 512)
        return dict(op=op, T=size(1, 16384), E=e, top_k=rng.randint(1, min(8, e)),
                    scoring=rng.choice(("softmax", "sigmoid", "sqrt_softplus")),
                    renormalize=rng.random() < 0.6, scale=rng.choice((1.0, 2.5)), dtype=dtype)
    more = dict(bias=rng.random() < 0.4) if op == "wgrad" else {}
    if dtype == "f32":  # exact products of float32, any size
        return dict(op=op, M=size(1, 2048), E=size(1, 32), N=size(16, 1024), K=size(16, 1024),
                    dtype=dtype, **more)
    return dict(op=op, M=size(1, 16384), E=size(1, 64), N=size(8, 512, 8), K=size(8, 512, 8),
                dtype=dtype, **more)


# ----------------------------------------------------------------- the inputs
def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    dt = TYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "tokens":
        # routes to random experts, some fuller than others, in rows sorted by expert
        T, K, H = c["T"], c["top_k"], c["H"]
        z = _randn(g, T, c["E"]) + _randn(g, c["E"])
        ids = z.topk(K, dim=1).indices.flatten()
        order = torch.sort(ids, stable=True).indices
        s["route_to_row"] = torch.empty_like(order, dtype=torch.int32)
        s["route_to_row"][order] = torch.arange(T * K, device="cuda", dtype=torch.int32)
        s["topk_weights"] = torch.softmax(_randn(g, T, K), 1)
        s["d_out"] = _randn(g, T, H, dtype=dt)
        s["expert_out"] = _randn(g, T * K, H, dtype=dt)
        s["d_expert_input"] = _randn(g, T * K, H, dtype=dt)
        return s
    if c["op"] in ("save", "act"):
        # a product's rows: columns of unequal strength, a few past the clamps
        n = wide(c)
        p = torch.randn((c["M"], n), generator=g, device="cuda")
        p *= 0.5 + 3.0 * torch.rand(n, generator=g, device="cuda") ** 4
        if c["op"] == "save":
            s["p"] = p.to(dt)
        else:
            s["codes"], s["scales"] = quantize_e4m3(p)
            s["d_act"] = _randn(g, c["M"], c["F"], dtype=dt)
        return s
    if c["op"] in ("dgrad", "wgrad"):
        M, E, N, K = c["M"], c["E"], c["N"], c["K"]
        share = torch.softmax(0.7 * _randn(g, E), 0)  # uneven experts, some without a row
        counts = torch.bincount(torch.multinomial(share, M, replacement=True, generator=g),
                                minlength=E)
        s["seg_end"] = counts.cumsum(0).to(torch.int32)
        s["ends"] = counts.cumsum(0).tolist()
        s["d_out"] = _randn(g, M, N, dtype=dt)
        if c["op"] == "wgrad":
            s["a"] = _randn(g, M, K, dtype=dt)
        else:
            s["w"] = torch.empty((E, N, K), dtype=dt, device="cuda")
            for e in range(E):
                s["w"][e] = _randn(g, N, K, std=K ** -0.5, dtype=dt)
        return s
    T, E, K = c["T"], c["E"], c["top_k"]
    s["logits"] = _randn(g, T, E, dtype=dt)
    s["topk_ids"] = s["logits"].float().topk(K, dim=1).indices.sort(1).values.to(torch.int32)
    s["d_weights"] = _randn(g, T, K)
    return s


# ----------------------------------------------------------------- plain forms
def _power(e):
    """2^e for integers -127 <= e <= 127."""
    bits = torch.where(e == -127, 1 << 22, (e + 127) << 23)
    return bits.to(torch.int32).view(torch.float32)


def quantize_e4m3(x):
    x = torch.nn.functional.pad(x.float(), (0, padded(x.shape[-1]) - x.shape[-1]))
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(-1)
    m, e = torch.frexp(top)  # top = m 2^e, 1/2 <= m < 1; 448 = 7/8 2^9
    e = torch.where(top > 0, e - 9 + (m > 0.875), -127).clamp(min=-127)
    v = (b * _power(-e).unsqueeze(-1)).clamp(-448, 448)
    scales = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return v.flatten(-2).to(torch.float8_e4m3fn), scales


def _values(codes, scales, n):
    bits = scales.view(torch.uint8).to(torch.int32)
    s = torch.where(bits == 0, 1 << 22, bits << 23).to(torch.int32).view(torch.float32)
    return (codes.float().unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)[:, :n]


def _pair(p, c):
    """Gate and up of the activation's argument: stacked, or interleaved (swiglu)."""
    if c["act"] == "relu":
        return p, None
    if c["act"] == "swiglu":
        return p[:, 0::2], p[:, 1::2]
    return p[:, :c["F"]], p[:, c["F"]:]


def _cdf(x):
    return 0.5 * torch.erfc(x * -(0.5 ** 0.5))


def _act(p, c):
    gate, up = _pair(p, c)
    if c["act"] == "relu":
        return gate.clamp(min=0)
    if c["act"] == "gelu":
        return gate * _cdf(gate) * up
    if c["act"] == "silu":
        return gate * torch.sigmoid(gate) * up
    gate, up = gate.clamp(max=LIMIT), up.clamp(-LIMIT, LIMIT)
    return gate * torch.sigmoid(ALPHA * gate) * (up + BETA)


def _act_gradient(p, d, c):
    gate, up = _pair(p, c)
    if c["act"] == "relu":
        return torch.where(gate > 0, d, 0.0)
    if c["act"] == "gelu":
        cdf, pdf = _cdf(gate), torch.exp(-0.5 * gate * gate) * (2 * math.pi) ** -0.5
        return torch.cat((d * up * (cdf + gate * pdf), d * gate * cdf), 1)
    if c["act"] == "silu":
        sig = torch.sigmoid(gate)
        return torch.cat((d * up * sig * (1 + gate * (1 - sig)), d * gate * sig), 1)
    low, mid = gate.clamp(max=LIMIT), up.clamp(-LIMIT, LIMIT)
    sig = torch.sigmoid(ALPHA * low)
    d_gate = torch.where(gate <= LIMIT, d * (mid + BETA) * sig * (1 + ALPHA * low * (1 - sig)), 0.0)
    d_up = torch.where(up.abs() <= LIMIT, d * low * sig, 0.0)
    return torch.stack((d_gate, d_up), 2).flatten(1)


def _route_gradient(z, ids, g, c):
    if c["scoring"] == "softmax":
        score = torch.softmax(z, 1)
    elif c["scoring"] == "sigmoid":
        score = torch.sigmoid(z)
    else:
        score = torch.sqrt(torch.nn.functional.softplus(z))
    s = score.gather(1, ids)
    if c["renormalize"]:
        total = s.sum(1, keepdim=True)
        d_s = (g - (g * s).sum(1, keepdim=True) / total) / total
    else:
        d_s = g
    d_score = torch.zeros_like(z).scatter_add(1, ids, c["scale"] * d_s)
    if c["scoring"] == "softmax":
        return score * (d_score - (d_score * score).sum(1, keepdim=True))
    if c["scoring"] == "sigmoid":
        return d_score * score * torch.sigmoid(-z)
    return d_score * torch.sigmoid(z) / (2 * score)


def _plain(s):
    c = s["case"]
    dt = TYPES[c["dtype"]]
    if c["op"] == "tokens":
        T, K, H = c["T"], c["top_k"], c["H"]
        rows, d = s["route_to_row"], s["d_out"].float().unsqueeze(1)
        d_expert_out = torch.empty_like(s["expert_out"])
        d_expert_out[rows] = (s["topk_weights"].unsqueeze(2) * d).to(dt).view(T * K, H)
        d_weights = (s["expert_out"][rows].float().view(T, K, H) * d).sum(2)
        d_hidden = s["d_expert_input"][rows].float().view(T, K, H).sum(1).to(dt)
        return {"d_expert_out": d_expert_out, "d_weights": d_weights, "d_hidden": d_hidden}
    if c["op"] == "save":
        p = s["p"].float()
        codes, scales = quantize_e4m3(p)
        return {"act": _act(p, c).to(dt), "codes": codes, "scales": scales}
    if c["op"] == "act":
        p = _values(s["codes"], s["scales"], wide(c))
        return {"d_p": _act_gradient(p, s["d_act"].float(), c).to(dt), "act": _act(p, c).to(dt)}
    if c["op"] == "route":
        z = s["logits"].float()
        return {"d_logits": _route_gradient(z, s["topk_ids"].long(), s["d_weights"], c).to(dt)}
    starts = [0] + s["ends"][:-1]
    d = s["d_out"]
    if c["op"] == "dgrad":
        d_a = torch.empty((c["M"], c["K"]), dtype=dt, device="cuda")
        for e, (lo, hi) in enumerate(zip(starts, s["ends"])):
            if hi > lo:
                d_a[lo:hi] = d[lo:hi].float() @ s["w"][e].float()
        return {"d_a": d_a}
    out = {"d_w": torch.empty((c["E"], c["N"], c["K"]), dtype=dt, device="cuda")}
    if c["bias"]:
        out["d_bias"] = torch.empty((c["E"], c["N"]), dtype=dt, device="cuda")
    for e, (lo, hi) in enumerate(zip(starts, s["ends"])):
        rows = d[lo:hi].float()
        out["d_w"][e] = rows.t() @ s["a"][lo:hi].float()
        if c["bias"]:
            out["d_bias"][e] = rows.sum(0)
    return out


# ----------------------------------------------------------------- the framework's calls
def _act_params(moe, act):
    if act == "swiglu":
        return moe.act_params(moe.MOE_ACT_SWIGLU, swiglu_fusion=1, limit=LIMIT, alpha=ALPHA,
                              beta=BETA)
    return moe.act_params({"silu": moe.MOE_ACT_SILU_AND_MUL, "gelu": moe.MOE_ACT_GELU_AND_MUL,
                           "relu": moe.MOE_ACT_RELU}[act])


def _calls(s):
    from mixture_experts_ffn_gb300 import moe

    c = s["case"]
    if c["op"] == "tokens":
        d_expert_out, d_weights = moe.moe_combine_backward(
            s["d_out"], s["expert_out"], s["topk_weights"], s["route_to_row"])
        d_hidden = moe.moe_permute_backward(s["d_expert_input"], s["route_to_row"], c["top_k"])
        return {"d_expert_out": d_expert_out, "d_weights": d_weights, "d_hidden": d_hidden}
    if "ws" not in s:  # a program's workspace and parameters, kept from call to call
        if c["op"] in ("save", "act"):
            s["ws"], s["act"] = None, _act_params(moe, c["act"])
        elif c["op"] == "route":
            s["ws"] = None
            s["route"] = moe.route_params(c["top_k"], c["scoring"], c["renormalize"],
                                          routed_scaling_factor=c["scale"])
        else:
            need = moe.MOE_STATUS_BYTES if c["op"] == "dgrad" else \
                moe.moe_grouped_gemm_wgrad_workspace_size(c["M"], c["N"], c["K"], c["E"])
            s["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
    if c["op"] == "save":
        act, codes, scales = moe.moe_act_checkpoint(s["p"], s["act"])
        return {"act": act, "codes": codes, "scales": scales}
    if c["op"] == "act":
        d_p, act = moe.moe_act_backward(s["codes"], s["d_act"], s["act"], scales=s["scales"])
        return {"d_p": d_p, "act": act}
    if c["op"] == "route":
        return {"d_logits": moe.moe_route_backward(s["logits"], s["topk_ids"], s["d_weights"],
                                                   s["route"])}
    if c["op"] == "dgrad":
        return {"d_a": moe.moe_grouped_gemm_dgrad(s["d_out"], s["w"], s["seg_end"], ws=s["ws"])}
    d_w, d_bias = moe.moe_grouped_gemm_wgrad(s["d_out"], s["a"], s["seg_end"], bias=c["bias"],
                                             ws=s["ws"])
    return {"d_w": d_w, "d_bias": d_bias} if c["bias"] else {"d_w": d_w}


def run(state):
    return _calls(state) if own else _plain(state)


# ----------------------------------------------------------------- what a pass needs
def work(case):
    c = case
    b = BYTES[c["dtype"]]
    if c["op"] == "tokens":
        rows, tokens = c["T"] * c["top_k"] * c["H"], c["T"] * c["H"]
        return {"bytes": b * (3 * rows + 2 * tokens) + 16 * c["T"] * c["top_k"],
                "flops": 4 * rows}
    if c["op"] in ("save", "act"):
        n, a = c["M"] * wide(c), c["M"] * c["F"]
        mx = c["M"] * padded(wide(c)) * (1 + 1 / 32)
        return {"bytes": mx + n * b + a * b * (1 if c["op"] == "save" else 2),
                "flops": (15 if c["op"] == "save" else 25) * a}
    if c["op"] == "route":
        read = c["E"] if c["scoring"] == "softmax" and not c["renormalize"] else c["top_k"]
        return {"bytes": c["T"] * ((c["E"] + read) * b + 8 * c["top_k"]),
                "flops": c["T"] * (2 * c["E"] + 20 * c["top_k"])}
    M, E, N, K = c["M"], c["E"], c["N"], c["K"]
    flops = 2 * M * N * K
    if c["op"] == "dgrad":
        return {"bytes": b * (M * (N + K) + min(E, M) * N * K), "flops": flops}
    return {"bytes": b * (M * (N + K) + E * N * (K + (1 if c["bias"] else 0))),
            "flops": flops + (M * N if c["bias"] else 0)}


# ----------------------------------------------------------------- the definition in 64 bits
def _x_checkpoint(v):
    """v [R, n] float64 -> (codes as numbers [R, padded], scales [R, padded / 32])."""
    R, n = v.shape
    out = torch.zeros(R, padded(n), dtype=torch.float64, device=v.device)
    out[:, :n] = v
    out = out.view(R, -1, 32)
    amax = out.abs().amax(2)
    low = torch.floor(torch.log2(amax.clamp(min=2.0 ** -149)))
    low = low + (torch.exp2(low + 1) <= amax).double() - (torch.exp2(low) > amax).double()
    ex = low - 8 + (amax > 448 * torch.exp2(low - 8)).double()
    ex = torch.where(amax > 0, ex, torch.full_like(ex, -127.0)).clamp(min=-127.0)
    sc = torch.exp2(ex)
    z = out / sc.unsqueeze(2)  # 3 mantissa bits down to 2^-6, then steps of 2^-9
    unit = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -30))).clamp(min=-6.0) - 3)
    return (torch.round(z / unit) * unit).clamp(-448.0, 448.0).view(R, -1), sc


def _x_act(p, c):
    """The activation of p's rows (float64) as a function that differentiation can follow."""
    F = c["F"]
    if c["act"] == "relu":
        return torch.relu(p)
    if c["act"] == "swiglu":
        x, y = torch.clamp(p[:, ::2], max=LIMIT), torch.clamp(p[:, 1::2], -LIMIT, LIMIT)
        return x / (1.0 + torch.exp(-ALPHA * x)) * (y + BETA)
    x, y = p.split(F, 1)
    if c["act"] == "silu":
        return x / (1.0 + torch.exp(-x)) * y
    return x * (0.5 + 0.5 * torch.erf(x / math.sqrt(2.0))) * y


def _x_weights(z, ids, c):
    if c["scoring"] == "softmax":
        s = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    elif c["scoring"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-z))
    else:
        s = torch.sqrt(torch.log(1.0 + torch.exp(z)))
    s = torch.take_along_dim(s, ids, 1)
    return c["scale"] * (s / s.sum(1, keepdim=True) if c["renormalize"] else s)


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "tokens":
        T, K, H = c["T"], c["top_k"], c["H"]
        to = s["route_to_row"].long().view(T, K)
        d = s["d_out"].double()
        d_y = torch.empty(T * K, H, dtype=torch.float64, device="cuda")
        d_w = torch.empty(T, K, dtype=torch.float64, device="cuda")
        d_h = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for k in range(K):
            d_y[to[:, k]] = d * s["topk_weights"][:, k:k + 1].double()
            d_w[:, k] = torch.einsum("th,th->t", d, s["expert_out"][to[:, k]].double())
            d_h += s["d_expert_input"][to[:, k]].double()
        return {"d_expert_out": d_y, "d_weights": d_w, "d_hidden": d_h}
    if c["op"] == "save":
        parts = []
        for p in s["p"].split(8192):
            p = p.double()
            parts.append((_x_act(p, c), *_x_checkpoint(p)))
        return dict(zip(("act", "codes", "scales"), (torch.cat(x) for x in zip(*parts))))
    if c["op"] == "act":
        parts = []
        at = torch.exp2(s["scales"].view(torch.uint8).double() - 127.0)
        for codes, sc, d in zip(s["codes"].split(8192), at.split(8192), s["d_act"].split(8192)):
            p = (codes.double().view(codes.shape[0], -1, 32) * sc.unsqueeze(2)).flatten(1)
            p = p[:, :wide(c)].clone().requires_grad_()
            a = _x_act(p, c)
            parts.append((torch.autograd.grad(a, p, d.double())[0], a.detach()))
        return dict(zip(("d_p", "act"), (torch.cat(x) for x in zip(*parts))))
    if c["op"] == "route":
        z = s["logits"].double().requires_grad_()
        w = _x_weights(z, s["topk_ids"].long(), c)
        return {"d_logits": torch.autograd.grad(w, z, s["d_weights"].double())[0]}
    owner = torch.searchsorted(s["seg_end"].long(), torch.arange(c["M"], device="cuda"), right=True)
    if c["op"] == "dgrad":
        d_a = torch.empty(c["M"], c["K"], dtype=torch.float64, device="cuda")
        for e in owner.unique().tolist():
            at = (owner == e).nonzero().flatten()
            d_a[at] = torch.matmul(s["d_out"][at].double(), s["w"][e].double())
        return {"d_a": d_a}
    d_w = torch.zeros(c["E"], c["N"], c["K"], dtype=torch.float64, device="cuda")
    d_b = torch.zeros(c["E"], c["N"], dtype=torch.float64, device="cuda")
    for e in owner.unique().tolist():
        at = (owner == e).nonzero().flatten()
        d = s["d_out"][at].double()
        d_w[e] = torch.einsum("mn,mk->nk", d, s["a"][at].double())
        d_b[e] = torch.einsum("mn->n", d)
    return {"d_w": d_w, "d_bias": d_b} if c["bias"] else {"d_w": d_w}
