"""Measured cases of the 8-bit linear path: activations and weights in E4M3 with one E8M0
scale for every 128 consecutive values along K.

Operators: quantization of a 16-bit matrix; the root-mean-square norm with the residual's
addition and 8-bit output; the block-scaled 8-bit matrix product; and the gated pair of
projections (gate, up, activation, product, 8-bit output).  Each has a plain form of
elementary torch operations, the framework's call, and its definition in 64 bits.

Formats: codes float8_e4m3fn [rows][K]; scales one E8M0 byte per group of 128 (the last group
of a row may be short), rows padded with zero bytes to a multiple of four.  A group's scale is
the smallest power of two 2^e with max|y| <= 448 2^e (byte e + 127; 0 for a group of zeros).
"""

import math

import torch

own = False

GROUP = 128
LARGEST = 2.0 * 4096 * 2 * 11008 * 4096       # flops of the largest listed case


def listed():
    return [
        # attention output of a 4096-token prompt, before the output projection
        dict(name="quantize_prompt", op="quantize", M=4096, K=4096, dtype="bf16"),
        # a caption's 77 tokens at the SANA-like width: 17.5 groups a row
        dict(name="quantize_caption", op="quantize", M=77, K=2240, dtype="fp16"),
        # one token between two layers: latency
        dict(name="norm_token", op="norm", M=1, K=4096, dtype="bf16", residual=True),
        # a prompt between two layers
        dict(name="norm_prompt", op="norm", M=8192, K=4096, dtype="bf16", residual=True),
        # an odd number of tokens at the PixArt-like width, first norm of a network (no residual yet)
        dict(name="norm_odd", op="norm", M=1155, K=1152, dtype="fp16", residual=False),
        # down-projection of one token: the weights' bytes
        dict(name="linear_token", op="linear", M=1, N=4096, K=11008, dtype="bf16", bias=False),
        # q, k and v of 37 sequences that each add a token
        dict(name="linear_batch", op="linear", M=37, N=6144, K=4096, dtype="bf16", bias=True),
        # down-projection of a prompt
        dict(name="linear_prompt", op="linear", M=4096, N=4096, K=11008, dtype="bf16", bias=False),
        # fc1 of the PixArt-like block, two images
        dict(name="linear_image", op="linear", M=8192, N=4608, K=1152, dtype="fp16", bias=True),
        # gate and up of one token
        dict(name="gated_token", op="gated", M=1, F=11008, K=4096, act="silu"),
        # a ragged batch of 203 tokens at the SANA-like widths: both K and F end inside a group
        dict(name="gated_odd", op="gated", M=203, F=5600, K=2240, act="gelu_tanh"),
        # gate and up of a prompt: the largest
        dict(name="gated_prompt", op="gated", M=4096, F=11008, K=4096, act="silu"),
    ]


def draw(rng):
    def size(lo, hi, step):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))

    op = rng.choice(["quantize", "norm", "linear", "linear", "gated", "gated"])
    M = size(1, 8192, 1)
    dtype = rng.choice(["bf16", "fp16"])
    K = size(128, 11008, 16)
    if op == "quantize":
        return dict(op=op, M=M, K=K, dtype=dtype)
    if op == "norm":
        return dict(op=op, M=M, K=K, dtype=dtype, residual=rng.random() < 0.7)
    if op == "linear":
        N = size(128, 11008, 16)
        M = max(1, min(M, int(LARGEST / (2.0 * N * K))))
        return dict(op=op, M=M, N=N, K=K, dtype=dtype, bias=rng.random() < 0.5)
    F = size(128, 11008, 16)
    M = max(1, min(M, int(LARGEST / (4.0 * F * K))))
    return dict(op=op, M=M, F=F, K=K, act=rng.choice(["silu", "gelu", "gelu_tanh"]))


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def _scale_cols(K):
    return 4 * ((K + 511) // 512)


# ------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(M, K, g):
    """Unit Gaussian values with a mean for each token and a few outlier channels."""
    x = torch.randn(M, K, device="cuda", generator=g)
    x += 0.5 * torch.randn(M, 1, device="cuda", generator=g)
    loud = torch.randperm(K, device="cuda", generator=g)[:12]
    x[:, loud] *= 20.0
    return x


def _weights(N, K, g):
    return torch.randn(N, K, device="cuda", generator=g) * K ** -0.5


def prepare(case, seed):
    g = _generator(seed)
    op, M, K = case["op"], case["M"], case["K"]
    s = dict(case=case)
    if op in ("quantize", "norm"):
        s["X"] = _activations(M, K, g).to(_dtype(case["dtype"]))
        if op == "norm":
            s["gamma"] = (1.0 + 0.2 * torch.randn(K, device="cuda", generator=g)).to(_dtype(case["dtype"]))
            if case["residual"]:
                s["residual"] = (3.0 * _activations(M, K, g)).to(_dtype(case["dtype"]))
        return s
    rows = case["N"] if op == "linear" else 2 * case["F"]
    s["xcodes"], s["xscales"] = _quantize(_activations(M, K, g))
    s["wcodes"], s["wscales"] = _quantize(_weights(rows, K, g))
    if op == "linear" and case["bias"]:
        s["bias"] = torch.randn(rows, device="cuda", generator=g).to(_dtype(case["dtype"]))
    return s


# ------------------------------------------------------------------------- plain form

def _quantize(y):
    """float32 [M][K] -> (float8_e4m3fn [M][K], uint8 [M][scale columns])."""
    M, K = y.shape
    G = (K + GROUP - 1) // GROUP
    y = torch.nn.functional.pad(y, (0, G * GROUP - K)).reshape(M, G, GROUP)
    top = y.abs().amax(dim=2)
    frac, ex = torch.frexp(top)                              # top = frac 2^ex, 0.5 <= frac < 1
    e = torch.where(frac <= 0.875, ex - 9, ex - 8)           # 448 = 0.875 2^9
    e = torch.where(top > 0, e, torch.full_like(e, -127)).clamp(min=-127)
    unit = ((127 - e) << 23).to(torch.int32).view(torch.float32)                 # 2^-e
    codes = (y * unit[:, :, None]).to(torch.float8_e4m3fn).reshape(M, G * GROUP)[:, :K].contiguous()
    scales = torch.zeros(M, _scale_cols(K), dtype=torch.uint8, device=y.device)
    scales[:, :G] = (e + 127).to(torch.uint8)
    return codes, scales


def _values(codes, scales):
    """The float32 values that codes and scales stand for."""
    K = codes.shape[1]
    s = scales.view(torch.float8_e8m0fnu).to(torch.float32).repeat_interleave(GROUP, dim=1)[:, :K]
    return codes.to(torch.float32) * s


def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _as_values(codes, scales):
    return {"codes": codes, "scales": scales.view(torch.float8_e8m0fnu)}


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import w4a4_post_quantization_amd as kq
        if op == "quantize":
            return _as_values(*kq.quantize_fp8(s["X"]))
        if op == "norm":
            codes, scales, h = kq.rmsnorm_quantize_fp8(s["X"], s["gamma"], eps=1e-6, residual=s.get("residual"))
            return dict(_as_values(codes, scales), residual=h)
        if op == "linear":
            return kq.fp8_linear(s["xcodes"], s["xscales"], s["wcodes"], s["wscales"], bias=s.get("bias"),
                                 dtype=_dtype(c["dtype"]))
        return _as_values(*kq.fp8_gated_linear(s["xcodes"], s["xscales"], s["wcodes"], s["wscales"], act=c["act"]))
    if op == "quantize":
        return _as_values(*_quantize(s["X"].float()))
    if op == "norm":
        h, out = s["X"].float(), None
        if "residual" in s:
            h = h + s["residual"].float()
            out = h.to(s["X"].dtype)
        y = h * (1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + 1e-6)) * s["gamma"].float()
        return dict(_as_values(*_quantize(y)), residual=out)
    y = _values(s["xcodes"], s["xscales"]) @ _values(s["wcodes"], s["wscales"]).t()
    if op == "linear":
        if "bias" in s:
            y = y + s["bias"].float()
        return y.to(_dtype(c["dtype"]))
    return _as_values(*_quantize(_act(y[:, : c["F"]], c["act"]) * y[:, c["F"]:]))


# ------------------------------------------------------------------------- cost and definition

def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "quantize":
        return {"bytes": 3.0 * M * K + M * _scale_cols(K), "flops": 3.0 * M * K}
    if case["op"] == "norm":
        return {"bytes": (7.0 if case["residual"] else 3.0) * M * K + M * _scale_cols(K) + 2.0 * K, "flops": 8.0 * M * K}
    if case["op"] == "linear":
        N = case["N"]
        return {"bytes": (M + N) * (K + _scale_cols(K)) + 2.0 * M * N + (2.0 * N if case["bias"] else 0.0),
                "flops": 2.0 * M * N * K}
    F = case["F"]
    return {"bytes": (M + 2.0 * F) * (K + _scale_cols(K)) + M * (F + _scale_cols(F)), "flops": 4.0 * M * F * K + 10.0 * M * F}


def _pow2(e):
    """2^e in float64 for whole e in the normal range, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_codes(y):
    """The values of the E4M3 codes and of the scales of float64 rows, from the definition."""
    M, K = y.shape
    cols = []
    codes = torch.empty_like(y)
    for k in range(0, K, GROUP):
        part = y[:, k:k + GROUP]
        top = part.abs().max(dim=1).values
        e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 448.0)).clamp(min=-127.0)
        unit = _pow2(e)
        v = part / unit[:, None]
        step = _pow2(torch.floor(torch.log2(torch.clamp(v.abs(), min=2.0 ** -6))) - 3.0)
        codes[:, k:k + GROUP] = torch.round(v / step) * step
        cols.append(unit)
    cols += [torch.full_like(cols[0], 2.0 ** -127)] * (_scale_cols(K) - len(cols))
    return {"codes": codes, "scales": torch.stack(cols, dim=1)}


def exact(case, seed):
    op, K = case["op"], case["K"]
    if work(case)["flops"] > 4e14:      # a float64 product of that size takes too long
        return None
    s = prepare(case, seed)
    if op == "quantize":
        return _exact_codes(s["X"].double())
    if op == "norm":
        h = s["X"].double()
        if "residual" in s:
            h = h + s["residual"].double()
        rms = torch.sqrt(torch.sum(h ** 2, dim=1) / K + 1e-6)
        return dict(_exact_codes(h / rms[:, None] * s["gamma"].double()), residual=h if "residual" in s else None)

    def dense(codes, scales):
        v = codes.to(torch.float64)
        for j, k in enumerate(range(0, K, GROUP)):
            v[:, k:k + GROUP] *= _pow2(scales[:, j:j + 1].to(torch.int64) - 127)
        return v

    y = torch.matmul(dense(s["xcodes"], s["xscales"]), dense(s["wcodes"], s["wscales"]).T)
    if op == "linear":
        return y + s["bias"].double() if "bias" in s else y
    g, u = y[:, : case["F"]], y[:, case["F"]:]
    if case["act"] == "silu":
        a = g * torch.sigmoid(g)
    elif case["act"] == "gelu":
        a = g * 0.5 * torch.erfc(-g / math.sqrt(2.0))
    else:
        a = g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))
    return _exact_codes(a * u)
