"""Cases, plain forms and float64 references of the 8-bit (E4M3, one power-of-two scale per
128-element block) operators: the root-mean-square norm with an 8-bit output, the
block-scaled matrix product, its gated form, and the feed-forward block made of the three.

An 8-bit block holds E4M3 codes c and one scale 2^e, e the smallest exponent for which no
value of the block exceeds 448 * 2^e. Activations have a block for each token and 128
features, weights one for each 128 outputs x 128 inputs; a last block may be shorter.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128
EPS = 1e-6


# ---------------------------------------------------------------------------- the cases --
def listed():
    return [
        # one decoded token: the residual stream's update and norm ahead of a projection
        {"name": "norm_token", "op": "norm", "M": 1, "K": 4096, "res": "bf16"},
        # a ragged batch of tokens, a width that ends inside a block, the stream kept in fp32
        {"name": "norm_ragged", "op": "norm", "M": 333, "K": 2080, "res": "f32"},
        # a long prompt: pure memory traffic
        {"name": "norm_prompt", "op": "norm", "M": 8192, "K": 8192, "res": "bf16"},
        # a projection for one decoded token: the weights are read once, nothing else counts
        {"name": "linear_token", "op": "linear", "M": 1, "K": 4096, "N": 4096, "out": "bf16"},
        # a handful of tokens through the fc1 shape of the repository's PixArt workload
        {"name": "linear_few", "op": "linear", "M": 24, "K": 1152, "N": 4608, "out": "f32"},
        # a chunk of a prompt, no size a multiple of a tile
        {"name": "linear_ragged", "op": "linear", "M": 1000, "K": 2080, "N": 1936, "out": "bf16"},
        # the PixArt fc1 workload itself
        {"name": "linear_fc1", "op": "linear", "M": 4096, "K": 1152, "N": 4608, "out": "bf16"},
        # a long prompt through a wide square projection: the tensor cores' rate
        {"name": "linear_prompt", "op": "linear", "M": 8192, "K": 8192, "N": 8192, "out": "bf16"},
        # gate and up projections for a small decode batch
        {"name": "gated_few", "op": "gated", "M": 8, "K": 4096, "N": 12288, "out": "bf16"},
        # the same for a long prompt
        {"name": "gated_prompt", "op": "gated", "M": 4096, "K": 4096, "N": 12288, "out": "bf16"},
        # the whole feed-forward block for one decoded token
        {"name": "ffn_token", "op": "ffn", "M": 1, "K": 2048, "N": 8192, "res": "bf16", "out": "bf16"},
        # and for a prompt of an odd length
        {"name": "ffn_prompt", "op": "ffn", "M": 2125, "K": 2304, "N": 9216, "res": "f32", "out": "bf16"},
    ]


def draw(rng):
    def size(lo, hi, step):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(step, int(round(v / step)) * step)

    op = rng.choice(["norm", "linear", "linear", "gated", "ffn"])
    while True:
        M, K = size(1, 8192, 1), size(256, 12288, 32)
        if op == "norm":
            return {"op": op, "M": M, "K": min(K, 8192), "res": rng.choice(["none", "bf16", "f32"])}
        c = {"op": op, "M": M, "K": K, "N": size(256, 12288, 32 if op == "ffn" else 16),
             "out": rng.choice(["bf16", "bf16", "f32"])}
        if op == "ffn":
            # the 8-bit values inside the block sit next to rounding borders: bf16 output
            c |= {"res": rng.choice(["none", "bf16", "f32"]), "out": "bf16"}
        if work(c)["flops"] <= 0.9e12:
            return c


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    res = {"none": 0, "bf16": 2, "f32": 4}[case.get("res", "none")]
    if op == "norm":
        return {"bytes": M * K * (2 + 2 * res + 2) + 4 * K, "flops": 6 * M * K}
    N, out = case["N"], {"bf16": 2, "f32": 4}[case["out"]]
    if op == "ffn":
        return {"bytes": M * K * (2 + 2 * res + out) + 4 * K + 3 * N * K, "flops": 6 * M * N * K}
    mats = 2 if op == "gated" else 1
    return {"bytes": 2 * M * K + mats * N * K + M * N * out, "flops": 2 * mats * M * N * K}


# ------------------------------------------------------------------------- 8-bit blocks --
def pow2(e):
    """2^e in float64 for whole numbers e, built from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def block_exponent(amax):
    """The smallest e with amax <= 448 * 2^e, at least -127; -127 for a block of zeros."""
    mant, p = torch.frexp(amax.double())               # amax = mant * 2^p, 0.5 <= mant < 1
    e = p - 9 + (mant > 0.875).to(p.dtype)             # 448 = 0.875 * 2^9
    return torch.where(amax == 0, torch.full_like(e, -127), e.clamp(min=-127))


def quantize_rows(v):
    """The values that rows v [M, K] (float32) stand for after the 8-bit encoding."""
    M, K = v.shape
    kb = -(-K // BLOCK)
    b = torch.nn.functional.pad(v, (0, kb * BLOCK - K)).view(M, kb, BLOCK)
    s = pow2(block_exponent(b.abs().amax(-1, keepdim=True)))
    codes = (b.double() / s).float().to(torch.float8_e4m3fn)
    return (codes.float() * s.float()).view(M, kb * BLOCK)[:, :K]


def quantize_weight(w):
    """E4M3 codes [N, K] and scale bytes [N / 128, K / 128] (exponent + 127) of w [N, K]."""
    N, K = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    b = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(nb, BLOCK, kb, BLOCK)
    e = block_exponent(b.abs().amax((1, 3)))
    codes = (b.double() / pow2(e)[:, None, :, None]).float().to(torch.float8_e4m3fn)
    codes = codes.view(torch.uint8).reshape(nb * BLOCK, kb * BLOCK)[:N, :K].contiguous()
    return codes.view(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def decode_weight(w, dtype):
    codes, scales = w
    s = pow2(scales.to(torch.int64) - 127).to(dtype)
    s = s.repeat_interleave(BLOCK, 0)[:codes.shape[0]].repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]
    return codes.to(dtype) * s


# --------------------------------------------------------------------------- the inputs --
def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def inputs(case, seed):
    """Activations as they leave a transformer's block (a scale of its own for each token and
    a few channels much larger than the rest), weights that keep the scale, norm gains near 1."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    M, K, N, op = case["M"], case["K"], case.get("N", 0), case["op"]
    s = {}
    x = torch.randn(M, K, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(M, 1, generator=g, device="cuda"))
    x[:, torch.randint(0, K, (max(1, K // 256),), generator=g, device="cuda")] *= 20
    s["x"] = x.to(torch.bfloat16)
    if op in ("norm", "ffn"):
        s["gamma"] = 1 + 0.25 * torch.randn(K, generator=g, device="cuda")
        s["residual"] = None
        if case["res"] != "none":
            s["residual"] = (2 * torch.randn(M, K, generator=g, device="cuda")).to(_dtype(case["res"]))

    def weight(n, k):
        return quantize_weight((torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k))
                               .to(torch.bfloat16).float())

    if op != "norm":
        s["w"] = weight(N, K)
    if op in ("gated", "ffn"):
        s["wu"] = weight(N, K)
    if op == "ffn":
        s["wd"] = weight(K, N)
    return s


def prepare(case, seed):
    s = {"case": dict(case), **inputs(case, seed)}
    M, K, N, op = case["M"], case["K"], case.get("N", 0), case["op"]
    if op == "norm":
        s["values"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    else:
        s["y"] = torch.empty(M, K if op == "ffn" else N, dtype=_dtype(case["out"]), device="cuda")
    if own:
        # what a program that serves the model keeps: the layers, their packed weights and a
        # workspace for its largest batch
        import w4a4_post_quantization_token_b200 as kq

        def buffer(n):
            return torch.empty(n, dtype=torch.uint8, device="cuda")

        def packed(layer, w, wu=None):
            buf = buffer(kq.fp8_weights_bytes(layer))
            kq.fp8_weights_pack(layer, *w, buf, *(wu or ()))
            return buf

        if op == "norm":
            s["act"] = buffer(kq.fp8_act_bytes(K, M))
        else:
            s["layer"] = kq.Fp8Layer(K, N, gated=op != "linear")
            s["weights"] = packed(s["layer"], s["w"], s.get("wu"))
            if op == "ffn":
                s["down"] = kq.Fp8Layer(N, K)
                s["down_weights"] = packed(s["down"], s["wd"])
                s["ws"] = buffer(kq.fp8_ffn_bytes(s["layer"], s["down"], M))
            else:
                s["act"] = buffer(kq.fp8_act_bytes(K, M))
    return s


# --------------------------------------------------------------------------- one pass ---
def run(state):
    op = state["case"]["op"]
    if own:
        return run_own(state, op)
    if op == "norm":
        y = norm(state)
        state["values"].copy_(quantize_rows(y))
        return {"residual": state["residual"], "values": state["values"]}
    if op == "linear":
        return state["y"].copy_(quantize_rows(state["x"].float()) @ decode_weight(state["w"], torch.float32).T)
    v = state["x"].float() if op == "gated" else norm(state)
    v = quantize_rows(v)
    gate = v @ decode_weight(state["w"], torch.float32).T
    up = v @ decode_weight(state["wu"], torch.float32).T
    h = gate / (1 + torch.exp(-gate)) * up
    if op == "gated":
        return state["y"].copy_(h)
    state["y"].copy_(quantize_rows(h) @ decode_weight(state["wd"], torch.float32).T)
    return {"residual": state["residual"], "y": state["y"]}


def norm(state):
    """h = x + residual (kept in the residual's type), h / rms(h) * gamma in float32, the mean
    square in float64: the 8-bit codes are decided next to borders."""
    h = state["x"].float()
    if state["residual"] is not None:
        state["residual"].copy_(h + state["residual"].float())
        h = state["residual"].float()
    r = torch.rsqrt(h.double().square().mean(-1, keepdim=True) + EPS).float()
    return h * r * state["gamma"]


def run_own(state, op):
    import w4a4_post_quantization_token_b200 as kq
    case = state["case"]
    if op == "norm":
        kq.fp8_rmsnorm_act(state["x"], state["gamma"], EPS, state["act"], residual=state["residual"])
        kq.fp8_act_unpack(case["K"], state["act"], case["M"], values=state["values"])
        return {"residual": state["residual"], "values": state["values"]}
    out = kq.OUT_BF16 if case["out"] == "bf16" else kq.OUT_F32
    if op == "ffn":
        kq.fp8_ffn(state["layer"], state["weights"], state["down"], state["down_weights"], state["x"],
                   state["gamma"], EPS, state["y"], state["ws"], out, residual=state["residual"])
        return {"residual": state["residual"], "y": state["y"]}
    kq.fp8_linear(state["layer"], state["weights"], state["x"], state["y"], state["act"], out)
    return state["y"]


# ------------------------------------------------------------------- float64 reference ---
def nearest_e4m3(v):
    """The E4M3 value nearest to v (float64, |v| <= 448): steps of 2^-3 relative to the power
    of two below, no finer than 2^-9, ties to the even multiple."""
    _, p = torch.frexp(v)
    step = pow2((p - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def blocks64(v):
    """The values an 8-bit encoding of rows v (float64) stands for, from the definition."""
    parts = []
    for k in range(0, v.shape[1], BLOCK):
        b = v[:, k:k + BLOCK]
        top = b.abs().amax(-1, keepdim=True)
        safe = torch.where(top == 0, torch.ones_like(top), top)
        e = torch.ceil(torch.log2(safe / E4M3_MAX)).clamp(min=-127)
        # log2 rounds: settle the exponent by the inequality that defines it
        e = torch.where(safe > E4M3_MAX * torch.exp2(e), e + 1, e)
        e = torch.where((safe <= E4M3_MAX * torch.exp2(e - 1)) & (e > -127), e - 1, e)
        s = pow2(e)
        parts.append(nearest_e4m3(b / s) * s)
    return torch.cat(parts, 1)


def exact(case, seed):
    s = inputs(case, seed)
    op = case["op"]
    v, res = s["x"].double(), None
    if op in ("norm", "ffn"):
        if s["residual"] is not None:
            # the stream's own rounding is part of the operator: one fp32 sum, kept in its type
            res = (v + s["residual"].double()).float().to(s["residual"].dtype)
            v = res.double()
        v = v / torch.sqrt((v * v).sum(-1, keepdim=True) / v.shape[1] + EPS) * s["gamma"].double()
    q = blocks64(v)
    if op == "norm":
        return {"residual": res, "values": q}
    y = torch.matmul(q, decode_weight(s["w"], torch.float64).T)
    if op == "linear":
        return y
    h = y * torch.sigmoid(y) * torch.matmul(q, decode_weight(s["wu"], torch.float64).T)
    if op == "gated":
        return h
    return {"residual": res, "y": torch.matmul(blocks64(h), decode_weight(s["wd"], torch.float64).T)}
