"""GPU: the 8-bit operators against the float64 oracle.

Codes and scales are compared bit for bit (both sides decide them from the same float32 values).
Products: the decoded operands are exact in float64 and each product of two codes is exact in the
tensor core, so a result may be off by the fp32 accumulation alone: one rounding (or truncation,
2^-23 of the running sum) for each 32-element step, K / 32 of them, plus the final rounding of
the output type. The running sum is at most sum |a||b|.
"""
import numpy as np
import pytest

from oracle import fp8

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _t(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _bf16(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def _np(t):
    return t.detach().double().cpu().numpy()


def tokens(M, K, seed):
    """bf16 rows of very different sizes with a few large channels."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.exp(2 * rng.standard_normal((M, 1)))
    x[:, rng.integers(0, K, max(1, K // 200))] *= 20
    return _bf16(x)


def weight(K, N, seed):
    """bf16 [K, N] whose 128 x 128 pieces have scales of their own."""
    rng = np.random.default_rng(seed + 77)
    w = rng.standard_normal((K, N)) / np.sqrt(K)
    w *= np.repeat(np.repeat(np.exp2(rng.integers(-3, 4, (-(-K // 128), -(-N // 128)))), 128, 0), 128, 1)[:K, :N]
    return _bf16(w)


def buf(n):
    import torch
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def unpack(kq, act, M, K):
    c, s = buf(M * K), buf(M * -(-K // 128))
    kq.fp8_act_unpack(K, act, M, c, s)
    return c.cpu().numpy().reshape(M, K), s.cpu().numpy().reshape(M, -1)


def packed(kq, L, W, Wu=None):
    """Prepared weights and the decoded [N, K] values of each matrix."""
    w = buf(kq.fp8_weights_bytes(L))
    enc = [fp8.encode_weight(_np(m)) for m in (W, Wu) if m is not None]
    parts = [_t(a) for e in enc for a in e]
    kq.fp8_weights_pack(L, parts[0], parts[1], w, *parts[2:])
    return w, [fp8.decode_weight(*e) for e in enc]


def accumulation(A, W):
    """Bound on the fp32 accumulation error of A W^T (see the module's docstring)."""
    return (A.shape[1] / 32 + 2) * 2.0 ** -23 * (np.abs(A) @ np.abs(W).T)


HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


# ------------------------------------------------------------------------------ codes ----
@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (130, 128), (7, 160), (33, 1152), (2, 2080), (1, 4096), (5, 8224),
                                 (2, 36864)])
def test_quantize_bit_exact(cuda_device, M, K):
    import torch
    import w4a4_post_quantization_token_b200 as kq
    X = tokens(M, K, M + K)
    X[0, :32] = 0
    act = buf(kq.fp8_act_bytes(K, M))
    kq.fp8_quantize_act(X.cuda(), act)
    c, s = unpack(kq, act, M, K)
    rc, rs = fp8.encode_rows(_np(X))
    np.testing.assert_array_equal(s, rs)
    np.testing.assert_array_equal(c, rc)
    for dt in (torch.bfloat16, torch.float32):
        v = torch.empty(M, K, dtype=dt, device="cuda")
        kq.fp8_act_unpack(K, act, M, values=v)
        np.testing.assert_array_equal(_np(v), fp8.decode_rows(rc, rs))
    # and back through the canonical parts
    act2 = buf(kq.fp8_act_bytes(K, M))
    kq.fp8_act_pack(K, _t(rc), _t(rs), M, act2)
    c2, s2 = unpack(kq, act2, M, K)
    np.testing.assert_array_equal(c2, rc)
    np.testing.assert_array_equal(s2, rs)


def test_quantize_every_bf16_magnitude(cuda_device):
    """Rows that hold every finite bf16 pattern, each beside a maximum of its own exponent."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    bits = np.arange(0x7F80, dtype=np.uint16)
    bits = np.concatenate([bits, bits | 0x8000])
    K = 128
    bits = np.resize(bits, (-(-bits.size // K)) * K).reshape(-1, K)
    X = torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16)
    act = buf(kq.fp8_act_bytes(K, X.shape[0]))
    kq.fp8_quantize_act(X.cuda(), act)
    c, s = unpack(kq, act, X.shape[0], K)
    rc, rs = fp8.encode_rows(_np(X))
    np.testing.assert_array_equal(s, rs)
    np.testing.assert_array_equal(c, rc)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_non_finite_blocks_are_nan(cuda_device, bad):
    import torch
    import w4a4_post_quantization_token_b200 as kq
    M, K, N = 4, 320, 32
    X = tokens(M, K, 3)
    X[1, 200] = bad
    act = buf(kq.fp8_act_bytes(K, M))
    kq.fp8_quantize_act(X.cuda(), act)
    c, s = unpack(kq, act, M, K)
    rc, rs = fp8.encode_rows(_np(X))
    np.testing.assert_array_equal(s, rs)
    np.testing.assert_array_equal(c, rc)
    L = kq.Fp8Layer(K, N)
    w, (Wd,) = packed(kq, L, weight(K, N, 0))
    Y = torch.zeros(M, N, device="cuda")
    kq.fp8_gemm(L, w, act, M, Y)
    y = _np(Y)
    assert np.all(np.isnan(y[1])) and np.all(np.isfinite(y[[0, 2, 3]]))


@pytest.mark.parametrize("K,N", [(32, 16), (128, 128), (160, 144), (1152, 400), (96, 1040)])
def test_prepare_weights_bit_exact(cuda_device, K, N):
    import w4a4_post_quantization_token_b200 as kq
    W, Wu = weight(K, N, 1), weight(K, N, 2)
    L = kq.Fp8Layer(K, N, gated=True)
    w = buf(kq.fp8_weights_bytes(L))
    kq.fp8_prepare_weights(L, W.cuda(), w, Wu.cuda())
    ns = -(-N // 128) * -(-K // 128)
    got = [buf(N * K), buf(ns), buf(N * K), buf(ns)]
    kq.fp8_weights_unpack(L, w, *got)
    for m, c, s in ((W, got[0], got[1]), (Wu, got[2], got[3])):
        rc, rs = fp8.encode_weight(_np(m))
        np.testing.assert_array_equal(c.cpu().numpy().reshape(N, K), rc)
        np.testing.assert_array_equal(s.cpu().numpy().reshape(rs.shape), rs)
    w2 = buf(kq.fp8_weights_bytes(L))
    kq.fp8_weights_pack(L, got[0], got[1], w2, got[2], got[3])
    got2 = [buf(N * K), buf(ns), buf(N * K), buf(ns)]
    kq.fp8_weights_unpack(L, w2, *got2)
    for a, b in zip(got, got2):
        np.testing.assert_array_equal(a.cpu().numpy(), b.cpu().numpy())


# ------------------------------------------------------------------------------- norm ----
@pytest.mark.parametrize("res", [None, "bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 32), (5, 160), (130, 1152), (3, 4096), (2, 6176), (2, 12288), (1, 32768)])
def test_rmsnorm_bit_exact(cuda_device, M, K, res):
    import torch
    import w4a4_post_quantization_token_b200 as kq
    rng = np.random.default_rng(K + M)
    X = tokens(M, K, K)
    X[0, :64] = 0
    gamma = (1 + 0.25 * rng.standard_normal(K)).astype(np.float32)
    R = round_ = None
    if res:
        R = torch.from_numpy(3 * rng.standard_normal((M, K)).astype(np.float32))
        R = R.to(torch.bfloat16) if res == "bf16" else R
        round_ = (lambda h: torch.from_numpy(h).to(torch.bfloat16).float().numpy()) if res == "bf16" else None
    act = buf(kq.fp8_act_bytes(K, M))
    Rg = None if R is None else R.clone().cuda()
    kq.fp8_rmsnorm_act(X.cuda(), _t(gamma), EPS, act, residual=Rg)
    y, h = fp8.rmsnorm(_np(X), gamma, EPS, None if R is None else _np(R), round_)
    rc, rs = fp8.encode_rows(y)
    c, s = unpack(kq, act, M, K)
    if res:
        np.testing.assert_array_equal(_np(Rg), h.astype(np.float64))
    np.testing.assert_array_equal(s, rs)
    np.testing.assert_array_equal(c, rc)


def test_rmsnorm_zero_and_overflowing_rows(cuda_device):
    """A row of zeros stays zero; a sum that leaves bf16 makes its row NaN and no other."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    M, K = 3, 256
    X = tokens(M, K, 9)
    X[0] = 0
    R = torch.zeros(M, K, dtype=torch.bfloat16)
    X[1, 5] = R[1, 5] = 3e38
    act = buf(kq.fp8_act_bytes(K, M))
    Rg = R.cuda()
    kq.fp8_rmsnorm_act(X.cuda(), torch.ones(K, device="cuda"), EPS, act, residual=Rg)
    c, s = unpack(kq, act, M, K)
    assert np.all(c[0] == 0) and np.all(s[0] == 0)
    assert np.isinf(_np(Rg)[1, 5]) and s[1, 0] == 0xFF
    assert not np.any(s[2] == 0xFF)


def test_pitched_rows_and_untouched_neighbours(cuda_device):
    """X, the residual and Y as column slices of wider tensors; nothing outside is written."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    M, K, N = 37, 160, 144
    wide = torch.full((M + 3, K + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    X = tokens(M, K, 1).cuda()
    wide[:M, 16:16 + K] = X
    R = torch.randn(M, K)
    wr = torch.full((M + 3, K + 32), 5.0, device="cuda")
    wr[:M, 8:8 + K] = R.cuda()
    gamma = torch.rand(K, device="cuda")
    a, b = buf(kq.fp8_act_bytes(K, M)), buf(kq.fp8_act_bytes(K, M))
    Rc = R.cuda()
    kq.fp8_rmsnorm_act(X, gamma, EPS, a, residual=Rc)
    kq.fp8_rmsnorm_act(wide[:M, 16:16 + K], gamma, EPS, b, residual=wr[:M, 8:8 + K])
    for u, v in zip(unpack(kq, a, M, K), unpack(kq, b, M, K)):
        np.testing.assert_array_equal(u, v)
    np.testing.assert_array_equal(_np(wr[:M, 8:8 + K]), _np(Rc))
    assert torch.all(wr[M:] == 5) and torch.all(wr[:, :8] == 5) and torch.all(wr[:, 8 + K:] == 5)
    L = kq.Fp8Layer(K, N)
    w, _ = packed(kq, L, weight(K, N, 4))
    for dt, flag, M2 in ((torch.float32, kq.OUT_F32, M), (torch.bfloat16, kq.OUT_BF16, M), (torch.bfloat16, kq.OUT_BF16, 300)):
        X2 = tokens(M2, K, 2).cuda()
        act = buf(kq.fp8_act_bytes(K, M2))
        Y = torch.empty(M2, N, dtype=dt, device="cuda")
        wy = torch.full((M2 + 5, N + 48), 3.0, dtype=dt, device="cuda")
        kq.fp8_linear(L, w, X2, Y, act, flag)
        kq.fp8_linear(L, w, X2, wy[:M2, 16:16 + N], act, flag)
        assert torch.equal(wy[:M2, 16:16 + N], Y)
        assert torch.all(wy[M2:] == 3) and torch.all(wy[:, :16] == 3) and torch.all(wy[:, 16 + N:] == 3)


# --------------------------------------------------------------------------- products ----
SHAPES = [(1, 32, 16), (1, 4096, 256), (3, 96, 48), (16, 512, 128), (17, 544, 144), (32, 1152, 272), (33, 128, 400),
          (64, 640, 128), (65, 2080, 256), (127, 160, 272), (128, 384, 128), (129, 1024, 144), (200, 12288, 160),
          (257, 1152, 528), (300, 96, 1040), (520, 736, 784), (1, 12288, 1040), (5, 8192, 640),
          (2100, 160, 2320), (1300, 640, 4112),         # several tiles for each CTA pair
          (20, 2304, 9488), (31, 12288, 144), (16, 160, 272),
          (65, 4096, 400), (100, 2080, 1936), (300, 1120, 144), (256, 12288, 528), (512, 8192, 656)]   # K shared by pairs


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear(cuda_device, M, K, N, out):
    import torch
    import w4a4_post_quantization_token_b200 as kq
    X, W = tokens(M, K, K + N), weight(K, N, M)
    L = kq.Fp8Layer(K, N)
    w, (Wd,) = packed(kq, L, W)
    act = buf(kq.fp8_act_bytes(K, M))
    Y = torch.full((M, N), float("nan"), dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    kq.fp8_linear(L, w, X.cuda(), Y, act, kq.OUT_BF16 if out == "bf16" else kq.OUT_F32)
    assert kq.fp8_last_device_error(act) == 0
    A = fp8.decode_rows(*fp8.encode_rows(_np(X)))
    ref = A @ Wd.T
    acc = accumulation(A, Wd)
    assert np.all(np.abs(_np(Y) - ref) <= HALF[out] * (np.abs(ref) + acc) + acc + 1e-37)


def gated_bound(z, u, zerr, uerr, kind):
    """|act'| <= 1.13 (GELU; SiLU 1.10) and fp32 evaluation of act within 2^-19 of |act| (exp and
    the quotient a few ulps, the exponent's rounding 2^-24 |z| log2 e with |z| <= 20 before act
    leaves the linear range)."""
    a = np.abs(fp8.activation(z, kind))
    return 1.13 * zerr * (np.abs(u) + uerr) + a * uerr + 2.0 ** -19 * a * np.abs(u)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("M,K,N", [(1, 32, 16), (2, 4096, 128), (16, 160, 144), (20, 512, 272), (64, 1152, 256),
                                   (65, 96, 400), (130, 2080, 272), (300, 640, 528), (1, 8192, 640), (1100, 160, 2080),
                                   (700, 544, 4016), (100, 4096, 528), (257, 2080, 160), (300, 8192, 800)])
def test_gated(cuda_device, M, K, N, kind):
    import torch
    import w4a4_post_quantization_token_b200 as kq
    X, W, Wu = tokens(M, K, K), weight(K, N, 1), weight(K, N, 2)
    L = kq.Fp8Layer(K, N, gated=True, activation=kind)
    w, (Wd, Wud) = packed(kq, L, W, Wu)
    act = buf(kq.fp8_act_bytes(K, M))
    A = fp8.decode_rows(*fp8.encode_rows(_np(X)))
    z, u = A @ Wd.T, A @ Wud.T
    ref = fp8.activation(z, kind) * u
    bound = gated_bound(z, u, accumulation(A, Wd), accumulation(A, Wud), kind)
    for out, dt, flag in (("f32", torch.float32, kq.OUT_F32), ("bf16", torch.bfloat16, kq.OUT_BF16)):
        Y = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
        kq.fp8_linear(L, w, X.cuda(), Y, act, flag)
        assert kq.fp8_last_device_error(act) == 0
        assert np.all(np.abs(_np(Y) - ref) <= HALF[out] * (np.abs(ref) + bound) + bound + 1e-37)
    if N % 32:
        return
    # 8-bit output: half a step of the E4M3 grid under the block's own scale, which holds the
    # block's largest value and is no larger than it needs to be
    h = buf(kq.fp8_act_bytes(N, M))
    kq.fp8_quantize_act(X.cuda(), act)
    kq.fp8_gated_act(L, w, act, M, h)
    c, s = unpack(kq, h, M, N)
    scale = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 128, 1)[:, :N]
    got = fp8.decode_rows(c, s)
    assert np.all(np.abs(got - ref) <= 2.0 ** -4 * (np.abs(ref) + bound) + 2.0 ** -10 * scale + bound)
    pad = np.zeros((M, s.shape[1] * 128))
    for sign in (1, -1):
        pad[:, :N] = np.abs(ref) + sign * bound
        top = pad.reshape(M, -1, 128).max(2)
        e = np.array([fp8.exponent_of(t) if t > 0 else -127 for t in top.ravel()]).reshape(top.shape) + 127
        assert np.all(s <= e) if sign == 1 else np.all(s >= e)


# ------------------------------------------------------------------- the block, whole ----
def make_ffn(kq, K, N, seed=0):
    G, D = kq.Fp8Layer(K, N, gated=True), kq.Fp8Layer(N, K)
    gw, (Wg, Wu) = packed(kq, G, weight(K, N, seed), weight(K, N, seed + 1))
    dw, (Wd,) = packed(kq, D, weight(N, K, seed + 2))
    return G, gw, D, dw, Wg, Wu, Wd


@pytest.mark.parametrize("res", [None, "bf16", "f32"])
@pytest.mark.parametrize("M,K,N", [(1, 256, 512), (9, 1152, 608), (100, 160, 288), (260, 512, 1056), (2, 2080, 288),
                                   (4, 1120, 160), (1, 12288, 64), (12, 1024, 160), (3, 32, 32)])
def test_ffn_is_its_parts(cuda_device, M, K, N, res):
    """The block gives what its three calls give, bit for bit, and is near the float64 chain."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    G, gw, D, dw, Wg, Wu, Wd = make_ffn(kq, K, N)
    X = tokens(M, K, 5)
    gamma = torch.rand(K) + 0.5
    R = None if res is None else torch.randn(M, K).to(torch.bfloat16 if res == "bf16" else torch.float32)
    R1, R2 = (None, None) if R is None else (R.clone().cuda(), R.clone().cuda())
    ws = buf(kq.fp8_ffn_bytes(G, D, M))
    Y = torch.empty(M, K, device="cuda")
    kq.fp8_ffn(G, gw, D, dw, X.cuda(), gamma.cuda(), EPS, Y, ws, residual=R1)
    assert kq.fp8_last_device_error(ws) == 0
    a, h = buf(kq.fp8_act_bytes(K, M)), buf(kq.fp8_act_bytes(N, M))
    Y2 = torch.empty(M, K, device="cuda")
    kq.fp8_rmsnorm_act(X.cuda(), gamma.cuda(), EPS, a, residual=R2)
    kq.fp8_gated_act(G, gw, a, M, h)
    kq.fp8_gemm(D, dw, h, M, Y2)
    assert torch.equal(Y, Y2) and (R is None or torch.equal(R1, R2))
    round_ = (lambda v: torch.from_numpy(v).to(torch.bfloat16).float().numpy()) if res == "bf16" else None
    y, _ = fp8.rmsnorm(_np(X), gamma.numpy(), EPS, None if R is None else _np(R), round_)
    A = fp8.decode_rows(*fp8.encode_rows(y))
    H = fp8.gated(A, Wg, Wu)
    ref = fp8.decode_rows(*fp8.encode_rows(H)) @ Wd.T
    # H is off by d = (K / 32) 2^-23 or so; a share 2 d / 2^-4 of its codes sits that close to a
    # border and moves by a step of 2^-3: sqrt(32 d) / 8 relative, at most 4e-3 for K = 1152
    d = (K / 32 + 8) * 2.0 ** -23
    err = np.linalg.norm(_np(Y) - ref) / np.linalg.norm(ref)
    assert err <= np.sqrt(32 * d) / 8 + 1e-6


@pytest.mark.parametrize("M", [3, 70])
def test_buffers_on_16_byte_boundaries(cuda_device, M):
    """Every device pointer 16 bytes past a 256-byte boundary gives the same results."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    K, N = 288, 160

    def off(t):
        raw = torch.zeros(t.numel() * t.element_size() + 16, dtype=torch.uint8, device="cuda")
        v = raw[16:].view(t.dtype).view(t.shape)
        assert v.data_ptr() % 256 == 16
        return v.copy_(t)

    got = []
    for move in (lambda t: t, off):
        X, R, g = move(tokens(M, K, 1).cuda()), move(torch.ones(M, K, device="cuda")), move(torch.full((K,), 0.5, device="cuda"))
        L = kq.Fp8Layer(K, N)
        w = move(buf(kq.fp8_weights_bytes(L)))
        kq.fp8_prepare_weights(L, move(weight(K, N, 2).cuda()), w)
        act = move(buf(kq.fp8_act_bytes(K, M)))
        V, F = move(torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")), move(torch.zeros(M, K, device="cuda"))
        Y, Z = move(torch.zeros(M, N, device="cuda")), move(torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"))
        kq.fp8_quantize_act(X, act)
        kq.fp8_act_unpack(K, act, M, values=V)
        kq.fp8_rmsnorm_act(X, g, EPS, act, residual=R)
        kq.fp8_act_unpack(K, act, M, values=F)
        kq.fp8_gemm(L, w, act, M, Y)
        kq.fp8_linear(L, w, X, Z, act, kq.OUT_BF16)
        got.append([t.clone() for t in (V, R, F, Y, Z)])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_ffn_without_norm(cuda_device):
    import torch
    import w4a4_post_quantization_token_b200 as kq
    M, K, N = 21, 256, 160
    G, gw, D, dw, *_ = make_ffn(kq, K, N)
    X = tokens(M, K, 6).cuda()
    ws = buf(kq.fp8_ffn_bytes(G, D, M))
    Y, Y2 = (torch.empty(M, K, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kq.fp8_ffn(G, gw, D, dw, X, None, EPS, Y, ws, kq.OUT_BF16)
    a, h = buf(kq.fp8_act_bytes(K, M)), buf(kq.fp8_act_bytes(N, M))
    kq.fp8_quantize_act(X, a)
    kq.fp8_gated_act(G, gw, a, M, h)
    kq.fp8_gemm(D, dw, h, M, Y2, kq.OUT_BF16)
    assert torch.equal(Y, Y2)


@pytest.mark.parametrize("M", [1, 40, 600])
def test_graph_replay_and_side_stream(cuda_device, M):
    """A captured block replays on new inputs; a block on another stream gives the same."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    K, N = 512, 544
    G, gw, D, dw, *_ = make_ffn(kq, K, N)
    gamma = torch.rand(K, device="cuda")
    X, R = tokens(M, K, 1).cuda(), torch.randn(M, K, device="cuda")
    X0, R0 = X.clone(), R.clone()
    ws = buf(kq.fp8_ffn_bytes(G, D, M))
    Y = torch.empty(M, K, device="cuda")
    kq.fp8_ffn(G, gw, D, dw, X, gamma, EPS, Y, ws, residual=R)
    torch.cuda.synchronize()
    want, wantR = Y.clone(), R.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kq.fp8_ffn(G, gw, D, dw, X, gamma, EPS, Y, ws, residual=R)
    for k in range(3):
        X2, R2 = tokens(M, K, 10 + k).cuda(), torch.randn(M, K, device="cuda")
        X.copy_(X2); R.copy_(R2)
        g.replay()
        Ye, Re, wse = torch.empty_like(Y), R2.clone(), buf(ws.numel())
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        kq.fp8_ffn(G, gw, D, dw, X2, gamma, EPS, Ye, wse, residual=Re, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        assert torch.equal(Y, Ye) and torch.equal(R, Re)
    X.copy_(X0); R.copy_(R0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, want) and torch.equal(R, wantR)


def test_calls_follow_one_another(cuda_device):
    """Many dependent calls on the same buffers without a wait between them."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    K = N = 512
    L = kq.Fp8Layer(K, N)
    w, _ = packed(kq, L, weight(K, N, 3))
    outs = []
    for wait in (True, False):
        X = tokens(24, K, 8).cuda()
        act = buf(kq.fp8_act_bytes(K, 24))
        Y = torch.empty(24, N, dtype=torch.bfloat16, device="cuda")
        for _ in range(30):
            kq.fp8_linear(L, w, X, Y, act, kq.OUT_BF16)
            X, Y = Y, X
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        outs.append(X.clone())
    assert torch.equal(*outs) and torch.isfinite(outs[0].float()).all()


def test_repacked_weights_are_read_at_once(cuda_device):
    """New weights written into the same buffer directly before a call are the ones it uses."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    M, K, N = 8, 1024, 512
    L = kq.Fp8Layer(K, N)
    X = tokens(M, K, 2).cuda()
    act = buf(kq.fp8_act_bytes(K, M))
    kq.fp8_quantize_act(X, act)
    filled = act.clone()
    parts = [[_t(a) for a in fp8.encode_weight(_np(weight(K, N, s)))] for s in (1, 2)]
    want = []
    for p in parts:
        w = buf(kq.fp8_weights_bytes(L))
        kq.fp8_weights_pack(L, *p, w)
        torch.cuda.synchronize()
        Y = torch.empty(M, N, device="cuda")
        kq.fp8_linear(L, w, X, Y, act)
        want.append(Y)
    w = buf(kq.fp8_weights_bytes(L))
    for _ in range(10):
        for p, y in zip(parts, want):
            Y = torch.empty(M, N, device="cuda")
            kq.fp8_weights_pack(L, *p, w)
            kq.fp8_gemm(L, w, filled, M, Y)
            Y2 = torch.empty(M, N, device="cuda")
            kq.fp8_weights_pack(L, *p, w)
            kq.fp8_linear(L, w, X, Y2, act)
            torch.cuda.synchronize()
            assert torch.equal(Y, y) and torch.equal(Y2, y)


@pytest.mark.parametrize("M", [1, 7, 40, 90])
def test_output_on_the_input(cuda_device, M):
    """Y in X's own buffer, and Y as other columns of the tensor that X is a part of."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    K = N = 512
    L = kq.Fp8Layer(K, N)
    w, _ = packed(kq, L, weight(K, N, 1))
    X = tokens(M, K, 3).cuda()
    act = buf(kq.fp8_act_bytes(K, M))
    want = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    kq.fp8_linear(L, w, X, want, act, kq.OUT_BF16)
    inplace = X.clone()
    kq.fp8_linear(L, w, inplace, inplace, act, kq.OUT_BF16)
    both = torch.cat([X, torch.zeros_like(X)], 1)
    kq.fp8_linear(L, w, both[:, :K], both[:, K:], act, kq.OUT_BF16)
    assert torch.equal(inplace, want) and torch.equal(both[:, K:], want) and torch.equal(both[:, :K], X)
    G, gw, D, dw, *_ = make_ffn(kq, K, 544)
    gamma = torch.rand(K, device="cuda")
    ws = buf(kq.fp8_ffn_bytes(G, D, M))
    kq.fp8_ffn(G, gw, D, dw, X, gamma, EPS, want, ws, kq.OUT_BF16)
    inplace = X.clone()
    kq.fp8_ffn(G, gw, D, dw, inplace, gamma, EPS, inplace, ws, kq.OUT_BF16)
    assert torch.equal(inplace, want)
    R = torch.randn(M, K, device="cuda").to(torch.bfloat16)
    R1, R2 = R.clone(), R.clone()
    kq.fp8_ffn(G, gw, D, dw, X, gamma, EPS, want, ws, kq.OUT_BF16, residual=R1)
    kq.fp8_ffn(G, gw, D, dw, X, gamma, EPS, X, ws, kq.OUT_BF16, residual=R2)
    assert torch.equal(X, want) and torch.equal(R1, R2) and not torch.equal(R1, R)


@pytest.mark.parametrize("M", [2, 50, 130])
def test_two_streams_at_once(cuda_device, M):
    """Blocks on two streams, each with a workspace of its own, do not disturb each other."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    K, N = 1024, 2048
    G, gw, D, dw, *_ = make_ffn(kq, K, N)
    gamma = torch.rand(K, device="cuda")
    Xs = [tokens(M, K, 20 + i).cuda() for i in range(2)]
    want = []
    for X in Xs:
        Y = torch.empty(M, K, device="cuda")
        kq.fp8_ffn(G, gw, D, dw, X, gamma, EPS, Y, buf(kq.fp8_ffn_bytes(G, D, M)))
        want.append(Y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Xs]
    got = [torch.empty(20, M, K, device="cuda") for _ in Xs]
    spaces = [buf(kq.fp8_ffn_bytes(G, D, M)) for _ in Xs]
    torch.cuda.synchronize()
    for k in range(20):
        for i, X in enumerate(Xs):
            kq.fp8_ffn(G, gw, D, dw, X, gamma, EPS, got[i][k], spaces[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert kq.fp8_last_device_error(spaces[i]) == 0
        assert all(torch.equal(got[i][k], want[i]) for k in range(20))


def test_two_graphs_share_a_workspace(cuda_device):
    """Two captured layers that use one workspace, replayed in turn on one stream."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    cases = []
    act = buf(max(kq.fp8_act_bytes(1024, 70), kq.fp8_act_bytes(2048, 5)))
    for M, K, N in ((70, 1024, 512), (5, 2048, 256)):
        L = kq.Fp8Layer(K, N)
        w, _ = packed(kq, L, weight(K, N, K))
        X, Y = tokens(M, K, M).cuda(), torch.empty(M, N, device="cuda")
        kq.fp8_linear(L, w, X, Y, act)
        torch.cuda.synchronize()
        want = Y.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kq.fp8_linear(L, w, X, Y, act)
        cases.append((g, Y, want, X, w))
    for _ in range(5):
        for g, Y, *_ in cases:
            Y.zero_()
            g.replay()
        torch.cuda.synchronize()
        for _, Y, want, *_ in cases:
            assert torch.equal(Y, want)


@pytest.mark.parametrize("M", [2, 200])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gate_far_from_zero(cuda_device, M, kind):
    """Gates of +-1e4 and beyond: the activation is its limit (0 or the gate itself), never NaN."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    K, N = 64, 128
    X = torch.zeros(M, K, dtype=torch.bfloat16)
    X[0::2, 0], X[1::2, 0], X[:, 1] = 1e4, -1e4, 2.0
    W, Wu = torch.zeros(K, N, dtype=torch.bfloat16), torch.zeros(K, N, dtype=torch.bfloat16)
    W[0] = 8.0
    Wu[1] = 1.0
    L = kq.Fp8Layer(K, N, gated=True, activation=kind)
    w, (Wd, Wud) = packed(kq, L, W, Wu)
    Y = torch.empty(M, N, device="cuda")
    kq.fp8_linear(L, w, X.cuda(), Y, buf(kq.fp8_act_bytes(K, M)))
    A = fp8.decode_rows(*fp8.encode_rows(_np(X)))
    z, u = A @ Wd.T, A @ Wud.T
    assert np.all(np.abs(z) > 7e4)
    np.testing.assert_allclose(_np(Y), np.where(z > 0, z, 0) * u, rtol=2.0 ** -18, atol=1e-30)


@pytest.mark.parametrize("M", [8, 200])
def test_silu_in_fp32(cuda_device, M):
    """fp32 outputs of a gated layer whose two products are exact hold the activation to a few fp32
    roundings, down to gates where it leaves the normal range.

    exp(-|z|) is within 2 ulps (2^-22), the sum 1 + exp within 2^-24 and half of the exponential's
    error (2^-23), the product z exp (for z < 0) within 2^-22 and a rounding of 2^-24, the quotient
    within 2 ulps (2^-22), the product with u within 2^-24: (4 + 1 + 2 + 1 + 4 + 1) 2^-24 together.
    Where the exponential is subnormal its 2 ulps are 2^-148, times z; the product there is half of
    2^-149 off, the quotient 2 of them, both times u, and the result another half."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    K, N = 32, 128
    n = torch.arange(N)
    X, W, Wu = torch.zeros(M, K), torch.zeros(K, N), torch.zeros(K, N)
    X[:, 0], X[:, 1] = (torch.arange(M) % 8 + 1).float(), 1.0
    sign = 1.0 - 2.0 * (n % 2)
    W[0] = sign * (8 + n // 2 % 8) * torch.exp2((n // 16 % 4).float()) / 8      # 1 .. 15
    W[1] = sign * (n % 5) / 8
    Wu[1] = 3.0
    X, W, Wu = (t.to(torch.bfloat16) for t in (X, W, Wu))
    L = kq.Fp8Layer(K, N, gated=True)
    w, (Wd, Wud) = packed(kq, L, W, Wu)
    Y = torch.empty(M, N, device="cuda")
    kq.fp8_linear(L, w, X.cuda(), Y, buf(kq.fp8_act_bytes(K, M)))
    A = fp8.decode_rows(*fp8.encode_rows(_np(X)))
    z, u = A @ Wd.T, A @ Wud.T
    np.testing.assert_array_equal(z, _np(X) @ _np(W))       # nothing was rounded on the way
    assert z.min() < -100 and z.max() > 100 and np.all(u == 3)
    ref = fp8.activation(z, "silu") * u
    bound = 13 * 2.0 ** -24 * np.abs(ref) + 2.0 ** -149 * ((2 * np.abs(z) + 2.5) * u + 1)
    assert np.all(np.abs(_np(Y) - ref) <= bound)


def run_short_of_a_k_tile(kq, M, K, N, how, k_tile):
    """The product with a k-tile's weights never loaded, then the ordinary one, on outputs filled with 0xAA
    bytes: (bytes after the first, bytes after the second, 0xAA everywhere), status, seconds."""
    import time

    import torch
    gated, blocks = how in ("8bit", "gated f32"), how == "8bit"
    out_dtype = kq.OUT_F32 if "f32" in how else kq.OUT_BF16
    L = kq.Fp8Layer(K, N, gated=gated)
    w = buf(kq.fp8_weights_bytes(L))
    W = [(torch.randn(K, N, device="cuda") / K ** 0.5).bfloat16() for _ in range(1 + gated)]
    kq.fp8_prepare_weights(L, W[0], w, W[1] if gated else None)
    X, act = tokens(M, K, 3).cuda(), buf(kq.fp8_act_bytes(K, M))
    kq.fp8_quantize_act(X, act)
    dt = torch.float32 if "f32" in how else torch.bfloat16
    out = torch.full((kq.fp8_act_bytes(N, M) if blocks else dt.itemsize * M * N,), 0xAA, dtype=torch.uint8, device="cuda")
    Y = None if blocks else out.view(dt).view(M, N)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    kq.fp8_debug_wait_timeout(L, w, act, M, k_tile, 5000, X=X if how == "fused" else None, Y=Y,
                              out_act=out if blocks else None, out_dtype=out_dtype)
    status = kq.fp8_last_device_error(act)
    seconds = time.perf_counter() - t0

    def parts():
        if blocks:
            return [torch.from_numpy(a) for a in unpack(kq, out, M, N)]
        return [out.view(M, -1).cpu()]

    short = parts()
    if blocks:
        kq.fp8_gated_act(L, w, act, M, out)
    elif how == "fused":
        kq.fp8_linear(L, w, X, Y, act, out_dtype)
    else:
        kq.fp8_gemm(L, w, act, M, Y, out_dtype)
    assert kq.fp8_last_device_error(act) == 0
    return short, parts(), status, seconds


@pytest.mark.parametrize("how,M,K,N", [
    ("gemm", 5, 640, 9488), ("gemm", 5, 8192, 640), ("gemm", 20, 12288, 144), ("gemm", 64, 2560, 9488), ("gemm", 64, 4096, 400),
    ("fused", 1, 4096, 256), ("fused", 20, 512, 272), ("fused", 2, 1152, 9488),
    ("8bit", 2, 4096, 128), ("8bit", 20, 8192, 288), ("8bit", 64, 4096, 544), ("8bit", 9, 1536, 9600), ("8bit", 40, 1536, 9600),
    ("gemm", 300, 1280, 528), ("gemm", 65, 4096, 400), ("gemm", 256, 12288, 528), ("gemm", 520, 1152, 656),
    ("8bit", 130, 2080, 288), ("8bit", 1100, 160, 2080)])
def test_a_wait_that_runs_out_leaves_the_outputs(cuda_device, how, M, K, N):
    """Whichever k-tile does not come, the call ends in time, reports it, and stores none of the sums
    that lack it; the context and the workspaces stay usable."""
    import w4a4_post_quantization_token_b200 as kq
    for k in (0, 1):
        short, whole, status, seconds = run_short_of_a_k_tile(kq, M, K, N, how, k)
        assert status == kq.ERR_DEVICE_TIMEOUT and 0.005 <= seconds < 2
        for s, w in zip(short, whole):
            assert bool((s == 0xAA).all()) and not bool((w == s).all())


@pytest.mark.parametrize("how,M,K,N,k", [("gemm", 2100, 160, 9296, 2), ("gemm", 2100, 160, 9296, 5), ("gemm", 1300, 640, 8208, 7),
                                         ("8bit", 1100, 160, 4064, 3), ("8bit", 2300, 544, 4064, 11)])
def test_tiles_before_a_wait_that_runs_out(cuda_device, how, M, K, N, k):
    """Several tiles for each CTA pair: those whose sums came before are stored, right, and no others."""
    import w4a4_post_quantization_token_b200 as kq
    short, whole, status, seconds = run_short_of_a_k_tile(kq, M, K, N, how, k)
    assert status == kq.ERR_DEVICE_TIMEOUT and 0.005 <= seconds < 2
    for s, w in zip(short, whole):
        left = s == 0xAA
        assert bool((left | (s == w)).all()) and 0.05 < left.double().mean() < 0.95


def test_a_k_tile_past_the_last_is_not_missed(cuda_device):
    import w4a4_post_quantization_token_b200 as kq
    for how, M in (("gemm", 5), ("8bit", 130), ("fused", 3), ("gemm", 200)):
        short, whole, status, _ = run_short_of_a_k_tile(kq, M, 640, 288, how, 1 << 40)
        assert status == 0 and all(bool((s == w).all()) for s, w in zip(short, whole))


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("M,K,N", [(17, 32, 32), (20, 512, 288), (31, 8192, 672), (32, 2080, 9632), (33, 64, 96), (48, 160, 416),
                                   (64, 4096, 544), (64, 1152, 9568), (12, 4096, 160), (16, 96, 9504)])
def test_8bit_output_of_few_tokens(cuda_device, M, K, N, kind):
    """Every token tile of the few-token kernel, K whole and split, last blocks of 32 to 96 outputs: codes
    within half a step of E4M3 under the block's own scale, which is the smallest that holds the
    block's largest value; nothing past the workspace is written."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    X, W, Wu = tokens(M, K, K + 1), weight(K, N, 3), weight(K, N, 4)
    L = kq.Fp8Layer(K, N, gated=True, activation=kind)
    w, (Wd, Wud) = packed(kq, L, W, Wu)
    act = buf(kq.fp8_act_bytes(K, M))
    A = fp8.decode_rows(*fp8.encode_rows(_np(X)))
    z, u = A @ Wd.T, A @ Wud.T
    ref = fp8.activation(z, kind) * u
    bound = gated_bound(z, u, accumulation(A, Wd), accumulation(A, Wud), kind)
    h = torch.full((kq.fp8_act_bytes(N, M + 64),), 0xAA, dtype=torch.uint8, device="cuda")
    kq.fp8_quantize_act(X.cuda(), act)
    kq.fp8_gated_act(L, w, act, M, h)
    assert kq.fp8_last_device_error(act) == 0
    c, s = unpack(kq, h, M, N)
    scale = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 128, 1)[:, :N]
    assert np.all(np.abs(fp8.decode_rows(c, s) - ref) <= 2.0 ** -4 * (np.abs(ref) + bound) + 2.0 ** -10 * scale + bound)
    pad = np.zeros((M, s.shape[1] * 128))
    for sign in (1, -1):
        pad[:, :N] = np.abs(ref) + sign * bound
        top = pad.reshape(M, -1, 128).max(2)
        e = np.array([fp8.exponent_of(t) if t > 0 else -127 for t in top.ravel()]).reshape(top.shape) + 127
        assert np.all(s <= e) if sign == 1 else np.all(s >= e)
    assert bool((h[kq.fp8_act_bytes(N, M):] == 0xAA).all())


def test_more_outputs_than_65535_blocks(cuda_device):
    """8.4 million outputs, 2049 copies of the same 4096: each copy's codes, scales and outputs are alike."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    K, n, copies = 32, 4096, 2049
    W = weight(K, n, 5).cuda()
    small, big = kq.Fp8Layer(K, n), kq.Fp8Layer(K, n * copies)
    ws, wb = buf(kq.fp8_weights_bytes(small)), buf(kq.fp8_weights_bytes(big))
    kq.fp8_prepare_weights(small, W, ws)
    kq.fp8_prepare_weights(big, W.repeat(1, copies), wb)
    cs, ss, cb, sb = buf(n * K), buf(n // 128), buf(n * K * copies), buf(n // 128 * copies)
    kq.fp8_weights_unpack(small, ws, cs, ss)
    kq.fp8_weights_unpack(big, wb, cb, sb)
    assert torch.equal(cb.view(copies, -1), cs.expand(copies, -1)) and torch.equal(sb.view(copies, -1), ss.expand(copies, -1))
    for M in (1, 66):
        X, act = tokens(M, K, 6).cuda(), buf(kq.fp8_act_bytes(K, M))
        Ys, Yb = (torch.zeros(M, w, dtype=torch.bfloat16, device="cuda") for w in (n, n * copies))
        kq.fp8_linear(small, ws, X, Ys, act, kq.OUT_BF16)
        kq.fp8_linear(big, wb, X, Yb, act, kq.OUT_BF16)
        assert kq.fp8_last_device_error(act) == 0
        assert torch.equal(Yb.view(M, copies, n), Ys[:, None].expand(M, copies, n)) and bool((Ys != 0).any())


def test_rows_of_more_than_2_28_features_are_refused(cuda_device):
    import torch
    import w4a4_post_quantization_token_b200 as kq
    K = (1 << 28) + 32
    with pytest.raises(kq.KQError):
        kq.fp8_quantize_act(torch.empty(1, K, dtype=torch.bfloat16, device="cuda"), buf(1 << 20))


LONG_SUMS = [("f32", 8, 24576, 9600), ("f32", 30, 24576, 9600), ("f32", 60, 24576, 9600), ("f32", 20, 66560, 272), ("f32", 300, 24576, 1040),
             ("f32", 300, 24576, 9616), ("f32", 1000, 16416, 4112), ("f32", 70, 35872, 144), ("gated f32", 8, 24576, 9600),
             ("gated f32", 30, 24576, 9600), ("gated f32", 60, 24576, 9600), ("gated f32", 2, 34816, 144), ("gated f32", 300, 24576, 1040),
             ("gated f32", 600, 8224, 9616)]


@pytest.mark.parametrize("kind,M,K,N", [(k, *c[1:]) for c in LONG_SUMS for k in (("silu", "gelu") if "gated" in c[0] else (None,))])
def test_fp32_outputs_of_long_sums(cuda_device, kind, M, K, N):
    """fp32 outputs stay within 1e-6, eight fp32 roundings, of float64 (relative norm) however long K is.

    A piece of the sum (8192 inputs, 4096 of a gated layer) is 7e-7 or 5e-7 off as the tensor core
    accumulates it; pieces of random signs add up like their errors do, so that the whole is off by as
    much, and by 2^-24 for each addition (8 at most here, 2e-7 together in the norm). Sums in one
    piece would be 2.6e-6 and 5e-6 off at 24576."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    gated = kind is not None
    L = kq.Fp8Layer(K, N, gated=gated, activation=kind or "silu")
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K)
    w = buf(kq.fp8_weights_bytes(L))
    Ws = [(torch.randn(K, N, generator=g, device="cuda") / K ** 0.5).bfloat16() for _ in range(1 + gated)]
    kq.fp8_prepare_weights(L, Ws[0], w, Ws[1] if gated else None)
    X, act = torch.randn(M, K, generator=g, device="cuda").bfloat16(), buf(kq.fp8_act_bytes(K, M))
    Y = torch.empty(M, N, device="cuda")
    kq.fp8_linear(L, w, X, Y, act)
    assert kq.fp8_last_device_error(act) == 0
    kq.fp8_quantize_act(X, act)
    A = torch.empty(M, K, device="cuda")
    kq.fp8_act_unpack(K, act, M, values=A)
    parts = [buf(N * K), buf(-(-N // 128) * -(-K // 128)), buf(N * K), buf(-(-N // 128) * -(-K // 128))]
    kq.fp8_weights_unpack(L, w, *parts[:2 + 2 * gated])
    z = []
    for c, s in (parts[:2], parts[2:])[:1 + gated]:
        V = c.view(torch.float8_e4m3fn).view(N, K).double()
        V *= torch.exp2(s.double() - 127).view(-(-N // 128), -1).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        z.append(A.double() @ V.T)
    ref = z[0]
    if gated:
        ref = (z[0] * torch.sigmoid(z[0]) if kind == "silu" else 0.5 * z[0] * torch.erfc(-z[0] / 2 ** 0.5)) * z[1]
    assert float((Y.double() - ref).norm() / ref.norm()) < 1e-6


@pytest.mark.parametrize("how,M,K,N,ks", [
    ("f32", 8, 24576, 9600, (3, 64, 191)), ("f32", 60, 24576, 9600, (64,)), ("f32", 20, 66560, 272, (64,)),
    ("gated f32", 30, 24576, 9600, (32, 100)), ("gated f32", 2, 34816, 144, (33,)), ("f32", 300, 24576, 9616, (64, 191)),
    ("gated f32", 600, 8224, 9616, (32, 64)), ("f32", 70, 35872, 144, (64, 69))])
def test_a_wait_that_runs_out_in_a_long_sum(cuda_device, how, M, K, N, ks):
    """The same in the first piece of a sum, at the start of another, and in the last."""
    import w4a4_post_quantization_token_b200 as kq
    for k in ks:
        short, whole, status, seconds = run_short_of_a_k_tile(kq, M, K, N, how, k)
        assert status == kq.ERR_DEVICE_TIMEOUT and seconds < 2
        for s, w in zip(short, whole):
            assert bool((s == 0xAA).all()) and not bool((w == s).all())


@pytest.mark.parametrize("kind,M,K,N", [(None, 4096, 256, 9216), (None, 2300, 96, 9600), (None, 3000, 288, 6160), (None, 2600, 12320, 9216),
                                        ("silu", 4096, 256, 4608), ("gelu", 2300, 96, 4112), ("silu", 1100, 8224, 9600)])
def test_accumulators_change_hands(cuda_device, kind, M, K, N):
    """Many tiles for each CTA pair with fp32 outputs, the epilogue that stores most, next to short sums, so
    that MMAs wait for accumulators to be read: every output right, and alike in 40 runs."""
    import torch
    import w4a4_post_quantization_token_b200 as kq
    L = kq.Fp8Layer(K, N, gated=kind is not None, activation=kind or "silu")
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    w, act = buf(kq.fp8_weights_bytes(L)), buf(kq.fp8_act_bytes(K, M))
    Ws = [(torch.randn(K, N, generator=g, device="cuda") / K ** 0.5).bfloat16() for _ in range(1 + L.gated)]
    kq.fp8_prepare_weights(L, Ws[0], w, Ws[1] if L.gated else None)
    kq.fp8_quantize_act(torch.randn(M, K, generator=g, device="cuda").bfloat16(), act)
    A = torch.empty(M, K, device="cuda")
    kq.fp8_act_unpack(K, act, M, values=A)
    ns = -(-N // 128) * -(-K // 128)
    parts = [buf(N * K), buf(ns), buf(N * K), buf(ns)]
    kq.fp8_weights_unpack(L, w, *parts[:2 + 2 * L.gated])
    z, acc = [], []
    for c, s in (parts[:2], parts[2:])[:1 + L.gated]:
        V = c.view(torch.float8_e4m3fn).view(N, K).double()
        V *= torch.exp2(s.double() - 127).view(-(-N // 128), -1).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        z.append(A.double() @ V.T)
        acc.append((K / 32 + 2) * 2.0 ** -23 * (A.double().abs() @ V.abs().T))
    ref, bound = z[0], acc[0]
    if L.gated:                                             # gated_bound, on the device
        a = z[0] * torch.sigmoid(z[0]) if kind == "silu" else 0.5 * z[0] * torch.erfc(-z[0] / 2 ** 0.5)
        ref = a * z[1]
        bound = 1.13 * acc[0] * (z[1].abs() + acc[1]) + a.abs() * acc[1] + 2.0 ** -19 * a.abs() * z[1].abs()
    bound = HALF["f32"] * (ref.abs() + bound) + bound + 1e-37
    want = torch.full((M, N), float("nan"), device="cuda")
    kq.fp8_gemm(L, w, act, M, want)
    assert bool(((want.double() - ref).abs() <= bound).all())
    Y = torch.empty_like(want)
    for _ in range(40):
        Y.fill_(float("nan"))
        kq.fp8_gemm(L, w, act, M, Y)
        assert torch.equal(Y, want)
    assert kq.fp8_last_device_error(act) == 0
