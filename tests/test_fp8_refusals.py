"""The 8-bit entry points refuse bad arguments on the host, before any CUDA call."""
import ctypes

import pytest
import torch

import w4a4_post_quantization_token_b200 as kq

OK = ctypes.c_void_p(0x100000)
OK2 = ctypes.c_void_p(0x900000)
ODD = ctypes.c_void_p(0x100008)
BIG = 1 << 40
lib = kq.lib


def L(K=64, N=64, gated=False):
    return kq.Fp8Layer(K, N, gated)


@pytest.mark.parametrize("K,N,status", [(0, 64, 1), (64, -16, 1), (48, 64, 2), (64, 40, 2)])
def test_shapes(K, N, status):
    d = L(K, N)
    assert kq.fp8_weights_bytes(d) == 0
    assert lib.kq_fp8_gemm(d.desc, OK, OK, 4, OK, 64, 0, None) == status
    assert lib.kq_fp8_prepare_weights(d.desc, OK, None, OK, None) == status
    assert lib.kq_fp8_weights_pack(d.desc, OK, OK, None, None, OK, None) == status


def test_descriptor_values():
    d = L()
    d._desc.gated = 2
    assert kq.fp8_weights_bytes(d) == 0
    d = L()
    d._desc.activation = 5
    assert kq.fp8_weights_bytes(d) == 0
    with pytest.raises(KeyError):
        kq.Fp8Layer(64, 64, True, "tanh")


def test_sizes():
    assert kq.fp8_act_bytes(64, 0) == 0 and kq.fp8_act_bytes(40, 4) == 0 and kq.fp8_act_bytes(0, 4) == 0
    assert kq.fp8_act_bytes(1152, 300) >= 300 * 1152 + 300 * 9
    assert kq.fp8_act_bytes(65536, 100000) > 65536 * 100000            # past 32 bits
    assert kq.fp8_weights_bytes(L(1152, 4608, True)) >= 2 * 1152 * 4608
    g, d = L(64, 96, True), L(96, 64)
    assert kq.fp8_ffn_bytes(g, d, 3) == kq.fp8_act_bytes(64, 3) + kq.fp8_act_bytes(96, 3)
    assert kq.fp8_ffn_bytes(g, d, 0) == 0 and kq.fp8_ffn_bytes(d, g, 3) == 0
    assert kq.fp8_ffn_bytes(g, L(64, 64), 3) == 0
    assert kq.fp8_ffn_bytes(L(64, 48, True), L(48, 64), 3) == 0         # 48 is no K of a layer


def quant(K=64, X=OK, ldx=64, M=4, act=OK, n=BIG):
    return lib.kq_fp8_quantize_act(K, X, ldx, M, act, n, None)


def test_quantize():
    assert quant(K=0) == 1 and quant(K=40) == 2
    assert quant(X=None) == 1 and quant(act=None) == 1 and quant(M=0) == 1 and quant(M=-1) == 1
    assert quant(ldx=63) == 1 and quant(ldx=68) == 3
    assert quant(X=ODD) == 3 and quant(act=ODD) == 3
    assert quant(n=kq.fp8_act_bytes(64, 4) - 1) == 5


def norm(K=64, X=OK, ldx=64, r=OK2, ldr=64, dt=0, g=OK, eps=1e-6, M=4, act=OK, n=BIG):
    return lib.kq_fp8_rmsnorm_act(K, X, ldx, r, ldr, dt, g, eps, M, act, n, None)


def test_rmsnorm():
    assert norm(K=40) == 2 and norm(K=32800, ldx=32800, ldr=32800) == 2
    assert norm(g=None) == 1 and norm(g=ODD) == 3
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert norm(eps=eps) == 1
    assert norm(dt=2) == 1 and norm(ldr=32) == 1 and norm(ldr=66) == 3 and norm(ldr=68, dt=1) == 3
    assert norm(r=ODD) == 3 and norm(X=None) == 1 and norm(M=0) == 1 and norm(n=10) == 5


def test_gemm_and_linear():
    d = L()
    g = lambda w=OK, a=OK2, M=4, Y=OK, ldy=64, dt=0: lib.kq_fp8_gemm(d.desc, w, a, M, Y, ldy, dt, None)
    assert g(w=None) == 1 and g(a=None) == 1 and g(M=0) == 1 and g(Y=None) == 1 and g(dt=2) == 1
    assert g(ldy=63) == 1 and g(ldy=66) == 3 and g(ldy=68, dt=1) == 3
    assert g(w=ODD) == 3 and g(a=ODD) == 3 and g(Y=ODD) == 3
    f = lambda w=OK, X=OK, ldx=64, M=4, Y=OK, ldy=64, dt=0, a=OK2, n=BIG: \
        lib.kq_fp8_linear(d.desc, w, X, ldx, M, Y, ldy, dt, a, n, None)
    assert f(w=None) == 1 and f(X=None) == 1 and f(ldx=32) == 1 and f(M=0) == 1 and f(dt=3) == 1
    assert f(n=64) == 5 and f(X=ODD) == 3 and f(w=ODD) == 3 and f(a=ODD) == 3


def test_gated():
    d, plain = L(64, 64, True), L()
    h = lambda d=d, w=OK, a=OK, M=4, o=OK2, n=BIG: lib.kq_fp8_gated_act(d.desc, w, a, M, o, n, None)
    assert h(d=plain) == 1 and h(w=None) == 1 and h(a=None) == 1 and h(o=None) == 1 and h(M=0) == 1
    assert h(a=OK2) == 1                                               # in place
    assert h(d=L(64, 48, True)) == 2 and h(o=ODD) == 3 and h(n=8) == 5
    assert lib.kq_fp8_prepare_weights(d.desc, OK, None, OK, None) == 1
    assert lib.kq_fp8_prepare_weights(plain.desc, OK, OK, OK, None) == 1
    assert lib.kq_fp8_weights_pack(d.desc, OK, OK, None, None, OK, None) == 1
    assert lib.kq_fp8_weights_pack(plain.desc, OK, OK, OK, OK, OK, None) == 1


def ffn(g=None, d=None, gw=OK, dw=OK, X=OK, r=None, gm=OK, eps=1e-6, M=4, Y=OK, ldy=64, dt=0, ws=OK2, n=BIG, ldx=64):
    g, d = g or L(64, 96, True), d or L(96, 64)
    return lib.kq_fp8_ffn(g.desc, gw, d.desc, dw, X, ldx, r, 64, 0, gm, eps, M, Y, ldy, dt, ws, n, None)


def test_ffn():
    assert ffn(g=L(64, 96)) == 1 and ffn(d=L(96, 64, True)) == 1 and ffn(d=L(64, 64)) == 1
    assert ffn(gw=None) == 1 and ffn(dw=None) == 1 and ffn(X=None) == 1 and ffn(ws=None) == 1 and ffn(Y=None) == 1
    assert ffn(M=0) == 1 and ffn(eps=0.0) == 1 and ffn(dt=2) == 1 and ffn(ldx=8) == 1 and ffn(ldy=8) == 1
    assert ffn(gm=None, r=OK) == 1
    assert ffn(n=100) == 5 and ffn(ws=ODD) == 3 and ffn(gm=ODD) == 3 and ffn(r=ODD) == 3


def test_last_error():
    assert lib.kq_fp8_last_device_error(None, None) == 1
    assert lib.kq_fp8_last_device_error(ODD, None) == 3


def test_binding_checks():
    X, act = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        kq.fp8_quantize_act(X, act)
    with pytest.raises(ValueError, match="CUDA"):
        kq.fp8_linear(L(), act, X, X, act, kq.OUT_BF16)
    with pytest.raises(ValueError, match="gated layers"):
        kq.fp8_prepare_weights(L(64, 64, True), X, act)
    with pytest.raises(ValueError, match="unsupported"):
        kq.fp8_gemm(L(40, 64), act, act, 4, X)


def test_debug_wait_timeout():
    d, plain = L(64, 64, True), L()

    def t(d=plain, w=OK, X=None, ldx=0, M=4, Y=OK, ldy=64, dt=0, a=OK2, n=BIG, o=None, on=0, k=0, us=1000):
        return lib.kq_fp8_debug_wait_timeout(d.desc, w, X, ldx, M, Y, ldy, dt, a, n, o, on, k, us, None)

    assert t(k=-1) == 1 and t(us=0) == 1 and t(us=1000001) == 1 and t(w=None) == 1 and t(a=None) == 1 and t(M=0) == 1
    assert t(Y=None) == 1 and t(dt=2) == 1 and t(ldy=66) == 3 and t(X=ODD, ldx=64) == 3 and t(X=OK, ldx=32) == 1
    assert t(n=64) == 5 and t(d=L(40, 64)) == 2
    assert t(o=OK, on=BIG, Y=None) == 1                                 # not gated
    assert t(d=d, o=OK, on=BIG) == 1 and t(d=d, o=OK2, on=BIG, Y=None) == 1 and t(d=d, o=OK, on=64, Y=None) == 5
    assert t(d=d, o=OK, on=BIG, X=OK, ldx=64, Y=None) == 1


def test_sizes_past_32_bits():
    """Sizes that the C ABI's 32-bit fields cannot hold are refused, not cut to their low bits."""
    far = (1 << 32) + 64
    for K, N in ((far, 64), (64, far), (-far, 64), (1 << 31, 64)):
        with pytest.raises(ValueError, match="32 bits"):
            kq.Fp8Layer(K, N)
    g, d = L(64, 96, True), L(96, 64)
    for M in (far, 1 << 31, 1 - far):
        assert kq.fp8_act_bytes(64, M) == 0 and kq.fp8_act_bytes(M, 4) == 0 and kq.fp8_ffn_bytes(g, d, M) == 0
    act, Y = torch.zeros(1 << 16, dtype=torch.uint8), torch.empty(far, 64, device="meta")
    wide, tall = (torch.empty(n, k, dtype=torch.bfloat16, device="meta") for n, k in ((1, far), (far, 64)))
    with pytest.raises(ValueError, match=f"needs {64 * far}"):
        kq.fp8_act_pack(64, act, act, far, act)
    calls = [lambda: kq.fp8_act_unpack(64, act, far),
             lambda: kq.fp8_act_unpack(far, act, 4), lambda: kq.fp8_gemm(L(), act, act, far, Y),
             lambda: kq.fp8_gated_act(g, act, act, far, act), lambda: kq.fp8_quantize_act(wide, act),
             lambda: kq.fp8_quantize_act(tall, act), lambda: kq.fp8_rmsnorm_act(tall, torch.ones(64), 1e-6, act),
             lambda: kq.fp8_linear(L(), act, tall, Y, act), lambda: kq.fp8_ffn(g, act, d, act, tall, None, 1e-6, Y, act)]
    for f in calls:
        with pytest.raises(ValueError, match="32 bits"):
            f()


def test_widest_layers():
    top = 1 << 28
    assert kq.fp8_weights_bytes(L(top, 16)) > top * 16 and kq.fp8_weights_bytes(L(32, top)) > top * 32
    assert kq.fp8_weights_bytes(L(top + 32, 16)) == 0 and kq.fp8_weights_bytes(L(32, top + 16)) == 0
    assert kq.fp8_act_bytes(top, 1) > top and kq.fp8_act_bytes(top + 32, 1) == 0
    assert quant(K=top + 32, ldx=top + 32) == 2
    assert lib.kq_fp8_gemm(L(32, top + 16).desc, OK, OK2, 1, OK, top + 16, 0, None) == 2
