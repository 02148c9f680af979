"""Which products from codes go to the few-token kernel: the sizes measured on
both sides, by the library's own rule (a C++ function of it)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def pays():
    import w8a8_int8_quantized_token_amd as w8

    name = "few_tokens_pay_from_codes"
    rule = getattr(w8.lib, f"_ZN4w8a8{len(name)}{name}Elllb")
    rule.restype, rule.argtypes = ctypes.c_bool, [ctypes.c_int64] * 3 + [ctypes.c_bool]
    return rule


# (tokens, channels, K, gated) where the tiled kernel was the faster one, and where it was not
TILED = [(1, 256, 64, False), (16, 8192, 64, False), (8, 4096, 128, False), (1, 8192, 256, False), (16, 12288, 320, False),
         (1, 12288, 512, False), (16, 16384, 512, False), (16, 16384, 640, False), (1, 32768, 768, False), (32, 256, 256, False),
         (17, 65536, 4096, False), (16, 65536, 4096, False), (1, 256, 64, True), (16, 4096, 128, True), (1, 12288, 256, True),
         (16, 8192, 512, True), (16, 14336, 704, True), (32, 32768, 2048, True)]
FEW = [(1, 2048, 256, False), (16, 4096, 320, False), (1, 8192, 512, False), (16, 8192, 640, False), (1, 8192, 768, False),
       (16, 16384, 832, False), (1, 65536, 1024, False), (16, 4096, 4096, False), (32, 16384, 4096, False), (8, 4096, 11008, False),
       (1, 4096, 512, True), (16, 1000, 320, True), (16, 32768, 1024, True), (1, 65536, 4096, True), (32, 12288, 4096, True)]


@pytest.mark.parametrize("M,N,K,gated", TILED)
def test_tiled(pays, M, N, K, gated):
    assert not pays(M, N, K, gated)


@pytest.mark.parametrize("M,N,K,gated", FEW)
def test_few_tokens(pays, M, N, K, gated):
    assert pays(M, N, K, gated)
