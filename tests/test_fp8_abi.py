"""Refusals of the 8-bit floating-point and routing entry points, on the host before anything
is enqueued (no GPU needed), and of their Python binding."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x100008)


@pytest.fixture(scope="module")
def lib():
    from int4_quantized_b200 import _build

    _build.build()
    import int4_quantized_b200 as q4

    return q4.lib()


@pytest.mark.parametrize("xt,x_rows,K,rows,R,flags,ptr,expect", [
    (3, 4, 128, False, 4, 0, True, 1),           # type
    (0, 4, 128, False, 4, 2, True, 1),           # unknown flag
    (0, -1, 128, False, -1, 0, True, 1),         # negative rows
    (0, 4, 0, False, 4, 0, True, 1),             # no columns
    (0, 4, 128, False, 5, 0, True, 1),           # R without a row list
    (0, 4, 128, True, -1, 0, True, 1),
    (0, 4, (1 << 30) + 1, False, 4, 0, True, 2),
    (0, 1 << 28, 1 << 12, False, 1 << 28, 0, True, 2),  # 2^33 blocks
    (0, 4, 128, False, 4, 0, False, 1),          # null pointers
    (0, 0, 128, False, 0, 0, False, 0),          # empty
    (0, 0, 128, True, 9, 0, True, 0),            # no row to take
])
def test_pack(lib, xt, x_rows, K, rows, R, flags, ptr, expect):
    p = FAKE if ptr else None
    assert lib.q4_fp8_pack(p, xt, x_rows, K, FAKE if rows else None, R, None, flags, p, p, None, None) == expect


@pytest.mark.parametrize("wt,E,N,K,ptr,expect", [
    (9, 1, 128, 128, True, 1), (0, -1, 128, 128, True, 1), (0, 1, -1, 128, True, 1), (0, 1, 128, 0, True, 1),
    (0, 1, (1 << 30) + 1, 128, True, 2), (0, 1 << 30, 1 << 10, 128, True, 2), (0, 1, 128, 128, False, 1),
    (0, 0, 128, 128, False, 0), (0, 3, 0, 128, False, 0),
])
def test_pack_weights(lib, wt, E, N, K, ptr, expect):
    p = FAKE if ptr else None
    assert lib.q4_fp8_pack_weights(p, wt, E, N, K, p, p, None, None) == expect


@pytest.mark.parametrize("M,N,K,yt,x,w,expect", [
    (1, 128, 128, 3, FAKE, FAKE, 1),             # type of y
    (-1, 128, 128, 0, FAKE, FAKE, 1), (1, -1, 128, 0, FAKE, FAKE, 1), (1, 128, 0, 0, FAKE, FAKE, 1),
    (1, 128, 136, 0, FAKE, FAKE, 2),             # K % 16
    (1, 128, 128, 0, ODD, FAKE, 2), (1, 128, 128, 0, FAKE, ODD, 2),
    ((1 << 30) + 1, 128, 128, 0, FAKE, FAKE, 2), (1, (1 << 30) + 1, 128, 0, FAKE, FAKE, 2),
    (1, 128, 128, 0, None, FAKE, 1), (1, 128, 128, 0, FAKE, None, 1),
    (0, 128, 128, 0, None, None, 0), (1, 0, 128, 0, None, None, 0),
])
def test_gemm(lib, M, N, K, yt, x, w, expect):
    assert lib.q4_fp8_gemm(x, FAKE, M, w, FAKE, N, K, FAKE, yt, None, None) == expect


@pytest.mark.parametrize("R,E,N,K,off,expect", [
    (4, 2, 128, 128, None, 1),                   # no offsets
    (4, -1, 128, 128, FAKE, 1), (4, 1025, 128, 128, FAKE, 2), (4, 1024, 1 << 22, 128, FAKE, 2),
    (4, 2, 128, 8, FAKE, 2), (0, 2, 128, 128, None, 0), (4, 0, 128, 128, None, 0),
])
def test_gemm_grouped(lib, R, E, N, K, off, expect):
    assert lib.q4_fp8_gemm_grouped(FAKE, FAKE, R, off, E, FAKE, FAKE, N, K, FAKE, 0, None, None) == expect


@pytest.mark.parametrize("bits,T,k,E,ptr,expect", [
    (16, 4, 2, 8, True, 1), (32, -1, 2, 8, True, 1), (32, 4, 0, 8, True, 1), (64, 4, 2, 0, True, 1),
    (32, 4, 2, 1025, True, 2), (32, 1 << 30, 2, 8, True, 2), (32, 4, 2, 8, False, 1),
])
def test_sort(lib, bits, T, k, E, ptr, expect):
    p = FAKE if ptr else None
    assert lib.q4_moe_sort(p, bits, T, k, E, p, p, p, None) == expect


@pytest.mark.parametrize("t,T,k,D,R,ptr,expect", [
    (5, 4, 2, 64, 8, True, 1), (0, -1, 2, 64, 8, True, 1), (0, 4, 0, 64, 8, True, 1), (0, 4, 2, 0, 8, True, 1),
    (0, 4, 2, 64, -1, True, 1), (0, 4, 2, (1 << 30) + 1, 8, True, 2), (0, 4, 2, 64, 1 << 31, True, 2),
    (0, 1 << 30, 2, 64, 8, True, 2), (0, 4, 2, 64, 8, False, 1), (0, 0, 2, 64, 8, False, 0),
])
def test_combine(lib, t, T, k, D, R, ptr, expect):
    p = FAKE if ptr else None
    assert lib.q4_moe_combine(p, t, R, D, p, None, T, k, p, None) == expect
    assert lib.q4_moe_combine_backward(p, p, t, R, D, p, p, T, k, p, p, None) == expect


@pytest.mark.parametrize("t,T,D,R,ptr,expect", [
    (5, 4, 64, 8, True, 1), (0, -1, 64, 8, True, 1), (0, 4, 0, 8, True, 1), (0, 4, 64, -1, True, 1),
    (0, 4, 64, 1 << 31, True, 2), (0, 4, 1 << 24, (1 << 31) - 1, True, 2), (0, 4, 64, 8, False, 1),
    (0, 4, 64, 0, False, 0), (0, 0, 64, 8, False, 0),
])
def test_gather(lib, t, T, D, R, ptr, expect):
    p = FAKE if ptr else None
    assert lib.q4_moe_gather(p, t, T, D, p, R, p, None) == expect


def test_binding_refuses_cpu_tensors():
    import torch

    import int4_quantized_b200 as q4

    x = torch.zeros(4, 128)
    c, s = x.to(torch.float8_e4m3fn), torch.zeros(4, 1)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: q4.fp8_pack(x), lambda: q4.fp8_pack_weights(x), lambda: q4.fp8_gemm(c, s, c, s),
                 lambda: q4.fp8_gemm_grouped(c, s, c[None], s[None], i[0]), lambda: q4.moe_sort(i, 4),
                 lambda: q4.moe_gather(x, i[:, 0]), lambda: q4.moe_combine(x, i),
                 lambda: q4.moe_combine_backward(x, x, i, x), lambda: q4.Fp8Experts(c, s, c, s)):
        with pytest.raises(TypeError):
            call()
