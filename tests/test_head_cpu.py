"""Refusals of the low-precision linear layer's entry points that need no GPU:
the C ABI checks its arguments on the host before anything is queued."""

import ctypes

import pytest
import torch

from communication_avoiding_mixed_amd import binding as B

P = ctypes.c_void_p(4096)  # an aligned address that no refused call reads
ODD = ctypes.c_void_p(4097)


def refused(rc, text):
    assert rc == B.EINVAL
    assert text in B.load().casgd_last_error().decode()


def test_padded_row_length():
    lib = B.load()
    assert [lib.casgd_mx_ld(c) for c in (1, 128, 129, 2000)] == [128, 128, 256, 2048]
    assert [B.mx_ld(c) for c in (1, 128, 129, 2000)] == [128, 128, 256, 2048]
    assert lib.casgd_mx_ld(0) == -1 and lib.casgd_mx_ld(2 ** 31) == -1


@pytest.mark.parametrize("args,text", [
    ((P, B.FP8, 4, 64, 64, B.MX4, P, P), "element type"),
    ((P, B.BF16, -1, 64, 64, B.MX4, P, P), "rows out of range"),
    ((P, B.BF16, 4, 0, 64, B.MX4, P, P), "columns out of range"),
    ((P, B.BF16, 4, 64, 63, B.MX4, P, P), "row stride"),
    ((P, B.BF16, 4, 64, 64, 2, P, P), "format"),
    ((None, B.BF16, 4, 64, 64, B.MX4, P, P), "NULL"),
    ((P, B.BF16, 4, 64, 64, B.MX4, None, P), "NULL"),
    ((P, B.BF16, 4, 64, 64, B.MX4, P, None), "NULL"),
    ((P, B.BF16, 4, 64, 64, B.MX4, ODD, P), "aligned"),
    ((P, B.BF16, 4, 64, 64, B.MX8, P, ODD), "aligned")])
def test_quantise_refusals(args, text):
    x, ty, rows, cols, stride, fmt, codes, scales = args
    refused(B.load().casgd_mx_quantize(*args, None), text)
    refused(B.load().casgd_mx_dequantize(codes, scales, fmt, rows, cols, x, ty, stride, None), text)


def test_product_refusals():
    lib = B.load()
    assert lib.casgd_mx4_linear_workspace(4, 64, 8) == 0 and lib.casgd_mx4_linear_workspace(4, 0, 8) == -1
    need = lib.casgd_mx4_linear_workspace(400, 64, 8)
    assert need >= 400 * (64 + 4)
    ok = (P, B.BF16, 400, 64, 64, P, P, 8, P, B.BF16, 8, P, need, None)

    def linear(at, value, text):
        refused(lib.casgd_mx4_linear(*ok[:at], value, *ok[at + 1:]), text)

    linear(0, None, "NULL"), linear(8, None, "NULL"), linear(11, None, "NULL"), linear(5, None, "NULL")
    linear(1, 3, "element type"), linear(9, 7, "element type"), linear(4, 63, "row stride"), linear(10, 7, "row stride")
    linear(12, need - 1, "workspace"), linear(11, ODD, "aligned"), linear(5, ODD, "aligned"), linear(7, 0, "columns")
    linear(7, 2 ** 27, "row stride")
    refused(lib.casgd_mx4_linear(P, B.BF16, 4, 64, 64, P, P, 2 ** 27, P, B.BF16, 2 ** 27, P, need, None), "2^26")
    refused(lib.casgd_mx4_linear(P, B.BF16, 4, 2 ** 25, 2 ** 25, P, P, 8, P, B.BF16, 8, P, need, None), "2^24")


def test_gradient_refusals():
    lib = B.load()
    assert lib.casgd_mx_grad_workspace(0, 4, 8, 64, P, B.FP32, 8) == 0
    assert lib.casgd_mx_grad_workspace(0, 4, 8, 64, P, B.FP8, 8) == -1
    m, n, k = 4000, 4000, 1600
    need = lib.casgd_mx_grad_workspace(0, m, n, k, P, B.FP32, n)
    assert need >= 2 * n * 1664 + 3 * 2 * m * n
    ok = (P, B.FP32, m, n, n, P, P, k, P, B.FP32, k, P, need, None)

    def grad_input(at, value, text):
        refused(lib.casgd_mx4_grad_input(*ok[:at], value, *ok[at + 1:]), text)

    for at in (0, 5, 6, 8, 11):
        grad_input(at, None, "NULL")
    grad_input(1, B.FP8, "element type"), grad_input(9, 9, "element type"), grad_input(4, n - 1, "row stride")
    grad_input(10, k - 1, "row stride"), grad_input(12, need - 1, "workspace"), grad_input(11, ODD, "aligned")
    grad_input(2, 2 ** 30, "rows")
    need = lib.casgd_mx_grad_workspace(1, m, n, k, P, B.FP32, n)
    okw = (P, B.FP32, m, n, n, P, P, k, P, B.FP32, k, 0, P, need, None)

    def grad_weight(at, value, text):
        refused(lib.casgd_mx8_grad_weight(*okw[:at], value, *okw[at + 1:]), text)

    for at in (0, 5, 6, 8, 12):
        grad_weight(at, None, "NULL")
    grad_weight(1, B.FP8, "element type"), grad_weight(9, 9, "element type"), grad_weight(4, n - 1, "row stride")
    grad_weight(10, k - 1, "row stride"), grad_weight(13, need - 1, "workspace"), grad_weight(12, ODD, "aligned")
    refused(lib.casgd_mx4_grad_input(P, B.BF16, 4, 2 ** 23, 2 ** 23, P, P, 64, P, B.BF16, 64, P, need, None), "2^22")


def test_preference_refusals():
    lib = B.load()
    assert lib.casgd_pref_workspace(10) == 80 and lib.casgd_pref_workspace(-1) == -1
    ok = [P, B.FP32, 6, 9, 9, P, P, 1, None, B.LOGISTIC, 0.1, 0.0, 0, P, P, P, P, P, P, 48, None]

    def loss(at, value, text):
        refused(lib.casgd_pref_loss(*ok[:at], value, *ok[at + 1:]), text)

    for at in (0, 5, 6, 13, 14, 15, 16, 17, 18):
        loss(at, None, "NULL")
    loss(1, B.FP8, "element type"), loss(4, 8, "row stride"), loss(7, 0, "pairs"), loss(9, B.POISSON, "logistic or squared")
    loss(10, 0.0, "beta"), loss(10, float("nan"), "beta"), loss(10, float("inf"), "beta"), loss(11, 1.5, "smoothing")
    loss(16, ODD, "aligned"), loss(19, 47, "workspace"), loss(2, 2 ** 30, "tokens")
    ok[9], ok[11] = B.SQUARED, 0.1
    refused(lib.casgd_pref_loss(*ok), "smoothing")
    refused(lib.casgd_token_logps(P, B.FP32, 6, 9, 9, None, P, None), "NULL")
    refused(lib.casgd_token_logps(P, B.FP32, 6, 9, 9, P, None, None), "NULL")
    refused(lib.casgd_pref_grad(P, B.FP32, 6, 9, 9, P, P, 1, P, P, None, P, 9, None), "NULL")
    refused(lib.casgd_pref_grad(P, B.FP32, 6, 9, 9, P, P, 1, P, P, P, P, 8, None), "row stride")
    refused(lib.casgd_pref_grad(P, B.FP32, 6, 9, 9, P, P, 1, P, P, P, P, 10, None), "in place")
    refused(lib.casgd_pref_grad(P, B.FP32, 6, 9, 9, P, P, 0, P, P, P, P, 9, None), "pairs")


def test_host_tensors_are_refused():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU"):
        B.mx_quantize(x, "mx4")
    with pytest.raises(ValueError, match="GPU"):
        B.MXMatrix("mx4", torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 64)
    with pytest.raises(ValueError, match="fit"):
        B.MXMatrix("mx4", torch.zeros(4, 60, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 64)
    with pytest.raises(ValueError, match="GPU"):
        B.token_logps(x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="loss"):
        B.pref_loss(x, None, None, loss="poisson")
