"""Scales that start where another operand of the 8-bit projections does are
refused (host-side, no GPU)."""
import pytest

from long_context_sparse_07_b200 import abi, build

P = 0x100000
BF, E4 = abi.CSA_BF16, abi.CSA_E4M3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.load()


def refused(lib, status):
    return status == -1 and b"scale must not overlap" in lib.csa_last_message()


@pytest.mark.parametrize("other", range(6))
def test_add_norm_quant(lib, other):
    x, residual, gamma, total, y, codes = (P * (i + 1) for i in range(6))
    scale = (x, residual, gamma, total, y, codes)[other]
    assert refused(lib, lib.csa_add_norm_quant(x, residual, gamma, BF, 4, 64, 1, 1e-6, total, y,
                                               codes, scale, None))


@pytest.mark.parametrize("other", range(2))
def test_quantize_weight(lib, other):
    assert refused(lib, lib.csa_quantize_weight(P, BF, 4, 32, 2 * P, (P, 2 * P)[other], None))


@pytest.mark.parametrize("other", range(5))
def test_fp8_proj(lib, other):
    ops = [P * (i + 1) for i in range(5)]
    A, As, W, Ws, out = ops
    assert refused(lib, lib.csa_fp8_proj(A, As, W, Ws, 4, 128, 128, 1, E4, out, ops[other], None))
