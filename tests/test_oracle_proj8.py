"""Pins of the 8-bit projections' oracle (oracle/proj8.py) and the refusals of
their C calls and bindings (host-side, no GPU)."""
import numpy as np
import pytest
import torch

from oracle import dequantize, proj8
from long_context_sparse_07_b200 import abi, build

F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- oracle pins

@pytest.mark.parametrize("rows,d", [(1, 16), (3, 128), (5, 144), (4, 400)])
def test_row_codes_match_torch_casts_and_bound(rows, d):
    gen = np.random.default_rng(rows + d)
    v = gen.standard_normal((rows, d)) * np.exp(gen.standard_normal((rows, 1)))
    v = v.astype(np.float32).astype(np.float64)
    codes, scales = proj8.quantize_rows(v)
    assert scales.shape == (rows, -(-d // 128))
    t = torch.from_numpy(v.astype(np.float32))
    for b in range(scales.shape[1]):
        part = t[:, b * 128:(b + 1) * 128]
        s = part.abs().amax(1, keepdim=True) / 448.0
        assert torch.equal(torch.from_numpy(scales[:, b]), s[:, 0])
        want = (part / s).clamp(-448, 448).to(F8).view(torch.uint8).numpy()
        assert np.array_equal(codes[:, b * 128:(b + 1) * 128], want)
    # half a step: 2^-4 of the value, or of the smallest step 2^-9 of the scale
    back = proj8.row_values(codes, scales)
    step = np.repeat(scales.astype(np.float64), 128, axis=1)[:, :d]
    assert (np.abs(back - v) <= np.maximum(np.abs(v) * 2.0 ** -4, step * 2.0 ** -10) *
            (1 + 2.0 ** -20)).all()


@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (130, 144), (300, 272)])
def test_weight_blocks_by_loops(N, K):
    W = np.random.default_rng(N).standard_normal((N, K)).astype(np.float32)
    codes, scales = proj8.quantize_weight(W)
    back = proj8.weight_values(codes, scales)
    for i in range(-(-N // 128)):
        for j in range(-(-K // 128)):
            blk = np.s_[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128]
            assert scales[i, j] == np.float32(np.abs(W[blk]).max()) / np.float32(448.0)
            assert np.abs(back[blk]).max() == pytest.approx(np.abs(W[blk]).max(), rel=1e-6)
            want = dequantize(codes[blk].reshape(1, -1), [[scales[i, j]]], codes[blk].size)
            assert np.array_equal(back[blk].reshape(1, -1), want)


def test_norm_and_product_by_loops():
    gen = np.random.default_rng(7)
    x, r, g = gen.standard_normal((3, 32)), gen.standard_normal((3, 32)), gen.standard_normal(32)
    s, v = proj8.add_norm(x, r, g, eps=0.5)
    for i in range(3):
        t = [x[i][j] + r[i][j] for j in range(32)]
        ms = sum(a * a for a in t) / 32 + 0.5
        assert np.allclose(s[i], t, rtol=1e-14)
        assert np.allclose(v[i], [t[j] / ms ** 0.5 * g[j] for j in range(32)], rtol=1e-13)
    assert np.array_equal(proj8.add_norm(x, normalise=False)[1], x)
    A, As = proj8.quantize_rows(gen.standard_normal((4, 256)))
    W, Ws = proj8.quantize_weight(gen.standard_normal((256, 128)))
    got = proj8.fp8_proj(A, As, W, Ws, groups=2)
    a, w = proj8.row_values(A, As), proj8.weight_values(W, Ws)
    for t in range(4):
        for j in range(256):
            lo = j // 128 * 128
            assert got[t, j] == pytest.approx(sum(a[t, lo + k] * w[j, k] for k in range(128)),
                                              rel=1e-11, abs=1e-11)


# ---------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.load()


P = 0x100000
BF, F, E4, E2 = abi.CSA_BF16, abi.CSA_F32, abi.CSA_E4M3, abi.CSA_E2M1


def test_add_norm_quant_refuses(lib):
    def call(x=P, residual=2 * P, gamma=3 * P, dt=BF, rows=4, d=64, norm=1, eps=1e-6, total=4 * P,
             y=None, codes=5 * P, scale=6 * P):
        return lib.csa_add_norm_quant(x, residual, gamma, dt, rows, d, norm, eps, total, y, codes,
                                      scale, None)

    assert call(x=None) == -1
    assert call(dt=E4) == -2
    assert call(rows=-1) == -1
    for d in (0, 8, 24, 65552):
        assert call(d=d) == -2, d
    assert call(eps=0.0) == -1
    assert call(norm=0) == -1 and b"gamma" in lib.csa_last_message()
    assert call(codes=None) == -1 and b"together" in lib.csa_last_message()
    assert call(scale=None) == -1
    assert call(total=None, codes=None, scale=None) == -1 and b"no output" in lib.csa_last_message()
    assert call(residual=None) == -1 and b"total" in lib.csa_last_message()
    for k in ("x", "residual", "total", "codes"):
        assert call(**{k: 9 * P + 8}) == -1 and b"aligned" in lib.csa_last_message(), k
    assert call(y=9 * P + 4) == -1
    assert call(gamma=3 * P + 2) == -1 and call(scale=6 * P + 2) == -1
    assert call(y=4 * P) == -1 and call(y=5 * P) == -1 and call(y=2 * P) == -1
    assert call(codes=P) == -1 and call(codes=2 * P) == -1
    # nothing to do: no device is touched
    assert call(rows=0, x=None, residual=None, total=None, codes=None, scale=None) == 0


def test_quantize_weight_refuses(lib):
    def call(W=P, dt=F, N=4, K=32, codes=2 * P, scale=3 * P):
        return lib.csa_quantize_weight(W, dt, N, K, codes, scale, None)

    assert call(W=None) == -1 and call(codes=None) == -1 and call(scale=None) == -1
    assert call(dt=E2) == -2 and call(N=-1) == -1
    assert call(K=0) == -2 and call(K=40) == -2
    assert call(W=P + 8) == -1 and call(codes=2 * P + 1) == -1 and call(scale=3 * P + 2) == -1
    assert call(codes=P) == -1
    assert call(N=0, W=None, codes=None, scale=None) == 0
    assert call(N=2 ** 30 + 1) == -1 and call(K=2 ** 30 + 16) == -1


def test_fp8_proj_refuses(lib):
    def call(A=P, As=2 * P, W=3 * P, Ws=4 * P, M=4, N=128, K=128, groups=1, dt=BF, out=5 * P,
             os=None):
        return lib.csa_fp8_proj(A, As, W, Ws, M, N, K, groups, dt, out, os, None)

    for k in ("A", "As", "W", "Ws", "out"):
        assert call(**{k: None}) == -1, k
    assert call(dt=E2) == -2
    assert call(M=-1) == -1 and call(M=2 ** 31) == -1 and call(N=0) == -1 and call(groups=0) == -1
    assert call(K=0) == -2 and call(K=24) == -2
    assert call(groups=2, N=120) == -2 and call(groups=2, K=144) == -2
    assert call(groups=2 ** 20, N=2 ** 20, K=128) == -1
    assert call(dt=E4, N=24, os=6 * P) == -2
    assert call(dt=E4) == -1 and b"out_scale" in lib.csa_last_message()
    assert call(os=6 * P) == -1
    for k in ("A", "W", "out"):
        assert call(**{k: 9 * P + 8}) == -1 and b"aligned" in lib.csa_last_message(), k
    for k in ("As", "Ws"):
        assert call(**{k: 9 * P + 2}) == -1 and b"aligned" in lib.csa_last_message(), k
    assert call(out=P) == -1 and b"overlap" in lib.csa_last_message()
    assert call(M=0, A=None, As=None, W=None, Ws=None, out=None) == 0
    assert call(N=2 ** 30 + 1) == -1 and call(K=2 ** 30 + 16) == -1
    assert call(groups=2, N=2 ** 30) == -1


def test_bindings_refuse_host_tensors_and_wrong_shapes():
    x = torch.zeros(2, 144, dtype=torch.bfloat16)
    c, s = torch.zeros(2, 144, dtype=F8), torch.zeros(2, 2)
    with pytest.raises(ValueError, match="CUDA"):
        abi.csa_add_norm_quant(x, codes=c, scale=s)
    with pytest.raises(ValueError, match="scale"):
        abi.csa_add_norm_quant(x, codes=c, scale=torch.zeros(2, 1))
    with pytest.raises(TypeError, match="residual"):
        abi.csa_add_norm_quant(x, residual=x.float(), codes=c, scale=s)
    with pytest.raises(ValueError, match="contiguous"):
        abi.csa_add_norm_quant(x.t().contiguous().t(), codes=c, scale=s)
    with pytest.raises(TypeError, match="codes"):
        abi.csa_quantize_weight(x, x, torch.zeros(1, 2))
    with pytest.raises(ValueError, match="scale"):
        abi.csa_quantize_weight(x, c, torch.zeros(2, 2))
    W, Ws = torch.zeros(256, 144, dtype=F8), torch.zeros(2, 2)
    out = torch.zeros(2, 256)
    with pytest.raises(ValueError, match="CUDA"):
        abi.csa_fp8_proj(c, s, W, Ws, out)
    with pytest.raises(ValueError, match="out is"):
        abi.csa_fp8_proj(c, s, W, Ws, torch.zeros(2, 128))
    with pytest.raises(ValueError, match="groups"):
        abi.csa_fp8_proj(c, s, W, Ws, out, groups=3)
    with pytest.raises(ValueError, match="W_scale"):
        abi.csa_fp8_proj(c, s, W, torch.zeros(256, 2), out)
