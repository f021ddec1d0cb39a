"""GPU parity of the 8-bit projection calls (csa_add_norm_quant,
csa_quantize_weight, csa_fp8_proj) against the float64 oracle.

Tolerances. U = 2^-24 is half a float32 step. A stored value is off by at most
half a step of its type: 2^-8 of it in bf16; in e4m3 2^-4 of it, or 2^-10 of
the scale where the code is subnormal.
* the norm: a sum of d squares over at least 32 lanes has chains of at most
  d / 32 + 64 additions, each off by U of the sum; the root halves that; eight
  more roundings (sum, mean, eps, root, quotient, two products): (d / 64 + 40) U.
* the product: at most 128 + nb additions and as many products, a step (2 U,
  for a sum that truncates) of the sum of magnitudes each.
"""
import numpy as np
import pytest
import torch

from oracle import proj8
from long_context_sparse_07_b200 import abi
from helpers import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
nb = proj8.blocks


def u8(t):
    return t.view(torch.uint8).cpu().numpy()


def rows_of(seed, rows, d, dt, spread=1.0):
    gen = np.random.default_rng(seed)
    v = gen.standard_normal((rows, d)) * np.exp(spread * gen.standard_normal((rows, 1)))
    return torch.from_numpy(v.astype(np.float32)).to(dt)


def check_codes(codes, scale, v, v_err, what):
    """Stored rows against float64 values v known to within v_err (absolute)."""
    s = scale.cpu().double().numpy()
    d = v.shape[1]
    amax = np.stack([np.abs(v[:, b * 128:(b + 1) * 128]).max(1) for b in range(nb(d))], 1)
    aerr = np.stack([v_err[:, b * 128:(b + 1) * 128].max(1) for b in range(nb(d))], 1)
    assert (np.abs(s * 448 - np.maximum(amax, 448 * 2.0 ** -126)) <= aerr + 4 * U * amax).all(), \
        what + ": scale"
    back = proj8.row_values(u8(codes), scale.cpu().numpy())
    step = np.repeat(s, 128, axis=1)[:, :d]
    tol = np.maximum(np.abs(v) * 2.0 ** -4, step * 2.0 ** -10) * (1 + 2.0 ** -20) + 1.25 * v_err
    err = np.abs(back - v)
    assert (err <= tol).all(), "%s: codes, worst %.3g of the bound" % (what, (err / tol).max())


# ---------------------------------------------------------------- norm

NORM_CASES = [
    # rows, d, dtype, residual, gamma, normalise
    (1, 16, torch.bfloat16, True, True, True),
    (1, 4096, torch.bfloat16, True, True, True),
    (8, 4096, torch.bfloat16, False, True, True),
    (33, 144, torch.float32, True, False, True),
    (5, 1040, torch.bfloat16, True, True, True),
    (7, 2064, torch.float32, False, True, True),
    (300, 512, torch.bfloat16, True, True, True),
    (3, 8192, torch.float32, True, True, True),
    (2, 16400, torch.bfloat16, True, True, True),
    (3, 32768, torch.bfloat16, False, False, False),
    (2, 65536, torch.float32, True, True, True),
    (2, 65520, torch.bfloat16, True, True, True),
    (1000, 64, torch.bfloat16, True, False, False),
    (129, 256, torch.float32, False, False, False),
    # many rows longer than a block's threads hold at once
    (200, 9216, torch.bfloat16, True, True, True),
    (170, 16400, torch.bfloat16, False, True, True),
    (160, 8208, torch.float32, True, False, True),
    # one long row over a cluster whose last block is short
    (1, 16640, torch.float32, True, True, True),
    (3, 8336, torch.bfloat16, True, True, True),
    # rows that share a warp
    (70, 80, torch.bfloat16, True, True, True),
    (131, 128, torch.float32, False, True, True),
    (3000, 240, torch.bfloat16, True, True, True),
]


@pytest.mark.parametrize("rows,d,dt,res,gam,norm", NORM_CASES)
def test_add_norm_quant_matches_oracle(rows, d, dt, res, gam, norm):
    x = rows_of(rows + d, rows, d, dt)
    r = rows_of(rows + d + 1, rows, d, dt) if res else None
    g = torch.from_numpy(np.random.default_rng(d).standard_normal(d).astype(np.float32)) \
        if gam and norm else None
    s, v = proj8.add_norm(x, r, g, norm)
    xd = x.to(DEV)
    total = torch.full((rows + 1, d), 7.0, device=DEV, dtype=dt) if res else None
    y = torch.full((rows + 1, d), 7.0, device=DEV, dtype=dt)
    codes = torch.full((rows + 1, d), 77, device=DEV, dtype=torch.uint8)
    scale = torch.full((rows + 1, nb(d)), 7.0, device=DEV)
    abi.csa_add_norm_quant(xd, r.to(DEV) if res else None, g.to(DEV) if g is not None else None,
                           norm, total=total[:rows] if res else None, y=y[:rows],
                           codes=codes[:rows], scale=scale[:rows])
    abi.csa_get_error()
    assert torch.equal(xd.cpu(), x)
    rel = (d / 64 + 40) * U if norm else 2 * U
    if res:
        assert (np.abs(to_np(total[:rows]) - s) <= (HALF[dt] + 2 * U) * np.abs(s)).all()
        assert (total[rows] == 7).all()
    assert (np.abs(to_np(y[:rows]) - v) <= (HALF[dt] + rel) * np.abs(v)).all()
    check_codes(codes[:rows], scale[:rows], v, rel * np.abs(v), "norm")
    if dt == torch.float32:
        # y is the very float32 row that is stored: codes and scales are exact
        c, sc = proj8.quantize_rows(to_np(y[:rows]))
        assert np.array_equal(u8(codes[:rows]), c) and np.array_equal(scale[:rows].cpu().numpy(), sc)
    # rows behind the last one stay as they were
    assert (y[rows] == 7).all() and (codes[rows] == 77).all() and (scale[rows] == 7).all()


def test_add_norm_quant_outputs_alone_and_in_place():
    rows, d = 65, 1040
    x, r = rows_of(1, rows, d, torch.bfloat16).to(DEV), rows_of(2, rows, d, torch.bfloat16).to(DEV)
    ref = [torch.empty_like(x), torch.empty_like(x), torch.empty(rows, d, device=DEV, dtype=F8),
           torch.empty(rows, nb(d), device=DEV)]
    abi.csa_add_norm_quant(x, r, total=ref[0], y=ref[1], codes=ref[2], scale=ref[3])
    # the sum written over the residual, the normed rows over x
    x2, r2 = x.clone(), r.clone()
    abi.csa_add_norm_quant(x2, r2, total=r2, y=x2)
    assert torch.equal(r2, ref[0]) and torch.equal(x2, ref[1])
    # the sum written over x, codes alone
    x3 = x.clone()
    c, s = torch.empty_like(ref[2]), torch.empty_like(ref[3])
    abi.csa_add_norm_quant(x3, r, total=x3, codes=c, scale=s)
    assert torch.equal(x3, ref[0])
    assert np.array_equal(u8(c), u8(ref[2])) and torch.equal(s, ref[3])
    # sum alone
    t = torch.empty_like(x)
    abi.csa_add_norm_quant(x, r, normalise=False, total=t)
    assert torch.equal(t, ref[0])
    # leading dimensions, and a row's result on its own
    c3 = torch.empty(5, 13, d, device=DEV, dtype=torch.uint8)
    s3 = torch.empty(5, 13, nb(d), device=DEV)
    abi.csa_add_norm_quant(x.view(5, 13, d), r.view(5, 13, d), codes=c3, scale=s3)
    assert np.array_equal(c3.view(rows, d).cpu().numpy(), u8(ref[2]))
    one, os = torch.empty(1, d, device=DEV, dtype=F8), torch.empty(1, nb(d), device=DEV)
    abi.csa_add_norm_quant(x[40:41], r[40:41], codes=one, scale=os)
    assert np.array_equal(u8(one[0]), u8(ref[2][40])) and torch.equal(os[0], ref[3][40])
    abi.csa_get_error()


def test_add_norm_quant_special_values():
    d = 272
    x = rows_of(3, 6, d, torch.float32)
    x[0] = 0.0
    x[1, 5] = float("nan")
    x[2, 130] = float("inf")
    x[3, 128:256] = 0.0
    x[4] *= 2.0 ** -130          # subnormal inputs: the scale's floor
    xd = x.to(DEV)
    y = torch.empty(6, d, device=DEV)
    c, s = torch.empty(6, d, device=DEV, dtype=F8), torch.empty(6, 3, device=DEV)
    abi.csa_add_norm_quant(xd, normalise=False, y=y, codes=c, scale=s)
    cf = c.float().cpu()
    assert (cf[0] == 0).all() and (s[0] == 2.0 ** -126).all()
    assert cf[1, :128].isnan().all() and not cf[1, 128:].isnan().any() and s[1, 0].isnan()
    assert s[2, 1] == float("inf") and cf[2, 130].isnan() and (cf[2, 131:256] == 0).all()
    assert not cf[2, 256:].isnan().any()
    assert s[3, 1] == 2.0 ** -126 and (cf[3, 128:256] == 0).all()
    assert (s[4] == 2.0 ** -126).all()
    want, sc = proj8.quantize_rows(to_np(xd[3:6]))
    assert np.array_equal(u8(c[3:6]), want) and np.array_equal(s[3:6].cpu().numpy(), sc)
    abi.csa_add_norm_quant(xd, y=y, codes=c, scale=s)
    assert (y[0] == 0).all() and (c.float()[0] == 0).all()
    assert y[1].isnan().all() and c.float()[1].isnan().all()
    assert not y[3:].isnan().any()
    abi.csa_get_error()


@pytest.mark.parametrize("rows,d", [(3, 64), (2, 4096), (2, 32768), (400, 20480)])
def test_add_norm_quant_sum_that_overflows_gives_zeros(rows, d):
    """Squares of 2^65 are beyond float32, those of 2^50 are not yet."""
    x = torch.full((rows, d), 2.0 ** 50, device=DEV)
    x[1] = 2.0 ** 65
    y, codes = torch.empty_like(x), torch.empty(rows, d, device=DEV, dtype=F8)
    scale = torch.empty(rows, nb(d), device=DEV)
    abi.csa_add_norm_quant(x, y=y, codes=codes, scale=scale)
    assert (y[1] == 0).all() and (codes[1].float() == 0).all() and (scale[1] == 2.0 ** -126).all()
    # all equal values: the norm is 1, off by the tolerance of the norm
    assert ((y[0] - 1).abs() <= (d / 64 + 40) * U).all()


# ---------------------------------------------------------------- weight

@pytest.mark.parametrize("N,K,dt", [
    (1, 16, torch.float32), (128, 128, torch.bfloat16), (130, 144, torch.bfloat16),
    (1000, 1040, torch.float32), (257, 4096, torch.bfloat16), (127, 2032, torch.float32),
])
def test_quantize_weight_is_the_oracles(N, K, dt):
    W = rows_of(N + K, N, K, dt, 0.3)
    W[N // 2, K // 2:] = 0.0
    want, wsc = proj8.quantize_weight(W)
    codes = torch.full((N + 1, K), 77, device=DEV, dtype=torch.uint8)
    scale = torch.full((nb(N) + 1, nb(K)), 7.0, device=DEV)
    abi.csa_quantize_weight(W.to(DEV), codes[:N], scale[:nb(N)])
    abi.csa_get_error()
    assert np.array_equal(codes[:N].cpu().numpy(), want)
    assert np.array_equal(scale[:nb(N)].cpu().numpy(), wsc)
    assert (codes[N] == 77).all() and (scale[nb(N)] == 7).all()


def test_quantize_weight_special_values():
    W = rows_of(5, 256, 256, torch.float32)
    W[3, 4] = float("nan")
    W[128:, :128] = 0.0
    W[130, 200] = -float("inf")
    c, s = torch.empty(256, 256, device=DEV, dtype=F8), torch.empty(2, 2, device=DEV)
    abi.csa_quantize_weight(W.to(DEV), c, s)
    cf, s = c.float().cpu(), s.cpu()
    assert s[0, 0].isnan() and cf[:128, :128].isnan().all()
    assert s[1, 0] == 2.0 ** -126 and (cf[128:, :128] == 0).all()
    assert s[1, 1] == float("inf") and cf[130, 200].isnan() and cf[128:, 128:].isnan().sum() == 1
    assert not cf[:128, 128:].isnan().any()


# ---------------------------------------------------------------- product

def operands(seed, M, N, K, groups=1):
    gen = np.random.default_rng(seed)
    A = gen.standard_normal((M, groups * K)) * np.exp(gen.standard_normal((M, 1)))
    W = gen.standard_normal((groups * N, K)) * np.exp(gen.standard_normal((groups * N, 1)))
    return proj8.quantize_rows(A) + proj8.quantize_weight(W.astype(np.float32))


def device(A, As, W, Ws):
    return (torch.from_numpy(A).to(DEV).view(F8), torch.from_numpy(As).to(DEV),
            torch.from_numpy(W).to(DEV).view(F8), torch.from_numpy(Ws).to(DEV))


def reference(A, As, W, Ws, groups):
    """The product in float64, and the bound of its float32 sums' error."""
    r = proj8.fp8_proj(A, As, W, Ws, groups)
    mags = proj8.fp8_proj(A & 0x7f, As, W & 0x7f, Ws, groups)
    return r, (2 * (128 + Ws.shape[1]) + 8) * 2 * U * mags


def run(ops, GN, dt, groups):
    M = ops[0].shape[0]
    out = torch.full((M + 1, GN), 7.0, device=DEV).to(dt)
    osc = torch.full((M + 1, nb(GN)), 7.0, device=DEV) if dt == F8 else None
    abi.csa_fp8_proj(*ops, out[:M], osc[:M] if osc is not None else None, groups=groups)
    abi.csa_get_error()
    assert (out[M].float() == 7).all() and (osc is None or (osc[M] == 7).all())
    return out[:M], osc[:M] if osc is not None else None


def check(out, osc, r, err, what):
    if osc is not None:
        check_codes(out, osc, r, err, what)
        return
    e = np.abs(to_np(out) - r)
    tol = err + HALF[out.dtype] * np.abs(r)
    assert np.isfinite(to_np(out)).all(), what
    assert (e <= tol).all(), "%s: worst %.3g of the bound" % (what, (e / np.maximum(tol, 1e-300)).max())


PROJ_CASES = [
    # M, N, K, groups
    (1, 1, 16, 1), (1, 16, 128, 1), (1, 1024, 4096, 1), (2, 300, 272, 1), (8, 512, 1024, 1),
    (15, 1040, 144, 1), (16, 128, 2048, 1), (17, 129, 400, 1), (33, 640, 640, 1),
    (64, 2048, 512, 1), (65, 256, 256, 1), (100, 1000, 2064, 1), (127, 130, 1024, 1),
    (128, 256, 128, 1), (129, 272, 1040, 1), (200, 16, 8192, 1), (256, 512, 2048, 1),
    (257, 768, 384, 1), (333, 1000, 2064, 1), (700, 2064, 528, 1), (1025, 1168, 64, 1),
    (3, 128, 256, 3), (40, 256, 128, 5), (130, 384, 256, 2), (520, 128, 512, 4),
    (300, 1024, 4096, 2), (1, 1024, 4096, 8), (2500, 4112, 272, 1),
]


@pytest.mark.parametrize("M,N,K,groups", PROJ_CASES)
def test_fp8_proj_matches_oracle(M, N, K, groups):
    host = operands(M + N + K, M, N, K, groups)
    ops = device(*host)
    r, err = reference(*host, groups)
    for dt in (torch.bfloat16, torch.float32) + ((F8,) if N % 16 == 0 else ()):
        out, osc = run(ops, groups * N, dt, groups)
        check(out, osc, r, err, "M %d N %d K %d groups %d %s" % (M, N, K, groups, dt))


@pytest.mark.parametrize("M,N,K", [(130, 65, 144), (601, 501, 272), (4097, 2047, 144),
                                   (4096, 2041, 272)])
def test_fp8_proj_result_rows_of_any_length(M, N, K):
    """Rows that are not whole 16-byte pieces, in single tiles and in pairs'; the
    value behind the last row stays."""
    host = operands(M + N, M, N, K)
    ops, (r, err) = device(*host), reference(*host, 1)
    for dt in (torch.bfloat16, torch.float32):
        out, _ = run(ops, N, dt, 1)
        check(out, None, r, err, "M %d N %d K %d %s" % (M, N, K, dt))


@pytest.mark.parametrize("M,N,K", [(5, 256, 400), (200, 300, 272), (600, 2048, 256)])
def test_fp8_proj_zero_rows_blocks_and_special_codes(M, N, K):
    A, As, W, Ws = operands(91 + M, M, N, K)
    A[1] = 0
    W[7] = 0x80                                  # -0
    A[0, 3] = 0x7f                               # NaN: all of row 0
    As[2, 1] = np.inf                            # an infinite block of row 2
    Ws[0, 0] = 0.0
    As[3] = 2.0 ** -126
    ops = device(A, As, W, Ws)
    out, _ = run(ops, N, torch.float32, 1)
    got = to_np(out)
    assert np.isnan(got[0]).all() and not np.isfinite(got[2]).any()
    assert (got[1] == 0).all() and (got[[r for r in range(M) if r not in (0, 2)]][:, 7] == 0).all()
    fine = [r for r in range(M) if r not in (0, 2)]
    r, err = reference(A[fine], As[fine], W, Ws, 1)
    # below the smallest normal float32 a rounding is off by half a step of 2^-149, not relatively
    check_tol = err + U * np.abs(r) + 2.0 ** -140
    assert (np.abs(got[fine] - r) <= check_tol).all()
    if N % 16 == 0:
        c, s = run(ops, N, F8, 1)
        assert c.float()[0].isnan().all() and s[0].isnan().all()
        assert (c.float()[1] == 0).all() and (s[1] == 2.0 ** -126).all()


@pytest.mark.parametrize("M,N,K", [(5, 272, 256), (30, 144, 2048), (60, 272, 2048),
                                   (200, 272, 128), (2500, 4112, 272)])
def test_fp8_proj_infinite_rows_behind_the_last_feature(M, N, K):
    """The last scale block holds 16 features: the tile's others, which are not
    there, leave the scale of a row with an infinite scale infinite (not NaN) and
    its finite neighbours alone."""
    A, As, W, Ws = operands(17 + M, M, N, K)
    A[3], W[:], As[3, 0] = 0x38, 0x38, np.inf     # ones: every sum of row 3 is positive
    c, s = run(device(A, As, W, Ws), N, F8, 1)
    assert torch.isinf(s[3]).all() and not c.float()[4].isnan().any()
    fine = [r for r in range(M) if r != 3]
    assert torch.isfinite(s[fine]).all()
    f32, _ = run(device(A, As, W, Ws), N, torch.float32, 1)
    assert torch.isposinf(f32[3]).all() and torch.isfinite(f32[fine]).all()


def test_fp8_proj_rows_do_not_depend_on_the_batch():
    """A token alone, in a small batch and in part of a large one is within the
    bound of the same product, and every call repeats exactly."""
    host = operands(12, 300, 512, 1024)
    A, As, W, Ws = device(*host)
    full, _ = run((A, As, W, Ws), 512, torch.float32, 1)
    again, _ = run((A, As, W, Ws), 512, torch.float32, 1)
    assert torch.equal(full, again)
    half, _ = run((A[100:300].contiguous(), As[100:300].contiguous(), W, Ws), 512, torch.float32, 1)
    one, _ = run((A[7:8], As[7:8], W, Ws), 512, torch.float32, 1)
    eight, _ = run((A[3:11], As[3:11], W, Ws), 512, torch.float32, 1)
    r, err = reference(*host, 1)
    for got, lo in ((half, 100), (one, 7), (eight, 3)):
        n = got.shape[0]
        assert (np.abs(to_np(got) - r[lo:lo + n]) <= err[lo:lo + n] + U * np.abs(r[lo:lo + n])).all()
    e2, _ = run((A[3:11], As[3:11], W, Ws), 512, torch.float32, 1)
    assert torch.equal(eight, e2)


def test_empty_calls_are_no_ops():
    e = torch.empty
    abi.csa_add_norm_quant(e(0, 64, device=DEV), codes=e(0, 64, device=DEV, dtype=F8),
                           scale=e(0, 1, device=DEV))
    abi.csa_quantize_weight(e(0, 64, device=DEV), e(0, 64, device=DEV, dtype=F8),
                            e(0, 1, device=DEV))
    _, _, W, Ws = device(*operands(1, 1, 128, 64))
    abi.csa_fp8_proj(e(0, 64, device=DEV, dtype=F8), e(0, 1, device=DEV), W, Ws,
                     e(0, 128, device=DEV))
    abi.csa_get_error()


# ---------------------------------------------------------------- streams, graphs, size

def test_streams_and_graph_replay():
    """The three calls in a row on a side stream, two streams at once, and a
    captured graph replayed over new inputs, give the plain run's results."""
    M, d, N = 70, 1040, 768
    gen = torch.Generator().manual_seed(3)
    xs = [torch.randn(M, d, generator=gen).to(DEV, torch.bfloat16) for _ in range(3)]
    W = (torch.randn(N, d, generator=gen) * 0.05).to(DEV, torch.bfloat16)

    def bufs():
        return dict(c=torch.empty(M, d, device=DEV, dtype=F8), s=torch.empty(M, nb(d), device=DEV),
                    wc=torch.empty(N, d, device=DEV, dtype=F8),
                    ws=torch.empty(nb(N), nb(d), device=DEV),
                    out=torch.empty(M, N, device=DEV, dtype=torch.bfloat16))

    def chain(x, b, stream=None):
        abi.csa_add_norm_quant(x, codes=b["c"], scale=b["s"], stream=stream)
        abi.csa_quantize_weight(W, b["wc"], b["ws"], stream=stream)
        abi.csa_fp8_proj(b["c"], b["s"], b["wc"], b["ws"], b["out"], stream=stream)

    ref = []
    for x in xs:
        b = bufs()
        chain(x, b)
        ref.append(b["out"])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    b1, b2 = bufs(), bufs()
    for _ in range(5):
        chain(xs[0], b1, s1)
        with torch.cuda.stream(s2):
            chain(xs[1], b2)
    torch.cuda.synchronize()
    assert torch.equal(b1["out"], ref[0]) and torch.equal(b2["out"], ref[1])
    x, b = xs[0].clone(), bufs()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain(x, b)
    for i in (2, 0, 1):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b["out"], ref[i])
    abi.csa_get_error()


@pytest.mark.parametrize("n", [1, 8, 24, 300, 3000])
def test_calls_in_a_row_wait_for_each_other(n):
    """Each call reads what the one before it wrote and overwrites what the one
    before that read, weights among them; launched one behind the other, in a
    stream or a graph, they give the bits they give with a wait between them."""
    d, rounds = 1024, 12
    gen = torch.Generator().manual_seed(n)
    Ws = [(torch.randn(d, d, generator=gen) / d ** 0.5).to(DEV, torch.bfloat16) for _ in range(2)]
    x0 = torch.randn(n, d, generator=gen).to(DEV, torch.bfloat16)
    x, y = torch.empty_like(x0), torch.empty_like(x0)
    w8, ws = torch.empty(d, d, device=DEV, dtype=F8), torch.empty(8, 8, device=DEV)
    h8, hs = torch.empty(n, d, device=DEV, dtype=F8), torch.empty(n, 8, device=DEV)
    u8s = torch.empty(n, d, device=DEV, dtype=F8), torch.empty(n, 8, device=DEV)
    log = torch.empty(rounds, n, d, device=DEV, dtype=torch.bfloat16)

    def chain(wait):
        x.copy_(x0)
        wait()
        for r in range(rounds):
            for call in (lambda: abi.csa_quantize_weight(Ws[r % 2], w8, ws),
                         lambda: abi.csa_add_norm_quant(x, codes=h8, scale=hs),
                         lambda: abi.csa_fp8_proj(h8, hs, w8, ws, *u8s),
                         lambda: abi.csa_fp8_proj(*u8s, w8, ws, y),
                         lambda: abi.csa_add_norm_quant(y, residual=x, total=x, y=log[r])):
                call()
                wait()

    chain(torch.cuda.synchronize)
    want = log.clone()
    assert torch.isfinite(want.float()).all() and want.float().abs().max() > 1
    for _ in range(3):
        log.zero_()
        chain(lambda: None)
        assert torch.equal(log, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(lambda: None)
    for _ in range(3):
        log.zero_()
        graph.replay()
        assert torch.equal(log, want)
    abi.csa_get_error()


def test_captured_fork_and_join():
    """Two streams of a captured step, with copies and other kernels between the
    calls, and a call that waits for both."""
    n, d = 70, 512
    gen = torch.Generator().manual_seed(3)
    x = [torch.randn(n, d, generator=gen).to(DEV, torch.bfloat16) for _ in range(2)]
    Wt = (torch.randn(d, d, generator=gen) / d ** 0.5).to(DEV)
    w8, ws = torch.empty(d, d, device=DEV, dtype=F8), torch.empty(4, 4, device=DEV)
    h = [(torch.empty(n, d, device=DEV, dtype=F8), torch.empty(n, 4, device=DEV)) for _ in x]
    o = [torch.empty(n, d, device=DEV, dtype=torch.bfloat16) for _ in x]
    both, out = torch.empty_like(o[0]), torch.empty(n, d, device=DEV)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        abi.csa_quantize_weight(Wt, w8, ws)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            abi.csa_add_norm_quant(x[1], codes=h[1][0], scale=h[1][1])
            abi.csa_fp8_proj(*h[1], w8, ws, o[1])
        abi.csa_add_norm_quant(x[0], codes=h[0][0], scale=h[0][1])
        abi.csa_fp8_proj(*h[0], w8, ws, o[0])
        both.copy_(o[0])
        main.wait_stream(side)
        abi.csa_add_norm_quant(both, residual=o[1], total=both, codes=h[0][0], scale=h[0][1])
        out.zero_()
        abi.csa_fp8_proj(*h[0], w8, ws, out)

    step()
    torch.cuda.synchronize()
    want = out.clone()
    assert want.abs().max() > 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        graph.replay()
    assert torch.equal(out, want)
    for _ in range(20):
        step()
    assert torch.equal(out, want)
    abi.csa_get_error()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_buffers_that_start_inside_a_sector(dt):
    """16-byte aligned buffers give the bits of 32-byte aligned ones."""
    def shifted(t, by=16):
        raw = torch.zeros(t.numel() * t.element_size() + 64, device=DEV, dtype=torch.uint8)
        at = by + -raw.data_ptr() % 32
        out = raw[at:at + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        assert out.data_ptr() % 32 == by % 32
        return out.copy_(t)

    for rows, d in ((5, 144), (9, 4096), (300, 10256), (3, 20480)):
        x, r = (rows_of(i, rows, d, dt).to(DEV) for i in (1, 2))
        g = torch.rand(d + 1, device=DEV)[1:]
        got = []
        for by in (0, 16):
            for norm in (True, False):
                t, y = shifted(torch.zeros_like(x), by), shifted(torch.zeros_like(x), by)
                c = torch.empty(rows, d, device=DEV, dtype=F8)
                s = torch.empty(rows, nb(d), device=DEV)
                abi.csa_add_norm_quant(shifted(x, by), shifted(r, by), g if norm else None, norm,
                                       total=t, y=y, codes=c, scale=s)
                got.append([v.clone() for v in (t, y, c.view(torch.uint8), s)])
            c, s = torch.empty(rows, d, device=DEV, dtype=F8), torch.empty(nb(rows), nb(d), device=DEV)
            abi.csa_quantize_weight(shifted(x, by), c, s)
            got.append([c.view(torch.uint8), s])
        for one, two in zip(got[:3], got[3:]):
            assert all(torch.equal(p, q) for p, q in zip(one, two))
    abi.csa_get_error()


def test_offsets_past_32_bits():
    """More than 2^32 bytes and 2^31 values of input: the last rows are right."""
    rows, d = 70000, 32768
    x = torch.zeros(rows, d, device=DEV, dtype=torch.bfloat16)
    tail = rows_of(4, 3, d, torch.bfloat16)
    x[-3:] = tail.to(DEV)
    codes = torch.empty(rows, d, device=DEV, dtype=F8)
    scale = torch.empty(rows, nb(d), device=DEV)
    abi.csa_add_norm_quant(x, normalise=False, codes=codes, scale=scale)
    abi.csa_get_error()
    want, wsc = proj8.quantize_rows(to_np(tail))
    assert np.array_equal(u8(codes[-3:]), want) and np.array_equal(scale[-3:].cpu().numpy(), wsc)
    assert (scale[:-3] == 2.0 ** -126).all() and (codes[rows // 2].float() == 0).all()
    del x
    N = 32896
    _, _, W, Ws = operands(8, 1, N, 256)
    Wd, Wsd = torch.from_numpy(W).to(DEV).view(F8), torch.from_numpy(Ws).to(DEV)
    A2, As2 = codes[:, :256].contiguous(), scale[:, :2].contiguous()
    out = torch.empty(rows, N, device=DEV, dtype=torch.bfloat16)
    abi.csa_fp8_proj(A2, As2, Wd, Wsd, out)
    abi.csa_get_error()
    r, err = reference(u8(A2[-3:]), As2[-3:].cpu().numpy(), W, Ws, 1)
    check(out[-3:], None, r, err, "large")
    assert (out[rows // 2] == 0).all()
    del out
    # inputs past 2^31 bytes: wide rows
    _, _, W, Ws = operands(9, 1, 128, d)
    out = torch.empty(rows, 128, device=DEV)
    abi.csa_fp8_proj(codes, scale, torch.from_numpy(W).to(DEV).view(F8),
                     torch.from_numpy(Ws).to(DEV), out)
    abi.csa_get_error()
    r, err = reference(u8(codes[-3:]), scale[-3:].cpu().numpy(), W, Ws, 1)
    check(out[-3:], None, r, err, "wide")
