"""The 8-bit product through each of its kernels (which one a call takes is asked
of the library, so that no change of its rules leaves a kernel untested):
results of every type, special values, the codes' rounding, waits that expire,
calls by several threads.

Tolerances as in test_gpu_proj8, or none: where sums are exact in float32, or
where one call's result is another's operand, the outputs are equal bit for bit.
"""
import threading
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import test_gpu_proj8 as proj8
from long_context_sparse_07_b200 import abi, build
from test_gpu_proj8 import DEV, F8, check, device, nb, operands, reference

gpu = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


# ---------------------------------------------------------------- every kernel

# kernel, M, N, K, groups: cut tiles and blocks on every side; several groups,
# of whole and (384 features) half tiles of a pair. Up to 8 tokens with e4m3
# results take the 16-token clusters.
FORMS = [
    ("few", 5, 300, 400, 1), ("few", 8, 128, 256, 3),
    ("cluster16", 13, 272, 400, 1), ("cluster16", 16, 256, 128, 3),
    ("cluster32", 31, 272, 400, 1), ("cluster32", 20, 384, 256, 2),
    ("cluster64", 60, 272, 2064, 1), ("cluster64", 100, 128, 2048, 3),
    ("tiles", 300, 400, 272, 1), ("tiles", 200, 384, 256, 2),
    ("pairs", 4097, 2032, 272, 1), ("pairs", 2300, 384, 256, 3), ("pairs", 4096, 1024, 128, 2),
]


def form(M, N, K, groups, dt):
    return abi.csa_debug_fp8_proj_form(M, N, K, groups, dt)


def test_every_kernel_is_reached_with_every_result_and_groups():
    build.build()
    seen = {(form(M, N, K, G, dt), dt, G > 1) for _, M, N, K, G in FORMS
            for dt in (BF, F) + ((F8,) if N % 16 == 0 else ())}
    want = {(f, dt, g) for f in abi.FP8_PROJ_FORMS for dt in (BF, F, F8) for g in (False, True)}
    assert seen == want - {("few", F8, False), ("few", F8, True)}
    for bad in ((4, 128, 24, 1), (4, 120, 128, 2), (-1, 128, 128, 1), (4, 0, 128, 1)):
        with pytest.raises(abi.CsaError):
            form(*bad, BF)
    with pytest.raises(abi.CsaError):
        form(4, 24, 128, 1, F8)


@pytest.mark.parametrize("M,N", [(256, 2048), (333, 1000), (1000, 384), (64, 8192)])
def test_long_or_unaligned_rows_over_few_tiles_take_clusters(M, N):
    build.build()
    assert form(M, N, 2048, 1, BF) == "tiles"
    for K in (2064, 2576, 4096, 4112, 8192):
        assert form(M, N, K, 1, BF) == "cluster64", K


@gpu
@pytest.mark.parametrize("kernel,M,N,K,groups", FORMS)
def test_every_kernel_matches_oracle(kernel, M, N, K, groups):
    host = operands(M + N + K, M, N, K, groups)
    ops = device(*host)
    r, err = reference(*host, groups)
    for dt in (BF, F) + ((F8,) if N % 16 == 0 else ()):
        assert form(M, N, K, groups, dt) == (kernel if M > 8 or dt != F8 else "cluster16")
        out, osc = proj8.run(ops, groups * N, dt, groups)
        check(out, osc, r, err, "%s %s" % (kernel, dt))


# special values need two blocks of inputs, an infinite scale a last scale block
# that is cut
SPECIAL = [(5, 272, 400, "few"), (13, 272, 400, "cluster16"), (31, 272, 400, "cluster32"),
           (60, 272, 2064, "cluster64"), (300, 400, 272, "tiles"), (4097, 1936, 400, "pairs")]


@gpu
@pytest.mark.parametrize("M,N,K,kernel", SPECIAL)
def test_special_values_through_every_kernel(M, N, K, kernel):
    assert form(M, N, K, 1, F) == kernel
    proj8.test_fp8_proj_zero_rows_blocks_and_special_codes(M, N, K)
    proj8.test_fp8_proj_infinite_rows_behind_the_last_feature(M, N, K)


@gpu
@pytest.mark.parametrize("kernel,M,N,K,groups", FORMS)
def test_a_rows_result_does_not_depend_on_other_rows(kernel, M, N, K, groups):
    """Other rows' codes and scales changed, to NaN and infinity among others:
    the rows that stay have the same bits."""
    A, As, W, Ws = operands(M + N, M, N, K, groups)
    gen = np.random.default_rng(K)
    keep = np.zeros(M, bool)
    keep[gen.choice(M, max(1, M // 5), replace=False)] = keep[M - 1] = True
    B, Bs = gen.integers(0, 256, A.shape, dtype=np.uint8), As * gen.choice([0.0, 1e30, 3.0], As.shape)
    Bs[gen.random(As.shape) < 0.1], Bs[gen.random(As.shape) < 0.1] = np.inf, np.nan
    B[keep], Bs[keep] = A[keep], As[keep]
    for dt in (BF, F) + ((F8,) if N % 16 == 0 else ()):
        one, s1 = proj8.run(device(A, As, W, Ws), groups * N, dt, groups)
        two, s2 = proj8.run(device(B, Bs.astype(np.float32), W, Ws), groups * N, dt, groups)
        assert torch.equal(one[keep].view(torch.uint8), two[keep].view(torch.uint8))
        assert dt != F8 or torch.equal(s1[keep], s2[keep])


# ---------------------------------------------------------------- e4m3 results

@gpu
@pytest.mark.parametrize("M,N,K,groups", [
    (5, 256, 16, 1), (31, 144, 144, 1), (60, 256, 2048, 1), (700, 400, 16, 1),
    (2300, 384, 128, 3),
])
def test_e4m3_results_on_a_tie_round_to_even(M, N, K, groups):
    """Sums that are exact in float32, over scales whose reciprocals are not:
    r = k t with a scale of k, t halfway between two codes."""
    gen = np.random.default_rng(M)
    base = gen.integers(8, 16, (groups * N,)) * 2.0 ** gen.integers(-7, 5, groups * N)
    half = 2.0 ** (np.floor(np.log2(base)) - 4)      # half a step of the code
    base[::16], half[::16] = 448.0, 0.0               # every scale's block has one
    A = np.zeros((M, groups, K))
    A[:, :, :2] = 1.0
    W = np.zeros((groups * N, K))
    W[:, 0], W[:, 1] = base, half

    def f8(v):
        t = torch.from_numpy(v).to(F8)
        assert np.array_equal(t.double().numpy(), v)
        return t.to(DEV)

    k = np.arange(1, M + 1, dtype=np.float32)
    As = torch.from_numpy(k).to(DEV)[:, None].expand(M, groups * nb(K)).contiguous()
    out = torch.empty(M, groups * N, device=DEV, dtype=F8)
    scale = torch.empty(M, nb(groups * N), device=DEV)
    abi.csa_fp8_proj(f8(A.reshape(M, -1)), As, f8(W),
                     torch.ones(nb(groups * N), nb(K), device=DEV), out, scale, groups=groups)
    abi.csa_get_error()
    assert (scale.cpu().numpy() == k[:, None]).all()
    want = torch.from_numpy(base + half).to(F8)       # to nearest, ties to even
    assert not np.array_equal(want.double().numpy(), base + half)
    assert torch.equal(out.cpu().view(torch.uint8),
                       want.view(torch.uint8)[None].expand(M, groups * N))


@gpu
@pytest.mark.parametrize("M,N,K,groups", [
    (12, 512, 1024, 1), (32, 1040, 400, 1), (64, 272, 2048, 1), (1000, 2032, 272, 1),
    (4096, 2048, 272, 1), (2300, 384, 256, 3),
])
def test_e4m3_results_are_the_storage_of_the_float32_results(M, N, K, groups):
    """The same kernel's float32 results, stored by csa_add_norm_quant."""
    ops = device(*operands(M + N, M, N, K, groups))
    GN = groups * N
    r = torch.empty(M, GN, device=DEV)
    abi.csa_fp8_proj(*ops, r, groups=groups)
    want = torch.empty(M, GN, device=DEV, dtype=F8), torch.empty(M, nb(GN), device=DEV)
    abi.csa_add_norm_quant(r, normalise=False, codes=want[0], scale=want[1])
    got = torch.empty_like(want[0]), torch.empty_like(want[1])
    abi.csa_fp8_proj(*ops, *got, groups=groups)
    abi.csa_get_error()
    assert torch.equal(got[1], want[1])
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8))


# ---------------------------------------------------------------- waits

@gpu
def test_lanes_of_a_warp_give_up_together():
    """A wait that one lane of a warp gives up is given up by all 32, whatever
    the others see (and in bounded time)."""
    abi.load()
    abi.csa_get_error()
    abi.csa_debug_wait_probe(1_000_000)
    with pytest.raises(abi.CsaError, match="kernel 8, detail 0 32") as ei:
        abi.csa_get_error()
    assert ei.value.status == -4
    assert abi.csa_get_error() == 0


# ---------------------------------------------------------------- threads

@gpu
def test_calls_from_several_threads():
    """Threads that call at the same time, each on its stream, through the few-token,
    cluster, single-tile and pair kernels, get the bits of a call alone."""
    shapes = [(5, 512, 1024, 1), (24, 512, 1024, 1), (300, 512, 512, 1), (2300, 384, 128, 3)]
    work = []
    for i, (M, N, K, G) in enumerate(shapes):
        ops = device(*operands(i, M, N, K, G))
        want = torch.empty(M, G * N, device=DEV)
        abi.csa_fp8_proj(*ops, want, groups=G)
        work.append((ops, G, want))
    torch.cuda.synchronize()
    start = threading.Barrier(8, timeout=60)

    def run(t):
        stream = torch.cuda.Stream()
        outs = [torch.empty_like(w[2]) for w in work]
        start.wait()
        for r in range(20):
            ops, G, _ = work[(t + r) % len(work)]
            abi.csa_fp8_proj(*ops, outs[(t + r) % len(work)], groups=G, stream=stream)
        stream.synchronize()
        return [torch.equal(o, w[2]) for o, w in zip(outs, work)]

    with ThreadPoolExecutor(8) as pool:
        assert all(all(same) for same in pool.map(run, range(8)))
    abi.csa_get_error()
