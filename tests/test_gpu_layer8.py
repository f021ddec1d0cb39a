"""A whole CSA layer with 8-bit projections on the GPU (path.CsaLayer8): every
stage against the float64 oracle on that stage's own inputs, so that no stage's
rounding hides another's error, and the projections of single tokens against
the prompt's. Tolerances as in test_gpu_proj8 (the products, the norm) and
test_gpu_pipeline (the attention path)."""
import numpy as np
import pytest
import torch

from oracle import proj8
from long_context_sparse_07_b200 import abi, path, workloads as W
from helpers import sample_rows, to_np
from test_gpu_pipeline import run_csa
from test_gpu_proj8 import F8, HALF, U, check_codes, reference, u8

pytestmark = pytest.mark.gpu


def layer_weights(w):
    d = {k: torch.from_numpy(np.ascontiguousarray(v)) for k, v in W.layer_draws(w).items()}
    H = d.pop("H")
    return H, {k: v.to(torch.bfloat16) if k.startswith("W_") else v for k, v in d.items()}


def check_product(what, A8, W8, out, out_scale=None, groups=1):
    r, err = reference(u8(A8[0]), A8[1].cpu().numpy(), u8(W8[0]), W8[1].cpu().numpy(), groups)
    out = out.reshape(r.shape)
    if out_scale is not None:
        check_codes(out, out_scale.reshape(r.shape[0], -1), r, err, what)
    else:
        e = np.abs(to_np(out) - r)
        assert (e <= err + HALF[out.dtype] * np.abs(r)).all(), what


@pytest.mark.parametrize("idx_dtype,rope", [("e4m3", 0), ("bf16", 0), ("e4m3", 64)])
def test_layer_stages_match_oracle(idx_dtype, rope):
    n, g, dg, dout = 768, 4, 256, 1040
    w = W.scaled(W.WORKLOADS["csa_bf16_n4096"], n=n, idx_dtype=idx_dtype)
    H, weights = layer_weights(w)
    gen = torch.Generator().manual_seed(5)
    x = H[:n].to(torch.bfloat16)
    res = torch.randn(x.shape, generator=gen).to(torch.bfloat16)
    gamma = 1 + 0.1 * torch.randn(x.shape[1], generator=gen)
    Wg = (0.02 * torch.randn(g * dg, w.h * w.c // g, generator=gen)).to(torch.bfloat16)
    Wo = 0.02 * torch.randn(dout, g * dg, generator=gen)
    L = path.CsaLayer8(w, x, weights, res, gamma, Wg=Wg, Wo=Wo, g=g, rope_dims=rope)
    L.step()
    abi.csa_get_error()
    P, ops = L.proj, L.proj.ops
    d = x.shape[1]
    s, v = proj8.add_norm(x, res, gamma)
    assert (np.abs(to_np(L.total) - s) <= (2.0 ** -8 + 2 * U) * np.abs(s)).all()
    check_codes(*P.h8, v, (d / 64 + 40) * U * np.abs(v), "hidden")
    for nm, wn in P.FROM_H:
        check_product(nm, P.h8, P.W[wn], ops[nm])
    check_product("wI", P.h8, P.W["W_w"], ops["wI"])
    check_product("cQ", P.h8, P.W["W_DQ"], *P.cq8)
    if not rope:                              # the step turns q in place
        check_product("q", P.cq8, P.W["W_UQ"], ops["q"])
    check_product("qI", P.cq8, P.W["W_IUQ"], ops["qI"], ops.get("qI_scale"))
    # the attention path on the very operands that the projections wrote
    if not rope:
        host = {k: t.cpu() for k, t in L.core.d.items()}
        run_csa(w, sample_rows(n, w.m, 64), ops=host)
        p2 = path.CsaPrefill(w, host)
        p2.step()
        assert torch.equal(p2.out, L.core.out) and torch.equal(p2.idx, L.core.idx)
    o = to_np(L.core.out).reshape(n, -1)
    check_codes(*L.o8, o, 2 * U * np.abs(o), "heads")
    check_product("u", L.o8, L.Wg, *L.u8, groups=g)
    check_product("out", L.u8, L.Wo, L.out)
    assert L.result() is L.out and [k for k, _ in L.phases()][-1] == "proj_out"


def test_projections_of_single_tokens_and_a_captured_step():
    """A decode step's projections (8 tokens, then one) agree with the prompt's
    within both calls' bounds, and a captured step replays them bit for bit."""
    w = W.scaled(W.WORKLOADS["csa_bf16_n4096"], n=200, idx_dtype="e4m3")
    H, weights = layer_weights(w)
    x = H[:200].to("cuda", torch.bfloat16)
    full = path.Projections8(w, weights)
    full.step(x)
    for lo, hi in ((17, 25), (150, 151)):
        few = path.Projections8(w, weights, n=hi - lo)
        xs = x[lo:hi].clone()
        few.step(xs)
        # the same hidden states: a row's norm does not depend on its batch
        assert np.array_equal(u8(few.h8[0]), u8(full.h8[0][lo:hi]))
        for nm, wn in few.FROM_H + (("wI", "W_w"),):
            r, err = reference(u8(few.h8[0]), few.h8[1].cpu().numpy(), u8(few.W[wn][0]),
                               few.W[wn][1].cpu().numpy(), 1)
            for t in (few.ops[nm], full.ops[nm][lo:hi]):
                assert (np.abs(to_np(t) - r) <= err + HALF[t.dtype] * np.abs(r)).all(), nm
        check_product("q", few.cq8, few.W["W_UQ"], few.ops["q"])
        check_product("qI", few.cq8, few.W["W_IUQ"], few.ops["qI"], few.ops["qI_scale"])
        want = {k: t.clone() for k, t in few.ops.items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            few.step(xs)
        for t in few.ops.values():
            t.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, t in few.ops.items():
            assert torch.equal(t.view(torch.uint8), want[k].view(torch.uint8)), k
    abi.csa_get_error()


def test_layer_refuses_workloads_it_cannot_write():
    w = W.WORKLOADS["csa_fp32_n256"]
    with pytest.raises(ValueError, match="bf16"):
        path.Projections8(w, {})
    with pytest.raises(ValueError, match="128"):
        path.Projections8(W.scaled(W.WORKLOADS["csa_bf16_n4096"], idx_dtype="e4m3", cI=64), {})
