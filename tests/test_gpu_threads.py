"""Calls that are the first CUDA call of their thread (a server's worker, say):
such a thread has no current context yet, and each call gives the bits it gives
on the main thread."""
import threading

import numpy as np
import pytest
import torch

from long_context_sparse_07_b200 import abi, path, workloads as W
from test_gpu_proj8 import DEV, F8, device, nb, operands

pytestmark = pytest.mark.gpu


def in_new_thread(f, *args):
    """f(*args) on a thread that has made no CUDA call."""
    raised = []

    def run():
        try:
            f(*args)
        except Exception as e:
            raised.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if raised:
        raise raised[0]


@pytest.mark.parametrize("M,N,K,groups", [(5, 512, 1024, 1), (13, 512, 1024, 1), (60, 256, 2048, 1),
                                          (300, 512, 512, 1), (2300, 384, 128, 3)])
@pytest.mark.parametrize("dt", [torch.bfloat16, F8])
def test_product(M, N, K, groups, dt):
    ops = device(*operands(M, M, N, K, groups))

    def call(res, stream):
        abi.csa_fp8_proj(*ops, *res, groups=groups, stream=stream)

    def result():
        out = torch.zeros(M, groups * N, device=DEV).to(dt)
        return (out, torch.zeros(M, nb(groups * N), device=DEV)) if dt == F8 else (out,)

    want, got = result(), result()
    s = torch.cuda.current_stream().cuda_stream
    call(want, s)
    torch.cuda.synchronize()
    in_new_thread(call, got, s)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    abi.csa_get_error()


def test_steps_of_the_path_and_the_output_projection():
    """Each phase of a prefill, with a fused selection too, and of an HCA prefill
    on a thread of its own, and csa_grouped_out_proj."""
    s = torch.cuda.current_stream().cuda_stream
    w = W.scaled(W.WORKLOADS["csa_bf16_n4096"], n=1024, idx_dtype="e4m3")
    ops = W.csa_operands(w)
    wh = W.scaled(W.WORKLOADS["hca_bf16_n65536"], n=1024)
    for make in (lambda: path.CsaPrefill(w, ops), lambda: path.CsaPrefill(w, ops, fused=True),
                 lambda: path.HcaPrefill(wh, W.hca_operands(wh))):
        p, q = make(), make()
        p.step(s)
        torch.cuda.synchronize()
        for _, f in q.phases():
            in_new_thread(f, s)
            torch.cuda.synchronize()
        assert torch.equal(p.result(), q.result())
    gen = np.random.default_rng(3)
    o, Wg, Wo = (torch.from_numpy(gen.standard_normal(sh).astype(np.float32)).to(DEV, torch.bfloat16)
                 for sh in ((70, 8, 64), (4 * 256, 128), (256, 1024)))
    want = torch.empty(70, 256, device=DEV, dtype=torch.bfloat16)
    u, got = torch.empty(70, 1024, device=DEV, dtype=torch.bfloat16), torch.empty_like(want)
    abi.csa_grouped_out_proj(o, Wg, Wo, 4, u, want)
    torch.cuda.synchronize()
    in_new_thread(abi.csa_grouped_out_proj, o, Wg, Wo, 4, u, got, s)
    torch.cuda.synchronize()
    assert torch.equal(want, got)
    abi.csa_get_error()
