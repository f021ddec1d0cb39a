"""csa_add_norm_quant: what an infinity in a row gives."""
import numpy as np
import pytest
import torch

from long_context_sparse_07_b200 import abi
from test_gpu_proj8 import DEV, F8, nb, rows_of

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("rows,d,dt", [(6, 272, F), (6, 272, BF), (3, 4096, BF), (2, 20480, BF),
                                       (400, 20480, BF), (160, 8208, F), (300, 10256, BF)])
def test_infinity(rows, d, dt):
    """As the header states it, with and without the norm, in a row with finite
    neighbours."""
    x = rows_of(rows, rows, d, dt)
    x[1, 130] = float("inf")
    y = torch.empty(rows, d, device=DEV, dtype=dt)
    c, s = torch.empty(rows, d, device=DEV, dtype=F8), torch.empty(rows, nb(d), device=DEV)
    abi.csa_add_norm_quant(x.to(DEV), y=y, codes=c, scale=s)
    cf, yf, other = c.float().cpu(), y.float().cpu(), np.arange(d) // 128 != 1
    place = np.arange(d) == 130
    assert yf[1, 130].isnan() and (yf[1][~place] == 0).all()
    assert cf[1, 128:256].isnan().all() and (cf[1][other] == 0).all()
    blocks = np.arange(nb(d)) != 1
    assert s[1, 1].isnan() and (s[1].cpu()[blocks] == 2.0 ** -126).all()
    rest = np.arange(rows) != 1
    assert yf[rest].isfinite().all() and cf[rest].isfinite().all()
    abi.csa_add_norm_quant(x.to(DEV), normalise=False, codes=c, scale=s)
    cf = c.float().cpu()
    assert s[1, 1] == float("inf") and s[1].cpu()[blocks].isfinite().all()
    assert cf[1, 130].isnan() and (cf[1, 128:256][np.arange(128) != 2] == 0).all()
    assert cf[1][other].isfinite().all() and cf[rest].isfinite().all()
    abi.csa_get_error()
