"""csa_add_norm_quant where a block of threads takes several rows one after the
other, and what an infinity in a row gives. Tolerances as in test_gpu_proj8."""
import numpy as np
import pytest
import torch

import test_gpu_proj8 as proj8
from long_context_sparse_07_b200 import abi
from test_gpu_proj8 import DEV, F8, nb, rows_of

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32

# rows of which a block takes a third: at most 740, 148, 1480 and 148 of these
# widths are resident at once (148 SMs, the blocks that their registers allow)
LOOPS = [(1537, 2064, F, True), (1537, 2064, F, False), (1000, 8192, F, True),
         (1000, 8192, F, False), (5000, 1040, BF, True), (5000, 1040, BF, False),
         (600, 9216, BF, True), (600, 9216, BF, False)]


@pytest.mark.parametrize("rows,d,dt,res", LOOPS)
def test_rows_in_turn_match_oracle(rows, d, dt, res):
    proj8.test_add_norm_quant_matches_oracle(rows, d, dt, res, True, True)


@pytest.mark.parametrize("rows,d,dt,res", LOOPS)
def test_rows_in_turn_in_place_and_alone(rows, d, dt, res):
    """total over residual and y over x, and each row in a call of few rows, give
    the same bits."""
    x = rows_of(rows, rows, d, dt).to(DEV)
    r = rows_of(rows + 1, rows, d, dt).to(DEV) if res else None
    g = torch.rand(d, device=DEV) + 0.5

    def call(x, r, total, y):
        n = x.shape[0]
        c, s = torch.empty(n, d, device=DEV, dtype=F8), torch.empty(n, nb(d), device=DEV)
        abi.csa_add_norm_quant(x, r, g, total=total, y=y, codes=c, scale=s)
        return c.view(torch.uint8), s

    total, y = torch.empty_like(x) if res else None, torch.empty_like(x)
    c, s = call(x, r, total, y)
    x2, r2 = x.clone(), r.clone() if res else None
    c2, s2 = call(x2, r2, r2, x2)
    assert torch.equal(x2, y) and torch.equal(c2, c) and torch.equal(s2, s)
    assert not res or torch.equal(r2, total)
    # rows of up to 8192 are summed alike whatever the number of rows
    if d <= 8192:
        for lo in (0, rows // 2, rows - 3):
            part = slice(lo, lo + 3)
            y3 = torch.empty(3, d, device=DEV, dtype=dt)
            c3, s3 = call(x[part], r[part] if res else None, None, y3)
            assert torch.equal(y3, y[part]) and torch.equal(c3, c[part]) and torch.equal(s3, s[part])
    abi.csa_get_error()


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
