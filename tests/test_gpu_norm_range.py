"""The norm's gradient near the ends of fp32's range: the sum over a row, which a mean follows, is larger than
what comes of it. Within the bounds of test_gpu_norm."""
import pytest
import torch

import routing_permute_mxfp8_amd as rp
from gpu_support import say
from oracle import dense
from test_gpu_norm import EPS, TYPES, check_backward, f64, on, rows_of, weight_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [100, 500, 1001, 1024, 7168, 16384])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [1e36, 1e-33])
def test_gradients_of_any_size(cols, dtype, size):
    """Gradients whose products with xh, added over a row, pass fp32's largest value while their mean and all
    results are far from it; and tiny ones, whose sum must not lose bits. fp16 rows: 5e3 and 1e-5 (a and
    xh dot are at most 1.2 x 5e3 x 2.5 and 5 x 1.3 x 5e3, rstd 1.2: all results are fp16 numbers)."""
    if dtype == torch.float16:
        size = 5e3 if size > 1 else 1e-5
    say(f"rms_norm_backward {cols} columns {dtype}, gradients of {size:g}")
    h, w = rows_of(20, cols, dtype, spread=0.1), weight_of(cols, torch.float32)
    sign = torch.sign(h.double())   # every product with xh is positive
    gy = (sign * size * (1 + 0.2 * torch.rand((20, cols), generator=torch.Generator().manual_seed(3)).double())).to(dtype)
    rstd = torch.from_numpy(dense.rms_norm(f64(h), f64(w), EPS)[1]).float()
    got = rp.rms_norm_backward(on(gy), on(h), on(w), on(rstd))
    assert bool(got[1].isfinite().all())
    check_backward(gy, h, w, rstd, None, got)
