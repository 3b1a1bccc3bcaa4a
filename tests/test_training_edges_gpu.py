"""Edges of the training operators (GPU): eps = 0 and rows that leave a block
part empty, values whose squares are near the smallest float, constant rows,
the widths at which a path ends."""
import pytest
import torch

import _train64 as ref
from _train64 import TYPES, close, make
from row_wise_rmsnorm_fwd_gb300 import binding, build

pytestmark = pytest.mark.gpu

PATHS = [None, {"path": "twopass"}]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    yield
    torch.cuda.synchronize()


def rms_bwd(dy, x, w, eps, options=None):
    got = binding.rmsnorm_bwd_ex(*(None if v is None else v.cuda() for v in (dy, x, w)), eps=eps,
                                 options=options)
    want, tol = ref.rmsnorm_bwd(dy, x, w, eps)
    for g, r, e, n in zip(got, want, tol, ("dx", "dw")):
        close(g, r, e, f"{n} of {tuple(x.shape)}")


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("hidden", [16, 64, 333, 512, 768, 1001, 2048, 2050, 4096, 5120, 8192, 8200])
def test_rmsnorm_backward_with_eps_zero(hidden, t, options):
    """The rows that a block lacks add nothing to dw, although their sum of
    squares is 0."""
    for rows in (1, 2, 3, 4, 5, 7, 8, 9, 13, 16, 17):
        x, dy = make((rows, hidden), t, rows, std=2.0), make((rows, hidden), t, rows + 50)
        rms_bwd(dy, x, make((hidden,), t, 3, mean=1.0, std=0.1), 0.0, options)
        if rows == 3:
            rms_bwd(dy, x, None, 0.0, options)
