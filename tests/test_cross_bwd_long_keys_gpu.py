"""GPU tests of attn_bwd_cross in fp16 over keys so many that P is below fp16's
normal numbers."""
import pytest
import torch

from tests import cross_bounds
from tests.test_cross_bwd_gpu import dout, run, saved
from tests.test_cross_gpu import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Nq,Nk,d", [(4, 131072, 64), (150, 40000, 64), (3, 300000, 128)])
def test_dv_keeps_its_digits(Nq, Nk, d):
    """P of nearly equal scores is 1 / Nk.  It is multiplied by 2^15, so half a step
    of its subnormal numbers is 2^-40."""
    q, k, v = make(1, 1, 1, Nq, Nk, d, torch.float16, seed=Nq, scale=0.1)
    do = dout(q, torch.float16, 5, 500.0)
    got = run(q, k, v, *saved(q, k, v, None, d ** -0.5), do, None)
    want, tol = cross_bounds.gradients(q, k, v, do, None, d ** -0.5, 2.0 ** -40, values=True,
                                       p_floor=2.0 ** -40)
    cross_bounds.within(got, want, tol)
