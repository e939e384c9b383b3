"""Use of the training operators beyond single calls on one stream: the drift of long sums."""
import pytest
import torch

import matrix_orthogonalising_optimizer_gb300 as pkg
from test_ops import gen


@pytest.mark.gpu
def test_long_sums_have_no_bias():
    """The mean relative error of sums of 140000 positive terms, more than are left in one
    chain of tensor-core additions.  Rounding the results averages out over 10^6 of them
    (2^-9 / 1000); truncated additions do not, and are to stay below 2^-13."""
    n, d = 140000, 1024
    g = gen(4)
    x = torch.rand(n, d, generator=g, device="cuda").mul_(1 / 32).bfloat16()
    dy = torch.rand(n, d, generator=g, device="cuda").bfloat16()
    wg, wu, wd = (torch.rand(d, d, generator=g, device="cuda").mul_(1 / 32).bfloat16() for _ in range(3))
    _, saved, h = pkg.gated_ffn(x, wg, wu, wd, save="compact")
    dwd = pkg.gated_ffn_backward(dy, x, wg, wu, wd, saved, h)[3].double()
    want = torch.zeros(d, d, device="cuda", dtype=torch.double)
    for i in range(0, n, 20000):
        want += dy[i:i + 20000].double().T @ h[i:i + 20000].double()
    assert abs(float(((dwd - want) / want).mean())) <= 2.0 ** -13
