"""What kda_latent_decode8 leaves of weights far below a row's largest."""
import math

import pytest
import torch

from tests import latent8_helpers as h8
from tests.test_gpu_latent8 import run_decode8

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


# A weight's last part ends 2^-21 below the largest one of the 16,384 tokens that are summed together, so each of them is off by 2^-22 at
# most and the sum by 2^-8 max |x| where all are (the log-sum-exp counts them as they are); 2^-12 is a weight's rounding otherwise, 2^-8 of
# the output its own.
@pytest.mark.parametrize("below", [12.0, 19.5, 21.5, 22.5, 26.0])
@pytest.mark.parametrize("first", [True, False])
def test_one_token_that_outweighs_16383_others(below, first):
    dl, n, R, H = 256, 16384, 304, 32  # two requests to a CTA: each is summed in one
    x = torch.zeros(n, dl + 64)
    x[:, :dl] = torch.randint(0, 2, (n, dl), generator=torch.Generator().manual_seed(4)) * 2.0 - 1.5
    x[:, dl] = 8.0
    x[0 if first else n - 1, dl] = 0
    cache = h8.poisoned_pages(n // 64, 64, dl)
    rows = torch.cat([h8.put(cache, dl, j, slice(0, 64), x[64 * j:64 * j + 64]) for j in range(n // 64)])
    table = torch.arange(n // 64, dtype=torch.int32, device=DEV).expand(R, -1).contiguous()
    q = torch.zeros(R, 1, H, dl + 64, dtype=BF, device=DEV)
    q[..., dl] = -1
    scale = below * math.log(2) / 8
    out, lse = run_decode8(q, cache, table, torch.full((R,), n, dtype=torch.int32, device=DEV), dl, scale)
    z = -rows[:, dl] * scale
    p = torch.softmax(z, 0)
    want, mag = p @ rows[:, :dl], p @ rows[:, :dl].abs()
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -8 * rows[:, :dl].abs().amax() + 2.0 ** -12 * mag
    assert ((out.double().cpu() - want).abs() <= tol).all()
    assert (lse.double().cpu() - torch.logsumexp(z, 0)).abs().max() <= 1e-5 + 2.0 ** -17 * below
