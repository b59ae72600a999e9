"""Group norm over sequences with tokens far from the others (a first token's large
activations) and long sums of equal terms, held to the common bar."""

import pytest
import torch

from tests.test_gpu_gdr import _say
from tests.test_gpu_mixer_limits import near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", [None, "before"])
@pytest.mark.parametrize("T", [9, 1000, 16384, 262145])
@pytest.mark.parametrize("what", ["first token", "every 256th token", "equal squares"])
def test_outliers(what, T, gate):
    import mamba_selective_scan_ssm_amd as ssm
    _say("group_norm outliers", what, T, gate)
    D, G = 32, 4
    g = torch.Generator("cuda").manual_seed(110)
    x = torch.randn(1, T, D, device="cuda", generator=g)
    z = torch.randn(1, T, D, device="cuda", generator=g) + 2 if gate else None
    if what == "first token":
        x[:, 0] += 1000
    elif what == "every 256th token":
        x[:, ::256] += 1000
    else:
        x = 1.1 * x.sign()
    for center in (True, False):
        y, _, _ = ssm.group_norm_fwd(x, G, z=z, gate=gate, per_token=False, center=center)
        u = x.double() * (torch.nn.functional.silu(z.double()) if gate else 1)
        u = u.view(1, T, G, D // G)
        u = u - u.mean((1, 3), keepdim=True) if center else u
        near(y, (u * (u.square().mean((1, 3), keepdim=True) + 1e-5).rsqrt()).view(1, T, D), (what, T, center))
