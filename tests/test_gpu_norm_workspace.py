"""A per-token group norm allocates its results and little else."""

import pytest
import torch

from tests import mixer_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,dtype", [(4096, torch.bfloat16), (5120, torch.bfloat16), (4096, torch.float32)])
def test_rms_norm_allocates_its_results(D, dtype):
    import mamba_selective_scan_ssm_amd as ssm
    print("[case] group_norm allocations", D, dtype, flush=True)
    g = torch.Generator().manual_seed(100)
    x, w = torch.randn(4, 512, D, generator=g).to(dtype), 1 + 0.2 * torch.randn(D, generator=g)
    xd, wd = x.cuda(), w.cuda()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    y, _, rstd = ssm.group_norm_fwd(xd, 1, wd, center=False)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before <= 2 * y.numel() * y.element_size()
    ref.close(y, ref.norm(x.double(), 1, w.double(), center=False), "y")
    # unaligned: the other path, with its workspace
    xo = torch.empty(x.numel() + 1, dtype=dtype, device="cuda")[1:].view(x.shape)
    xo.copy_(xd)
    yo, _, _ = ssm.group_norm_fwd(xo, 1, wd, center=False)
    torch.cuda.synchronize()
    ref.close(yo, ref.norm(x.double(), 1, w.double(), center=False), "y of unaligned x")
