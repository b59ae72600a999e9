"""Sizes at which the gated delta rule and the group norm take another path or
refuse, on the host (a rejected call never reaches the device)."""

import ctypes
import os

import pytest

import mamba_selective_scan_ssm_amd as ssm

OK, UNSUPPORTED = 0, 2
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssm.LIB_PATH):
        pytest.skip("libssmscan.so not built")
    return ssm.lib()


def test_chunks_within_a_grid(lib):
    """2^23 workgroups of 512 threads are a dimension's 2^32: from there on by tokens,
    whose workspace does not follow the alignment."""
    size = lib.ssm_gdr_bwd_workspace_size
    by_chunks = [(65535, 32, 127, 1, 1, 8, BF16), (1, 1 << 28, 1, 1, 1, 8, BF16)]
    by_tokens = [(65535, 32, 129, 1, 1, 8, BF16), (65529, 32, 128, 1, 1, 8, BF16), (1, 1 << 29, 1, 1, 1, 8, BF16)]
    for c in by_chunks:
        assert 0 < size(*c, 1) != size(*c, 0) > 0, c
    for c in by_tokens:
        assert size(*c, 1) == size(*c, 0) > 0, c


def test_norm_channels(lib):
    """Fewer than 2^31 channels, whatever the rows."""
    P = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(12)]

    def fwd(S, T, D, G):
        return lib.ssm_group_norm_fwd(S, T, D, G, F32, P[0], None, None, None, 1e-5, 0, 0, 0, P[1], None, None, None, 0,
                                      None)

    def bwd(S, T, D, G):
        return lib.ssm_group_norm_bwd(S, T, D, G, F32, *P[:7], 1e-5, 0, 0, 0, *P[7:11], None, 0, None)
    assert fwd(0, 1, (1 << 31) - 1, 1) == OK
    for f in (fwd, bwd):
        assert f(0, 1, 1 << 31, 1) == UNSUPPORTED
        assert f(2, 1, 1 << 30, 1) == UNSUPPORTED
