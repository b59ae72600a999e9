"""Sizes at which the gated delta rule takes another path."""

import os

import pytest

import mamba_selective_scan_ssm_amd as ssm

BF16 = 1


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
