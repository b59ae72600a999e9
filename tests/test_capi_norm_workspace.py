"""The group norm asks for the workspace of the path that a call takes, on the host
(a rejected call never reaches the device)."""

import ctypes
import os

import pytest

import mamba_selective_scan_ssm_amd as ssm

WORKSPACE = 3
F32, BF16 = 0, 1
P = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssm.LIB_PATH):
        pytest.skip("libssmscan.so not built")
    return ssm.lib()


def test_rows_need_none(lib):
    """Per token, a group in registers: nothing forwards, and backwards less than the
    channels' sums of 1024 blocks of rows."""
    fwd, bwd = lib.ssm_group_norm_fwd_workspace_size_ex, lib.ssm_group_norm_bwd_workspace_size_ex
    for W, dt in ((4096, BF16), (5120, BF16), (10240, BF16), (4096, F32), (5120, F32)):
        assert fwd(1 << 15, 1, W, 1, dt, 1) == 0, (W, dt)
    for W, dt in ((4096, BF16), (6144, BF16), (4096, F32)):
        assert 0 < bwd(1 << 15, 1, W, 1, dt, 1) <= 8 * 1024 * W, (W, dt)
    # single elements of more than 2048 channels, over sequences, and more than the registers hold:
    # two sums an element, or of 8 tokens
    assert fwd(64, 1, 4096, 1, BF16, 0) >= 8 * 64 * 4096
    assert fwd(64, 1, 10248, 1, BF16, 1) >= 8 * 64 * 10248
    assert fwd(8, 64, 512, 4, BF16, 1) >= 8 * 8 * 8 * 512
    assert fwd(64, 1, 4097, 1, BF16, 1) == fwd(64, 1, 4097, 1, BF16, 0) > 0  # no whole pieces


def test_the_most_of_any_type_and_alignment(lib):
    for S, T, D, G in ((7, 1, 4096, 1), (7, 1, 6144, 2), (64, 1, 640, 8), (3, 40, 640, 32), (5, 1, 8192, 1), (9, 1, 4097, 1),
                       (2, 1, 20000, 1)):
        for f in ("fwd", "bwd"):
            most = getattr(lib, f"ssm_group_norm_{f}_workspace_size")(S, T, D, G)
            each = [getattr(lib, f"ssm_group_norm_{f}_workspace_size_ex")(S, T, D, G, dt, al) for dt in (F32, BF16)
                    for al in (0, 1)]
            assert most == max(each), (f, S, T, D, G)
    assert lib.ssm_group_norm_fwd_workspace_size_ex(64, 1, 20000, 1, F32, 2) == 0
    assert lib.ssm_group_norm_fwd_workspace_size_ex(64, 1, 20000, 1, 7, 1) == 0


def test_a_call_is_held_to_its_own(lib):
    def fwd(x, D, dt, ws_len):
        return lib.ssm_group_norm_fwd(64, 1, D, 1, dt, x, None, None, None, 1e-5, 0, 0, 0, P[1], None, None, P[2], ws_len,
                                      None)
    need = lib.ssm_group_norm_fwd_workspace_size_ex(64, 1, 4096, 1, BF16, 0)
    off = ctypes.c_void_p(P[0].value + 2)
    assert fwd(off, 4096, BF16, need - 1) == WORKSPACE
    assert fwd(P[0], 10248, BF16, lib.ssm_group_norm_fwd_workspace_size_ex(64, 1, 10248, 1, BF16, 1) - 1) == WORKSPACE
