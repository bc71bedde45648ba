"""Calls of the operators around a scan whose work exceeds what a launch can hold (2^32 threads
along a dimension): refused as unsupported, before anything is enqueued.  No GPU: the addresses
are never dereferenced."""
import pytest

from chunked_linear_recurrence_amd import ssd

P = [(1 << 46) + (k << 41) for k in range(32)]      # aligned, 2 TiB apart
WS = 1 << 41
UNSUPPORTED = 4


def lib():
    try:
        return ssd.lib()
    except RuntimeError:
        pytest.skip("libssdscan.so not built")


def conv(b, L, C, W=4):
    return ssd.ConvDims(b, L, C, W, 0, L * C, C, L * C, C)


def sel(b, L, D, N):
    return ssd.SelectiveDims(b, L, D, N, 1, 0, 0, *([L * D, D] * 3 + [L * N, N] * 2 + [L * D, D]))


def conv_bwd(d):
    return lib().ssd_conv_bwd(d, *P[:11], 0, P[11], WS, None)


def sel_bwd(d):
    return lib().ssd_selective_bwd(d, *P[:21], 16, P[21], WS, None)


CASES = {
    "conv_fwd": lambda: lib().ssd_conv_fwd(conv(1 << 24, 1, 1), *P[:7], 0, None),
    "conv_step": lambda: lib().ssd_conv_step(conv(1 << 28, 1, 64), *P[:6], 0, None),
    "conv_bwd": lambda: conv_bwd(conv(1 << 24, 1, 1)),
    "conv_bwd, sums": lambda: conv_bwd(conv(1, 1, 1 << 26)),
    "selective_fwd": lambda: lib().ssd_selective_fwd(sel(1 << 26, 1, 1, 16), *P[:13], 16, P[13], WS, None),
    "selective_step": lambda: lib().ssd_selective_step(sel(1 << 20, 1, 1024, 16), *P[:11], 16, None),
    "selective_bwd": lambda: sel_bwd(sel(1 << 24, 1, 1, 16)),
    "selective_bwd, sums for B and C": lambda: sel_bwd(sel(1, 1 << 25, 64, 64)),
    "selective_bwd, sums for A": lambda: sel_bwd(sel(1, 1, 64 * 63551, 64)),
    "norm_fwd": lambda: lib().ssd_norm_fwd(ssd.NormDims(1 << 22, 8193, 0, 0, 8193, 8193), *P[:3], 1e-5, *P[3:6], None),
    "norm_bwd": lambda: lib().ssd_norm_bwd(ssd.NormDims(1 << 22, 8193, 0, 0, 8193, 8193), *P[:9], WS, None),
    "norm_bwd, sums": lambda: lib().ssd_norm_bwd(ssd.NormDims(1, (1 << 27) - 1, 0, 0, 0, 0), *P[:9], WS, None),
}


@pytest.mark.parametrize("name", CASES)
def test_work_beyond_a_launch_is_refused(name):
    assert CASES[name]() == UNSUPPORTED, lib().ssd_last_error_message()
    assert b"grid" in lib().ssd_last_error_message()
