"""What a product kept in float32 for its backward refuses (no GPU: every call fails before anything
is enqueued)."""
import pytest
import torch

from chunked_linear_recurrence_amd import ssd
from test_ffn_checks import P, dims, gated_fwd, lib, linear_fwd

z = torch.zeros
WIDE = ssd.SSD_FLAG_PRE_F32


def test_flags():
    for fwd in (linear_fwd, gated_fwd):
        assert fwd(dims(), flags=8 | 32 | WIDE) == 2 and fwd(dims(), flags=8 | 64 | WIDE) == 2
    assert gated_fwd(dims(), flags=WIDE) == 2                       # an activation is needed
    L = lib()
    assert L.ssd_linear_bwd_workspace_bytes(dims(), 8 | WIDE) == L.ssd_linear_bwd_workspace_bytes(dims(), 8)
    assert L.ssd_linear_bwd_workspace_bytes(dims(), WIDE) == L.ssd_linear_bwd_workspace_bytes(dims(), 0)


def test_alignment_and_extent():
    """bfloat16 [40, 16] (gated [40, 32]) in float32: 4 bytes an element, 2560 (5120) in all."""
    for fwd, n in ((linear_fwd, 40 * 16 * 4), (gated_fwd, 40 * 32 * 4)):
        assert fwd(dims(dtype=1), flags=8 | WIDE, pre=P[5] + 2) == 5
        assert fwd(dims(dtype=1), flags=8 | WIDE, pre=P[4] - n + 4) == 8
    L = lib()
    for name, n in (("ssd_linear_bwd", 40 * 16 * 4), ("ssd_gated_bwd", 40 * 32 * 4)):
        def bwd(pre):
            return getattr(L, name)(dims(dtype=1), P[0], P[1], P[2], pre, P[4], P[5], P[6], 8 | WIDE, P[7], 1 << 33, None)
        assert bwd(P[3] + 2) == 5 and bwd(P[4] - n + 4) == 8


def test_binding():
    lib()
    x, w = z(5, 8).bfloat16(), z(6, 8).bfloat16()
    for call, msg in ((lambda: ssd.linear_fwd(x, w, act="silu", keep=torch.float16), "keep must be"),
                      (lambda: ssd.gated_fwd(x, w, keep=torch.float64), "keep must be"),
                      (lambda: ssd.gated_fwd(x.float(), w.float(), keep=torch.bfloat16), "keep must be"),
                      (lambda: ssd.linear_bwd(z(5, 6).bfloat16(), x, w, None, z(5, 6).half(), act="silu"), "pre has dtype"),
                      (lambda: ssd.linear_bwd(z(5, 6), x.float(), w.float(), None, z(5, 6).bfloat16(), act="silu"), "pre has dtype"),
                      (lambda: ssd.gated_bwd(z(5, 3).bfloat16(), x, w, None, z(5, 5)), "pre has shape"),
                      (lambda: ssd.gated_bwd(z(5, 3).bfloat16(), x, w, None, z(5, 6)), "CUDA device")):
        with pytest.raises(ValueError, match=msg):
            call()
