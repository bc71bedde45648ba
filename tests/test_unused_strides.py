"""Strides over a dimension of one element are never used and so refuse nothing and choose
nothing: a view of one row, or of one token, may carry any there."""
import pytest
import torch

from chunked_linear_recurrence_amd import ssd
from test_block_checks import P, conv_dims, conv_fwd, lib, sel_dims, sel_fwd

ALIAS, WORKSPACE, MISALIGNED, SHAPE = 8, 6, 5, 2


def sel_bwd(d):
    return lib().ssd_selective_bwd(d, *P[:21], 16, P[21], 0, None)


def test_one_row_or_one_token_refuses_no_stride():
    """The calls get as far as the check after the strides'."""
    assert sel_fwd(sel_dims(b=1, dtype=1, over={6: 641, 8: 17}), n=0) == WORKSPACE         # batch strides of B and C
    assert sel_bwd(sel_dims(L=1, dtype=1, over={7: 17, 9: 33})) == WORKSPACE               # token strides
    assert sel_bwd(sel_dims(b=1, L=1, dtype=1, over={k: 35 for k in (6, 7, 8, 9)})) == WORKSPACE
    assert sel_bwd(sel_dims(L=1, over={k: 1 << 40 for k in (1, 3, 5, 7, 9, 11)})) == WORKSPACE
    assert sel_fwd(sel_dims(b=1, over={0: -1, 4: -9}), n=0) == WORKSPACE
    assert conv_fwd(conv_dims(b=1, xs=(-7, 16)), y=P[0]) == ALIAS
    assert conv_fwd(conv_dims(L=1, xs=(640, -16)), y=P[0]) == ALIAS
    assert lib().ssd_norm_fwd(ssd.NormDims(1, 32, 0, 0, -1, 0), P[0], None, None, 1e-5, P[0], None, None, None) == ALIAS


def test_strides_that_are_used_are_still_checked():
    assert sel_fwd(sel_dims(dtype=1, over={6: 641}), n=0) == MISALIGNED
    assert sel_fwd(sel_dims(b=1, dtype=1, over={7: 17}), n=0) == MISALIGNED
    assert sel_bwd(sel_dims(L=1, dtype=1, over={6: 641})) == MISALIGNED
    assert conv_fwd(conv_dims(b=1, xs=(640, -16)), y=P[0]) == SHAPE


@pytest.mark.gpu
def test_one_token_out_of_odd_rows():
    """One token's B and C, in bfloat16, on 4 bytes in a row of an odd number of elements."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)
    row, x = randn(1, 1, 35), randn(1, 1, 70)
    A = -torch.rand(70, 16, generator=gen, device="cuda") * 4
    outs = []
    for B, C in ((row[..., :16], row[..., 16:32]), (row[..., :16].contiguous(), row[..., 16:32].contiguous())):
        a = (x, x, A, B.unflatten(-1, (1, 16)), C.unflatten(-1, (1, 16)), None, x, None)
        y, f, kept = ssd.selective_fwd(*a, keep=True)
        outs.append([y, f] + [t for t in ssd.selective_bwd(x, *a, kept) if t is not None])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(*outs))
