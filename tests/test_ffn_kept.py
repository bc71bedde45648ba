"""What the functions with gradients keep for a backward: nothing where none can follow.  No GPU:
the library is replaced by one that records its arguments."""
import pytest
import torch

from chunked_linear_recurrence_amd import block, ssd

z = torch.zeros


@pytest.fixture
def calls(monkeypatch):
    """The arguments of every entry point called, by name."""
    seen = {}

    class Library:
        def __getattr__(self, name):
            def entry(*args):
                seen[name] = args
                return 64 if name.endswith("_bytes") else 0
            return entry
    monkeypatch.setattr(ssd, "lib", lambda: Library())
    monkeypatch.setattr(ssd, "_elsewhere", lambda t, stream: None)
    monkeypatch.setattr(ssd, "_current", lambda t: 0)
    return seen


def kept(calls):
    """Whether pre was asked for by linear and gated, and stats by residual_norm."""
    return [calls["ssd_linear_fwd"][6] is not None, calls["ssd_gated_fwd"][5] is not None,
            calls["ssd_residual_norm_fwd"][10] is not None]


def run(x, w, one):
    y = block.linear(x, w, act="silu")
    h = block.gated(x, w)
    n, total = block.residual_norm(x, pre_weight=one)
    return y, h, n, total


def test_kept_where_a_backward_can_follow(calls):
    for given in range(3):
        t = [z(5, 8), z(6, 8), z(8)]
        t[given].requires_grad_(True)
        run(*t)
        assert kept(calls) == [given < 2, given < 2, given != 1], given


def test_nothing_kept_without_gradients(calls):
    t = [z(5, 8).requires_grad_(True), z(6, 8).requires_grad_(True), z(8).requires_grad_(True)]
    for context in (torch.no_grad(), torch.inference_mode()):
        with context:
            out = run(*t)
        assert kept(calls) == [False] * 3 and not any(v.requires_grad for v in out)
    run(z(5, 8), z(6, 8), z(8))
    assert kept(calls) == [False] * 3


def test_tangents_are_refused(calls):
    """Forward mode has no formula here: a call that dropped the tangent would answer with none."""
    one, w = z(8), z(6, 8)
    with torch.autograd.forward_ad.dual_level():
        x = torch.autograd.forward_ad.make_dual(z(5, 8), torch.ones(5, 8))
        for grad in (True, False):
            for f in (lambda: block.linear(x, w), lambda: block.gated(x, w), lambda: block.residual_norm(x, pre_weight=one)):
                with torch.set_grad_enabled(grad), pytest.raises(NotImplementedError, match="jvp"):
                    f()


def test_what_is_no_tensor_is_named(calls):
    for grad in (True, False):
        with torch.set_grad_enabled(grad):
            for f, msg in ((lambda: block.linear([1.0], z(6, 8)), "x must be a torch.Tensor"),
                           (lambda: block.linear(z(5, 8), [1.0]), "weight must be a torch.Tensor"),
                           (lambda: block.gated(None, z(6, 8)), "x must be a torch.Tensor"),
                           (lambda: block.residual_norm(None, pre_weight=z(8)), "branch must be a torch.Tensor")):
                with pytest.raises(ValueError, match=msg):
                    f()
