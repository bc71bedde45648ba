"""Every tensor of the caller that a binding call writes has its version moved on, so that a
backward that saved the tensor's old values raises instead of reading the new ones.  The
library is replaced by one that does nothing: no GPU."""
import pytest
import torch

from chunked_linear_recurrence_amd import block, ssd


class _Library:
    """Every entry point succeeds; sizes are 64 bytes."""

    def __getattr__(self, name):
        return lambda *args: 64 if name.endswith("_bytes") else 0


@pytest.fixture(autouse=True)
def binding(monkeypatch):
    monkeypatch.setattr(ssd, "lib", lambda: _Library())
    monkeypatch.setattr(ssd, "_elsewhere", lambda t, stream: None)
    monkeypatch.setattr(ssd, "_current", lambda t: 0)
    monkeypatch.setattr(ssd, "_stream", lambda stream: None)
    monkeypatch.setattr(ssd, "_same_device", lambda **tensors: None)


def z(*shape):
    return torch.zeros(*shape)


B, L, C, W, N, H, P = 2, 5, 8, 4, 16, 2, 4


def sel(step):
    lead = (B,) if step else (B, L)
    return z(*lead, C), z(*lead, C), z(C, N), z(*lead, 1, N), z(*lead, 1, N), z(C), z(*lead, C), z(C)


def layer(step=False):
    lead = (B,) if step else (B, L)
    return z(*lead, H, P), z(*lead, H), z(H), z(*lead, 1, N), z(*lead, 1, N), z(H)


def stack():
    x, dt, A, Bm, Cm, D = layer()
    return x, dt, A[None], Bm, Cm, D[None]


CALLS = {   # name: (call, tensors that it writes), all of them the caller's
    "conv_fwd": lambda y, s: ssd.conv_fwd(z(B, L, C), z(C, W), y=y, final_state=s),
    "conv_fwd in place": lambda y, s: ssd.conv_fwd(z(B, L, C), z(C, W), None, s, y=y, final_state=s),
    "conv_step": lambda y, s: ssd.conv_step(z(B, C), z(C, W), None, s, y=y),
    "conv_step out": lambda y, s: ssd.conv_step(z(B, C), z(C, W), None, z(B, W - 1, C), y=y, state_out=s),
    "selective_fwd": lambda y, s: ssd.selective_fwd(*sel(False), y=y, final_state=s),
    "selective_fwd in place": lambda y, s: ssd.selective_fwd(*sel(False), s, y=y, final_state=s),
    "selective_step": lambda y, s: ssd.selective_step(*sel(True), s, y=y),
    "selective_step out": lambda y, s: ssd.selective_step(*sel(True), z(B, C, N), y=y, state_out=s),
    "norm_fwd": lambda y, s: ssd.norm_fwd(z(L, C), y=y),
    "fwd": lambda y, s: ssd.fwd(*layer(), y=y, final_state=s),
    "fwd in place": lambda y, s: ssd.fwd(*layer(), s, y=y, final_state=s),
    "fwd_noalloc": lambda y, s: ssd.fwd_noalloc(*layer(), y=y, final_state=s),
    "segmented": lambda y, s: ssd.segmented(*stack(), s, 5, y=y),
    "horizontal": lambda y, s: ssd.horizontal(*stack(), s),
    "step": lambda y, s: ssd.step(*layer(True), s, y=y),
}


def outputs(name):
    if name.startswith("conv"):
        return z(B, C) if "step" in name else z(B, L, C), z(B, W - 1, C)
    if name.startswith("selective"):
        return z(B, C) if "step" in name else z(B, L, C), z(B, C, N)
    if name == "norm_fwd":
        return z(L, C), None
    if name in ("segmented", "horizontal"):
        return z(B, L, H, P) if name == "segmented" else None, z(1, B, H, P, N)
    return z(B, H, P) if name == "step" else z(B, L, H, P), z(B, H, P, N)


@pytest.mark.parametrize("name", CALLS)
def test_written_tensors_have_a_new_version(name):
    written = outputs(name)
    CALLS[name](*written)
    for t in written:
        assert t is None or t._version > 0, name


def test_a_state_that_is_not_written_keeps_its_version():
    s = z(B, W - 1, C)
    ssd.conv_step(z(B, C), z(C, W), None, s, state_out=z(B, W - 1, C))
    ssd.conv_fwd(z(B, L, C), z(C, W), None, s)
    h = z(B, C, N)
    ssd.selective_step(*sel(True), h, state_out=z(B, C, N))
    ssd.selective_fwd(*sel(False), h)
    assert s._version == 0 and h._version == 0


def test_backward_after_a_step_has_moved_the_saved_state_raises():
    """The convolution's backward reads the state that entered it."""
    x, w, s = z(B, L, C).requires_grad_(True), z(C, W), z(B, W - 1, C)
    for write in (lambda: ssd.conv_step(z(B, C), w, None, s),
                  lambda: ssd.conv_fwd(z(B, L, C), w, None, s, final_state=s),
                  lambda: ssd.conv_step(z(B, C), w, None, z(B, W - 1, C), state_out=s)):
        y, _ = block.conv(x, w, None, s)
        write()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
