"""The products where they are cut, joined and laid out in each of their ways: the same bits at every
call."""
import pytest
import torch

from chunked_linear_recurrence_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.float32, torch.bfloat16]

# rows, inner, outer, and what the forward's workspace shows of its path: more than nothing where K is
# split, both operands where they are laid out anew, less than that where they pass through registers
PATHS = {
    "direct, K ends in a step": (130, 200, 264, None),
    "through registers": (150, 131, 70, "registers"),
    "K split and joined": (100, 4096, 64, "split"),
    "laid out anew": (2561, 2047, 2051, "laid out"),
    "tiles of 256": (2901, 200, 2840, None),
}


def make(m, k, n, dtype, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device=DEV) * std).to(dtype)
    return r(m, k), r(n, k, std=k ** -0.5), r(n, std=0.3), r(m, n), r(m, n)


def check_path(m, k, n, dtype, path, gated):
    dims = ssd.ProductDims(m, k, n, ssd._DTYPE_CODE[dtype], 0, k, n, n)
    L = ssd.lib()
    got = (L.ssd_gated_fwd_workspace_bytes if gated else L.ssd_linear_fwd_workspace_bytes)(dims)
    both = (m + n * (2 if gated else 1)) * k * (2 if dtype == torch.bfloat16 else 4)
    if path == "split":
        assert got > 0
    elif path == "laid out":
        assert got >= both
    elif path == "registers":
        assert got < both


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("path", PATHS)
def test_gated_calls_repeat_bit_for_bit(path, dtype):
    m, k, n, kind = PATHS[path]
    f = n // 2
    check_path(m, k, f, dtype, kind if kind != "registers" else None, True)
    x, w, b, _, _ = make(m, k, 2 * f, dtype, 1)
    dh = make(m, 1, f, dtype, 2)[4]
    first = None
    for _ in range(4):
        h, pre = ssd.gated_fwd(x, w, b, keep=True)
        got = (h, pre) + ssd.gated_bwd(dh, x, w, b, pre)
        first = first or got
        assert all(torch.equal(p, q) for p, q in zip(first, got))
