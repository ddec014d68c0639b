"""One workspace, made for the largest batch, for products of every smaller one."""
import pytest
import torch

import sparse_delta_codec_amd as pulse

pytestmark = pytest.mark.gpu


def operands(m, n, k, form):
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    codes = lambda *s: torch.randint(0, 127, s, device="cuda", generator=gen).to(torch.uint8)  # noqa: E731
    scales = lambda *s: torch.rand(s, device="cuda", generator=gen)  # noqa: E731
    inner, out = (k, n) if form == "nt" else (n, k)
    up = lambda v: (v + 127) // 128  # noqa: E731
    return codes(m, inner), scales(m, up(inner)), codes(n, k), scales(up(n), up(k)), torch.empty((m, out), dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("n,k,form", [(640, 5120, "nt"), (7168, 5120, "nt"), (1040, 4112, "nn"), (4112, 8208, "nn")])
def test_smaller_batches(n, k, form):
    sizes = [2000, 1024, 300, 129, 128, 96, 40, 20, 8, 1]
    shared = pulse.fp8_gemm_workspace(sizes[0], n, k, form)
    refused = 0
    for m in sizes:
        x, sx, w, sw, y = operands(m, n, k, form)
        pulse.fp8_block_gemm(x, sx, w, sw, y, pulse.fp8_gemm_workspace(m, n, k, form), form=form)
        want = y.clone()
        y.fill_(-1)
        shared.fill_(255)
        pulse.fp8_block_gemm(x, sx, w, sw, y, shared, form=form)
        assert torch.equal(y, want)
        try:  # with none, a product that needs one is refused, and the others are the same
            y.fill_(-1)
            pulse.fp8_block_gemm(x, sx, w, sw, y, form=form)
            assert torch.equal(y, want)
        except RuntimeError:
            refused += 1
            assert (y == -1).all()
    assert refused  # (some of them go through the workspace)
