"""Operands at the border of what the operators take."""
import pytest
import torch

from all_movement_amd import moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_columns_of_one_buffer_as_input_and_output():
    gen = torch.Generator().manual_seed(1)
    for dt in (torch.bfloat16, torch.float32):
        buf = torch.randn(90, 160, generator=gen).to(dt).to(DEV)
        y, out = buf[:, :64], buf[:30, 64:128]
        place = torch.randperm(90, generator=gen).to(torch.int32).view(30, 3).to(DEV)
        w = torch.rand(30, 3, generator=gen).to(DEV)
        want = moe.combine(y.contiguous(), place, w)
        edge = buf[:, 128:].clone()
        assert torch.equal(moe.combine(y, place, w, out=out), want)
        assert torch.equal(buf[:, 128:], edge) and torch.equal(buf[:30, 64:128], want)
    buf = torch.randn(70, 104, generator=gen).to(torch.bfloat16).to(DEV)
    wt = torch.randn(2, 40, 64, generator=gen).to(torch.bfloat16).to(DEV)
    c = torch.tensor([30, 40], dtype=torch.int32, device=DEV)
    want = moe.gmm(buf[:, :64].contiguous(), wt, c)
    before = buf[:, :64].clone()
    moe.gmm(buf[:, :64], wt, c, out=buf[:, 64:])
    assert torch.equal(buf[:, 64:], want) and torch.equal(buf[:, :64], before)
