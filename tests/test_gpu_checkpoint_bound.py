"""How far a checkpoint's values are off: by the group's largest magnitude over
127, or 2^-127 where that is more, and by less than 2^122 at the top."""

import pytest
import torch

import ring_allreduce_rs_amd as ar

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
def test_bound(t):
    # a row, one group, for each power of two that a largest magnitude can begin with, and the
    # largest numbers
    tops = [1.3 * 2.0 ** k for k in range(-133, 127)]
    tops += [2.0 ** -128, 2.0 ** -127, 1.984375 * 2.0 ** 127, 1.9921875 * 2.0 ** 127,
             torch.finfo(t).max]
    g = torch.Generator().manual_seed(4)
    x = torch.rand((len(tops), 32), generator=g, dtype=torch.float64) * 2 - 1
    x[:, 0] = 1.0
    x = (x * torch.tensor(tops, dtype=torch.float64)[:, None]).to(t)
    saved = ar.save_8bit(x.cuda())
    x = x.double()
    m = x.abs().amax(1, keepdim=True)
    full = m > 1.984375 * 2.0 ** 127
    for back in (torch.bfloat16, torch.float32):
        off = (ar.restore_8bit(saved, back).double().cpu() - x).abs()
        assert bool((off <= torch.where(full, 2.0 ** 122, torch.clamp(m / 127, min=2.0 ** -127))).all())
        # both ends of it are met: over m / 127 below, over half a scale at the top
        small = (m < 2.0 ** -127) & (m > 0)
        assert bool((off > m / 127)[small.expand_as(off)].any())
        assert bool((off > 2.0 ** 121)[full.expand_as(off)].any())
    # a scale of 0, as nothing saves it
    zero = ar.Saved8(torch.full((2, 40), 5, dtype=torch.int8, device="cuda"),
                     torch.zeros((2, 2), dtype=torch.uint8, device="cuda"))
    assert not ar.restore_8bit(zero, t).any()
