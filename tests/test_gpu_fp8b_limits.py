"""GPU parity of the FP8 blocks of 128 where their numbers end: every border
between two codes under every mantissa of a block's scale."""
import numpy as np
import pytest
import torch

import oracle as O
from ragged_grouped_gemm_gb300 import api

pytestmark = pytest.mark.gpu


def _quantise(x):
    codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(x.shape[0], api.fp8_scale_ld(x.shape[1]), device="cuda")
    api.moe_quantize_fp8_rows(x.cuda(), codes, scales)
    torch.cuda.synchronize()
    return codes, scales


@pytest.mark.parametrize("exponent", [0, 15, -30, -66, -104, -126, 120])
def test_quantise_rows_every_mantissa_of_the_scale(exponent):
    """A block's largest magnitude takes all 128 bf16 mantissas of a binade, so its scale has every
    mantissa it can have; the others run through every bf16 magnitude down to amax / 2^21, past the
    smallest code (2^-9 of a scale that is amax / 448).  Whether a quotient lies just below
    or above a power of two, where the codes' spacing changes, depends on the scale's mantissa."""
    blocks = []
    for m in range(128):
        top = ((exponent + 127) << 7) + m                              # bf16 bits of amax
        bits = torch.arange(max(top - 21 * 128, 0), top + 1, dtype=torch.int32)
        v = (bits << 16).view(torch.float32)
        v = torch.cat([v, -v])
        v = torch.nn.functional.pad(v, (0, -v.numel() % 127)).view(-1, 127)
        amax = torch.tensor([top << 16], dtype=torch.int32).view(torch.float32)
        blocks.append(torch.cat([amax.expand(v.shape[0], 1), v], 1))
    x = torch.cat(blocks).to(torch.bfloat16)
    codes, scales = _quantise(x)
    rc, rs = O.fp8_rows_quantize(x.float().numpy())
    np.testing.assert_array_equal(scales[:, :1].cpu().numpy().view(np.uint32), rs.view(np.uint32))
    wrong = codes.cpu().numpy() != rc
    r, c = np.nonzero(wrong)
    assert not wrong.any(), (int(wrong.sum()), [(float(x[i, 0]), float(x[i, j]), int(codes[i, j]), int(rc[i, j]))
                                                for i, j in zip(r[:4], c[:4])])
