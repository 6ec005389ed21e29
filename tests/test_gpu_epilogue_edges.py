"""The products with an epilogue at the end of K: what stands in other rows' scales stays there."""
import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv
from test_gpu_epilogue import extras, operands, run

pytestmark = pytest.mark.gpu
NAN_SCALE = 0x7F


def scale_at(row, block, K):
    """Byte of a row's 16-value block in the 128x4 layout."""
    groups = (K // 16 + 3) // 4
    return (((row >> 7) * groups + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
            (block & 3))


# every schedule: streaming, clusters, split-K, SM pairs (whole and half tiles); K with one,
# two and three steps in its last stage
SHAPES = [(2, 19200, 576), (2, 19200, 64), (4, 1030, 640), (4, 1030, 192), (300, 520, 2624),
          (300, 520, 576), (300, 520, 704), (2500, 2064, 192), (2500, 2064, 64)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("prepared", [False, True])
def test_nan_scales_stay_in_their_row_and_column(M, N, K, prepared):
    a, sfa, b, sfb, alpha = operands("nvfp4", M, N, K)
    bias, res = extras(M, N, False, True, True)
    clean = run("nvfp4", (a, sfa, b, sfb, alpha), M, N, K, bias, "none", False, res, prepared)
    # the first scales of the row tile after row 72's (and the last row's neighbour below)
    bad_n = [200, N - 1]
    bad_m = [200] if M > 200 else []
    sfa, sfb = sfa.clone(), sfb.clone()
    for block in range(4):
        for n in bad_n:
            sfb[scale_at(n, block, K)] = NAN_SCALE
        for m in bad_m:
            sfa[scale_at(m, block, K)] = NAN_SCALE
    y = run("nvfp4", (a, sfa, b, sfb, alpha), M, N, K, bias, "none", False, res, prepared)
    torch.cuda.synchronize()
    assert nv.last_device_status() == nv.OK
    bad = torch.zeros(M, N, dtype=torch.bool, device=y.device)
    bad[:, bad_n] = True
    bad[bad_m, :] = True
    assert torch.isnan(y[bad]).all()
    assert torch.equal(y[~bad].view(torch.int16), clean[~bad].view(torch.int16))
