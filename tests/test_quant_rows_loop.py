"""rom_quant_rows with more rows than its persistent CTAs take at once: every
form of the kernel goes round, with a remainder that no CTA or warp fills."""
import pytest
import torch

from lowbit_util import rows_to_8bit
from mixture_experts_projections_b200 import rom

gpu = pytest.mark.gpu


# On 148 SMs one round takes 37888 rows of up to 64 columns (a quarter of a warp
# each), 18944 of 128, 9472 of 512; 4736 of 1000 (64 threads each), 592 of 8192 and
# of 16384 (512 threads), 1036 of 8200 (288).
@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,K", [(40003, 64), (39001, 56), (19003, 128), (9601, 256), (9601, 512), (9599, 264),
                                    (5003, 1000), (601, 8192), (1051, 8200), (601, 16384)])
def test_every_row_of_every_round(rows, K, dtype):
    g = torch.Generator().manual_seed(K)
    x = (torch.randn(rows, K, generator=g) * 10.0 ** torch.randint(-20, 20, (rows, 1), generator=g)).to(dtype)
    bad = [0, rows // 2 + 1, rows - 1]  # rows without a scale, the last round's among them
    x[bad[0], 1], x[bad[1], K - 1], x[bad[2], K // 2] = float("nan"), float("inf"), -float("inf")
    x[rows - 2] = 0
    q, s = rom.quant_rows(x.cuda())
    rq, rs = rows_to_8bit(x)
    q, s = q.cpu(), s.cpu()
    keep = torch.ones(rows, dtype=torch.bool)
    keep[bad] = False
    assert torch.equal(q.view(torch.uint8)[keep], rq.view(torch.uint8)[keep]) and torch.equal(s[keep], rs[keep])
    assert s[bad].isnan().all() and q[bad].float().isnan().all()
