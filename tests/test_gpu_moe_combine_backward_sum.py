"""moe_combine_backward's router-weight gradient over long rows.

Products and sums in FP64, rounded once: 2^-24 |dw| for the rounding, and H 2^-53 sum |dy d| for the kernel's
sums and as much for the reference's.  Rows whose products cancel show a sum that was rounded on the way.
"""
import pytest
import torch

import precision_moe_gemm_amd as pmg
from helpers import gpu_ready

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ready(), reason="needs a GPU")]


@pytest.mark.parametrize("T,k,H", [(5, 2, 8), (9, 4, 64), (7, 3, 520), (61, 8, 768), (33, 2, 2048), (17, 4, 8200),
                                   (5, 2, 65536), (2, 1, 1 << 20)])
@pytest.mark.parametrize("ty", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("td", [torch.bfloat16, torch.float32])
def test_one_rounding(T, k, H, ty, td):
    print(f"[combine backward] T={T} k={k} H={H} {ty} {td}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(73)
    dy = torch.randn((T, H), generator=g, device="cuda").to(ty)
    d = torch.randn((T * k, H), generator=g, device="cuda").to(td)
    # the second half of each row near the first's negative, so that most of the sum cancels
    d[:, H // 2:] = -(d[:, :H // 2].float() * (1 + 0.01 * torch.randn((T * k, H // 2), generator=g, device="cuda"))).to(td)
    dy[:, H // 2:] = dy[:, :H // 2]
    row = torch.randperm(T * k, generator=g, device="cuda").int()
    _, dw = pmg.moe_combine_backward(dy, d, row, k, want_dd=False)
    terms = dy.double().repeat_interleave(k, 0) * d.double()[row.long()]
    want, size = terms.sum(1), terms.abs().sum(1)
    err = (dw.double().view(-1) - want).abs()
    assert bool((err <= 2.0 ** -24 * want.abs() + 2 * H * 2.0 ** -53 * size).all()), float((err / want.abs()).max())
    _, both = pmg.moe_combine_backward(dy, d, row, k)
    assert torch.equal(both, dw)
