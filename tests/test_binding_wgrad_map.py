"""bf16_grouped_gemm_wgrad refuses a routing map that it would not use (no GPU needed)."""
import pytest
import torch

import precision_moe_gemm_amd as pmg


@pytest.mark.parametrize("kw", [{"row_to_tk": torch.zeros(8, dtype=torch.int32)}, {"k": 2},
                                {"row_to_tk": torch.zeros(8, dtype=torch.int32), "k": 2}])
def test_a_map_without_an_operand_to_gather(kw):
    g = torch.zeros(8, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="gather"):
        pmg.bf16_grouped_gemm_wgrad(g, g, torch.zeros(3, dtype=torch.int32), **kw)
