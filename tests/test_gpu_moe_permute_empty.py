"""moe_permute of a batch without tokens needs no workspace, like the short lists beside it."""
import pytest
import torch

import precision_moe_gemm_amd as pmg
from helpers import gpu_ready

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ready(), reason="needs a GPU")]


@pytest.mark.parametrize("E", [1, 7, 128, 1000, 1024])
def test_no_tokens_no_workspace(E):
    lib, stream = pmg.load_library(), torch.cuda.current_stream().cuda_stream
    k = min(E, 4)
    assert pmg.moe_permute_workspace_size(16, k, E) == 0
    for dtype in (0, 1):
        for ws, size in ((None, 0), (torch.full((256,), 7, dtype=torch.uint8, device="cuda"), 16)):
            off = torch.full((E + 3,), -5, dtype=torch.int32, device="cuda")
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            assert lib.moe_permute(None, dtype, 0, 64, None, k, E, None, off.data_ptr(), None, None,
                                   None if ws is None else ws.data_ptr(), size, err.data_ptr(), stream) == 0
            torch.cuda.synchronize()
            assert not off[:E + 1].any() and (off[E + 1:] == -5).all() and int(err) == 0
            assert ws is None or (ws == 7).all()
    # a buffer sized for the largest of the program's short batches serves its empty one
    none = torch.empty(pmg.moe_permute_workspace_size(16, k, E), dtype=torch.uint8, device="cuda")
    ids = torch.empty((0, k), dtype=torch.int32, device="cuda")
    for x in (None, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")):
        got = pmg.moe_permute(x, ids, E, workspace=none)
        assert got["expert_offsets"].shape == (E + 1,) and not got["expert_offsets"].any()


def test_captured():
    off = torch.full((129,), 3, dtype=torch.int32, device="cuda")
    ids = torch.empty((0, 8), dtype=torch.int32, device="cuda")
    out = {"expert_offsets": off}
    pmg.moe_permute(None, ids, 128, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pmg.moe_permute(None, ids, 128, out=out)
    for _ in range(3):
        off.fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert not off.any()
