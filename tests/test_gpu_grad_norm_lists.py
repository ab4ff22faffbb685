"""The norm over long lists of tensors: the values, and that it reads a list as fast as the same bytes in few tensors.

Values as in test_gpu_grad_clip.py: squares are exact and summed in FP64, so the norm is one rounding off
(2^-24, and 2^-40 for the sums).
"""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as pmg
from helpers import gpu_ready

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ready(), reason="needs a GPU")]

U = 2.0 ** -24


def exact_norm(grads):
    return float(torch.stack([(g.double() ** 2).sum() for g in grads]).sum().sqrt())


@pytest.mark.parametrize("sizes", [
    # several launches of many pieces each (a piece holds 16384 float32), the last one's tensors few and large or small
    [50_000 + 17 * j for j in range(1000)],
    [60_001] * 96 + [1] * 96 + [5_000_003],
    [1] * 96 + [3_000_001] * 3 + [0] * 200 + [40_000] * 150,
    [1 + j % 5 for j in range(3000)],
], ids=["thousand", "few_last", "few_first", "tiny"])
def test_values(sizes):
    print(f"[norm] {len(sizes)} tensors, {sum(sizes)} elements", flush=True)
    g = torch.Generator(device="cuda").manual_seed(72)
    grads = [torch.randn(n, generator=g, device="cuda").to(torch.bfloat16 if j % 3 == 1 else torch.float32)
             for j, n in enumerate(sizes)]
    want = exact_norm(grads)
    ws = torch.full((pmg.grad_workspace_size(len(grads)),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN as doubles
    norm = pmg.grad_norm(grads, workspace=ws)
    assert abs(float(norm) - want) <= (U + 2.0 ** -40) * want
    assert torch.equal(pmg.grad_norm(grads), norm)                       # what the workspace held is not read
    # the list the other way round, whose launches have other grids: the same up to the norm's rounding
    assert abs(float(pmg.grad_norm(grads[::-1], workspace=ws)) - want) <= (U + 2.0 ** -40) * want
    clipped, out = pmg.grad_clip(grads, 1.0, workspace=ws)
    assert torch.equal(clipped, norm)
    c = 1.0 / (want + 1e-6)
    for j in range(0, len(grads), 37):
        rel, least = (2 * U, 2.0 ** -150) if grads[j].dtype == torch.float32 else (2.0 ** -8 + 2 * U, 2.0 ** -134)
        ref = grads[j].double() * c
        assert bool(((out[j].double() - ref).abs() <= 1.001 * rel * ref.abs() + least).all()), j
    _, same = pmg.grad_clip(grads, 1.0, out=grads, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(same, out))


def _replay_us(grads):
    """The device's time for one norm: the shortest of ten replays of a graph, which the host does not slow down."""
    norm = torch.empty(1, device="cuda")
    ws = torch.empty(pmg.grad_workspace_size(len(grads)), dtype=torch.uint8, device="cuda")
    pmg.grad_norm(grads, norm=norm, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pmg.grad_norm(grads, norm=norm, workspace=ws)
    best = float("inf")
    for _ in range(10):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


def test_a_long_list_keeps_the_device_busy():
    """1 GiB as 4 tensors and as 4096: 43 launches, each of 96 tensors of four pieces.  A launch that fills the
    device reads its 25 MB in about the time that a launch itself takes (5 us); one with a 43rd of the
    workgroups that fill it takes many times as long.  Allowed: 15 us a launch above the few tensors' time."""
    flat = torch.empty(1 << 28, device="cuda").normal_()
    few = _replay_us(list(flat.chunk(4)))
    many = _replay_us(list(flat.chunk(4096)))
    print(f"[norm] 1 GiB as 4 tensors {few:.0f} us, as 4096 {many:.0f} us", flush=True)
    assert many <= few + 43 * 15.0


def test_captured_and_replayed():
    """A list of several launches: each replay starts its partial sums anew."""
    g = torch.Generator(device="cuda").manual_seed(74)
    grads = [torch.randn(20_000 + 13 * j, generator=g, device="cuda") for j in range(300)]
    out = [torch.empty_like(x) for x in grads]
    norm = torch.empty(1, device="cuda")
    ws = torch.empty(pmg.grad_workspace_size(len(grads)), dtype=torch.uint8, device="cuda")
    pmg.grad_clip(grads, 1.0, out=out, norm=norm, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pmg.grad_clip(grads, 1.0, out=out, norm=norm, workspace=ws)
    for scale in (1.0, 0.25, 3.0):
        for x in grads:
            x.mul_(scale)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        want, clipped = pmg.grad_clip(grads, 1.0)
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(out, clipped))
