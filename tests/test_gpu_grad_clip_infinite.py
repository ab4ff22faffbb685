"""grad_norm and grad_clip where the norm is not a number of float32.

max_norm = inf takes the norm alone: factor 1 whatever the norm, so that the tensors stay (in place: their bits)
or are copied.  With a finite max_norm the factor comes from the FP64 norm: 0 where that is inf, NaN where it is
NaN, and above 0 where only the float32 result overflows.
"""
import math

import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as pmg
from oracle import gradients as og
from helpers import gpu_ready

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ready(), reason="needs a GPU")]

INF, NAN = float("inf"), float("nan")
# at most two pieces of 64 KB take one launch, more two; then a list of more than one launch's tensors
SIZES = {"one_launch": [1000, 33], "two_launches": [1000, 70_001, 200_003], "long_list": [300 + j for j in range(230)]}


def bits(t):
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def tensors(sizes, value, where):
    """Both types in turn, `value` at one element of tensor `where`."""
    g = torch.Generator(device="cuda").manual_seed(71)
    out = [torch.randn(n, generator=g, device="cuda").to(torch.bfloat16 if j % 2 else torch.float32)
           for j, n in enumerate(sizes)]
    out[where][7] = value
    return out


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("where", [0, 1, -1])
def test_infinite_limit_leaves_the_tensors(name, value, where):
    print(f"[clip] {name} {value} in {where}", flush=True)
    grads = tensors(SIZES[name], value, where)
    before = [bits(g).clone() for g in grads]
    norm, out = pmg.grad_clip(grads, INF)
    assert bool(norm.isnan()) == math.isnan(value) and bool(norm.isinf()) != math.isnan(value)
    for g, o in zip(grads, out):
        assert o.data_ptr() != g.data_ptr()
        # a NaN is copied as a NaN
        assert torch.equal(g.isnan(), o.isnan()) and torch.equal(bits(g)[~g.isnan()], bits(o)[~o.isnan()])
    # outputs that lie differently towards a 16-byte boundary
    aside = [torch.empty(g.numel() + 1, dtype=g.dtype, device="cuda")[1:] for g in grads]
    pmg.grad_clip(grads, INF, out=aside)
    for g, o in zip(grads, aside):
        assert torch.equal(g.isnan(), o.isnan()) and torch.equal(bits(g)[~g.isnan()], bits(o)[~o.isnan()])
    pmg.grad_clip(grads, INF, out=grads)
    assert all(torch.equal(b, bits(g)) for b, g in zip(before, grads))


@pytest.mark.parametrize("name", SIZES)
def test_finite_limits(name):
    for value in (INF, -INF, NAN):
        for max_norm in (0.0, 1.0, 3e38):
            grads = tensors(SIZES[name], value, 1)
            norm, out = pmg.grad_clip(grads, max_norm)
            assert bool(norm.isnan()) == math.isnan(value)
            for g, o in zip(grads, out):
                assert torch.equal(o.isnan(), torch.ones_like(g, dtype=torch.bool) if math.isnan(value) else g.isinf())
                assert not o[~o.isnan()].any()


@pytest.mark.parametrize("name", SIZES)
def test_a_norm_beyond_float32_alone(name):
    """The FP64 norm is finite, so is the factor: 1 with max_norm = inf, else max_norm / norm."""
    grads = [torch.full((n,), 3e38, device="cuda") for n in SIZES[name]]
    norm, out = pmg.grad_clip(grads, INF)
    assert bool(norm.isinf()) and all(torch.equal(g, o) for g, o in zip(grads, out))
    norm, out = pmg.grad_clip(grads, 1.0)
    want = og.norm([g.double().cpu().numpy() for g in grads])
    assert bool(norm.isinf()) and math.isfinite(want)
    for g, o in zip(grads, out):
        # the product rounded to float32: 2^-24, and the FP64 factor
        assert np.allclose(o.double().cpu().numpy(), float(g[0]) / want, rtol=2.0 ** -24 + 2.0 ** -40, atol=0)
