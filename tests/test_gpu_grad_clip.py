"""grad_norm and grad_clip against float64.

The squares are exact and their sums in float64, so the norm is one rounding off (2^-24, and 2^-40 for the
sums); a clipped float32 value is off by the factor's rounding and the product's (2 2^-24), a bf16 one by
2^-8 more; values near the type's least one by half of its step (2^-150, 2^-134).
"""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as pmg
import workloads as W
from oracle import gradients as og
from helpers import assert_within, gpu_ready, host

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ready(), reason="needs a GPU")]

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def tensors(spec, seed, scale=1.0, offset=0):
    """Device tensors of (size, type), each starting `offset` elements into an allocation."""
    out = []
    for j, (n, t) in enumerate(spec):
        v = torch.from_numpy((scale * W.rng(seed, j).standard_normal(n + offset)).astype(np.float32)).to("cuda").to(DT[t])
        out.append(v[offset:])
    return out


def f64(t):
    return t.double().cpu().numpy()


def check(grads, max_norm, out=None):
    want_n, want = og.clip([f64(g) for g in grads], max_norm)
    before = [g.clone() for g in grads]
    # the norm's own rounding: half a float32 step, which below 2^-126 is 2^-149 / 2 whatever the value
    near = np.array([(U + 2.0 ** -40) * want_n + 2.0 ** -150])
    assert_within(host(pmg.grad_norm(grads)), np.array([want_n]), near, "norm")
    norm, got = pmg.grad_clip(grads, max_norm, out=out)
    assert_within(host(norm), np.array([want_n]), near, "norm of clip")
    for g, b, o, w in zip(grads, before, got, want):
        if o.data_ptr() != g.data_ptr():
            assert torch.equal(g, b)
        rel, least = (2 * U, 2.0 ** -150) if g.dtype == torch.float32 else (2.0 ** -8 + 2 * U, 2.0 ** -134)
        assert_within(f64(o), w, (rel * 1.001) * np.abs(w) + least, "clipped")
    return norm, got


SPECS = {
    "one": [(1, "f32")],
    "one_bf16": [(1, "bf16")],
    "two": [(1000, "bf16"), (0, "f32"), (333, "f32")],
    "two_pieces": [(30_000, "f32")],
    "two_full_pieces": [(65_550, "bf16")],
    "small": [(3, "bf16"), (0, "f32"), (5, "f32"), (8, "bf16"), (4, "f32"), (7, "f32"), (9, "bf16"), (64, "f32")],
    "odd": [(1021, "f32"), (4099, "bf16"), (16385, "f32"), (32769, "bf16"), (65537, "f32")],
    "many": [(1 + 37 * j % 900, "f32" if j % 3 else "bf16") for j in range(230)],
    "pieces": [(400_003, "f32"), (1_000_001, "bf16"), (131_072, "f32")],
    "table_and_one": [(17, "f32")] * 96 + [(1_000_000, "bf16")],
    "empty": [(0, "f32"), (0, "bf16")],
    "none": [],
}


@pytest.mark.parametrize("name", SPECS)
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_norm_and_clip(name, offset):
    print(f"[clip] {name} offset {offset}", flush=True)
    grads = tensors(SPECS[name], 41, offset=offset)
    for max_norm in (0.7, 1e9, 0.0, float("inf")):
        norm, out = check(grads, max_norm)
        if max_norm >= 1e9:
            assert all(torch.equal(a, b) for a, b in zip(grads, out))
        if max_norm == 0.0:
            assert all(not o.any() for o in out)
    # outputs that lie differently towards a 16-byte boundary
    check(grads, 0.7, out=tensors(SPECS[name], 42, offset=(offset + 1) % 4))
    ref = [o.clone() for o in pmg.grad_clip(grads, 0.7)[1]]
    keep = [g.data_ptr() for g in grads]
    _, got = pmg.grad_clip(grads, 0.7, out=grads)                    # in place
    assert [o.data_ptr() for o in got] == keep and all(torch.equal(a, b) for a, b in zip(got, ref))
    _, got = pmg.grad_clip(grads, 1e9, out=grads)                    # nothing to clip
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_neighbours_are_left_alone():
    """Views into one flat buffer: what lies between them stays."""
    flat = torch.randn(5000, device="cuda")
    before = flat.clone()
    cut = [(1, 4), (7, 8), (9, 1000), (1003, 2999), (3001, 4998)]
    pmg.grad_clip([flat[a:b] for a, b in cut], 0.1, out=[flat[a:b] for a, b in cut])
    inside = torch.zeros(5000, dtype=torch.bool, device="cuda")
    for a, b in cut:
        inside[a:b] = True
    assert torch.equal(flat[~inside], before[~inside])
    assert (flat[inside] != before[inside]).all()


def test_extreme_values():
    big = torch.full((1000,), 3e38, device="cuda")
    norm, out = pmg.grad_clip([big], 1.0)        # the squares' sum is far above float32's range
    want = 3e38 * 1000 ** 0.5
    assert norm.isinf().all() == (want > 3.4028235e38)
    assert_within(f64(out[0]), f64(big) / want, 3 * U * f64(big) / want, "clipped")
    tiny = torch.full((1000,), 1e-42, device="cuda")
    check([tiny, torch.full((9,), 1e-40, device="cuda").bfloat16()], 1e-43)
    x = torch.randn(100, device="cuda")
    x[3] = float("inf")
    norm, out = pmg.grad_clip([x], 1.0)
    assert norm.isinf().all() and out[0][3].isnan() and not out[0][:3].any()
    x[4] = float("nan")
    norm, out = pmg.grad_clip([x, torch.ones(5, device="cuda").bfloat16()], 1.0)
    assert norm.isnan().all() and all(o.isnan().all() for o in out)
    neg = torch.tensor([-1], dtype=torch.int16, device="cuda").view(torch.bfloat16)     # a NaN of all ones
    assert pmg.grad_norm([neg]).isnan().all()


def test_same_bits_every_time_and_the_same_tensor_twice():
    g = tensors(SPECS["odd"], 43)
    ref = pmg.grad_norm(g)
    for _ in range(3):
        assert torch.equal(pmg.grad_norm(g), ref)
        assert torch.equal(pmg.grad_clip(g, 1.0)[0], ref)
    two = og.norm([f64(g[0]), f64(g[0])])
    assert abs(float(pmg.grad_norm([g[0], g[0]])) - two) <= (U + 2.0 ** -40) * two
    for bad in ([g[0], g[0]], [g[2][:100], g[2][50:200]]):
        with pytest.raises(pmg.NVFP4Error):
            pmg.grad_clip(bad, 1.0, out=bad)


def test_shapes_and_refusals():
    g = [torch.randn(3, 4, 5, device="cuda"), torch.randn((), device="cuda")]
    norm, out = pmg.grad_clip(g, 1.0)
    assert out[0].shape == (3, 4, 5) and out[1].shape == ()
    given = torch.empty(1, device="cuda")
    ws = torch.empty(pmg.grad_workspace_size(2), dtype=torch.uint8, device="cuda")
    assert pmg.grad_norm(iter(g), norm=given, workspace=ws) is given and torch.equal(given, norm)
    with pytest.raises(pmg.NVFP4Error, match="workspace"):
        pmg.grad_norm(g, workspace=ws[:64])
    with pytest.raises(ValueError, match="contiguous"):
        pmg.grad_norm([g[0].transpose(0, 1)])
    with pytest.raises(ValueError, match="outputs for"):
        pmg.grad_clip(g, 1.0, out=[g[0]])
    with pytest.raises(ValueError, match="sizes and types"):
        pmg.grad_clip(g, 1.0, out=[g[0], torch.randn(2, device="cuda")])
    for bad in (-1.0, float("nan")):
        with pytest.raises(pmg.NVFP4Error):
            pmg.grad_clip(g, bad)


def test_sizes_past_32_bits():
    n = 2 ** 31 + 12345
    print(f"[clip] {n} bf16 elements", flush=True)
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    x[-5:] = 3.0
    x[2 ** 31 - 2:2 ** 31 + 2] = 2.0
    norm, out = pmg.grad_clip([x], 1.0)
    want = (5 * 9 + 4 * 4) ** 0.5
    assert abs(float(norm) - want) <= 2 * U * want
    c = 1 / (want + 1e-6)
    assert torch.allclose(out[0][-5:].double(), torch.full((5,), 3 * c, dtype=torch.float64, device="cuda"), rtol=2.0 ** -8 + 2 * U)
    assert int((out[0] != 0).sum()) == 9
