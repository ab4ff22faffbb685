"""The instances that only operands beyond the 256 MB last-level cache reach, and long routing lists with rows of
more than a wavefront's group, compared in full.

dgu, dd, rows: bit for bit.  Sums in FP64 of terms within 2^-49 of theirs, rounded once (the SwiGLU's dw and the
combine's): 2^-24 |dw| + 2^-40 sum |terms|.  A clipped float32 value is the FP64 product rounded once, 2^-24 (and
the factor's own 2^-40).
"""
import pytest
import torch

import precision_moe_gemm_amd as pmg
from helpers import gpu_ready

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ready(), reason="needs a GPU")]

U = 2.0 ** -24
CACHE = 256 << 20
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def maps(T, k, seed, lost):
    """row_to_tk (2^31 - 1 behind the last row), tk_to_row (-1: no row), rows, router weights."""
    g = gen(seed)
    R = T * k
    order = torch.randperm(R, generator=g, device="cuda").int()
    n = R - int(lost * R)
    r2t = torch.full((R,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    r2t[:n] = order[:n]
    t2r = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    t2r[order[:n].long()] = torch.arange(n, dtype=torch.int32, device="cuda")
    return r2t, t2r, n, torch.rand((T, k), generator=g, device="cuda")


def filled(shape, dtype):
    size = 4 if dtype == F32 else 2
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.view(torch.int32 if size == 4 else torch.int16).fill_(-0x5A5B)
    return t


def same(a, b):
    kind = torch.int32 if a.dtype == F32 else torch.int16
    return torch.equal(a.view(kind), b.view(kind))


@pytest.mark.parametrize("T,k,I", [(3175, 7, 768), (16001, 4, 264), (131101, 8, 16)])
def test_swiglu_backward_weights(T, k, I):
    R = T * k
    assert 16 * I * R >= CACHE
    print(f"[swiglu backward] {R} rows of {I}", flush=True)
    r2t, t2r, n, w = maps(T, k, 81, 0.1)
    g = gen(82)
    gu = 2 * torch.randn((R, 2 * I), generator=g, device="cuda")
    dh = torch.randn((R, I), generator=g, device="cuda")
    off = torch.tensor([0, n // 3, n], dtype=torch.int32, device="cuda")
    dgu, dw = pmg.swiglu_backward_weights(gu, dh, off, w, r2t, t2r, dgu=filled((R, 2 * I), BF16))
    assert same(pmg.swiglu_backward(gu, dh, off, w.view(-1), r2t, dgu=filled((R, 2 * I), BF16)), dgu)
    assert same(dgu[n:], filled((R - n, 2 * I), BF16))
    # the same rows in slices that the caches hold
    step = (CACHE // (16 * I)) // 3
    for a in range(0, n, step):
        b = min(n, a + step)
        part = pmg.swiglu_backward(gu[a:b], dh[a:b], torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
                                   w.view(-1)[r2t[a:b].long()].contiguous(),
                                   torch.arange(b - a, dtype=torch.int32, device="cuda"))
        assert same(part, dgu[a:b]), a
    gd, ud = gu[:n, :I].double(), gu[:n, I:].double()
    terms = dh[:n].double() * (gd / (1 + torch.exp(-gd))) * ud
    want, size = torch.zeros(R, dtype=torch.float64, device="cuda"), torch.zeros(R, dtype=torch.float64, device="cuda")
    want[r2t[:n].long()], size[r2t[:n].long()] = terms.sum(1), terms.abs().sum(1)
    assert bool(((dw.double().view(-1) - want).abs() <= U * want.abs() + 2.0 ** -40 * size).all())
    assert not dw.view(-1)[t2r < 0].any()


# at most 8 elements a lane (one piece) and several pieces ahead; groups of 16, 32 and 64 lanes
@pytest.mark.parametrize("H", [72, 512, 520, 2056])
@pytest.mark.parametrize("ty", [BF16, F32])
@pytest.mark.parametrize("td", [BF16, F32])
def test_combine_backward(H, ty, td):
    k = 3
    size = 4 if td == F32 else 2
    T = CACHE // (H * size * k) + 7                     # either of d and dd alone is beyond the cache
    R = T * k
    print(f"[combine backward] {R} rows of {H} {td}, dy {ty}", flush=True)
    r2t, t2r, n, w = maps(T, k, 83, 0.1)
    g = gen(84)
    dy = torch.randn((T, H), generator=g, device="cuda").to(ty)
    d = torch.randn((R, H), generator=g, device="cuda").to(td)
    dd, dw = pmg.moe_combine_backward(dy, d, t2r, k, w, dd=filled((R, H), td))
    entry = r2t[:n].long()
    assert same(dd[:n], (w.view(-1)[entry, None] * dy.float()[entry // k]).to(td))
    assert same(dd[n:], filled((R - n, H), td))
    want = torch.zeros(R, dtype=torch.float64, device="cuda")
    total = torch.zeros(R, dtype=torch.float64, device="cuda")
    for a in range(0, n, 1 << 16):
        e = entry[a:a + (1 << 16)]
        terms = dy[e // k].double() * d[a:a + e.numel()].double()
        want[e], total[e] = terms.sum(1), terms.abs().sum(1)
    assert bool(((dw.double().view(-1) - want).abs() <= U * want.abs() + 2.0 ** -40 * total).all())
    assert not dw.view(-1)[t2r < 0].any()
    only, _ = pmg.moe_combine_backward(dy, None, t2r, k, w, dd=filled((R, H), td))
    assert same(only, dd)
    _, alone = pmg.moe_combine_backward(dy, d, t2r, k, w, want_dd=False)
    assert torch.equal(alone, dw)


@pytest.mark.parametrize("offset", [0, 1])
def test_clip_float32(offset):
    sizes = [33_554_433, 12_345, 40_000_001]
    assert 4 * sum(sizes) >= CACHE
    print(f"[clip] {sum(sizes)} float32 elements, offset {offset}", flush=True)
    g = gen(85)
    grads = [torch.randn(n + offset, generator=g, device="cuda")[offset:] for n in sizes]
    before = [x.clone() for x in grads]
    want = float(torch.stack([(x.double() ** 2).sum() for x in grads]).sum().sqrt())
    norm, out = pmg.grad_clip(grads, 1.0)
    assert abs(float(norm) - want) <= (U + 2.0 ** -40) * want
    c = 1.0 / (want + 1e-6)
    for x, b, o in zip(grads, before, out):
        assert torch.equal(x, b)
        ref = x.double() * c
        assert bool(((o.double() - ref).abs() <= (U + 2.0 ** -40) * ref.abs() + 2.0 ** -150).all())
    _, inplace = pmg.grad_clip(grads, 1.0, out=grads)
    assert all(torch.equal(a, b) for a, b in zip(inplace, out))


# count tables beyond what a workgroup scans, rows of 16 bytes to more than a wavefront holds (256 words)
@pytest.mark.parametrize("T,E,k,H,dtype", [(9000, 300, 32, 264, F32), (40000, 128, 8, 520, BF16), (33000, 512, 4, 2056, BF16),
                                           (40001, 128, 8, 1032, F32), (20000, 1000, 31, 136, BF16), (70000, 300, 3, 256, BF16)])
def test_permute_long_lists(T, E, k, H, dtype):
    print(f"[permute] T={T} E={E} k={k} H={H} {dtype}", flush=True)
    R = T * k
    assert -(-R // 2048) * E > 4096
    g = gen(86)
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1)[1].int()
    ids[torch.rand((T, k), generator=g, device="cuda") < 0.02] = -1
    x = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    out = {"rows": filled((R, H), dtype), "row_to_tk": torch.full((R,), -9, dtype=torch.int32, device="cuda")}
    got = pmg.moe_permute(x, ids, E, out=out)
    flat = ids.view(-1)
    order = torch.where(flat < 0, E, flat).argsort(stable=True)
    n = int((flat >= 0).sum())
    assert torch.equal(got["row_to_tk"][:n], order[:n].int()) and (got["row_to_tk"][n:] == -9).all()
    assert torch.equal(got["expert_offsets"][1:], torch.bincount(flat[flat >= 0], minlength=E).cumsum(0).int())
    back = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    back[order[:n]] = torch.arange(n, dtype=torch.int32, device="cuda")
    assert torch.equal(got["tk_to_row"], back)
    assert same(got["rows"][:n], x[order[:n] // k])
    assert same(got["rows"][n:], filled((R - n, H), dtype))


def test_permute_past_32_bits_in_full():
    T, k, E, H = 70000, 4, 8, 8192
    print(f"[permute] {T * k} rows of {H}", flush=True)
    g = gen(87)
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1)[1].int()
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    got = pmg.moe_permute(x, ids, E)
    order = ids.view(-1).argsort(stable=True)
    assert torch.equal(got["row_to_tk"], order.int())
    for a in range(0, T * k, 1 << 16):
        assert same(got["rows"][a:a + (1 << 16)], x[order[a:a + (1 << 16)] // k]), a
