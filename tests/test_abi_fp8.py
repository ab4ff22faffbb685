"""Host checks of the FP8 and BF16 weight-gradient entry points: every refusal returns its
status before anything is enqueued (no device pointer is ever dereferenced, no GPU needed)."""
import pytest
import torch

import precision_moe_gemm_amd as pmg

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_LAUNCH, ERR_ARG = range(7)
P = 0x100000   # aligned, never dereferenced


def test_quantize_rows(lib):
    f = lib.fp8_quantize_rows
    call = lambda **kw: f(kw.get("x", P), kw.get("dt", 0), kw.get("rows", 4), kw.get("K", 256), kw.get("off", None),
                          kw.get("E", 0), kw.get("codes", P), kw.get("scales", P), None)
    assert call(dt=2) == ERR_ARG
    for kw in ({"K": 24}, {"K": 0}, {"K": 65552}, {"rows": -1}, {"rows": 1 << 28}, {"rows": 1 << 31}, {"off": P, "E": 0}, {"off": P, "E": 1025}):
        assert call(**kw) == ERR_SHAPE, kw
    for n in ("x", "codes", "scales"):
        assert call(**{n: None}) == ERR_NULL
        assert call(**{n: P + 8}) == ERR_ALIGN
    assert call(rows=0, x=None, codes=None, scales=None) == OK


def test_quantize_weights(lib):
    f = lib.fp8_quantize_weights
    call = lambda **kw: f(kw.get("w", P), kw.get("E", 2), kw.get("N", 256), kw.get("K", 256), kw.get("c", P),
                          kw.get("s", P), kw.get("ct", P), kw.get("st", P), None)
    for kw in ({"K": 40}, {"N": 0}, {"N": 24}, {"N": (1 << 20) + 16}, {"E": 65536}, {"E": -1}, {"N": 65552}):
        assert call(**kw) == ERR_SHAPE, kw
    for kw in ({"w": None}, {"c": None, "ct": None}, {"s": None}, {"st": None}):
        assert call(**kw) == ERR_NULL, kw
    for n in ("w", "c", "s", "ct", "st"):
        assert call(**{n: P + 4}) == ERR_ALIGN, n
    assert call(E=0, w=None, c=None, s=None, ct=None, st=None) == OK


def test_swiglu_quantize(lib):
    f = lib.fp8_swiglu_quantize
    call = lambda **kw: f(kw.get("gu", P), kw.get("dt", 1), kw.get("R", 8), kw.get("I", 64), kw.get("off", P),
                          kw.get("E", 4), kw.get("tw", None), kw.get("map", None), kw.get("c", P), kw.get("s", P),
                          kw.get("h", None), None)
    assert call(dt=3) == ERR_ARG
    for kw in ({"I": 40}, {"I": 65552}, {"R": -1}, {"R": 1 << 28}, {"E": 0}, {"E": 1025}):
        assert call(**kw) == ERR_SHAPE, kw
    for kw in ({"gu": None}, {"off": None}, {"c": None}, {"s": None}, {"tw": P}):
        assert call(**kw) == ERR_NULL, kw
    for kw in ({"gu": P + 8}, {"c": P + 8}, {"s": P + 8}, {"h": P + 8}):
        assert call(**kw) == ERR_ALIGN, kw
    assert call(R=0, gu=None, off=None, c=None, s=None) == OK


def test_grouped_gemm(lib):
    f, g = lib.fp8_grouped_gemm, lib.fp8_grouped_gemm_gather

    def both(**kw):
        v = dict(a=P, sa=P, T=4096, map=P, k=8, off=P, E=128, R=32768, w=P, sw=P, N=1536, K=2048, c=P, cd=0) | kw
        tail = [v["off"], v["E"], v["R"], v["w"], v["sw"], v["N"], v["K"], v["c"], v["cd"], None]
        got = {g(v["a"], v["sa"], v["T"], v["map"], v["k"], *tail)}
        if not {"T", "map", "k"} & set(kw):
            got.add(f(v["a"], v["sa"], *tail))
        assert len(got) == 1
        return got.pop()

    assert both(cd=2) == ERR_ARG
    for kw in ({"E": 0}, {"E": 1025}, {"R": -1}, {"R": 1 << 30}, {"K": 2056}, {"K": 0}, {"K": 65552}, {"N": 0},
               {"N": (1 << 20) + 1}, {"k": 0}, {"k": 33}, {"T": 0}, {"T": -1}, {"T": 1 << 21}):
        assert both(**kw) == ERR_SHAPE, kw
    for kw in ({"a": None}, {"sa": None}, {"off": None}, {"w": None}, {"sw": None}, {"c": None}, {"map": None}):
        assert both(**kw) == ERR_NULL, kw
    for n in ("a", "sa", "w", "sw", "c"):
        assert both(**{n: P + 4}) == ERR_ALIGN, n
    assert f(None, None, None, 128, 0, None, None, 1536, 2048, None, 0, None) == OK
    assert g(None, None, 0, None, 8, None, 128, 0, None, None, 1536, 2048, None, 0, None) == OK


def test_wgrad(lib):
    f = lib.bf16_grouped_gemm_wgrad
    call = lambda **kw: f(kw.get("g", P), kw.get("gr", 64), kw.get("gk", 0), kw.get("x", P), kw.get("xr", 64),
                          kw.get("xk", 0), kw.get("map", None), kw.get("off", P), kw.get("E", 4), kw.get("R", 64),
                          kw.get("M", 128), kw.get("N", 128), kw.get("c", P), kw.get("cd", 0), None)
    assert call(cd=5) == ERR_ARG
    for kw in ({"E": 0}, {"E": 1025}, {"R": -1}, {"M": 0}, {"M": 12}, {"N": 4}, {"N": (1 << 20) + 8}, {"gk": -1},
               {"xk": 33}, {"gr": 63}, {"xr": 63}, {"gk": 2, "gr": 0, "map": P}, {"gk": 1, "gr": 1 << 25, "map": P}):
        assert call(**kw) == ERR_SHAPE, kw
    for kw in ({"g": None}, {"x": None}, {"off": None}, {"c": None}, {"xk": 2}):
        assert call(**kw) == ERR_NULL, kw
    for kw in ({"g": P + 8}, {"x": P + 8}, {"c": P + 8}):
        assert call(**kw) == ERR_ALIGN, kw


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    u8 = torch.zeros(4, 256, dtype=torch.uint8)
    for call in (lambda: pmg.fp8_quantize_rows(x), lambda: pmg.fp8_quantize_weights(x.view(1, 4, 256)),
                 lambda: pmg.fp8_swiglu_quantize(x, off), lambda: pmg.bf16_grouped_gemm_wgrad(x, x, off),
                 lambda: pmg.fp8_grouped_gemm(u8, x.float(), off, u8.view(2, 2, 256), x.float())):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(TypeError):
        pmg.fp8_quantize_rows(x.half())
    with pytest.raises(TypeError):
        pmg.fp8_grouped_gemm(x, x.float(), off, u8.view(2, 2, 256), x.float())
    with pytest.raises(TypeError):
        pmg.bf16_grouped_gemm_wgrad([1.0], x, off)
