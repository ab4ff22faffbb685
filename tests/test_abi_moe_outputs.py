"""Outputs that are an input or another output are refused before anything is enqueued (no GPU needed)."""
import pytest

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_LAUNCH, ERR_ARG = range(7)
P = [0x100000 * (j + 1) for j in range(12)]   # aligned, never dereferenced


@pytest.mark.parametrize("T", [4, 4096])      # a short list, a long one
@pytest.mark.parametrize("same", [("ids", "off"), ("ids", "r2t"), ("ids", "t2r"), ("off", "r2t"), ("off", "t2r"), ("r2t", "t2r"),
                                  ("x", "rows")])
def test_permute(lib, T, same):
    a = dict(zip(("x", "ids", "rows", "off", "r2t", "t2r", "ws"), P))
    a[same[1]] = a[same[0]]
    for x, rows in ((a["x"], a["rows"]), (None, None)):
        if x is None and same == ("x", "rows"):
            continue
        assert lib.moe_permute(x, 0, T, 64, a["ids"], 8, 128, rows, a["off"], a["r2t"], a["t2r"], a["ws"], 1 << 30,
                               None, None) == ERR_ARG


@pytest.mark.parametrize("same", [("gu", "dgu"), ("dh", "dgu"), ("w", "dw")])
def test_swiglu_backward_weights(lib, same):
    a = dict(zip(("gu", "dh", "off", "w", "r2t", "t2r", "dgu", "dw"), P))
    a[same[1]] = a[same[0]]
    assert lib.swiglu_backward_weights(a["gu"], a["dh"], 8, 64, a["off"], 4, a["w"], a["r2t"], a["t2r"], a["dgu"],
                                       a["dw"], None) == ERR_ARG
