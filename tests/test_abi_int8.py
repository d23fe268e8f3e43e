"""C-ABI checks of the int8 and scored-router entry points that need no GPU:
bad arguments are rejected before the device is touched."""

import os

import pytest
import torch

from block_diffusion_lm_tq4_amd import _lib, ops

OK, E_NULL, E_SHAPE, E_ALIGN, E_WS = 0, 1, 2, 3, 4
FAKE = 0x10000          # a non-null, 256-byte aligned address that is never touched
MIS = FAKE + 2


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libtq4.so is not built (run __graft_entry__.build())")
    return _lib.lib()


def test_sizes(L):
    assert L.tq4_int8_cache_size(8192, 2688) == 8192 * 2688 + 8192 * 4
    assert L.tq4_int8_cache_size(10, 96) == 10 * 128 + 40          # k padded to 64
    assert L.tq4_int8_cache_size(10, 33) == 0
    assert L.tq4_int8_cache_size(-1, 64) == 0
    assert L.tq4_int8_cache_size(10, 0) == 0
    assert L.tq4_int8_cache_size(10, 131072) > 0
    assert L.tq4_int8_cache_size(10, 131072 + 32) == 0             # int32 sums could overflow
    assert L.tq4_linear_int8_workspace_size(16, 2688, 8192) >= 16 * 2688 + 64
    assert L.tq4_linear_int8_workspace_size(0, 2688, 8192) == 0
    assert L.tq4_linear_int8_workspace_size(16, 2690, 8192) == 0


def test_cache_and_act_errors(L):
    for fn, args in ((L.tq4_int8_cache, (7,)), (L.tq4_int8_cache_bf16, ())):
        assert fn(FAKE, 8, 95, *args, FAKE, None) == E_SHAPE
        assert fn(FAKE, -1, 96, *args, FAKE, None) == E_SHAPE
        assert fn(FAKE, 8, 262144, *args, FAKE, None) == E_SHAPE
        assert fn(None, 8, 96, *args, FAKE, None) == E_NULL
        assert fn(FAKE, 8, 96, *args, None, None) == E_NULL
        assert fn(FAKE + 2, 8, 96, *args, FAKE, None) == E_ALIGN
        assert fn(FAKE, 8, 96, *args, FAKE + 4, None) == E_ALIGN
        assert fn(None, 0, 96, *args, None, None) == OK
    a = L.tq4_act_int8
    assert a(FAKE, 4, 48, FAKE, FAKE, None) == E_SHAPE
    assert a(FAKE, 4, 64, None, FAKE, None) == E_NULL
    assert a(FAKE, 4, 64, FAKE, None, None) == E_NULL
    assert a(FAKE + 2, 4, 64, FAKE, FAKE, None) == E_ALIGN
    assert a(FAKE, 4, 64, FAKE + 8, FAKE, None) == E_ALIGN
    assert a(FAKE, 4, 64, FAKE, FAKE + 2, None) == E_ALIGN
    assert a(None, 4, 0, None, None, None) == OK


@pytest.mark.parametrize("form", ["plain", "fp32", "bf16"])
def test_linear_errors(L, form):
    ws = L.tq4_linear_int8_workspace_size(100, 2688, 8192)
    far = FAKE + (1 << 24)

    def call(**kw):
        a = dict(dict(x=FAKE, m=100, k=2688, c=FAKE, n=8192, b=FAKE, r=far, y=FAKE, ws=FAKE,
                      wsb=ws), **kw)
        head = (a["x"], a["m"], a["k"], a["c"], a["n"])
        tail = (a["y"], a["ws"], a["wsb"], None)
        if form == "plain":
            return L.tq4_linear_int8(*head, *tail)
        fn = L.tq4_linear_int8_epilogue if form == "fp32" else L.tq4_linear_int8_epilogue_bf16
        return fn(*head, a["b"], a["r"], *tail)

    assert call(k=2690) == E_SHAPE
    assert call(k=262144) == E_SHAPE
    assert call(m=-1) == E_SHAPE
    assert call(n=1 << 31) == E_SHAPE
    assert call(x=None) == E_NULL
    assert call(c=None) == E_NULL
    assert call(y=None) == E_NULL
    assert call(x=MIS) == E_ALIGN
    assert call(c=FAKE + 4) == E_ALIGN
    assert call(y=FAKE + 1) == E_ALIGN
    assert call(ws=None) == E_WS
    assert call(wsb=ws - 1) == E_WS
    assert call(ws=FAKE + 16) == E_ALIGN
    assert call(m=0) == OK and call(n=0) == OK
    if form != "plain":
        elem = 4 if form == "fp32" else 2
        assert call(b=FAKE + 2) == E_ALIGN
        assert call(r=far + 1) == E_ALIGN
        assert call(r=FAKE + elem) == E_SHAPE                      # overlaps y without being y
        assert call(r=FAKE + 100 * 8192 * elem - elem) == E_SHAPE
        assert call(r=FAKE + 100 * 8192 * elem, ws=None) == E_WS
        assert call(r=FAKE, ws=None) == E_WS
        assert call(b=None, r=None, ws=None) == E_WS


def test_linear_quantized_errors(L):
    q = L.tq4_linear_int8_quantized
    assert q(FAKE, FAKE, 100, 2690, FAKE, 8192, FAKE, None) == E_SHAPE
    assert q(None, FAKE, 100, 2688, FAKE, 8192, FAKE, None) == E_NULL
    assert q(FAKE, None, 100, 2688, FAKE, 8192, FAKE, None) == E_NULL
    assert q(FAKE, FAKE, 100, 2688, None, 8192, FAKE, None) == E_NULL
    assert q(FAKE, FAKE, 100, 2688, FAKE, 8192, None, None) == E_NULL
    assert q(FAKE + 8, FAKE, 100, 2688, FAKE, 8192, FAKE, None) == E_ALIGN
    assert q(FAKE, FAKE + 2, 100, 2688, FAKE, 8192, FAKE, None) == E_ALIGN
    assert q(FAKE, FAKE, 100, 2688, FAKE + 8, 8192, FAKE, None) == E_ALIGN
    assert q(None, None, 0, 2688, None, 8192, None, None) == OK


def test_moe_errors(L):
    size = L.tq4_moe_grouped_int8_workspace_size
    ws = size(16, 6, 128, 1856, 2688)
    assert ws >= 16 * 2692 + 96 * (1856 * 3 + 4) + 96 * 2688 * 4
    assert size(16, 6, 128, 1850, 2688) == 0          # n1 % 32
    assert size(16, 7, 4, 64, 64) == 0                # topk > E
    assert size(16, 6, 513, 64, 64) == 0
    assert size(1 << 20, 6, 128, 1856, 2688) == 0     # t * kp reaches 2^31
    assert size(1 << 19, 8, 128, 1024, 64) == 0       # t * topk * n1p does

    def call(**kw):
        a = dict(dict(x=FAKE, t=16, k=2688, ids=FAKE, g=FAKE, topk=6, e=128, w1=FAKE, n1=1856,
                      w2=FAKE, out=FAKE, ws=FAKE, wsb=ws), **kw)
        return L.tq4_moe_grouped_int8(a["x"], a["t"], a["k"], a["ids"], a["g"], a["topk"], a["e"],
                                      a["w1"], a["n1"], a["w2"], a["out"], a["ws"], a["wsb"], None)

    for bad in (dict(topk=129), dict(topk=0), dict(e=513), dict(n1=1850), dict(k=2690),
                dict(t=-1), dict(k=0)):
        assert call(**bad) == E_SHAPE
    for name in ("x", "ids", "g", "w1", "w2", "out"):
        assert call(**{name: None}) == E_NULL
    for name, off in (("x", 2), ("ids", 2), ("g", 2), ("w1", 4), ("w2", 4), ("out", 8)):
        assert call(**{name: FAKE + off}) == E_ALIGN
    assert call(ws=None) == E_WS
    assert call(wsb=ws - 1) == E_WS
    assert call(ws=FAKE + 16) == E_ALIGN
    assert call(t=0) == OK


def test_router_scored_errors(L):
    def call(**kw):
        a = dict(dict(l=FAKE, t=4, e=128, topk=6, score=1, b=FAKE, g=8, kg=4, ids=FAKE, w=FAKE),
                 **kw)
        return L.tq4_moe_router_scored(a["l"], a["t"], a["e"], a["topk"], a["score"], a["b"],
                                       a["g"], a["kg"], 1, 2.5, a["ids"], a["w"], None)

    for bad in (dict(t=-1), dict(e=0), dict(e=513), dict(topk=0), dict(topk=129), dict(score=2),
                dict(score=-1), dict(g=0), dict(g=7), dict(kg=0), dict(kg=9),
                dict(topk=17, kg=1), dict(t=(1 << 33) + 1)):
        assert call(**bad) == E_SHAPE
    for name in ("l", "ids", "w"):
        assert call(**{name: None}) == E_NULL
    for name in ("l", "b", "ids", "w"):
        assert call(**{name: MIS}) == E_ALIGN
    assert call(t=0, l=None, ids=None, w=None) == OK


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    cache = torch.zeros(8 * 68, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device"):
        ops.linear_int8(x, cache, 8)
    with pytest.raises(ValueError, match="device"):
        ops.act_int8(x)
    with pytest.raises(ValueError, match="device"):
        ops.moe_router_scored(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError, match="device"):
        ops.moe_grouped_int8(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), cache,
                             cache, 1, 32)


def test_linear_output_may_not_be_its_input(L):
    """A residual that is x and an output that is x too: some rows would be read
    after others were stored."""
    far = FAKE + (1 << 30)
    for m, k, n in ((1, 64, 64), (40, 64, 64)):
        ws = L.tq4_linear_int8_workspace_size(m, k, n)
        for y in (FAKE, FAKE + 4, FAKE + 2 * m * k - 4, FAKE - 4):
            assert L.tq4_linear_int8(FAKE, m, k, far, n, y, 2 * far, ws, None) == E_SHAPE
            assert L.tq4_linear_int8_epilogue(FAKE, m, k, far, n, None, None, y, 2 * far, ws,
                                              None) == E_SHAPE
            assert L.tq4_linear_int8_epilogue_bf16(FAKE, m, k, far, n, None, y, y, 2 * far, ws,
                                                   None) == E_SHAPE
        for y in (FAKE, FAKE + m * k - 4, FAKE - 4):
            assert L.tq4_linear_int8_quantized(FAKE, 3 * far, m, k, far, n, y, None) == E_SHAPE
        assert L.tq4_linear_int8_quantized(3 * far, FAKE, m, k, far, n, FAKE, None) == E_SHAPE


def test_linear_row_limit(L):
    big = (1 << 24) + 1
    for m, n in ((big, 8), (8, big)):
        assert L.tq4_linear_int8_workspace_size(m, 64, n) == 0
        assert L.tq4_linear_int8(FAKE, m, 64, FAKE, n, FAKE, FAKE, 1 << 40, None) == E_SHAPE
        assert L.tq4_linear_int8_quantized(FAKE, FAKE, m, 64, FAKE, n, FAKE, None) == E_SHAPE
    assert L.tq4_linear_int8_workspace_size(1 << 24, 64, 8) > 0
    assert L.tq4_int8_cache_size(big, 64) == big * 68              # a cache may have more


def test_act_of_empty_rows(L):
    assert L.tq4_act_int8(None, 0, 0, None, None, None) == OK
    assert L.tq4_act_int8(None, 4, 0, None, None, None) == OK
    assert L.tq4_act_int8(None, 4, 0, None, MIS, None) == E_ALIGN
