"""C-ABI checks of the MXFP4 and router-training entry points that need no GPU: bad
arguments are rejected before the device is touched."""

import os

import pytest
import torch

from block_diffusion_lm_tq4_amd import _lib, ops

OK, E_NULL, E_SHAPE, E_ALIGN, E_WS = 0, 1, 2, 3, 4
FAKE = 0x10000          # a non-null, 256-byte aligned address that is never touched
FAR = FAKE + (1 << 30)
BIG = (1 << 24) + 1


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libtq4.so is not built (run __graft_entry__.build())")
    return _lib.lib()


def test_sizes(L):
    assert L.tq4_mxfp4_cache_size(8192, 2688) == 8192 * (1344 + 84)
    assert L.tq4_mxfp4_cache_size(10, 96) == 10 * (64 + 4)          # k padded to 128
    assert L.tq4_mxfp4_cache_size(3, 1856) == 3 * (960 + 60)
    assert L.tq4_mxfp4_cache_size(10, 33) == 0
    assert L.tq4_mxfp4_cache_size(-1, 64) == 0
    assert L.tq4_mxfp4_cache_size(10, 0) == 0
    assert L.tq4_mxfp4_cache_size(10, 1 << 20) > 0
    assert L.tq4_mxfp4_cache_size(10, (1 << 20) + 32) == 0
    assert L.tq4_mxfp4_cache_size(BIG, 64) == BIG * 68              # a cache may have more rows
    w = L.tq4_linear_mxfp4_workspace_size
    assert w(100, 2688, 8192) >= 100 * 1428
    assert w(1, 2688, 8192) == w(16, 2688, 8192) == 0               # quantized by the product
    assert w(0, 2688, 8192) == w(100, 2690, 8192) == 0
    assert w(BIG, 64, 8) == w(100, 64, BIG) == 0 and w(1 << 24, 64, 8) > 0
    b = L.tq4_moe_balance_workspace_size
    assert b(16, 128) == b(0, 1) == 0                               # one workgroup
    assert b(1024, 128) >= 16 * 4 * 257
    assert b(-1, 128) == b(16, 0) == b(16, 513) == 0


def test_cache_act_and_values_errors(L):
    for fn, args in ((L.tq4_mxfp4_cache, (7,)), (L.tq4_mxfp4_cache_bf16, ())):
        assert fn(FAKE, 8, 95, *args, FAKE, None) == E_SHAPE
        assert fn(FAKE, -1, 96, *args, FAKE, None) == E_SHAPE
        assert fn(FAKE, 8, 1 << 21, *args, FAKE, None) == E_SHAPE
        assert fn(FAKE, 1 << 31, 96, *args, FAKE, None) == E_SHAPE
        assert fn(None, 8, 96, *args, FAKE, None) == E_NULL
        assert fn(FAKE, 8, 96, *args, None, None) == E_NULL
        assert fn(FAKE + 2, 8, 96, *args, FAKE, None) == E_ALIGN
        assert fn(FAKE, 8, 96, *args, FAKE + 4, None) == E_ALIGN
        assert fn(None, 0, 96, *args, None, None) == OK
    a = L.tq4_act_mxfp4
    assert a(FAKE, 4, 48, FAKE, FAKE, None) == E_SHAPE
    for args in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None)):
        assert a(args[0], 4, 64, args[1], args[2], None) == E_NULL
    assert a(FAKE + 2, 4, 64, FAKE, FAKE, None) == E_ALIGN
    assert a(FAKE, 4, 64, FAKE + 8, FAKE, None) == E_ALIGN
    assert a(FAKE, 4, 64, FAKE, FAKE + 2, None) == E_ALIGN
    assert a(None, 4, 0, None, None, None) == a(None, 0, 64, None, None, None) == OK
    v = L.tq4_mxfp4_values
    assert v(FAKE, FAKE, 4, 48, FAKE, None) == E_SHAPE
    for args in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None)):
        assert v(args[0], args[1], 4, 64, args[2], None) == E_NULL
    assert v(FAKE + 8, FAKE, 4, 64, FAKE, None) == E_ALIGN
    assert v(FAKE, FAKE + 1, 4, 64, FAKE, None) == E_ALIGN
    assert v(FAKE, FAKE, 4, 64, FAKE + 8, None) == E_ALIGN
    assert v(None, None, 0, 64, None, None) == OK


@pytest.mark.parametrize("m", [16, 100])
@pytest.mark.parametrize("form", ["plain", "fp32", "bf16"])
def test_linear_errors(L, form, m):
    ws = L.tq4_linear_mxfp4_workspace_size(m, 2688, 8192)
    far = FAKE + (1 << 24)

    def call(**kw):
        a = dict(dict(x=FAR, m=m, k=2688, c=FAKE, n=8192, b=FAKE, r=far, y=FAKE, ws=FAKE,
                      wsb=ws), **kw)
        head = (a["x"], a["m"], a["k"], a["c"], a["n"])
        tail = (a["y"], a["ws"], a["wsb"], None)
        if form == "plain":
            return L.tq4_linear_mxfp4(*head, *tail)
        fn = L.tq4_linear_mxfp4_epilogue if form == "fp32" else L.tq4_linear_mxfp4_epilogue_bf16
        return fn(*head, a["b"], a["r"], *tail)

    for bad in (dict(k=2690), dict(k=1 << 21), dict(m=-1), dict(n=BIG), dict(m=BIG)):
        assert call(**bad) == E_SHAPE
    for name in ("x", "c", "y"):
        assert call(**{name: None}) == E_NULL
    assert call(x=FAR + 2) == E_ALIGN
    assert call(c=FAKE + 4) == E_ALIGN
    assert call(y=FAKE + 1) == E_ALIGN
    if ws:
        assert call(ws=None) == E_WS
        assert call(wsb=ws - 1) == E_WS
        assert call(ws=FAKE + 16) == E_ALIGN
    assert call(m=0) == OK and call(n=0) == OK
    elem = 2 if form == "bf16" else 4
    size = m * 8192 * elem
    for x in (FAKE, FAKE + 16, FAKE + size - 16, FAKE - 16):         # y overlaps x
        assert call(x=x) == E_SHAPE
    if form != "plain":
        assert call(b=FAKE + 2) == E_ALIGN
        assert call(r=far + 1) == E_ALIGN
        assert call(r=FAKE + elem) == E_SHAPE                        # overlaps y without being y
        assert call(r=FAKE + size - elem) == E_SHAPE


def test_linear_quantized_errors(L):
    q = L.tq4_linear_mxfp4_quantized
    assert q(FAR, FAR, 100, 2690, FAKE, 8192, FAKE, None) == E_SHAPE
    assert q(FAR, FAR, BIG, 64, FAKE, 8192, FAKE, None) == E_SHAPE
    assert q(None, FAR, 100, 2688, FAKE, 8192, FAKE, None) == E_NULL
    assert q(FAR, None, 100, 2688, FAKE, 8192, FAKE, None) == E_NULL
    assert q(FAR, FAR, 100, 2688, None, 8192, FAKE, None) == E_NULL
    assert q(FAR, FAR, 100, 2688, FAKE, 8192, None, None) == E_NULL
    assert q(FAR + 8, FAR, 100, 2688, FAKE, 8192, FAKE, None) == E_ALIGN
    assert q(FAR, FAR + 2, 100, 2688, FAKE, 8192, FAKE, None) == E_ALIGN
    assert q(FAR, FAR, 100, 2688, FAKE + 8, 8192, FAKE, None) == E_ALIGN
    assert q(FAKE, FAR, 100, 2688, FAR, 8192, FAKE, None) == E_SHAPE      # y over the codes
    assert q(FAR, FAKE + 64, 100, 2688, FAR, 8192, FAKE, None) == E_SHAPE  # or the scales
    assert q(None, None, 0, 2688, None, 8192, None, None) == OK


def test_moe_errors(L):
    size = L.tq4_moe_grouped_mxfp4_workspace_size
    ws = size(16, 6, 128, 1856, 2688)
    assert ws >= 16 * 1428 + 96 * 1020 + 96 * 2688 * 4
    assert size(16, 6, 128, 1850, 2688) == 0          # n1 % 32
    assert size(16, 7, 4, 64, 64) == 0                # topk > E
    assert size(16, 6, 513, 64, 64) == 0
    assert size(1 << 21, 6, 128, 1856, 2688) == 0     # t * kp / 2 reaches 2^31
    assert size(1 << 19, 8, 128, 1024, 64) == 0       # t * topk * n1p / 2 does
    assert size(16, 6, 128, 1856, 1 << 21) == 0

    def call(**kw):
        a = dict(dict(x=FAKE, t=16, k=2688, ids=FAKE, g=FAKE, topk=6, e=128, w1=FAKE, n1=1856,
                      w2=FAKE, out=FAKE, ws=FAKE, wsb=ws), **kw)
        return L.tq4_moe_grouped_mxfp4(a["x"], a["t"], a["k"], a["ids"], a["g"], a["topk"],
                                       a["e"], a["w1"], a["n1"], a["w2"], a["out"], a["ws"],
                                       a["wsb"], None)

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


def test_balance_errors(L):
    ws = L.tq4_moe_balance_workspace_size(400, 128)   # (up to 256 tokens need none)

    def call(**kw):
        a = dict(dict(l=FAKE, t=400, e=128, ids=FAKE, topk=6, score=0, loss=FAKE, c=FAKE, n=FAKE,
                      p=FAKE, ws=FAKE, wsb=ws), **kw)
        return L.tq4_moe_balance(a["l"], a["t"], a["e"], a["ids"], a["topk"], a["score"],
                                 a["loss"], a["c"], a["n"], a["p"], a["ws"], a["wsb"], None)

    for bad in (dict(t=-1), dict(e=0), dict(e=513), dict(topk=0), dict(topk=129), dict(score=2),
                dict(score=-1), dict(t=(1 << 31) // 6 + 1)):
        assert call(**bad) == E_SHAPE
    for name in ("l", "ids", "loss", "c", "n", "p"):
        assert call(**{name: None}) == E_NULL
        assert call(**{name: FAKE + 2}) == E_ALIGN
    assert call(ws=None) == E_WS
    assert call(wsb=ws - 1) == E_WS
    assert call(ws=FAKE + 16) == E_ALIGN
    assert call(t=0, loss=None) == E_NULL             # an empty batch still writes zeros


def test_router_backward_errors(L):
    def call(**kw):
        a = dict(dict(l=FAKE, t=40, e=128, ids=FAKE, topk=6, score=1, dg=FAKE, c=FAKE, n=FAKE,
                      dl=FAKE, out=FAR), **kw)
        return L.tq4_moe_router_backward(a["l"], a["t"], a["e"], a["ids"], a["topk"], a["score"],
                                         a["dg"], 1, 2.5, a["c"], a["n"], a["dl"], a["out"], None)

    for bad in (dict(t=-1), dict(e=0), dict(e=513), dict(topk=0), dict(topk=129), dict(score=2)):
        assert call(**bad) == E_SHAPE
    for name in ("l", "ids", "c", "n", "dl", "out"):
        assert call(**{name: None}) == E_NULL
    for name in ("l", "ids", "dg", "c", "n", "dl", "out"):
        assert call(**{name: FAR + (1 << 26) + 2}) == E_ALIGN
    far = FAR + (1 << 28)
    for bad in (dict(l=FAR), dict(l=FAR + 40 * 512 - 4), dict(l=FAR - 40 * 512 + 4),
                dict(ids=FAR + 400), dict(dg=FAR + 400), dict(ids=FAR - 40 * 24 + 4),
                dict(c=FAR + 400), dict(c=FAR - 512 + 4), dict(n=FAR), dict(dl=FAR + 400)):
        assert call(**dict(dict(l=far, ids=far, dg=far), **bad)) == E_SHAPE
    assert call(t=0, l=None, ids=None, out=None) == OK


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    cache = torch.zeros(8 * 68, dtype=torch.uint8)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: ops.linear_mxfp4(x, cache, 8), lambda: ops.act_mxfp4(x),
                 lambda: ops.mxfp4_values(cache.view(8, 68), cache.view(8, 68), 128),
                 lambda: ops.linear_mxfp4_quantized(cache.view(8, 68), cache, 64, cache, 8),
                 lambda: ops.mxfp4_cache_bf16(x),
                 lambda: ops.moe_grouped_mxfp4(x, ids, torch.zeros(4, 2), cache, cache, 1, 32),
                 lambda: ops.moe_balance(torch.zeros(4, 8), ids),
                 lambda: ops.moe_router_backward(torch.zeros(4, 8), ids)):
        with pytest.raises(ValueError, match="device"):
            call()


def test_mxfp4_abi_checks_pass_under_asan_and_ubsan():
    import subprocess
    import sys

    from test_abi_sanitized import ROOT, _hipcc, _stale
    if os.environ.get("TQ4_LIBRARY"):
        pytest.skip("already under the sanitizers")
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not available")
    from block_diffusion_lm_tq4_amd import build as B
    if _stale(B.SANITIZED_LIB):
        B.build_sanitized()
    runtime = subprocess.run([hipcc, "-print-file-name=libclang_rt.asan-x86_64.so"],
                             capture_output=True, text=True).stdout.strip()
    assert os.path.exists(runtime), runtime
    env = dict(os.environ)
    env.update(TQ4_LIBRARY=B.SANITIZED_LIB, LD_PRELOAD=runtime,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                          os.path.abspath(__file__)],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-4000:]
    assert "passed" in out and "ERROR: AddressSanitizer" not in out and "runtime error" not in out
