"""Refusals of the training entry points, on the CPU: every argument check of the C ABI runs before any
CUDA call (the addresses below are never followed), and the binding's checks before any call into
the library."""
import pytest
import torch

import fp32_accumulate_lm_b200 as lm
from fp32_accumulate_lm_b200 import _build
from test_binding_checks import FakeCuda

HID, W, BIAS, TGT = 0x10000000, 0x20000000, 0x30000000, 0x31000000
LOSS, LSE, WS = 0x32000000, 0x33000000, 0x400000000
GL, DH, DW, DB = 0x34000000, 0x50000000, 0x60000000, 0x70000000
PASSED = (0, 4, 5, 6)  # past every argument check


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return lm.load_library()


def forward(**kw):
    a = dict(h=HID, dt=0, rows=40, H=64, w=W, V=300, alpha=1.0, b=0, t=TGT, ignore=-100, z=0.0, red=2,
             loss=LOSS, lse=LSE, ws=WS, n=None)
    a.update(kw)
    n = a["n"]
    if n is None:
        n = 1 << 30
    return lm.lmhead_cross_entropy_f32(a["h"], a["dt"], a["rows"], a["H"], a["w"], a["V"], a["alpha"],
                                       a["b"], a["t"], a["ignore"], a["z"], a["red"], a["loss"],
                                       a["lse"], a["ws"], n, 0)


def backward(**kw):
    a = dict(h=HID, dt=0, rows=40, H=64, w=W, V=300, alpha=1.0, b=0, t=TGT, ignore=-100, z=0.0, red=2,
             lse=LSE, gl=GL, dh=DH, dw=DW, db=0, acc=0, ws=WS, n=1 << 30)
    a.update(kw)
    return lm.lmhead_cross_entropy_grad(a["h"], a["dt"], a["rows"], a["H"], a["w"], a["V"],
                                        a["alpha"], a["b"], a["t"], a["ignore"], a["z"], a["red"],
                                        a["lse"], a["gl"], a["dh"], a["dw"], a["db"], a["acc"],
                                        a["ws"], a["n"], 0)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), 2), (dict(H=0), 2), (dict(V=0), 2), (dict(H=60), 3), (dict(dt=2), 2),
    (dict(rows=2 ** 30), 2), (dict(V=2 ** 30), 2), (dict(H=2 ** 30), 2), (dict(red=3), 2),
    (dict(red=-1), 2), (dict(ignore=2 ** 31), 2), (dict(ignore=-2 ** 31 - 1), 2),
    (dict(h=0), 1), (dict(w=0), 1), (dict(t=0), 1), (dict(ws=0), 1), (dict(lse=0), 1),
    (dict(h=HID + 8), 3), (dict(w=W + 2), 3), (dict(b=BIAS + 1), 3), (dict(t=TGT + 2), 3),
    (dict(lse=LSE + 1), 3), (dict(ws=WS + 128), 3),
])
def test_both_directions_refuse(kw, want):
    assert forward(**kw) == want
    assert backward(**kw) == want


def test_valid_calls_reach_the_device():
    for kw in (dict(), dict(b=BIAS), dict(ignore=lm.IGNORE_NONE), dict(ignore=2 ** 31 - 1),
               dict(red=0), dict(dt=1)):
        assert forward(**kw) in PASSED
        assert backward(**kw) in PASSED


def test_forward_outputs():
    assert forward(loss=0) == 1 and forward(loss=LOSS + 2) == 3
    need = lm.cross_entropy_workspace_bytes(40, 64, 300)
    assert need > 0 and forward(n=need - 1) == 2 and forward(n=need) in PASSED
    assert forward(loss=LSE + 8) == 7                       # inside lse
    assert forward(red=0, loss=LSE - 156) == 7              # the rows' losses end inside lse
    assert forward(red=2, loss=LSE - 156) in PASSED         # the mean is one number
    assert forward(lse=HID + 64) == 7 and forward(loss=W + 4) == 7 and forward(lse=TGT) == 7
    assert forward(b=BIAS, lse=BIAS + 8) == 7
    assert forward(ws=HID - 256) == 7 and forward(ws=(LSE >> 8) << 8) == 7
    # rows == 0: the rows' form does nothing, the others write one number
    assert forward(rows=0, red=0, h=0, w=0, t=0, loss=0, lse=0, ws=0) == 0
    assert forward(rows=0, loss=0) == 1 and forward(rows=0, loss=LOSS + 1) == 3


def test_backward_outputs():
    need = lm.cross_entropy_grad_workspace_bytes(40, 64, 300)
    assert need > 0 and backward(n=need - 1) == 2 and backward(n=need) in PASSED
    assert backward(dh=0, dw=0, db=0) == 1
    for kw in (dict(dh=0), dict(dw=0), dict(dh=0, dw=0, db=DB), dict(acc=1, db=DB, b=BIAS)):
        assert backward(**kw) in PASSED
    assert backward(gl=0) == 1 and backward(gl=GL + 2) == 3
    assert backward(dh=DH + 8) == 3 and backward(dw=DW + 8) == 3 and backward(db=DB + 1) == 3
    assert backward(dh=HID) == 7 and backward(dw=W) == 7 and backward(dw=DH + 64) == 7
    assert backward(db=DW + 64) == 7 and backward(dh=LSE - 64) == 7 and backward(dh=TGT) == 7
    assert backward(ws=DW) == 7 and backward(ws=W) == 7
    assert backward(red=0, dh=GL - 5120 + 64) == 7
    # rows == 0 that accumulates changes nothing and needs nothing
    assert backward(rows=0, h=0, w=0, t=0, lse=0, gl=0, ws=0, acc=1) == 0


def test_workspace_sizes():
    for f in (lm.cross_entropy_workspace_bytes, lm.cross_entropy_grad_workspace_bytes):
        for bad in ((0, 64, 300), (4, 0, 300), (4, 64, 0), (-1, 64, 300), (2 ** 30, 64, 300),
                    (4, 64, 2 ** 30)):
            assert f(*bad) == 0
        assert f(40, 64, 300) % 256 == 0
        assert f(200, 64, 300, None) < f(200, 64, 300)      # no place for the packed rows
    # d of a piece at a time: far from the logits of a training batch
    assert lm.cross_entropy_grad_workspace_bytes(16384, 4096, 151936) < 16384 * 151936 * 2 // 3
    assert lm.cross_entropy_workspace_bytes(16384, 4096, 151936) < 16384 * 151936 * 2 // 10
    for bad in ((0, 300, 64), (4, 0, 64), (4, 300, 0), (2 ** 30, 300, 64)):
        assert lm.embedding_grad_workspace_bytes(*bad) == 0


def embed(**kw):
    a = dict(ids=TGT, n=10, w=W, dt=0, V=300, v0=0, H=64, out=DH)
    a.update(kw)
    return lm.lmhead_embedding(a["ids"], a["n"], a["w"], a["dt"], a["V"], a["v0"], a["H"], 1.0,
                               a["out"], 0)


def embed_grad(**kw):
    a = dict(d=HID, dt=0, ids=TGT, n=10, V=300, v0=0, H=64, dw=DW, acc=0, ws=WS, nb=1 << 28)
    a.update(kw)
    return lm.lmhead_embedding_grad(a["d"], a["dt"], a["ids"], a["n"], a["V"], a["v0"], a["H"], 1.0,
                                    a["dw"], a["acc"], a["ws"], a["nb"], 0)


def test_embedding_refuses():
    for f in (embed, embed_grad):
        assert f() in PASSED and f(dt=1) in PASSED
        assert f(dt=2) == 2 and f(n=-1) == 2 and f(V=0) == 2 and f(H=0) == 2 and f(H=60) == 3
        assert f(n=2 ** 30) == 2 and f(V=2 ** 30) == 2 and f(v0=-1) == 2
        assert f(v0=2 ** 31 - 300) in PASSED and f(v0=2 ** 31 - 299) == 2
        assert f(ids=0) == 1 and f(ids=TGT + 1) == 3
    assert embed(w=0) == 1 and embed(out=0) == 1 and embed(w=W + 8) == 3 and embed(out=DH + 8) == 3
    assert embed(out=W + 64) == 7 and embed(out=TGT) == 7
    assert embed(n=0, ids=0, w=0, out=0) == 0
    need = lm.embedding_grad_workspace_bytes(10, 300, 64)
    assert embed_grad(nb=need) in PASSED and embed_grad(nb=need - 1) == 2
    assert embed_grad(d=0) == 1 and embed_grad(dw=0) == 1 and embed_grad(ws=0) == 1
    assert embed_grad(d=HID + 8) == 3 and embed_grad(dw=DW + 4) == 3 and embed_grad(ws=WS + 8) == 3
    assert embed_grad(dw=HID) == 7 and embed_grad(dw=TGT) == 7 and embed_grad(ws=DW) == 7
    assert embed_grad(n=0, d=0, ids=0, ws=0, acc=1) == 0


# ---------------------------------------------------------------- the binding

BF16, F16, F32, I32, I64, U8 = (torch.bfloat16, torch.float16, torch.float32, torch.int32,
                                torch.int64, torch.uint8)
R, H, V = 4, 64, 256


class Strided(FakeCuda):
    def is_contiguous(self):
        return False


def head(**kw):
    a = dict(hidden=FakeCuda((R, H), BF16), W=FakeCuda((V, H), BF16), targets=FakeCuda((R,), I32),
             bias=FakeCuda((V,), BF16))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw", [
    dict(hidden=FakeCuda((R, H), F32)), dict(W=FakeCuda((V, H), F16)),
    dict(W=FakeCuda((V, H + 8), BF16)), dict(hidden=FakeCuda((2, 2, H), BF16)),
    dict(hidden=Strided((R, H), BF16)), dict(W=Strided((V, H), BF16)),
    dict(W=FakeCuda((V, H), BF16, 1)), dict(targets=FakeCuda((R,), I64)),
    dict(targets=FakeCuda((R + 1,), I32)), dict(targets=FakeCuda((R,), I32, 1)),
    dict(targets=Strided((R,), I32)), dict(bias=FakeCuda((V,), F32)),
    dict(bias=FakeCuda((V + 1,), BF16)), dict(bias=FakeCuda((V,), BF16, 1)),
])
def test_binding_refuses_wrong_heads(kw):
    a = head(**kw)
    with pytest.raises(ValueError):
        lm.cross_entropy_f32(a["hidden"], a["W"], a["targets"], bias=a["bias"])
    with pytest.raises(ValueError):
        lm.cross_entropy_grad(a["hidden"], a["W"], a["targets"], FakeCuda((R,), F32),
                              FakeCuda((), F32), bias=a["bias"])


def test_binding_refuses_wrong_outputs_and_gradients():
    a = head()
    args = (a["hidden"], a["W"], a["targets"])
    lse, one, each = FakeCuda((R,), F32), FakeCuda((), F32), FakeCuda((R,), F32)
    bad = [
        lambda: lm.cross_entropy_f32(*args, reduction="max"),
        lambda: lm.cross_entropy_f32(*args, out=(each, lse)),               # a mean is one number
        lambda: lm.cross_entropy_f32(*args, reduction="none", out=(one, lse)),
        lambda: lm.cross_entropy_f32(*args, out=(one, FakeCuda((R + 1,), F32))),
        lambda: lm.cross_entropy_f32(*args, out=(one, FakeCuda((R,), F32, 1))),
        lambda: lm.cross_entropy_grad(*args, FakeCuda((R,), BF16), one),
        lambda: lm.cross_entropy_grad(*args, FakeCuda((R,), F32, 1), one),
        lambda: lm.cross_entropy_grad(*args, lse, each),
        lambda: lm.cross_entropy_grad(*args, lse, one, reduction="none"),
        lambda: lm.cross_entropy_grad(*args, lse, FakeCuda((), F16)),
        lambda: lm.cross_entropy_grad(*args, lse, one, accumulate=True),    # into what?
        lambda: lm.cross_entropy_grad(*args, lse, one, out=(None, None, None)),
        lambda: lm.cross_entropy_grad(*args, lse, one, out=(None, FakeCuda((V, H), F32), None)),
        lambda: lm.cross_entropy_grad(*args, lse, one, out=(None, FakeCuda((V, H), BF16, 1), None)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_wrong_embeddings():
    ids, table = FakeCuda((6,), I32), FakeCuda((V, H), BF16)
    bad = [
        lambda: lm.embedding(FakeCuda((6,), I64), table),
        lambda: lm.embedding(FakeCuda((6,), I32, 1), table),
        lambda: lm.embedding(Strided((6,), I32), table),
        lambda: lm.embedding(ids, FakeCuda((V, H), F32)),
        lambda: lm.embedding(ids, FakeCuda((V,), BF16)),
        lambda: lm.embedding(ids, Strided((V, H), BF16)),
        lambda: lm.embedding(ids, table, out=FakeCuda((6, H + 8), BF16)),
        lambda: lm.embedding_grad(FakeCuda((5, H), BF16), ids, V),
        lambda: lm.embedding_grad(FakeCuda((6, H), F32), ids, V),
        lambda: lm.embedding_grad(FakeCuda((6, H), BF16), ids, V, accumulate=True),
        lambda: lm.embedding_grad(FakeCuda((6, H), BF16), ids, V, out=FakeCuda((V + 1, H), BF16)),
        lambda: lm.embedding_grad(FakeCuda((6, H), BF16, 1), ids, V),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 16

    a = head()
    for call in (lambda: lm.cross_entropy_f32(a["hidden"], a["W"], a["targets"], stream=Stream()),
                 lambda: lm.embedding(FakeCuda((6,), I32), a["W"], stream=Stream())):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_wrappers_run_nothing_on_the_host():
    h, w = torch.zeros(R, H, dtype=BF16), torch.zeros(V, H, dtype=BF16)
    t = torch.zeros(R, dtype=I32)
    for call in (lambda: lm.cross_entropy_f32(h, w, t), lambda: lm.embedding(t, w),
                 lambda: lm.linear_cross_entropy(h, w, t), lambda: lm.embed(t, w),
                 lambda: lm.embedding_grad(h, t, V)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        lm.linear_cross_entropy(h, w, t[:2])


