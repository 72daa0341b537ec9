"""Host-side checks of the rotary norm's C ABI (no GPU, no kernel is launched)."""
import ctypes

import pytest
import torch

import onnx_recurrent_layers_amd as rl
from tests.test_ssm_host import ARG, FAKE, SHAPE, UNSUPPORTED, filled, refused

WHO = "rotary norm: "


def desc(**kw):
    return rl.rnn_rotary_desc(**(dict(dtype=0, interleaved=0, epsilon=1e-6, rows=5, q_heads=3, k_heads=2, size=6, rotary=4, table=10) | kw))


@pytest.fixture
def handle():
    h = rl.rnn_rotary_create(desc())
    yield h
    rl.rnn_rotary_destroy(h)


@pytest.mark.parametrize("field,value,code", [
    ("dtype", 3, ARG), ("dtype", -1, ARG), ("interleaved", 2, ARG), ("epsilon", -1.0, ARG), ("epsilon", float("nan"), ARG),
    ("epsilon", float("inf"), ARG), ("rows", -1, SHAPE), ("q_heads", 0, SHAPE), ("k_heads", -1, SHAPE), ("size", 0, SHAPE), ("rotary", 3, SHAPE),
    ("rotary", 8, SHAPE), ("rotary", -2, SHAPE), ("table", -1, SHAPE), ("size", 513, UNSUPPORTED), ("rows", (1 << 30) + 1, UNSUPPORTED),
    ("table", (1 << 30) + 1, UNSUPPORTED),
])
def test_create_refuses(field, value, code):
    refused(lambda: rl.rnn_rotary_create(desc(**{field: value})), code, WHO, field)


def test_more_refused_sizes():
    refused(lambda: rl.rnn_rotary_create(desc(q_heads=(1 << 20) + 1)), UNSUPPORTED, WHO, "heads")
    refused(lambda: rl.rnn_rotary_create(desc(rows=1 << 30, q_heads=1 << 20, size=512, rotary=4)), SHAPE, WHO, "Q: size overflows")


def test_null_arguments(handle):
    lib = rl.load_library()
    assert lib.rnn_rotary_create(None, ctypes.byref(ctypes.c_void_p())) == ARG and rl.rnn_last_error() == WHO + "desc: NULL"
    assert lib.rnn_rotary_create(ctypes.byref(desc()), None) == ARG
    rl.rnn_rotary_destroy(None)
    for f, n in (("scratch_size", 2), ("encode", 3), ("encode_backward", 4)):
        assert getattr(lib, f"rnn_rotary_{f}")(None, *[None] * n) == ARG and rl.rnn_last_error() == WHO + "rotary: NULL"
    assert lib.rnn_rotary_encode(handle, None, None, None) == ARG and "operands: NULL" in rl.rnn_last_error()
    assert lib.rnn_rotary_encode_backward(handle, None, None, None, None) == ARG and "operands: NULL" in rl.rnn_last_error()
    assert lib.rnn_rotary_encode_backward(handle, ctypes.byref(rl.rnn_rotary_operands()), None, None, None) == ARG
    assert "gradients: NULL" in rl.rnn_last_error()


def test_operands_refused(handle):
    encode, backward = rl.rnn_rotary_encode, rl.rnn_rotary_encode_backward
    for name in ("Q", "K", "cos", "sin", "positions"):
        refused(lambda: encode(handle, filled("rotary", "operands", (name,))), ARG, WHO, f"{name}: NULL")
    for name in ("dQ_out", "dK_out"):
        refused(lambda: backward(handle, filled("rotary", "operands"), filled("rotary", "gradients", (name,))), ARG, WHO, f"{name}: NULL")
    for struct, call in (("operands", lambda t: encode(handle, t)), ("gradients", lambda t: backward(handle, filled("rotary", "operands"), t))):
        for name, kind in getattr(rl, f"rnn_rotary_{struct}")._fields_:
            for field, value, code, text in (("elem_offset", -1, ARG, "negative element offset"), ("ptr", None, ARG, "address not aligned"),
                                             ("row_stride", 3, SHAPE, "row_stride 3 below"), ("row_stride", 1 << 60, SHAPE, "size overflows")):
                if field == "row_stride" and kind is not rl.rnn_rows:
                    continue
                t = filled("rotary", struct)
                setattr(getattr(t, name), field, getattr(t, name).ptr + 2 if value is None else value)
                refused(lambda: call(t), code, WHO, f"{name}: {text}")
    for out, other in (("Q_out", "K"), ("K_out", "Q"), ("K_out", "Q_out"), ("Q_out", "cos")):
        t = filled("rotary", "operands")
        getattr(t, out).ptr = getattr(t, other).ptr
        refused(lambda: encode(handle, t), ARG, WHO, "the same memory as")
    t = filled("rotary", "operands")
    t.Q_out.ptr, t.Q_out.row_stride = t.Q.ptr, 40
    refused(lambda: encode(handle, t), ARG, WHO, "Q_out: the memory of its input at another row_stride")
    t = filled("rotary", "gradients")
    t.dQ.ptr = t.dQ_out.ptr
    refused(lambda: backward(handle, filled("rotary", "operands"), t), ARG, WHO, "dQ: the same memory as dQ_out")
    refused(lambda: backward(handle, filled("rotary", "operands"), filled("rotary", "gradients")), ARG, WHO, "scratch: NULL")
    refused(lambda: backward(handle, filled("rotary", "operands"), filled("rotary", "gradients"), FAKE + 64), ARG, WHO, "scratch: not 256-byte aligned")


def test_nothing_asked_for_is_nothing_done(handle):
    rl.rnn_rotary_encode(handle, filled("rotary", "operands", ("Q_out", "K_out")))
    g = rl.rnn_rotary_gradients()
    g.dQ_out.ptr = FAKE + (1 << 16)
    rl.rnn_rotary_encode_backward(handle, filled("rotary", "operands"), g)
    h = rl.rnn_rotary_create(desc(rows=0))
    rl.rnn_rotary_encode(h, filled("rotary", "operands"))
    rl.rnn_rotary_destroy(h)


def test_binding_refuses_tensors():
    op = rl.RotaryNorm(dtype="f16", rows=4, q_heads=3, k_heads=2, size=10, table=7, device="cuda:0")
    op._index = -1     # CPU tensors stand for the device's: nothing is launched

    def fill(**kw):
        return lambda: op._fill(op._forward, kw)

    refused(fill(Q=torch.zeros(4, 20, dtype=torch.float16)), SHAPE, WHO, "Q: shape")
    refused(fill(positions=torch.zeros(4, dtype=torch.int64)), ARG, WHO, "positions: type")
    refused(fill(cos=torch.zeros(7, 5, dtype=torch.float16)), ARG, WHO, "cos: type")
    refused(fill(sin=torch.zeros(7, 10)[:, ::2]), ARG, WHO, "sin: has to be contiguous")
    ops = rl.rnn_rotary_operands.from_buffer(fill(K=torch.zeros(4, 50, dtype=torch.float16)[:, 30:])())
    assert ops.K.row_stride == 50 and ops.Q.ptr is None
