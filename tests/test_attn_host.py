"""Host-side checks of linear attention's C ABI (no GPU, no kernel is
launched): descriptions and operands are refused with messages that name
operator and argument, and the binding's own checks of tensors."""
import ctypes

import pytest
import torch

import onnx_recurrent_layers_amd as rl
from tests.test_ssm_host import ARG, FAKE, SHAPE, UNSUPPORTED, filled, refused

WHO = "linear attention: "


def desc(**kw):
    return rl.rnn_attn_desc(**(dict(dtype=0, direction=0, layout=1, scale=1.0, seq=5, batch=3, heads=6, groups=2, key=4, value=8) | kw))


@pytest.fixture
def handle():
    h = rl.rnn_attn_create(desc())
    yield h
    rl.rnn_attn_destroy(h)


@pytest.mark.parametrize("field,value,code", [
    ("dtype", 3, ARG), ("dtype", -1, ARG), ("direction", 2, ARG), ("direction", 5, ARG), ("layout", 2, ARG), ("scale", float("nan"), ARG),
    ("scale", float("inf"), ARG), ("seq", -1, SHAPE), ("batch", -1, SHAPE), ("heads", 0, SHAPE), ("groups", 0, SHAPE), ("groups", 4, SHAPE),
    ("groups", 12, SHAPE), ("key", 0, SHAPE), ("value", 0, SHAPE), ("key", 257, UNSUPPORTED), ("value", 257, UNSUPPORTED),
    ("heads", (1 << 24) + 1, UNSUPPORTED), ("batch", (1 << 30) + 1, UNSUPPORTED), ("seq", (1 << 30) + 1, UNSUPPORTED),
])
def test_create_refuses(field, value, code):
    refused(lambda: rl.rnn_attn_create(desc(**{field: value})), code, WHO, field)


@pytest.mark.parametrize("fields,code", [
    (dict(seq=1 << 29, batch=1 << 29), SHAPE), (dict(batch=1 << 24, heads=2, seq=1), UNSUPPORTED),
    (dict(seq=1 << 30, batch=1 << 20, heads=1, groups=1, key=256), SHAPE),
])
def test_sizes_are_checked_in_64_bits(fields, code):
    refused(lambda: rl.rnn_attn_create(desc(**fields)), code, WHO, "")


def test_null_arguments(handle):
    lib = rl.load_library()
    assert lib.rnn_attn_create(None, ctypes.byref(ctypes.c_void_p())) == ARG and rl.rnn_last_error() == WHO + "desc: NULL"
    assert lib.rnn_attn_create(ctypes.byref(desc()), None) == ARG
    rl.rnn_attn_destroy(None)
    for f, n in (("scratch_size", 2), ("encode", 3), ("encode_backward", 4)):
        assert getattr(lib, f"rnn_attn_{f}")(None, *[None] * n) == ARG and rl.rnn_last_error() == WHO + "attn: NULL"
    assert lib.rnn_attn_encode(handle, None, None, None) == ARG and "operands: NULL" in rl.rnn_last_error()
    assert lib.rnn_attn_encode_backward(handle, None, None, None, None) == ARG and "operands: NULL" in rl.rnn_last_error()
    assert lib.rnn_attn_encode_backward(handle, ctypes.byref(rl.rnn_attn_operands()), None, None, None) == ARG
    assert "gradients: NULL" in rl.rnn_last_error()
    assert lib.rnn_attn_scratch_size(handle, None, None) == rl.RNN_OK and rl.rnn_last_error() == ""


def test_operands_refused(handle):
    encode, backward = rl.rnn_attn_encode, rl.rnn_attn_encode_backward
    for name in ("Q", "K", "V"):
        refused(lambda: encode(handle, filled("attn", "operands", (name,))), ARG, WHO, f"{name}: NULL")
    refused(lambda: backward(handle, filled("attn", "operands"), filled("attn", "gradients", ("dY",))), ARG, WHO, "dY: NULL")
    for struct, call in (("operands", lambda t: encode(handle, t)), ("gradients", lambda t: backward(handle, filled("attn", "operands"), t))):
        for name, kind in getattr(rl, f"rnn_attn_{struct}")._fields_:
            for field, value, code, text in (("elem_offset", -1, ARG, "negative element offset"), ("elem_offset", 1 << 60, SHAPE, "element offset overflows"),
                                             ("ptr", None, ARG, "address not aligned"), ("row_stride", 3, SHAPE, "row_stride 3 below"),
                                             ("row_stride", 1 << 60, SHAPE, "size overflows")):
                if field == "row_stride" and kind is not rl.rnn_rows:
                    continue
                t = filled("attn", struct)
                setattr(getattr(t, name), field, getattr(t, name).ptr + 2 if value is None else value)
                refused(lambda: call(t), code, WHO, f"{name}: {text}")
    for out, other in (("Y", "V"), ("Y", "Q"), ("final_state", "G")):
        t = filled("attn", "operands")
        getattr(t, out).ptr = getattr(t, other).ptr
        refused(lambda: encode(handle, t), ARG, WHO, f"{out}: the same memory as {other}")
    for out, other in (("dV", "dY"), ("dQ", "dY"), ("dK", "dQ"), ("d_initial_state", "d_final_state")):
        t = filled("attn", "gradients")
        getattr(t, out).ptr = getattr(t, other).ptr
        refused(lambda: backward(handle, filled("attn", "operands"), t), ARG, WHO, f"{out}: the same memory as {other}")
    refused(lambda: backward(handle, filled("attn", "operands"), filled("attn", "gradients")), ARG, WHO, "scratch: NULL")
    refused(lambda: backward(handle, filled("attn", "operands"), filled("attn", "gradients"), FAKE + 64), ARG, WHO, "scratch: not 256-byte aligned")


def test_nothing_asked_for_is_nothing_done(handle):
    """No output, or no batch row: success, with no launch and no scratch."""
    rl.rnn_attn_encode(handle, filled("attn", "operands", ("Y", "final_state")))
    g = rl.rnn_attn_gradients()
    g.dY.ptr = FAKE + (1 << 16)
    rl.rnn_attn_encode_backward(handle, filled("attn", "operands"), g)
    h = rl.rnn_attn_create(desc(batch=0))
    rl.rnn_attn_encode(h, filled("attn", "operands"))
    rl.rnn_attn_destroy(h)


def test_scratch_sizes(monkeypatch):
    def up(n):
        return (n + 255) // 256 * 256

    def sizes(**kw):
        h = rl.rnn_attn_create(desc(**kw))
        try:
            return rl.rnn_attn_scratch_size(h)
        finally:
            rl.rnn_attn_destroy(h)

    monkeypatch.delenv("RNN_ATTN_PIECE", raising=False)
    # tokens: each step's two sums and each row's product and sum; for shared queries a row of every head
    rows, one = up(3 * 6 * 4 * 4), up(3 * 6 * 4)
    assert sizes(seq=4) == (0, 2 * rows + 2 * one + up(4 * 3 * 6 * 4 * 4))
    assert sizes(seq=4, groups=6) == (0, 2 * rows + 2 * one)
    monkeypatch.setenv("RNN_ATTN_PIECE", "100")    # of 128 steps: two
    starts = up(3 * 6 * 2 * 4 * 8 * 4) + up(3 * 6 * 2 * 4)
    assert sizes(seq=200, groups=6) == (starts, 2 * starts + 2 * up(3 * 6 * 200 * 4) + 2 * up(3 * 6 * 2 * 4))
    monkeypatch.setenv("RNN_ATTN_PIECE", "1000")
    assert sizes(seq=200, groups=6) == (0, 2 * up(3 * 6 * 200 * 4) + 2 * up(3 * 6 * 4))


def test_binding_refuses_tensors():
    op = rl.LinearAttention(dtype="f16", seq=4, batch=3, heads=6, groups=2, key=5, value=7, device="cuda:0")
    op._index = -1     # CPU tensors stand for the device's: nothing is launched
    good = {"Q": torch.zeros(3, 4, 10, dtype=torch.float16)}

    def fill(**kw):
        return lambda: op._fill(op._forward, good | kw)

    fill()()
    refused(fill(Q=torch.zeros(3, 4, 2, 5, dtype=torch.float16)), SHAPE, WHO, "Q: shape")
    refused(fill(Q=torch.zeros(3, 4, 10)), ARG, WHO, "Q: type")
    refused(fill(G=torch.zeros(3, 4, 6, dtype=torch.float16)), ARG, WHO, "G: type")
    refused(fill(V=torch.zeros(3, 4, 84, dtype=torch.float16)[..., ::2]), ARG, WHO, "V: the elements of a row")
    refused(fill(initial_state=torch.zeros(3, 6, 7, 5).transpose(2, 3)), ARG, WHO, "initial_state: has to be contiguous")
    refused(lambda: op.encode({"X": torch.zeros(1)}), ARG, WHO, "X: unknown tensor")
    ops = rl.rnn_attn_operands.from_buffer(fill(V=torch.zeros(3, 4, 50, dtype=torch.float16)[..., 4:46])())
    assert ops.V.row_stride == 50 and ops.Q.row_stride == 0 and ops.K.ptr is None
