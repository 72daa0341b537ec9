"""Host-side checks of the state space operators' and layer normalization's C
ABI (no GPU, no kernel is launched): descriptions and operands are refused with
messages that name operator and argument, scratch sizes by hand, and the
binding's own checks of tensors."""
import ctypes

import pytest
import torch

import onnx_recurrent_layers_amd as rl

ARG, SHAPE, UNSUPPORTED = rl.RNN_ERR_ARG, rl.RNN_ERR_SHAPE, rl.RNN_ERR_UNSUPPORTED
FAKE = 1 << 20     # an address that no check reads


def conv_desc(**kw):
    return rl.rnn_conv_desc(**(dict(dtype=0, direction=0, layout=1, silu=1, seq=5, batch=3, channels=6, width=4) | kw))


def scan_desc(**kw):
    return rl.rnn_scan_desc(**(dict(dtype=0, direction=0, layout=1, delta_softplus=1, seq=5, batch=3, channels=6, state=4, groups=2) | kw))


def norm_desc(**kw):
    return rl.rnn_norm_desc(**(dict(dtype=0, epsilon=1e-5, rows=5, size=6) | kw))


OPS = {"conv": (rl.rnn_conv_create, rl.rnn_conv_destroy, conv_desc, "conv: "),
       "scan": (rl.rnn_scan_create, rl.rnn_scan_destroy, scan_desc, "scan: "),
       "norm": (rl.rnn_norm_create, rl.rnn_norm_destroy, norm_desc, "layer norm: ")}


def refused(call, code, start, needle):
    with pytest.raises(rl.RnnError) as err:
        call()
    assert err.value.code == code, err.value
    assert err.value.message.startswith(start) and needle in err.value.message, err.value
    return True


@pytest.mark.parametrize("op,field,value,code", [
    ("conv", "dtype", 3, ARG), ("conv", "dtype", -1, ARG), ("conv", "direction", 2, ARG), ("conv", "direction", 5, ARG),
    ("conv", "layout", 2, ARG), ("conv", "silu", 2, ARG), ("conv", "seq", -1, SHAPE), ("conv", "batch", -1, SHAPE),
    ("conv", "channels", 0, SHAPE), ("conv", "width", 0, SHAPE), ("conv", "width", 1, UNSUPPORTED), ("conv", "width", 9, UNSUPPORTED),
    ("conv", "channels", (1 << 24) + 1, UNSUPPORTED), ("conv", "batch", (1 << 30) + 1, UNSUPPORTED), ("conv", "seq", (1 << 30) + 1, UNSUPPORTED),
    ("scan", "dtype", 3, ARG), ("scan", "direction", 2, ARG), ("scan", "layout", -1, ARG), ("scan", "delta_softplus", 2, ARG),
    ("scan", "seq", -1, SHAPE), ("scan", "batch", -1, SHAPE), ("scan", "channels", 0, SHAPE), ("scan", "state", 0, SHAPE),
    ("scan", "state", 129, UNSUPPORTED), ("scan", "groups", 0, SHAPE), ("scan", "groups", 4, SHAPE), ("scan", "groups", 12, SHAPE),
    ("norm", "dtype", 3, ARG), ("norm", "epsilon", -1.0, ARG), ("norm", "epsilon", float("nan"), ARG), ("norm", "epsilon", float("inf"), ARG),
    ("norm", "rows", -1, SHAPE), ("norm", "size", 0, SHAPE), ("norm", "rows", 1 << 31, UNSUPPORTED), ("norm", "size", 1 << 25, UNSUPPORTED),
])
def test_create_refuses(op, field, value, code):
    create, _, desc, start = OPS[op]
    refused(lambda: create(desc(**{field: value})), code, start, field)


@pytest.mark.parametrize("op,fields,code", [
    ("conv", dict(seq=1 << 29, batch=1 << 29), SHAPE), ("scan", dict(seq=1 << 29, batch=1 << 29), SHAPE),
    ("scan", dict(seq=1 << 28, batch=1 << 10, channels=64), UNSUPPORTED), ("conv", dict(seq=1 << 28, batch=1 << 10, channels=64), UNSUPPORTED),
    ("norm", dict(rows=1 << 30, size=1 << 24), SHAPE), ("norm", dict(rows=1 << 29, size=64), UNSUPPORTED),
])
def test_sizes_are_checked_in_64_bits(op, fields, code):
    create, _, desc, start = OPS[op]
    refused(lambda: create(desc(**fields)), code, start, "")


@pytest.mark.parametrize("op", OPS)
def test_null_arguments(op):
    lib = rl.load_library()
    create, destroy, desc, start = OPS[op]
    assert getattr(lib, f"rnn_{op}_create")(None, ctypes.byref(ctypes.c_void_p())) == ARG
    assert rl.rnn_last_error() == start + "desc: NULL"
    assert getattr(lib, f"rnn_{op}_create")(ctypes.byref(desc()), None) == ARG
    destroy(None)
    for f in ("scratch_size", "encode", "encode_backward"):
        args = {"scratch_size": (None, None), "encode": (None, None, None), "encode_backward": (None, None, None, None)}[f]
        assert getattr(lib, f"rnn_{op}_{f}")(None, *args) == ARG
        assert rl.rnn_last_error() == f"{start}{op}: NULL"
    h = create(desc())
    try:
        assert getattr(lib, f"rnn_{op}_encode")(h, None, None, None) == ARG and "operands: NULL" in rl.rnn_last_error()
        assert getattr(lib, f"rnn_{op}_encode_backward")(h, None, None, None, None) == ARG and "operands: NULL" in rl.rnn_last_error()
        ops = getattr(rl, f"rnn_{op}_operands")()
        assert getattr(lib, f"rnn_{op}_encode_backward")(h, ctypes.byref(ops), None, None, None) == ARG
        assert "gradients: NULL" in rl.rnn_last_error()
        assert getattr(lib, f"rnn_{op}_scratch_size")(h, None, None) == rl.RNN_OK and rl.rnn_last_error() == ""
    finally:
        destroy(h)


def filled(op, struct, skip=()):
    """Every tensor at an address of its own."""
    t = getattr(rl, f"rnn_{op}_{struct}")()
    for i, (name, _) in enumerate(t._fields_):
        if name not in skip:
            getattr(t, name).ptr = FAKE + 4096 * (i + (64 if struct == "gradients" else 0))
    return t


REQUIRED = {"conv": (("X", "W"), ("dY",)), "scan": (("X", "delta", "A", "B", "C"), ("dY",)), "norm": (("X", "Scale"), ("dY",))}


@pytest.mark.parametrize("op", OPS)
def test_operands_refused(op):
    create, destroy, desc, start = OPS[op]
    encode, backward = getattr(rl, f"rnn_{op}_encode"), getattr(rl, f"rnn_{op}_encode_backward")
    h = create(desc())
    try:
        for name in REQUIRED[op][0]:
            refused(lambda: encode(h, filled(op, "operands", (name,))), ARG, start, f"{name}: NULL")
        for name in REQUIRED[op][1]:
            refused(lambda: backward(h, filled(op, "operands"), filled(op, "gradients", (name,))), ARG, start, f"{name}: NULL")
        for name, kind in getattr(rl, f"rnn_{op}_operands")._fields_:
            t = filled(op, "operands")
            getattr(t, name).elem_offset = -1
            refused(lambda: encode(h, t), ARG, start, f"{name}: negative element offset")
            t = filled(op, "operands")
            getattr(t, name).elem_offset = 1 << 60
            refused(lambda: encode(h, t), SHAPE, start, f"{name}: element offset overflows")
            t = filled(op, "operands")
            getattr(t, name).ptr += 2
            refused(lambda: encode(h, t), ARG, start, f"{name}: address not aligned")
            if kind is rl.rnn_rows:
                t = filled(op, "operands")
                getattr(t, name).row_stride = 3
                refused(lambda: encode(h, t), SHAPE, start, f"{name}: row_stride 3 below")
                t = filled(op, "operands")
                getattr(t, name).row_stride = 1 << 60
                refused(lambda: encode(h, t), SHAPE, start, f"{name}: size overflows")
        # an output on an input's memory
        for out, other in {"conv": (("Y", "X"),), "scan": (("Y", "X"), ("Y", "Z")), "norm": (("Y", "X"), ("Mean", "Scale"))}[op]:
            t = filled(op, "operands")
            getattr(t, out).ptr = getattr(t, other).ptr
            refused(lambda: encode(h, t), ARG, start, f"{out}: the same memory as {other}")
        for out, other in {"conv": (("dX", "dY"), ("d_initial_state", "d_final_state")), "norm": (("dX", "dY"),),
                           "scan": (("dX", "dY"), ("d_initial_state", "d_final_state"), ("dC", "dB"))}[op]:
            g = filled(op, "gradients")
            getattr(g, out).ptr = getattr(g, other).ptr
            refused(lambda: backward(h, filled(op, "operands"), g), ARG, start, f"{out}: the same memory as {other}")
        # scratch
        refused(lambda: backward(h, filled(op, "operands"), filled(op, "gradients")), ARG, start, "scratch: NULL")
        refused(lambda: backward(h, filled(op, "operands"), filled(op, "gradients"), FAKE + 64), ARG, start, "scratch: not 256-byte aligned")
        if op == "scan":
            refused(lambda: encode(h, filled(op, "operands")), ARG, start, "scratch: NULL")
    finally:
        destroy(h)


def test_scan_dz_needs_z():
    h = rl.rnn_scan_create(scan_desc())
    try:
        refused(lambda: rl.rnn_scan_encode_backward(h, filled("scan", "operands", ("Z",)), filled("scan", "gradients"), FAKE), ARG, "scan: ", "dZ: there is no Z")
    finally:
        rl.rnn_scan_destroy(h)


def test_norm_backward_needs_statistics():
    h = rl.rnn_norm_create(norm_desc())
    try:
        for name in ("Mean", "InvStdDev"):
            refused(lambda: rl.rnn_norm_encode_backward(h, filled("norm", "operands", (name,)), filled("norm", "gradients"), FAKE), ARG, "layer norm: ", f"{name}: NULL")
    finally:
        rl.rnn_norm_destroy(h)


def test_nothing_asked_for_is_nothing_done():
    """No output, or no batch row: success, with no launch and no scratch."""
    for op, outs in (("conv", ("Y", "final_state")), ("scan", ("Y", "final_state")), ("norm", ("Y", "Mean", "InvStdDev"))):
        create, destroy, desc, _ = OPS[op]
        h = create(desc())
        getattr(rl, f"rnn_{op}_encode")(h, filled(op, "operands", outs))
        g = getattr(rl, f"rnn_{op}_gradients")()
        g.dY.ptr = FAKE + (1 << 16)
        getattr(rl, f"rnn_{op}_encode_backward")(h, filled(op, "operands"), g)
        destroy(h)
        h = create(desc(**({"rows": 0} if op == "norm" else {"batch": 0})))
        getattr(rl, f"rnn_{op}_encode")(h, filled(op, "operands"))
        destroy(h)


def test_scratch_sizes(monkeypatch):
    def up(n):
        return (n + 255) // 256 * 256

    monkeypatch.delenv("RNN_SCAN_CHUNK", raising=False)
    h = rl.rnn_conv_create(conv_desc(seq=100, batch=2, channels=10, width=3))
    # 16 steps a thread, four threads a workgroup along time: 2 parts a row, (3 + 1) x 10 sums each
    assert rl.rnn_conv_scratch_size(h) == (0, up(2 * 2 * 4 * 10 * 4))
    rl.rnn_conv_destroy(h)
    h = rl.rnn_norm_create(norm_desc(rows=100, size=10))
    assert rl.rnn_norm_scratch_size(h) == (0, up(25 * 2 * 10 * 4))
    rl.rnn_norm_destroy(h)
    monkeypatch.setenv("RNN_SCAN_CHUNK", "32")
    h = rl.rnn_scan_create(scan_desc(seq=100, batch=2, channels=10, state=5, groups=2))
    # a row for what is not stored; 4 chunks, states padded to 8, segments of 16 steps, 2 channel blocks
    loc, total = up(2 * 4 * 8 * 10 * 4), up(2 * 4 * 10 * 4)
    assert rl.rnn_scan_scratch_size(h) == (
        up(10 * 4) + loc + total + up(2 * 8 * 10 * 4),
        up(10 * 4) + 2 * loc + total + up(2 * 7 * 8 * 10 * 4) + up(2 * 7 * 10 * 4) + up(2 * 2 * 100 * 2 * 8 * 4) + loc + up(2 * 4 * 2 * 10 * 4))
    rl.rnn_scan_destroy(h)
    monkeypatch.setenv("RNN_SCAN_CHUNK", "1000")
    h = rl.rnn_scan_create(scan_desc(seq=100, batch=2, channels=10, state=5, groups=2))
    assert rl.rnn_scan_scratch_size(h)[0] == up(10 * 4)
    rl.rnn_scan_destroy(h)
    h = rl.rnn_scan_create(scan_desc(seq=1))      # tokens
    assert rl.rnn_scan_scratch_size(h)[0] == 0
    rl.rnn_scan_destroy(h)


def test_recurrent_layers_refuse_bf16():
    from onnx_recurrent_layers_amd.synth import LayerSpec
    d = rl.make_desc(LayerSpec("LSTM", seq=5, batch=3, input=4, hidden=6))
    d.dtype = rl.DTYPES["bf16"]
    refused(lambda: rl.rnn_problem_create(d), ARG, "LSTM: ", "dtype")


@pytest.fixture
def scan():
    op = rl.SelectiveScan(dtype="f32", seq=4, batch=3, channels=6, state=4, device="cuda:0")
    op._index = -1     # (few steps take no scratch) CPU tensors stand for the device's: nothing is launched
    return op


def test_binding_refuses_tensors(scan):
    good = {"X": torch.zeros(3, 4, 6)}

    def fill(**kw):
        return lambda: scan._fill(scan._forward, good | kw)

    fill()()
    refused(fill(X=torch.zeros(4, 3, 6)), SHAPE, "scan: ", "X: shape")
    refused(fill(X=torch.zeros(3, 4, 6, dtype=torch.float16)), ARG, "scan: ", "X: type")
    refused(fill(X=torch.zeros(3, 4, 12)[..., ::2]), ARG, "scan: ", "X: the elements of a row")
    refused(fill(X=torch.zeros(4, 3, 6).transpose(0, 1)), ARG, "scan: ", "constant stride")
    refused(fill(X=torch.zeros(1, 1, 6).expand(3, 4, 6)), ARG, "scan: ", "X: its rows overlap")
    refused(fill(A=torch.zeros(4, 6).t()), ARG, "scan: ", "A: has to be contiguous")
    refused(lambda: scan.encode({"W": torch.zeros(1)}), ARG, "scan: ", "W: unknown tensor")
    x = torch.zeros(3, 4, 20)[..., 3:9]
    ops = rl.rnn_scan_operands.from_buffer(fill(X=x)())
    assert (ops.X.ptr, ops.X.elem_offset, ops.X.row_stride) == (x.data_ptr(), 0, 20) and ops.delta.ptr is None
    scan._index = 0
    refused(fill(), ARG, "scan: ", "X: on cpu")


def test_binding_refuses_another_devices_stream(scan):
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0

    refused(lambda: scan.encode({"X": torch.zeros(3, 4, 6)}, Stream()), ARG, "scan: ", "stream: on cuda:1, expected cuda:0")
