"""ONNX recurrent layers (RNN, GRU, LSTM) on MI355X (gfx950), and the operators
of a selective state space block with layer normalization.

A thin ctypes binding over the C ABI of ``include/rnn.h`` (library
``librnn_mi355x.so``, built in-tree by ``onnx_recurrent_layers_amd.build``).
The functions carry the C names and only marshal arguments: every stage of a
layer runs in the library's HIP kernels.  PyTorch supplies device memory and
the stream.  There is no fallback: when the library is missing, loading fails.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "librnn_mi355x.so")

RNN_OK, RNN_ERR_ARG, RNN_ERR_SHAPE, RNN_ERR_UNSUPPORTED, RNN_ERR_HIP = range(5)
CELLS = {"RNN": 0, "GRU": 1, "LSTM": 2}
DTYPES = {"f32": 0, "f16": 1, "bf16": 2}   # (bf16: the operators beside the recurrent layers)
DIRECTIONS = {"forward": 0, "reverse": 1, "bidirectional": 2}
ACTIVATIONS = {
    "Relu": 0, "Tanh": 1, "Sigmoid": 2, "Affine": 3, "LeakyRelu": 4, "ThresholdedRelu": 5,
    "ScaledTanh": 6, "HardSigmoid": 7, "Elu": 8, "Softsign": 9, "Softplus": 10,
}
ENGINES = {"auto": 0, "launch": 1, "persistent": 2}


class RnnError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"[{code}] {message}")
        self.code = code
        self.message = message


class rnn_activation(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("alpha", ctypes.c_float), ("beta", ctypes.c_float)]


class rnn_problem_desc(ctypes.Structure):
    _fields_ = [
        ("cell", ctypes.c_int32), ("dtype", ctypes.c_int32), ("direction", ctypes.c_int32),
        ("layout", ctypes.c_int32), ("seq", ctypes.c_int64), ("batch", ctypes.c_int64),
        ("input", ctypes.c_int64), ("hidden", ctypes.c_int64), ("clip", ctypes.c_float),
        ("input_forget", ctypes.c_int32), ("linear_before_reset", ctypes.c_int32),
        ("num_activations", ctypes.c_int32), ("activations", rnn_activation * 6),
        ("max_length", ctypes.c_int64), ("engine", ctypes.c_int32), ("x_bidirectional_y", ctypes.c_int32),
        ("xw_chunk_steps", ctypes.c_int64),
    ]


class rnn_tensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("elem_offset", ctypes.c_int64)]


OPERAND_NAMES = ("X", "W", "R", "B", "sequence_lens", "initial_h", "initial_c", "P", "Y", "Y_h", "Y_c")


class rnn_operands(ctypes.Structure):
    _fields_ = [(n, rnn_tensor) for n in OPERAND_NAMES]


class rnn_run_status(ctypes.Structure):
    _fields_ = [("persistent", ctypes.c_int32), ("fallback_workgroups", ctypes.c_int32),
                ("timed_out", ctypes.c_int32)]


class rnn_plan_info(ctypes.Structure):
    _fields_ = [("engine", ctypes.c_int32), ("steps", ctypes.c_int32), ("launches", ctypes.c_int32),
                ("step_blocks", ctypes.c_int32), ("step_launches", ctypes.c_int32),
                ("proj_products", ctypes.c_int32), ("step_products", ctypes.c_int32),
                ("xw_chunk_steps", ctypes.c_int32), ("xw_slots", ctypes.c_int32)]


class rnn_rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("elem_offset", ctypes.c_int64), ("row_stride", ctypes.c_int64)]


class rnn_conv_desc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("direction", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("silu", ctypes.c_int32), ("seq", ctypes.c_int64), ("batch", ctypes.c_int64),
                ("channels", ctypes.c_int64), ("width", ctypes.c_int64)]


class rnn_conv_operands(ctypes.Structure):
    _fields_ = [("X", rnn_rows), ("W", rnn_tensor), ("B", rnn_tensor), ("sequence_lens", rnn_tensor),
                ("initial_state", rnn_tensor), ("Y", rnn_rows), ("final_state", rnn_tensor)]


class rnn_conv_gradients(ctypes.Structure):
    _fields_ = [("dY", rnn_rows), ("d_final_state", rnn_tensor), ("dX", rnn_rows), ("dW", rnn_tensor),
                ("dB", rnn_tensor), ("d_initial_state", rnn_tensor)]


class rnn_scan_desc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("direction", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("delta_softplus", ctypes.c_int32), ("seq", ctypes.c_int64), ("batch", ctypes.c_int64),
                ("channels", ctypes.c_int64), ("state", ctypes.c_int64), ("groups", ctypes.c_int64)]


class rnn_scan_operands(ctypes.Structure):
    _fields_ = [("X", rnn_rows), ("delta", rnn_rows), ("A", rnn_tensor), ("B", rnn_rows), ("C", rnn_rows),
                ("D", rnn_tensor), ("Z", rnn_rows), ("delta_bias", rnn_tensor), ("sequence_lens", rnn_tensor),
                ("initial_state", rnn_tensor), ("Y", rnn_rows), ("final_state", rnn_tensor)]


class rnn_scan_gradients(ctypes.Structure):
    _fields_ = [("dY", rnn_rows), ("d_final_state", rnn_tensor), ("dX", rnn_rows), ("ddelta", rnn_rows),
                ("dA", rnn_tensor), ("dB", rnn_rows), ("dC", rnn_rows), ("dD", rnn_tensor), ("dZ", rnn_rows),
                ("ddelta_bias", rnn_tensor), ("d_initial_state", rnn_tensor)]


class rnn_norm_desc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("epsilon", ctypes.c_float), ("rows", ctypes.c_int64),
                ("size", ctypes.c_int64)]


class rnn_norm_operands(ctypes.Structure):
    _fields_ = [("X", rnn_rows), ("Scale", rnn_tensor), ("B", rnn_tensor), ("Y", rnn_rows), ("Mean", rnn_tensor),
                ("InvStdDev", rnn_tensor)]


class rnn_norm_gradients(ctypes.Structure):
    _fields_ = [("dY", rnn_rows), ("dX", rnn_rows), ("dScale", rnn_tensor), ("dB", rnn_tensor)]


# rnn_products: which arithmetic units carry a stage's products
PRODUCTS = {0: "f32 vector ALU", 1: "f32 matrix cores", 2: "f16 matrix cores", 3: "bf16x3 matrix cores"}


_lib = None


def load_library(path: str = LIB_PATH):
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m onnx_recurrent_layers_amd.build`")
    # One HIP runtime per process: when PyTorch supplies device memory and
    # streams, load it first so that this library binds to the same runtime.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    lib.rnn_problem_create.argtypes = [P(rnn_problem_desc), P(ctypes.c_void_p)]
    lib.rnn_problem_create.restype = ctypes.c_int
    lib.rnn_problem_destroy.argtypes = [ctypes.c_void_p]
    lib.rnn_problem_destroy.restype = None
    lib.rnn_scratch_size.argtypes = [ctypes.c_void_p, P(ctypes.c_size_t), P(ctypes.c_size_t)]
    lib.rnn_scratch_size.restype = ctypes.c_int
    lib.rnn_encode.argtypes = [ctypes.c_void_p, P(rnn_operands), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    lib.rnn_encode.restype = ctypes.c_int
    lib.rnn_encode_timed.argtypes = [ctypes.c_void_p, P(rnn_operands), ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, P(ctypes.c_void_p)]
    lib.rnn_encode_timed.restype = ctypes.c_int
    lib.rnn_validate_lengths.argtypes = [P(ctypes.c_int32), ctypes.c_int64, ctypes.c_int64, P(ctypes.c_int64)]
    lib.rnn_validate_lengths.restype = ctypes.c_int
    lib.rnn_problem_plan.argtypes = [ctypes.c_void_p, P(rnn_plan_info)]
    lib.rnn_problem_plan.restype = ctypes.c_int
    lib.rnn_encode_noalloc.argtypes = [ctypes.c_void_p, P(rnn_operands), ctypes.c_void_p]
    lib.rnn_encode_noalloc.restype = ctypes.c_int
    lib.rnn_read_run_status.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, P(rnn_run_status)]
    lib.rnn_read_run_status.restype = ctypes.c_int
    for op, desc, operands, gradients in (("conv", rnn_conv_desc, rnn_conv_operands, rnn_conv_gradients),
                                          ("scan", rnn_scan_desc, rnn_scan_operands, rnn_scan_gradients),
                                          ("norm", rnn_norm_desc, rnn_norm_operands, rnn_norm_gradients)):
        def declare(name, restype, *argtypes):
            f = getattr(lib, f"rnn_{op}_{name}")
            f.argtypes, f.restype = list(argtypes), restype
        declare("create", ctypes.c_int, P(desc), P(ctypes.c_void_p))
        declare("destroy", None, ctypes.c_void_p)
        declare("scratch_size", ctypes.c_int, ctypes.c_void_p, P(ctypes.c_size_t), P(ctypes.c_size_t))
        declare("encode", ctypes.c_int, ctypes.c_void_p, P(operands), ctypes.c_void_p, ctypes.c_void_p)
        declare("encode_backward", ctypes.c_int, ctypes.c_void_p, P(operands), P(gradients), ctypes.c_void_p,
                ctypes.c_void_p)
    lib.rnn_last_error.argtypes = []
    lib.rnn_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def hip_runtime():
    """The HIP runtime library this process uses (the one the library is bound to)."""
    load_library()
    for line in open("/proc/self/maps"):
        path = line.split()[-1]
        if os.path.basename(path).startswith("libamdhip64.so"):
            return ctypes.CDLL(path)
    return ctypes.CDLL("libamdhip64.so")


def rnn_last_error() -> str:
    return load_library().rnn_last_error().decode()


def _check(rc: int):
    if rc != RNN_OK:
        raise RnnError(rc, rnn_last_error())


def make_desc(spec, engine: str = "auto") -> rnn_problem_desc:
    """rnn_problem_desc from a layer description (``synth.LayerSpec`` fields)."""
    d = rnn_problem_desc()
    d.cell = CELLS[spec.cell]
    d.dtype = DTYPES[spec.dtype]
    d.direction = DIRECTIONS[spec.direction]
    d.layout = int(spec.layout)
    d.seq, d.batch, d.input, d.hidden = int(spec.seq), int(spec.batch), int(spec.input), int(spec.hidden)
    d.clip = float(spec.clip) if spec.clip is not None else 0.0
    d.input_forget = int(spec.input_forget)
    d.linear_before_reset = int(spec.linear_before_reset)
    acts = list(spec.activations)
    d.num_activations = len(acts)
    for i, (name, a, b) in enumerate(acts):
        d.activations[i].kind = ACTIVATIONS[name]
        d.activations[i].alpha = float(a)
        d.activations[i].beta = float(b)
    d.max_length = int(spec.max_length or 0)
    d.engine = ENGINES[engine]
    d.x_bidirectional_y = int(getattr(spec, "x_bidirectional_y", 0))
    d.xw_chunk_steps = int(getattr(spec, "xw_chunk_steps", 0))
    return d


def rnn_problem_create(desc: rnn_problem_desc) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(load_library().rnn_problem_create(ctypes.byref(desc), ctypes.byref(h)))
    return h


def rnn_problem_destroy(handle) -> None:
    load_library().rnn_problem_destroy(handle)


def rnn_scratch_size(handle):
    xw, st = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().rnn_scratch_size(handle, ctypes.byref(xw), ctypes.byref(st)))
    return xw.value, st.value


def rnn_problem_plan(handle) -> rnn_plan_info:
    info = rnn_plan_info()
    _check(load_library().rnn_problem_plan(handle, ctypes.byref(info)))
    return info


def rnn_read_run_status(handle, state_scratch_ptr: int, stream_ptr: int = 0) -> rnn_run_status:
    out = rnn_run_status()
    _check(load_library().rnn_read_run_status(handle, ctypes.c_void_p(state_scratch_ptr or None),
                                              ctypes.c_void_p(stream_ptr or None), ctypes.byref(out)))
    return out


def rnn_validate_lengths(lens, seq: int) -> int:
    import numpy as np
    arr = np.ascontiguousarray(np.asarray(lens, dtype=np.int32))
    mx = ctypes.c_int64()
    _check(load_library().rnn_validate_lengths(arr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                               arr.size, int(seq), ctypes.byref(mx)))
    return mx.value


def make_operands(tensors: dict, offsets: Optional[dict] = None) -> rnn_operands:
    """rnn_operands from device tensors (torch) keyed by ONNX names; ``offsets``
    gives element offsets into each tensor's storage (default 0)."""
    ops = rnn_operands()
    offsets = offsets or {}
    for name in OPERAND_NAMES:
        t = tensors.get(name)
        if t is None:
            continue
        tr = getattr(ops, name)
        tr.ptr = t.data_ptr()
        tr.elem_offset = int(offsets.get(name, 0))
    return ops


def rnn_encode(handle, operands: rnn_operands, xw_scratch_ptr: int, state_scratch_ptr: int,
               stream_ptr: int = 0) -> None:
    _check(load_library().rnn_encode(handle, ctypes.byref(operands), ctypes.c_void_p(xw_scratch_ptr or None),
                                     ctypes.c_void_p(state_scratch_ptr or None), ctypes.c_void_p(stream_ptr or None)))


def rnn_encode_noalloc(handle, operands: rnn_operands, stream_ptr: int = 0) -> None:
    """rnn_encode with the library's fixed scratch (no caller scratch)."""
    _check(load_library().rnn_encode_noalloc(handle, ctypes.byref(operands), ctypes.c_void_p(stream_ptr or None)))


NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024


def rnn_encode_timed(handle, operands: rnn_operands, xw_scratch_ptr: int, state_scratch_ptr: int,
                     stream_ptr: int, events) -> None:
    """rnn_encode plus hipEventRecord of five stage-boundary events (hipEvent_t
    handles as ints, or None) on the same stream."""
    ev = (ctypes.c_void_p * 5)(*[ctypes.c_void_p(e) if e else None for e in events])
    _check(load_library().rnn_encode_timed(handle, ctypes.byref(operands), ctypes.c_void_p(xw_scratch_ptr or None),
                                           ctypes.c_void_p(state_scratch_ptr or None),
                                           ctypes.c_void_p(stream_ptr or None), ev))


class Layer:
    """One created problem plus its scratch, for repeated encodes."""

    def __init__(self, spec, engine: str = "auto", device: str = "cuda"):
        import torch
        self.spec = spec
        self.handle = rnn_problem_create(make_desc(spec, engine))
        self.xw_bytes, self.state_bytes = rnn_scratch_size(self.handle)
        self.plan = rnn_problem_plan(self.handle)
        self.device = torch.device(device)
        self.xw = torch.empty(max(self.xw_bytes, 256), dtype=torch.uint8, device=self.device)
        self.state = torch.empty(max(self.state_bytes, 256), dtype=torch.uint8, device=self.device)
        # what the allocator hands out may still be in use by work queued on the
        # stream that it counts it to: another stream's call waits for that
        if self.device.type == "cuda":
            home = torch.cuda.current_stream(self.device)
            self._home = home.cuda_stream
            with torch.cuda.stream(home):
                self._ready = None if torch.cuda.is_current_stream_capturing() else home.record_event()

    def _take(self, stream):
        """The scratch, for a call on `stream`."""
        import torch
        if stream.cuda_stream == self._home:
            return
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return
        if self._ready is not None:
            stream.wait_event(self._ready)
        for memory in (self.xw, self.state):
            memory.record_stream(stream)     # (not reused, once this object is gone, before the call has run)

    def encode(self, tensors: dict, offsets: Optional[dict] = None, stream=None, events=None) -> None:
        import torch
        ops = make_operands(tensors, offsets)
        st = stream if stream is not None else torch.cuda.current_stream(self.device)
        self._take(st)
        xw = self.xw.data_ptr() if self.xw_bytes else 0
        if events is None:
            rnn_encode(self.handle, ops, xw, self.state.data_ptr(), st.cuda_stream)
        else:
            rnn_encode_timed(self.handle, ops, xw, self.state.data_ptr(), st.cuda_stream, events)

    def run_status(self, stream=None) -> rnn_run_status:
        """rnn_read_run_status of this layer's state scratch (waits for the stream)."""
        import torch
        st = stream if stream is not None else torch.cuda.current_stream(self.device)
        return rnn_read_run_status(self.handle, self.state.data_ptr() if self.state_bytes else 0, st.cuda_stream)

    def __del__(self):
        try:
            if getattr(self, "handle", None):
                rnn_problem_destroy(self.handle)
                self.handle = None
        except Exception:
            pass


# ---- the operators of a state space block, and layer normalization

def _create(name: str, desc) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(getattr(load_library(), name)(ctypes.byref(desc), ctypes.byref(h)))
    return h


def _scratch(name: str, handle):
    forward, backward = ctypes.c_size_t(), ctypes.c_size_t()
    _check(getattr(load_library(), name)(handle, ctypes.byref(forward), ctypes.byref(backward)))
    return forward.value, backward.value


def rnn_conv_create(desc: rnn_conv_desc) -> ctypes.c_void_p:
    return _create("rnn_conv_create", desc)


def rnn_conv_destroy(handle) -> None:
    load_library().rnn_conv_destroy(handle)


def rnn_conv_scratch_size(handle):
    return _scratch("rnn_conv_scratch_size", handle)


def rnn_conv_encode(handle, operands: rnn_conv_operands, scratch_ptr: int = 0, stream_ptr: int = 0) -> None:
    _check(load_library().rnn_conv_encode(handle, operands, scratch_ptr or None, stream_ptr or None))


def rnn_conv_encode_backward(handle, operands: rnn_conv_operands, gradients: rnn_conv_gradients, scratch_ptr: int = 0,
                             stream_ptr: int = 0) -> None:
    _check(load_library().rnn_conv_encode_backward(handle, operands, gradients, scratch_ptr or None,
                                                   stream_ptr or None))


def rnn_scan_create(desc: rnn_scan_desc) -> ctypes.c_void_p:
    return _create("rnn_scan_create", desc)


def rnn_scan_destroy(handle) -> None:
    load_library().rnn_scan_destroy(handle)


def rnn_scan_scratch_size(handle):
    return _scratch("rnn_scan_scratch_size", handle)


def rnn_scan_encode(handle, operands: rnn_scan_operands, scratch_ptr: int = 0, stream_ptr: int = 0) -> None:
    _check(load_library().rnn_scan_encode(handle, operands, scratch_ptr or None, stream_ptr or None))


def rnn_scan_encode_backward(handle, operands: rnn_scan_operands, gradients: rnn_scan_gradients, scratch_ptr: int = 0,
                             stream_ptr: int = 0) -> None:
    _check(load_library().rnn_scan_encode_backward(handle, operands, gradients, scratch_ptr or None,
                                                   stream_ptr or None))


def rnn_norm_create(desc: rnn_norm_desc) -> ctypes.c_void_p:
    return _create("rnn_norm_create", desc)


def rnn_norm_destroy(handle) -> None:
    load_library().rnn_norm_destroy(handle)


def rnn_norm_scratch_size(handle):
    return _scratch("rnn_norm_scratch_size", handle)


def rnn_norm_encode(handle, operands: rnn_norm_operands, scratch_ptr: int = 0, stream_ptr: int = 0) -> None:
    _check(load_library().rnn_norm_encode(handle, operands, scratch_ptr or None, stream_ptr or None))


def rnn_norm_encode_backward(handle, operands: rnn_norm_operands, gradients: rnn_norm_gradients, scratch_ptr: int = 0,
                             stream_ptr: int = 0) -> None:
    _check(load_library().rnn_norm_encode_backward(handle, operands, gradients, scratch_ptr or None,
                                                   stream_ptr or None))


class _Operator:
    """One created problem of the operators below plus its scratch (made by the
    first call, forward and backward, on that call's stream), for repeated
    calls.  The tensors of a call are torch tensors keyed by the C names; each
    one's shape, type and device are checked.  Sequence tensors may be views
    whose rows lie a constant stride apart (a slice of a wider projection); the
    others have to be contiguous.  Calls that overlap in time need an object
    each, since an object holds one scratch (so do graphs that replay at once),
    and an object is kept for as long as a graph replays its calls."""

    op = ""             # the C functions' middle name
    who = ""            # the name in messages
    operand_names = ()
    gradient_names = ()

    def _open(self, desc, device, shapes):
        import torch
        self._handle = None
        lib = load_library()
        self._destroy = getattr(lib, f"rnn_{self.op}_destroy")
        # (function objects of their own: a call's structs are filled as arrays of words)
        self._encode, self._encode_backward = lib[f"rnn_{self.op}_encode"], lib[f"rnn_{self.op}_encode_backward"]
        self._encode.argtypes = [ctypes.c_void_p] * 4
        self._encode_backward.argtypes = [ctypes.c_void_p] * 5
        self._handle = _create(f"rnn_{self.op}_create", desc)
        self.forward_bytes, self.backward_bytes = _scratch(f"rnn_{self.op}_scratch_size", self._handle)
        self.device = torch.device(device)
        if self.device.index is None:
            self.device = torch.device(self.device.type, torch.cuda.current_device())
        self._index = self.device.index
        # name -> (shape, torch type, row tensor)
        specs = shapes(torch, {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[self.dtype])
        self._specs = specs

        def layout(struct, names):   # struct's words, and of each of `names` (first word, shape, type, row tensor)
            return ctypes.c_uint64 * (ctypes.sizeof(struct) // 8), [(n, getattr(struct, n).offset // 8, *specs[n]) for n in names]

        self._forward = layout(self._operands, self.operand_names)
        self._inputs = layout(self._operands, self.input_names)
        self._grads = layout(self._gradients, self.gradient_names)
        self._forward_scratch = self._backward_scratch = None

    def _new_scratch(self, size, stream, raw):
        """Scratch and the stream that the allocator counts it to: the stream of
        the first call that takes it.  What the allocator hands out may still be
        in use by work queued on the stream that it counts the memory to (its
        last holder's), so on that stream only it may be written at once; calls
        after the first do not overlap with it."""
        import torch
        with torch.cuda.stream(stream):
            return torch.empty(size, dtype=torch.uint8, device=self.device), raw

    def _raw(self, stream):
        """The handle of a call's stream."""
        import torch
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self._index)   # (the handle alone: a Stream object takes 1.8 us)
        if stream.device.index != self._index:
            raise self._bad(RNN_ERR_ARG, f"stream: on {stream.device}, expected {self.device}")
        return stream.cuda_stream

    def _bad(self, code, text):
        return RnnError(code, f"{self.who}: {text}")

    def _fill(self, layout, tensors):
        """One C struct of a call: a tensor is its pointer, element offset 0 and, in rows, the stride."""
        words, fields = layout
        w, index = words(), self._index
        for name, at, shape, dtype, row in fields:
            t = tensors.get(name)
            if t is None:
                continue
            if t.shape != shape:
                raise self._bad(RNN_ERR_SHAPE, f"{name}: shape {tuple(t.shape)}, expected {shape}")
            if t.dtype is not dtype:
                raise self._bad(RNN_ERR_ARG, f"{name}: type {t.dtype}, expected {dtype}")
            if t.get_device() != index:
                raise self._bad(RNN_ERR_ARG, f"{name}: on {t.device}, expected {self.device}")
            if not t.is_contiguous() and t.numel():
                if not row:
                    raise self._bad(RNN_ERR_ARG, f"{name}: has to be contiguous")
                w[at + 2] = self._row_stride(name, t)
            w[at] = t.data_ptr()
        return w

    def _row_stride(self, name, t):
        """Elements from one row to the next, where all leading dimensions go by one stride."""
        size, stride = t.shape, t.stride()
        if size[-1] > 1 and stride[-1] != 1:
            raise self._bad(RNN_ERR_ARG, f"{name}: the elements of a row have to be contiguous")
        step = None
        for n, d in zip(reversed(size[:-1]), reversed(stride[:-1])):
            if n == 1:
                continue
            if step is None:
                step, rows = d, n
            elif d != step * rows:
                raise self._bad(RNN_ERR_ARG, f"{name}: its rows have to lie a constant stride apart, got {stride}")
            else:
                rows *= n
        if step is not None and step < size[-1]:
            raise self._bad(RNN_ERR_ARG, f"{name}: its rows overlap, stride {step}")
        return 0 if step is None else step

    def _capturing(self, stream):
        import torch
        with torch.cuda.stream(stream):
            return torch.cuda.is_current_stream_capturing()

    def _call(self, encode, structs, scratch, stream, raw):
        import torch
        ptr = None
        if scratch is not None:
            memory, home = scratch
            ptr = memory.data_ptr()
            if raw != home and not self._capturing(stream):
                # (not reused, once this object is gone, before the call has run)
                memory.record_stream(stream if stream is not None else torch.cuda.current_stream(self.device))
        if torch.cuda.current_device() == self._index:
            _check(encode(self._handle, *structs, ptr, raw or None))
        else:
            with torch.cuda.device(self.device):
                _check(encode(self._handle, *structs, ptr, raw or None))

    def _known(self, tensors):
        if not tensors.keys() <= self._specs.keys():
            raise self._bad(RNN_ERR_ARG, f"{min(tensors.keys() - self._specs.keys())}: unknown tensor")

    def encode(self, tensors: dict, stream=None) -> None:
        """Enqueue the operator on `stream` (default: the current one)."""
        self._known(tensors)
        ops, raw = self._fill(self._forward, tensors), self._raw(stream)
        if self._forward_scratch is None and self.forward_bytes:
            self._forward_scratch = self._new_scratch(self.forward_bytes, stream, raw)
        self._call(self._encode, (ops,), self._forward_scratch, stream, raw)

    def backward(self, tensors: dict, stream=None) -> None:
        """Enqueue the gradient.  `tensors` holds the forward pass's inputs too.
        The first call allocates its scratch, so it cannot be the captured one."""
        self._known(tensors)
        ops, grads, raw = self._fill(self._inputs, tensors), self._fill(self._grads, tensors), self._raw(stream)
        if self._backward_scratch is None and self.backward_bytes:
            if self._capturing(stream):
                raise self._bad(RNN_ERR_ARG, "scratch: call backward once before a graph captures it")
            self._backward_scratch = self._new_scratch(self.backward_bytes, stream, raw)
        self._call(self._encode_backward, (ops, grads), self._backward_scratch, stream, raw)

    def __del__(self):
        try:
            if getattr(self, "_handle", None):
                self._destroy(self._handle)
                self._handle = None
        except Exception:
            pass


class CausalConv(_Operator):
    """Short causal convolution (``rnn_conv_*``): one filter of ``width`` taps a
    channel over time, with SiLU or without, for prompts and (``seq = 1``, state
    carried) single tokens, and its gradient."""

    op, who = "conv", "conv"
    _operands, _gradients = rnn_conv_operands, rnn_conv_gradients
    operand_names = tuple(n for n, _ in rnn_conv_operands._fields_)
    input_names = operand_names[:-2]
    gradient_names = tuple(n for n, _ in rnn_conv_gradients._fields_)

    def __init__(self, dtype: str, seq: int, batch: int, channels: int, width: int = 4, silu: bool = True,
                 direction: str = "forward", layout: int = 1, device: str = "cuda"):
        self.dtype = dtype
        desc = rnn_conv_desc(DTYPES[dtype], DIRECTIONS[direction], int(layout), int(silu), int(seq), int(batch),
                             int(channels), int(width))

        def shapes(torch, dt):
            row = ((seq, batch, channels) if layout == 0 else (batch, seq, channels), dt, True)
            state = ((batch, width - 1, channels), dt, False)
            f32 = torch.float32
            return {"X": row, "W": ((channels, width), dt, False), "B": ((channels,), dt, False),
                    "sequence_lens": ((batch,), torch.int32, False), "initial_state": state, "Y": row,
                    "final_state": state, "dY": row, "d_final_state": state, "dX": row,
                    "dW": ((channels, width), f32, False), "dB": ((channels,), f32, False), "d_initial_state": state}

        self._open(desc, device, shapes)


class SelectiveScan(_Operator):
    """Selective scan (``rnn_scan_*``): the state space recurrence with a step
    size and input and output weights of each step, skip and gate, for prompts
    and (``seq = 1``, state carried) single tokens, and its gradient.  A, D,
    delta_bias, the states and the gradients of parameters are f32."""

    op, who = "scan", "scan"
    _operands, _gradients = rnn_scan_operands, rnn_scan_gradients
    operand_names = tuple(n for n, _ in rnn_scan_operands._fields_)
    input_names = operand_names[:-2]
    gradient_names = tuple(n for n, _ in rnn_scan_gradients._fields_)

    def __init__(self, dtype: str, seq: int, batch: int, channels: int, state: int, groups: int = 1,
                 delta_softplus: bool = True, direction: str = "forward", layout: int = 1, device: str = "cuda"):
        self.dtype = dtype
        desc = rnn_scan_desc(DTYPES[dtype], DIRECTIONS[direction], int(layout), int(delta_softplus), int(seq),
                             int(batch), int(channels), int(state), int(groups))

        def shapes(torch, dt):
            lead = (seq, batch) if layout == 0 else (batch, seq)
            f32 = torch.float32
            row, bc = (lead + (channels,), dt, True), (lead + (groups * state,), dt, True)
            chan, h = ((channels,), f32, False), ((batch, channels, state), f32, False)
            a = ((channels, state), f32, False)
            return {"X": row, "delta": row, "A": a, "B": bc, "C": bc, "D": chan, "Z": row, "delta_bias": chan,
                    "sequence_lens": ((batch,), torch.int32, False), "initial_state": h, "Y": row, "final_state": h,
                    "dY": row, "d_final_state": h, "dX": row, "ddelta": row, "dA": a, "dB": bc, "dC": bc, "dD": chan,
                    "dZ": row, "ddelta_bias": chan, "d_initial_state": h}

        self._open(desc, device, shapes)


class LayerNorm(_Operator):
    """Layer normalization (``rnn_norm_*``, the ONNX operator over the last
    axis) with its gradient.  X is [rows, size]; Mean and InvStdDev are f32,
    and the backward pass reads them."""

    op, who = "norm", "layer norm"
    _operands, _gradients = rnn_norm_operands, rnn_norm_gradients
    operand_names = tuple(n for n, _ in rnn_norm_operands._fields_)
    input_names = ("X", "Scale", "Mean", "InvStdDev")
    gradient_names = tuple(n for n, _ in rnn_norm_gradients._fields_)

    def __init__(self, dtype: str, rows: int, size: int, epsilon: float = 1e-5, device: str = "cuda"):
        self.dtype = dtype
        desc = rnn_norm_desc(DTYPES[dtype], float(epsilon), int(rows), int(size))

        def shapes(torch, dt):
            row, stat = ((rows, size), dt, True), ((rows,), torch.float32, False)
            col, grad = ((size,), dt, False), ((size,), torch.float32, False)
            return {"X": row, "Scale": col, "B": col, "Y": row, "Mean": stat, "InvStdDev": stat, "dY": row, "dX": row,
                    "dScale": grad, "dB": grad}

        self._open(desc, device, shapes)


def output_shapes(spec) -> dict:
    S, B, H = spec.seq, spec.batch, spec.hidden
    D = 2 if spec.direction == "bidirectional" else 1
    st = (D, B, H) if spec.layout == 0 else (B, D, H)
    return {"Y": (S, D, B, H) if spec.layout == 0 else (B, S, D, H), "Y_h": st, "Y_c": st}


def to_device(inputs: dict, device: str = "cuda") -> dict:
    """numpy inputs -> torch device tensors (same dtypes)."""
    import numpy as np
    import torch
    return {k: torch.from_numpy(np.ascontiguousarray(v)).to(device) for k, v in inputs.items()}


def run(spec, inputs: dict, engine: str = "auto", outputs=None, device: str = "cuda"):
    """Run one layer on device tensors (or numpy arrays, copied to the device);
    returns the requested outputs as torch tensors on the device."""
    import numpy as np
    import torch
    tens = {k: (torch.from_numpy(np.ascontiguousarray(v)).to(device) if isinstance(v, np.ndarray) else v)
            for k, v in inputs.items()}
    dt = torch.float32 if spec.dtype == "f32" else torch.float16
    shapes = output_shapes(spec)
    want = outputs if outputs is not None else spec.outputs
    outs = {}
    for n in want:
        if n == "Y_c" and spec.cell != "LSTM":
            continue
        outs[n] = torch.empty(shapes[n], dtype=dt, device=device)
    layer = Layer(spec, engine=engine, device=device)
    layer.encode({**tens, **outs})
    return outs
