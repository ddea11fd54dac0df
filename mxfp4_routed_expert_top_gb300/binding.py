"""Thin ctypes binding of libdfmoe.so (include/df_moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. torch tensors are accepted wherever the C call takes a pointer (their
data_ptr() is passed); streams are torch.cuda.Stream objects or raw handles.
There is no fallback: if the library is missing this module raises.
"""
import ctypes
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libdfmoe.so")

OK, EINVAL, ENOMEM, ECUDA, ESTATE, ERANGE, ETIMEOUT, EDEVICE = 0, -1, -2, -3, -4, -5, -6, -7
STACK_RMSNORM_RESIDUAL = 1
PREFILL_MMA_SYNC = 4
MXFP8_ACT = 8
PLANES = 16
KERNEL_KINDS = 18
BF16, F16, F32, E4M3 = 0, 1, 2, 3
_TYPES = {"bf16": (BF16, 2), "f16": (F16, 2), "f32": (F32, 4), "e4m3": (E4M3, 1)}  # and the bytes of an element
_TYPES.update({t[0]: t for t in _TYPES.values()})
_ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "swiglu": 4}
_GATES = {"none": 0, "channel": 1, "token": 2, "full": 3}
_SCORES = {"softmax": 0, "sigmoid": 1}

# every symbol the header declares (checked by the CPU tests)
SYMBOLS = [
    "df_moe_create", "df_moe_destroy", "df_moe_last_error",
    "df_moe_expert_span_bytes", "df_moe_span_bytes_for", "df_moe_load_experts",
    "df_moe_forward", "df_moe_forward_trace", "df_moe_forward_host", "df_moe_sync",
    "df_moe_step_router", "df_moe_step_topk", "df_moe_step_group",
    "df_moe_step_expert_gateup", "df_moe_step_expert_down",
    "df_moe_step_shared", "df_moe_step_rmsnorm", "df_moe_read_expert_span",
    "df_moe_timing_enable", "df_moe_timing_reset", "df_moe_timing_get",
    "df_moe_last_launch_count", "df_moe_route_noalloc",
    "df_moe_graph_create", "df_moe_graph_launch", "df_moe_graph_launch_count",
    "df_moe_graph_destroy", "df_moe_stream_read", "df_moe_create_cached",
    "df_moe_cache_stats", "df_moe_test_drop_arrival", "df_moe_step_mxfp8",
    "df_moe_permute_workspace", "df_moe_permute", "df_moe_permute_grad", "df_moe_unpermute",
    "df_moe_unpermute_grad", "df_moe_fp8_quantize", "df_moe_fp8_matmul", "df_moe_test_fp8_give_up",
    "df_moe_matmul", "df_moe_matmul_grad", "df_moe_test_matmul_give_up", "df_moe_block_norm",
    "df_moe_block_norm_grad", "df_moe_block_norm_grad_workspace", "df_moe_balance_loss",
    "df_moe_balance_loss_grad", "df_moe_balance_loss_workspace", "df_moe_packed",
]


class DfMoeError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("df_moe error %d: %s" % (code, msg))
        self.code = code


class Config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("n_shared", ctypes.c_int32), ("shared_inter", ctypes.c_int32),
                ("n_layers", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
                ("rms_eps", ctypes.c_float), ("flags", ctypes.c_uint32)]


class LayerWeights(ctypes.Structure):
    _fields_ = [("router", ctypes.c_void_p), ("experts", ctypes.c_void_p),
                ("expert_begin", ctypes.c_int32), ("expert_count", ctypes.c_int32),
                ("shared_gate", ctypes.c_void_p), ("shared_up", ctypes.c_void_p),
                ("shared_down", ctypes.c_void_p), ("src_is_device", ctypes.c_int32)]


_lib = None


def lib():
    """Loads libdfmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libdfmoe.so is not built; run __graft_entry__.build() "
                              "or python -m mxfp4_routed_expert_top_gb300.build")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.df_moe_create.argtypes = [ctypes.POINTER(Config), ctypes.c_int,
                                    ctypes.POINTER(vp)]
        L.df_moe_destroy.argtypes = [vp]; L.df_moe_destroy.restype = None
        L.df_moe_last_error.argtypes = [vp]; L.df_moe_last_error.restype = ctypes.c_char_p
        L.df_moe_expert_span_bytes.argtypes = [vp]
        L.df_moe_expert_span_bytes.restype = ctypes.c_size_t
        L.df_moe_span_bytes_for.argtypes = [i32, i32]
        L.df_moe_span_bytes_for.restype = ctypes.c_size_t
        L.df_moe_load_experts.argtypes = [vp, i32, ctypes.POINTER(LayerWeights), vp]
        L.df_moe_forward.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, vp]
        L.df_moe_forward_trace.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, vp, vp]
        L.df_moe_forward_host.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, vp]
        L.df_moe_sync.argtypes = [vp, vp]
        L.df_moe_step_router.argtypes = [vp, i32, vp, i32, vp, vp]
        L.df_moe_step_topk.argtypes = [vp, vp, i32, vp, vp, vp]
        L.df_moe_step_group.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp]
        L.df_moe_step_expert_gateup.argtypes = [vp, i32, vp, i32, vp, vp, vp]
        L.df_moe_step_expert_down.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp]
        L.df_moe_step_shared.argtypes = [vp, i32, vp, i32, vp, vp]
        L.df_moe_step_rmsnorm.argtypes = [vp, vp, i32, vp, vp]
        L.df_moe_step_mxfp8.argtypes = [vp, vp, i32, i32, vp, vp, vp]
        L.df_moe_read_expert_span.argtypes = [vp, i32, i32, vp]
        L.df_moe_timing_enable.argtypes = [vp, ctypes.c_int]
        L.df_moe_timing_reset.argtypes = [vp]
        L.df_moe_timing_get.argtypes = [vp, ctypes.c_int, ctypes.POINTER(ctypes.c_char_p),
                                        ctypes.POINTER(i64), ctypes.POINTER(ctypes.c_double)]
        L.df_moe_last_launch_count.argtypes = [vp]
        L.df_moe_route_noalloc.argtypes = [vp, i32, i32, vp, i32, i32, vp, vp, vp]
        L.df_moe_graph_create.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp,
                                          ctypes.POINTER(ctypes.c_void_p)]
        L.df_moe_graph_launch.argtypes = [vp, vp]
        L.df_moe_graph_launch_count.argtypes = [vp]
        L.df_moe_graph_destroy.argtypes = [vp]; L.df_moe_graph_destroy.restype = None
        L.df_moe_stream_read.argtypes = [vp, ctypes.c_size_t, vp, vp]
        L.df_moe_create_cached.argtypes = [ctypes.POINTER(Config), ctypes.c_int, i32,
                                           ctypes.POINTER(ctypes.c_void_p)]
        L.df_moe_cache_stats.argtypes = [vp, ctypes.POINTER(i64), ctypes.POINTER(i64),
                                         ctypes.POINTER(i64)]
        ci, sz = ctypes.c_int, ctypes.c_size_t
        L.df_moe_permute_workspace.argtypes = [i64, i32, i32]
        L.df_moe_permute_workspace.restype = sz
        L.df_moe_permute.argtypes = [ci, vp, i64, i32, i32, vp, i32, i64, i64, vp, i32, i64, vp, i64,
                                     vp, i64, vp, vp, vp, vp, sz, vp]
        L.df_moe_permute_grad.argtypes = [ci, vp, i32, i64, i64, vp, i64, i32, i64, vp, i64, vp]
        L.df_moe_unpermute.argtypes = [ci, vp, i32, i64, i64, vp, vp, i64, i32, i64, vp, i64, vp]
        L.df_moe_unpermute_grad.argtypes = [ci, vp, i64, vp, i32, i64, i64, vp, vp, i64, i32, i64,
                                            vp, i64, vp, vp]
        L.df_moe_fp8_quantize.argtypes = [ci, vp, i32, i64, i64, i64, vp, i64, vp, i64, vp]
        L.df_moe_fp8_matmul.argtypes = [ci, vp, i64, vp, i64, vp, i64, vp, vp, i32, i64, i64, i64,
                                        i32, vp, i32, i64, vp, vp]
        L.df_moe_test_fp8_give_up.argtypes = [i32]
        L.df_moe_test_matmul_give_up.argtypes = [i32]
        L.df_moe_packed.argtypes = [i32, ctypes.c_char_p]
        L.df_moe_block_norm_grad_workspace.argtypes = [i64, i64]
        L.df_moe_block_norm_grad_workspace.restype = sz
        L.df_moe_balance_loss_workspace.argtypes = [i64, i32, i64]
        L.df_moe_balance_loss_workspace.restype = sz
        for name in SYMBOLS:
            f = getattr(L, name)
            if f.restype is ctypes.c_int:  # default
                f.restype = ctypes.c_int
        _lib = L
    return _lib


def span_bytes_for(H, I):
    return lib().df_moe_span_bytes_for(H, I)


def route_noalloc(router, E, H, x, T, k, ids, weights, stream=None):
    """Router + top-k with no device allocation (df_moe_route_noalloc): for
    callers that must not allocate, e.g. an engine whose memory pools already
    own all of HBM. Same kernels and results as step_router + step_topk."""
    rc = lib().df_moe_route_noalloc(_ptr(router), E, H, _ptr(x), T, k, _ptr(ids),
                                    _ptr(weights), _stream(stream))
    if rc != OK:
        raise DfMoeError(rc, lib().df_moe_last_error(None).decode())


def _ptr(a):
    """Pointer of a torch tensor / numpy array / int / None."""
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if hasattr(a, "data_ptr"):
        return a.data_ptr()
    if hasattr(a, "ctypes"):
        return a.ctypes.data
    raise TypeError("cannot take the address of %r" % type(a))


def _stream(s):
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


class MoE:
    """Owns one df_moe handle. Methods mirror the C calls (df_moe_ prefix
    dropped) and raise DfMoeError on failure."""

    def __init__(self, hidden, n_experts, top_k, inter, n_shared, shared_inter,
                 n_layers=1, max_tokens=1, rms_eps=1e-6, flags=0, device=0, cache_slots=0):
        """cache_slots > 0: experts in pinned host memory, that many a layer
        in HBM (df_moe_create_cached)."""
        self.cfg = Config(hidden, n_experts, top_k, inter, n_shared, shared_inter,
                          n_layers, max_tokens, rms_eps, flags)
        h = ctypes.c_void_p()
        if cache_slots:
            rc = lib().df_moe_create_cached(ctypes.byref(self.cfg), device, cache_slots,
                                            ctypes.byref(h))
        else:
            rc = lib().df_moe_create(ctypes.byref(self.cfg), device, ctypes.byref(h))
        if rc != OK:
            raise DfMoeError(rc, lib().df_moe_last_error(None).decode())
        self.h = h
        self.device = device

    def close(self):
        if getattr(self, "h", None):
            lib().df_moe_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    def _check(self, rc):
        if rc != OK:
            raise DfMoeError(rc, lib().df_moe_last_error(self.h).decode())

    @property
    def span_bytes(self):
        return lib().df_moe_expert_span_bytes(self.h)

    def load_experts(self, layer, router=None, experts=None, expert_begin=0,
                     expert_count=0, shared=None, src_is_device=False, stream=None):
        """shared: list of (gate, up, down) per shared expert (or None)."""
        keep = []
        sg = su = sd = None
        if shared:
            n = len(shared)
            arr = lambda i: (ctypes.c_void_p * n)(*[_ptr(s[i]) for s in shared])
            sg, su, sd = arr(0), arr(1), arr(2)
            keep += [sg, su, sd]
        w = LayerWeights(_ptr(router), _ptr(experts), expert_begin, expert_count,
                         ctypes.cast(sg, ctypes.c_void_p) if sg else None,
                         ctypes.cast(su, ctypes.c_void_p) if su else None,
                         ctypes.cast(sd, ctypes.c_void_p) if sd else None,
                         1 if src_is_device else 0)
        self._check(lib().df_moe_load_experts(self.h, layer, ctypes.byref(w),
                                              _stream(stream)))

    def forward(self, x, T, out, ids, weights, residual=None, out_f32=None,
                stream=None):
        self._check(lib().df_moe_forward(self.h, _ptr(x), T, _ptr(residual), _ptr(out),
                                         _ptr(out_f32), _ptr(ids), _ptr(weights),
                                         _stream(stream)))

    def forward_trace(self, x, T, out, ids, weights, trace_x=None, trace_xn=None,
                      out_f32=None, stream=None):
        """Stack mode: forward that also records each layer's input x and its
        normalised form xn ([L][T][H] bf16 device buffers)."""
        self._check(lib().df_moe_forward_trace(self.h, _ptr(x), T, _ptr(out), _ptr(out_f32),
                                               _ptr(ids), _ptr(weights), _ptr(trace_x),
                                               _ptr(trace_xn), _stream(stream)))

    def forward_host(self, x, T, out, ids=None, weights=None, residual=None,
                     out_f32=None, stream=None):
        self._check(lib().df_moe_forward_host(self.h, _ptr(x), T, _ptr(residual),
                                              _ptr(out), _ptr(out_f32), _ptr(ids),
                                              _ptr(weights), _stream(stream)))

    def sync(self, stream=None):
        self._check(lib().df_moe_sync(self.h, _stream(stream)))

    def test_drop_arrival(self):
        """Test hook: the next forward's gate/up phase leaves one pipeline
        stage unfilled, so a bounded device wait runs out (ETIMEOUT)."""
        self._check(lib().df_moe_test_drop_arrival(self.h))

    def step_router(self, layer, x, T, logits, stream=None):
        self._check(lib().df_moe_step_router(self.h, layer, _ptr(x), T, _ptr(logits),
                                             _stream(stream)))

    def step_topk(self, logits, T, ids, weights, stream=None):
        self._check(lib().df_moe_step_topk(self.h, _ptr(logits), T, _ptr(ids),
                                           _ptr(weights), _stream(stream)))

    def step_group(self, ids, T, offs, tok, slot, n_union, stream=None):
        self._check(lib().df_moe_step_group(self.h, _ptr(ids), T, _ptr(offs), _ptr(tok),
                                            _ptr(slot), _ptr(n_union), _stream(stream)))

    def step_expert_gateup(self, layer, x, T, ids, hbuf, stream=None):
        self._check(lib().df_moe_step_expert_gateup(self.h, layer, _ptr(x), T, _ptr(ids),
                                                    _ptr(hbuf), _stream(stream)))

    def step_expert_down(self, layer, hbuf, T, ids, weights, y, stream=None):
        self._check(lib().df_moe_step_expert_down(self.h, layer, _ptr(hbuf), T, _ptr(ids),
                                                  _ptr(weights), _ptr(y), _stream(stream)))

    def step_shared(self, layer, x, T, y, stream=None):
        self._check(lib().df_moe_step_shared(self.h, layer, _ptr(x), T, _ptr(y),
                                             _stream(stream)))

    def step_rmsnorm(self, x, T, xn, stream=None):
        self._check(lib().df_moe_step_rmsnorm(self.h, _ptr(x), T, _ptr(xn),
                                              _stream(stream)))

    def step_mxfp8(self, v, rows, n, codes, scales, stream=None):
        """The library's MXFP8 rounding of fp32 rows v [rows][n]: E4M3 codes
        [rows][n] and E8M0 scales [rows][n/32]."""
        self._check(lib().df_moe_step_mxfp8(self.h, _ptr(v), rows, n, _ptr(codes), _ptr(scales),
                                            _stream(stream)))

    def read_expert_span(self, layer, expert, dst):
        self._check(lib().df_moe_read_expert_span(self.h, layer, expert, _ptr(dst)))

    def timing_enable(self, on=True):
        self._check(lib().df_moe_timing_enable(self.h, 1 if on else 0))

    def timing_reset(self):
        self._check(lib().df_moe_timing_reset(self.h))

    def timing(self):
        """{kernel kind name: (launches, total_ms)} since the last reset."""
        out = {}
        for kind in range(KERNEL_KINDS):
            name = ctypes.c_char_p()
            n = ctypes.c_int64()
            ms = ctypes.c_double()
            self._check(lib().df_moe_timing_get(self.h, kind, ctypes.byref(name),
                                                ctypes.byref(n), ctypes.byref(ms)))
            out[name.value.decode()] = (n.value, ms.value)
        return out

    def last_launch_count(self):
        return lib().df_moe_last_launch_count(self.h)

    def cache_stats(self):
        """(hits, misses, bytes copied host -> HBM) of the expert cache."""
        hits, misses, nbytes = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        self._check(lib().df_moe_cache_stats(self.h, ctypes.byref(hits), ctypes.byref(misses),
                                             ctypes.byref(nbytes)))
        return hits.value, misses.value, nbytes.value

    def graph(self, x, T, out, ids, weights, residual=None, out_f32=None):
        """A forward pass captured into a CUDA graph (df_moe_graph_create),
        bound to these buffers: replay with Graph.launch after changing the
        contents of x."""
        g = ctypes.c_void_p()
        self._check(lib().df_moe_graph_create(self.h, _ptr(x), T, _ptr(residual), _ptr(out),
                                              _ptr(out_f32), _ptr(ids), _ptr(weights),
                                              ctypes.byref(g)))
        return Graph(g)


class Graph:
    """Owns one df_moe_graph."""

    def __init__(self, g):
        self.g = g

    def launch(self, stream=None):
        rc = lib().df_moe_graph_launch(self.g, _stream(stream))
        if rc != OK:
            raise DfMoeError(rc, lib().df_moe_last_error(None).decode())

    def launch_count(self):
        return lib().df_moe_graph_launch_count(self.g)

    def close(self):
        if self.g:
            lib().df_moe_graph_destroy(self.g)
            self.g = None

    def __del__(self):
        self.close()


def stream_read(buf, nbytes, sink, stream=None):
    """Read-only streaming probe over nbytes of device memory (df_moe_stream_read)."""
    rc = lib().df_moe_stream_read(_ptr(buf), nbytes, _ptr(sink), _stream(stream))
    if rc != OK:
        raise DfMoeError(rc, lib().df_moe_last_error(None).decode())


# ---- the expert path's operators (no handle) ---------------------------------
# A decode step makes several of these calls with microseconds of work each, so
# the marshalling is kept short: one pass over the arrays, the C functions
# looked up once. A call runs on `stream`, or without one on the stream that
# torch has current on the arrays' device (between other work of the same
# program, and inside a capture); where all arrays are raw addresses, that is
# the legacy default stream.
_INT32 = 0x7fffffff  # what lies further from 0 is cut by the C call's 32-bit arguments, so refused here


class _Calls:
    """The C functions, each looked up at its first call."""

    def __getattr__(self, name):
        f = getattr(lib(), name)
        setattr(self, name, f)
        return f


_c = _Calls()


def _find_torch_stream(dev):
    global _torch_stream
    import torch  # the arrays are torch's, so torch is loaded
    _torch_stream = torch._C._cuda_getCurrentRawStream
    return _torch_stream(dev)


_torch_stream = _find_torch_stream  # from the first call on, torch's own


def _find_tensor_calls(a):
    global _get_device, _element_size, _data_ptr
    import sys
    torch = sys.modules.get("torch")
    if torch:
        _get_device, _element_size, _data_ptr = torch.Tensor.get_device, torch.Tensor.element_size, torch.Tensor.data_ptr
    raise TypeError


# Of a tensor (TypeError for what is none): torch's own from the second call on,
# which cost less than methods that are looked up.
_get_device = _element_size = _data_ptr = _find_tensor_calls


def _type(d):
    try:
        return _TYPES[d]
    except (KeyError, TypeError):
        raise DfMoeError(EINVAL, "dtype must be one of 'bf16', 'f16', 'f32', 'e4m3', not %r" % (d,)) from None


def _placer(layout, lead=None):
    """place(array, ..., size=0, other=0, gate_size=0, dgate_size=0) -> (device, address, ...):
    the one CUDA device that the torch tensors among the arrays lie on (-1, the
    current one, where there are only raw addresses), and the arrays' addresses (0
    for one that is absent). `layout`: the arrays' names, each with the bytes of an
    element, which a tensor's have to be (0: any): the library goes by the types
    that the call names, and would pass the end of a narrower array. `lead`: the
    array that the device is asked of first, where it is not the first.

    The function is written out here, without a loop, since a decode step's calls
    take microseconds: with a loop it cost 0.3 us more (seven arrays)."""
    names, sizes = zip(*(word.split(":") for word in layout.split()))
    checks = ["dev >= 0"]
    for a, n in zip(names, sizes):
        wide = {"0": "True", "gate_size": "(not gate_size or _element_size(gate) == gate_size)",
                "dgate_size": "(not dgate_size or _element_size(dgate) == dgate_size)"}.get(n, "_element_size(%s) == %s" % (a, n))
        checks.append(wide if a == names[0] and not lead else "(%s is None or _get_device(%s) == dev and %s)" % (a, a, wide))
    scope = {}
    exec("""
def place(%s, size=0, other=0, gate_size=0, dgate_size=0):
    try:  # all of them tensors on one device, or absent
        dev = _get_device(%s)
        if %s:
            return dev, %s
    except TypeError:
        pass
    return _place_any(%r, (%s,), (%s,))
""" % (", ".join(names), lead or names[0], " and ".join(checks),
       ", ".join("0 if %s is None else _data_ptr(%s)" % (a, a) for a in names), names, ", ".join(sizes), ", ".join(names)),
         globals(), scope)
    return scope["place"]


def _place_any(names, sizes, arrays):
    dev, out = -1, [-1]
    for i, a in enumerate(arrays):
        if a is None or a.__class__ is int:
            out.append(a or 0)
            continue
        try:
            d, p = a.get_device(), a.data_ptr()
        except AttributeError:
            raise DfMoeError(EINVAL, "every array must be in device memory") from None
        if d != dev:
            if d < 0:
                raise DfMoeError(EINVAL, "every array must be in device memory")
            if dev >= 0:
                raise DfMoeError(EINVAL, "arrays on different devices: %d and %d" % (dev, d))
            dev = d
        elif d < 0:
            raise DfMoeError(EINVAL, "every array must be in device memory")
        size = getattr(a, "element_size", None)
        if size and sizes[i] and size() != sizes[i]:
            if names[i] != "status" or size() < 4:  # of a wider one the first word is taken
                raise DfMoeError(EINVAL, "%s has elements of %d bytes, not of the %d that the call takes" %
                                 (names[i], size(), sizes[i]))
        out.append(p)
    out[0] = dev
    return out


def _int32(**sizes):
    """Refuses what a 32-bit argument would cut."""
    for name, v in sizes.items():
        if not -_INT32 - 1 <= v <= _INT32:
            raise DfMoeError(EINVAL, "%s = %d does not fit 32 bits" % (name, v))


def _failed(rc):
    raise DfMoeError(rc, lib().df_moe_last_error(None).decode())


_place_permute = _placer("ids:4 x:size rows:size offs:4 pos:4 src:4")
_place_permute_all = _placer("ids:4 x:size rows:size offs:4 pos:4 src:4 workspace:0 scales:4 rows_scales:4")
_place_permute_grad = _placer("drows:size pos:4 dx:size")
_place_unpermute = _placer("rows:size pos:4 weights:4 y:size")
_place_unpermute_grad = _placer("dy:size rows:size pos:4 weights:4 drows:size dweights:4")
_place_fp8_quantize = _placer("x:size codes:1 scales:4")
_place_fp8_matmul = _placer("x:1 xs:4 w:1 ws:4 offs:4 y:size status:4")


def permute_workspace(T, k, E):
    """Bytes of workspace that permute needs (df_moe_permute_workspace)."""
    if (k | E) >> 31:
        return 0
    return _c.df_moe_permute_workspace(T, k, E)


def permute(ids, T, k, E, x, dtype, H, rows, offs, pos, src, workspace=None, workspace_bytes=0,
            ldx=0, ldr=0, scales=None, n_scales=0, ld_scales=0, rows_scales=None, ld_rows_scales=0,
            stream=None):
    """Tokens sorted by expert (df_moe_permute): rows[pos[a]] = x[a // k]."""
    if (k | E | n_scales) >> 31:
        _int32(k=k, E=E, n_scales=n_scales)
    if workspace_bytes < 0:
        raise DfMoeError(EINVAL, "workspace_bytes is negative")
    dtype, n = _type(dtype)
    if workspace is None and scales is None and rows_scales is None:
        dev, i, x, r, o, q, s = _place_permute(ids, x, rows, offs, pos, src, n)
        w = xs = rs = None
    else:
        dev, i, x, r, o, q, s, w, xs, rs = _place_permute_all(ids, x, rows, offs, pos, src, workspace, scales, rows_scales, n)
    rc = _c.df_moe_permute(dev, i, T, k, E, x, dtype, H, ldx, xs, n_scales, ld_scales, r,
                           ldr, rs, ld_rows_scales, o, q, s, w, workspace_bytes, _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _failed(rc)


def permute_grad(drows, dtype, n_rows, pos, T, k, H, dx, ldr=0, ldx=0, stream=None):
    """Gradient of permute's x (df_moe_permute_grad)."""
    if k >> 31:
        _int32(k=k)
    dtype, n = _type(dtype)
    dev, r, q, y = _place_permute_grad(drows, pos, dx, n)
    rc = _c.df_moe_permute_grad(dev, r, dtype, n_rows, ldr, q, T, k, H, y, ldx,
                                _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _failed(rc)


def unpermute(rows, dtype, n_rows, pos, weights, T, k, H, y, ldr=0, ldy=0, stream=None):
    """Weighted rows back to their tokens (df_moe_unpermute)."""
    if k >> 31:
        _int32(k=k)
    dtype, n = _type(dtype)
    dev, r, q, w, y = _place_unpermute(rows, pos, weights, y, n)
    rc = _c.df_moe_unpermute(dev, r, dtype, n_rows, ldr, q, w, T, k, H, y, ldy,
                             _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _failed(rc)


def unpermute_grad(dy, rows, dtype, n_rows, pos, weights, T, k, H, drows, dweights, lddy=0, ldr=0,
                   lddr=0, stream=None):
    """Gradients of unpermute's rows and weights (df_moe_unpermute_grad)."""
    if k >> 31:
        _int32(k=k)
    dtype, n = _type(dtype)
    dev, g, r, q, w, dr, dw = _place_unpermute_grad(dy, rows, pos, weights, drows, dweights, n)
    rc = _c.df_moe_unpermute_grad(dev, g, lddy, r, dtype, n_rows, ldr, q, w, T, k, H, dr,
                                  lddr, dw, _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _failed(rc)


def fp8_quantize(x, dtype, M, K, codes, scales, ldx=0, ldc=0, lds=0, stream=None):
    """Rows as e4m3 codes with one fp32 scale per 128 (df_moe_fp8_quantize)."""
    dtype, n = _type(dtype)
    dev, x, c, s = _place_fp8_quantize(x, codes, scales, n)
    rc = _c.df_moe_fp8_quantize(dev, x, dtype, M, K, ldx, c, ldc, s, lds, _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _failed(rc)


def fp8_matmul(x, xs, w, ws, offs, G, M, N, K, y, dtype, transposed=False, ldx=0, ldxs=0, ldw=0,
               ldy=0, status=None, stream=None):
    """e4m3 rows times their group's e4m3 weights (df_moe_fp8_matmul)."""
    if G >> 31:
        _int32(G=G)
    dtype, n = _type(dtype)
    dev, x, xs, w, ws, o, y, st = _place_fp8_matmul(x, xs, w, ws, offs, y, status, n)
    rc = _c.df_moe_fp8_matmul(dev, x, ldx, xs, ldxs, w, ldw, ws, o, G, M, N, K,
                              1 if transposed else 0, y, dtype, ldy, st, _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _failed(rc)


def test_fp8_give_up(role):
    """Test hook: one role of the next fp8_matmul gives up (df_moe_test_fp8_give_up)."""
    rc = _c.df_moe_test_fp8_give_up(role)
    if rc:
        _failed(rc)


# ---- around the routed experts (no handle) -----------------------------------
# These calls have twenty arguments and more, of which ctypes takes 0.1 us each:
# they go as one block of 8-byte values (df_moe_packed). What a value cannot hold
# does not pack.
def _packer(call, layout):
    pack = struct.Struct(layout).pack

    def run(*args):
        try:
            block = pack(*args)
        except struct.error:
            raise DfMoeError(EINVAL, "an argument is not a number of 64 bits") from None
        rc = _c.df_moe_packed(call, block)
        if rc:
            _failed(rc)
    return run


_call_matmul = _packer(0, "20q")
_call_matmul_grad = _packer(1, "24q")
_call_block_norm = _packer(2, "10qdqd9q")
_call_block_norm_grad = _packer(3, "14qdqd15q")
_call_balance_loss = _packer(4, "12q2d8q")
_call_balance_loss_grad = _packer(5, "13q2d7q")


_place_matmul = _placer("x:size w:size y:other bias:size residual:other pre:size status:4")
_place_matmul_grad = _placer("dy:size x:size w:size dx:size dw:other dbias:other pre:size dz:size status:4")
_place_norm = _placer("u:size residual:size h:size n:size post_weight:other gate:gate_size pre_weight:other",
                      "residual if u is None else u")
_place_norm_grad = _placer("dh:size dn:size u:size h:size du:size dresidual:size post_weight:other dpost_weight:4 gate:gate_size "
                           "dgate:dgate_size pre_weight:other dpre_weight:4 workspace:0", "dn if dh is None else dh")
_place_balance = _placer("logits:size ids:4 loss:4 counts:4 tokens:4 workspace:0 probs:4 offs:4 mask:1 status:4")
_place_balance_grad = _placer("dloss:4 logits:size ids:4 counts:4 tokens:4 dlogits:size offs:4 mask:1 weights:4 dweights:4")

# By the names that a call gives: their codes, and the bytes of an element of the
# arrays of those types (of gates and their gradients by the kind of gate, too).
_PAIRS = [(a, i, n, b, j, o) for a, (i, n) in _TYPES.items() for b, (j, o) in _TYPES.items()]
_PRODUCT = {(a, b, c): (i, j, k, n, o) for a, i, n, b, j, o in _PAIRS for c, k in _ACTS.items()}
_NORM = {(a, b, c): (i, j, k, n, o, (0, o, 4, n)[k], (0, 4, 4, n)[k]) for a, i, n, b, j, o in _PAIRS for c, k in _GATES.items()}
_BALANCE = {(a, c): (i, k, n) for a, (i, n) in _TYPES.items() for c, k in _SCORES.items()}


def _unknown(types, kinds, name, v):
    """Names that are in no table."""
    for t in types:
        _type(t)
    raise DfMoeError(EINVAL, "%s must be one of %s, not %r" % (name, ", ".join(map(repr, kinds)), v)) from None


def matmul(x, w, dtype, M, N, K, y, out_dtype, bias=None, act="none", residual=None, pre=None, ldx=0,
           ldw=0, ldy=0, ldr=0, ldp=0, status=None, stream=None):
    """y = residual + act(x w' + bias) of 16-bit matrices (df_moe_matmul)."""
    try:
        t, o, a, size, other = _PRODUCT[dtype, out_dtype, act]
    except (KeyError, TypeError):
        _unknown((dtype, out_dtype), _ACTS, "act", act)
    dev, x, w, y, b, r, z, st = _place_matmul(x, w, y, bias, residual, pre, status, size, other)
    _call_matmul(dev, x, ldx, w, ldw, t, M, N, K, b, a, r, ldr, z, ldp, y, o, ldy, st,
                 _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream) or 0)


def matmul_grad(dy, x, w, dtype, M, N, K, dx=None, dw=None, dbias=None, grad_dtype="f32", act="none",
                pre=None, dz=None, lddy=0, ldx=0, ldw=0, lddx=0, lddw=0, ldp=0, lddz=0, status=None,
                stream=None):
    """Gradients of matmul's x, w and bias (df_moe_matmul_grad)."""
    try:
        t, g, a, size, other = _PRODUCT[dtype, grad_dtype, act]
    except (KeyError, TypeError):
        _unknown((dtype, grad_dtype), _ACTS, "act", act)
    dev, dy, x, w, dx, dw, db, z, dz, st = _place_matmul_grad(dy, x, w, dx, dw, dbias, pre, dz, status, size, other)
    _call_matmul_grad(dev, dy, lddy, x, ldx, w, ldw, t, M, N, K, a, z, ldp, dz, lddz, dx, lddx, dw, lddw, db, g, st,
                      _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream) or 0)


def test_matmul_give_up(role):
    """Test hook: one role of the next product gives up (df_moe_test_matmul_give_up)."""
    rc = _c.df_moe_test_matmul_give_up(role)
    if rc:
        _failed(rc)


def block_norm(u, residual, dtype, T, H, h=None, n=None, post=False, post_weight=None, gate=None,
               gate_kind="none", residual_scale=1.0, pre_weight=None, weight_dtype="f32", eps=1e-6, ldu=0,
               ldr=0, ldg=0, ldh=0, ldn=0, stream=None):
    """h = residual_scale residual + gate norm(u), n = norm(h) (df_moe_block_norm)."""
    try:
        t, w, kind, size, other, gate_size, _ = _NORM[dtype, weight_dtype, gate_kind]
    except (KeyError, TypeError):
        _unknown((dtype, weight_dtype), _GATES, "gate_kind", gate_kind)
    dev, u, r, h, n, q, g, v = _place_norm(u, residual, h, n, post_weight, gate, pre_weight, size, other, gate_size)
    _call_block_norm(dev, u, ldu, 1 if post else 0, q, kind, g, ldg, r, ldr, residual_scale, v, eps, T, H, t, w, h, ldh, n, ldn,
                     _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream) or 0)


def block_norm_grad_workspace(T, H):
    """Bytes of workspace that block_norm_grad needs (df_moe_block_norm_grad_workspace)."""
    if (T | H) >> 63 not in (0, -1):
        return 0
    return _c.df_moe_block_norm_grad_workspace(T, H)


def block_norm_grad(dh, dn, u, h, dtype, T, H, du=None, dresidual=None, post=False, post_weight=None,
                    dpost_weight=None, gate=None, gate_kind="none", dgate=None, residual_scale=1.0,
                    pre_weight=None, dpre_weight=None, weight_dtype="f32", eps=1e-6, workspace=None,
                    workspace_bytes=0, lddh=0, lddn=0, ldu=0, ldh=0, ldg=0, lddu=0, lddr=0, lddg=0,
                    stream=None):
    """Gradients of block_norm (df_moe_block_norm_grad)."""
    try:
        t, w, kind, size, other, gate_size, dgate_size = _NORM[dtype, weight_dtype, gate_kind]
    except (KeyError, TypeError):
        _unknown((dtype, weight_dtype), _GATES, "gate_kind", gate_kind)
    dev, dh, dn, u, h, du, dr, q, dq, g, dg, v, dv, ws = _place_norm_grad(
        dh, dn, u, h, du, dresidual, post_weight, dpost_weight, gate, dgate, pre_weight, dpre_weight, workspace, size, other,
        gate_size, dgate_size)
    if workspace_bytes < 0:
        raise DfMoeError(EINVAL, "workspace_bytes is negative")
    _call_block_norm_grad(dev, dh, lddh, dn, lddn, u, ldu, h, ldh, 1 if post else 0, q, kind, g, ldg, residual_scale, v, eps, T, H,
                          t, w, du, lddu, dr, lddr, dq, dg, lddg, dv, ws, workspace_bytes,
                          _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream) or 0)


def balance_loss_workspace(T, E, S=1):
    """Bytes of workspace that balance_loss needs (df_moe_balance_loss_workspace)."""
    if E >> 31 or (T | S) >> 63 not in (0, -1):
        return 0
    return _c.df_moe_balance_loss_workspace(T, E, S)


def balance_loss(logits, dtype, T, E, ids, k, loss, counts, tokens, workspace=None, workspace_bytes=0,
                 probs=None, offs=None, S=1, mask=None, score="softmax", coef=1.0, z_coef=0.0, ldl=0,
                 status=None, stream=None):
    """The router's balance loss and every expert's count, a sequence (df_moe_balance_loss)."""
    if (E | k) >> 31:
        _int32(E=E, k=k)
    if workspace_bytes < 0:
        raise DfMoeError(EINVAL, "workspace_bytes is negative")
    try:
        kind, sc, size = _BALANCE[dtype, score]
    except (KeyError, TypeError):
        _unknown((dtype,), _SCORES, "score", score)
    dev, z, i, lo, c, t, ws, p, o, m, st = _place_balance(logits, ids, loss, counts, tokens, workspace, probs, offs, mask,
                                                          status, size)
    _call_balance_loss(dev, z, kind, ldl, i, T, E, k, o, S, m, sc, coef, z_coef, lo, c, t, p, ws, workspace_bytes, st,
                       _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream) or 0)


def balance_loss_grad(dloss, logits, dtype, T, E, ids, k, counts, tokens, dlogits, offs=None, S=1,
                      mask=None, score="softmax", coef=1.0, z_coef=0.0, weights=None, dweights=None, ldl=0,
                      lddl=0, stream=None):
    """The gradient of the logits: the loss's and the routing weights' (df_moe_balance_loss_grad)."""
    if (E | k) >> 31:
        _int32(E=E, k=k)
    try:
        kind, sc, size = _BALANCE[dtype, score]
    except (KeyError, TypeError):
        _unknown((dtype,), _SCORES, "score", score)
    dev, g, z, i, c, t, d, o, m, w, dw = _place_balance_grad(dloss, logits, ids, counts, tokens, dlogits, offs, mask, weights,
                                                             dweights, size)
    _call_balance_loss_grad(dev, g, z, kind, ldl, i, T, E, k, o, S, m, sc, coef, z_coef, c, t, w, dw, d, lddl,
                            _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream) or 0)
