"""Thin ctypes binding of libdfmoe.so (include/df_moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. torch tensors are accepted wherever the C call takes a pointer (their
data_ptr() is passed); streams are torch.cuda.Stream objects or raw handles.
There is no fallback: if the library is missing this module raises.
"""
import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libdfmoe.so")

OK, EINVAL, ENOMEM, ECUDA, ESTATE, ERANGE, ETIMEOUT, EDEVICE = 0, -1, -2, -3, -4, -5, -6, -7
STACK_RMSNORM_RESIDUAL = 1
PREFILL_MMA_SYNC = 4
MXFP8_ACT = 8
PLANES = 16
KERNEL_KINDS = 18
BF16, F16, F32, E4M3 = 0, 1, 2, 3
_DTYPES = {"bf16": BF16, "f16": F16, "f32": F32, "e4m3": E4M3,
           BF16: BF16, F16: F16, F32: F32, E4M3: E4M3}

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
_INT32 = 0x7fffffff  # larger: cut by the C call's 32-bit arguments, so refused here


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


def _dtype(d):
    try:
        return _DTYPES[d]
    except (KeyError, TypeError):
        raise DfMoeError(EINVAL, "dtype must be one of 'bf16', 'f16', 'f32', 'e4m3', not %r" % (d,))


def _place(*arrays):
    """[device, address, address, ...]: the one CUDA device that the torch
    tensors among the arrays lie on (-1, the current one, where there are only
    raw addresses), and the arrays' addresses."""
    try:  # all of them tensors on one device
        out = [a.data_ptr() for a in arrays]
        dev = arrays[0].get_device()
        if dev >= 0:
            for a in arrays:
                if a.get_device() != dev:
                    break
            else:
                return [dev, *out]
    except AttributeError:
        pass
    return _place_any(arrays)


def _place_any(arrays):
    dev, out = -1, [-1]
    for a in arrays:
        if a is None or a.__class__ is int:
            out.append(a)
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
        out.append(p)
    out[0] = dev
    return out


def _int32(**sizes):
    """Refuses what a 32-bit argument would cut."""
    for name, v in sizes.items():
        if v > _INT32:
            raise DfMoeError(EINVAL, "%s = %d does not fit 32 bits" % (name, v))


def _failed(rc):
    raise DfMoeError(rc, lib().df_moe_last_error(None).decode())


def permute_workspace(T, k, E):
    """Bytes of workspace that permute needs (df_moe_permute_workspace)."""
    if (k | E) > _INT32:
        return 0
    return _c.df_moe_permute_workspace(T, k, E)


def permute(ids, T, k, E, x, dtype, H, rows, offs, pos, src, workspace=None, workspace_bytes=0,
            ldx=0, ldr=0, scales=None, n_scales=0, ld_scales=0, rows_scales=None, ld_rows_scales=0,
            stream=None):
    """Tokens sorted by expert (df_moe_permute): rows[pos[a]] = x[a // k]."""
    if (k | E | n_scales) > _INT32:
        _int32(k=k, E=E, n_scales=n_scales)
    if workspace_bytes < 0:
        raise DfMoeError(EINVAL, "workspace_bytes is negative")
    if workspace is None and scales is None and rows_scales is None:
        dev, i, x, r, o, q, s = _place(ids, x, rows, offs, pos, src)
        w = xs = rs = None
    else:
        dev, i, x, r, o, q, s, w, xs, rs = _place_any((ids, x, rows, offs, pos, src, workspace, scales,
                                                       rows_scales))
    rc = _c.df_moe_permute(dev, i, T, k, E, x, _dtype(dtype), H, ldx, xs, n_scales, ld_scales, r,
                           ldr, rs, ld_rows_scales, o, q, s, w, workspace_bytes, _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _failed(rc)


def permute_grad(drows, dtype, n_rows, pos, T, k, H, dx, ldr=0, ldx=0, stream=None):
    """Gradient of permute's x (df_moe_permute_grad)."""
    if k > _INT32:
        _int32(k=k)
    dev, r, q, y = _place(drows, pos, dx)
    rc = _c.df_moe_permute_grad(dev, r, _dtype(dtype), n_rows, ldr, q, T, k, H, y, ldx,
                                _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _failed(rc)


def unpermute(rows, dtype, n_rows, pos, weights, T, k, H, y, ldr=0, ldy=0, stream=None):
    """Weighted rows back to their tokens (df_moe_unpermute)."""
    if k > _INT32:
        _int32(k=k)
    dev, r, q, w, y = _place(rows, pos, weights, y)
    rc = _c.df_moe_unpermute(dev, r, _dtype(dtype), n_rows, ldr, q, w, T, k, H, y, ldy,
                             _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _failed(rc)


def unpermute_grad(dy, rows, dtype, n_rows, pos, weights, T, k, H, drows, dweights, lddy=0, ldr=0,
                   lddr=0, stream=None):
    """Gradients of unpermute's rows and weights (df_moe_unpermute_grad)."""
    if k > _INT32:
        _int32(k=k)
    dev, g, r, q, w, dr, dw = _place(dy, rows, pos, weights, drows, dweights)
    rc = _c.df_moe_unpermute_grad(dev, g, lddy, r, _dtype(dtype), n_rows, ldr, q, w, T, k, H, dr,
                                  lddr, dw, _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _failed(rc)


def fp8_quantize(x, dtype, M, K, codes, scales, ldx=0, ldc=0, lds=0, stream=None):
    """Rows as e4m3 codes with one fp32 scale per 128 (df_moe_fp8_quantize)."""
    dev, x, c, s = _place(x, codes, scales)
    rc = _c.df_moe_fp8_quantize(dev, x, _dtype(dtype), M, K, ldx, c, ldc, s, lds, _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _failed(rc)


def fp8_matmul(x, xs, w, ws, offs, G, M, N, K, y, dtype, transposed=False, ldx=0, ldxs=0, ldw=0,
               ldy=0, status=None, stream=None):
    """e4m3 rows times their group's e4m3 weights (df_moe_fp8_matmul)."""
    if G > _INT32:
        _int32(G=G)
    dev, x, xs, w, ws, o, y, st = _place(x, xs, w, ws, offs, y, status)
    rc = _c.df_moe_fp8_matmul(dev, x, ldx, xs, ldxs, w, ldw, ws, o, G, M, N, K,
                              1 if transposed else 0, y, _dtype(dtype), ldy, st, _torch_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _failed(rc)


def test_fp8_give_up(role):
    """Test hook: one role of the next fp8_matmul gives up (df_moe_test_fp8_give_up)."""
    rc = _c.df_moe_test_fp8_give_up(role)
    if rc:
        _failed(rc)
