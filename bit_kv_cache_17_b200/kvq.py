"""ctypes binding of libkvq.so: the entry points of include/kvq.h under the same names.

Argument marshalling only (tensor -> pointer, Python ints -> C arrays); every step of
the append / decode / dequant path runs in the library's CUDA kernels.  The library is
loaded at import and a missing library is an ImportError: there is no fallback path.
"""
import ctypes as C
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkvq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing; build it with `python -m bit_kv_cache_17_b200.build`")
_lib = C.CDLL(LIB_PATH)

# kvq_type (include/kvq.h)
TYPES = {
    "bf16": 0, "q2_0": 1, "q3_0": 2, "q4_0": 3, "q5_0": 4, "q6_0": 5, "q8_0": 6, "q4_1": 7,
    "kvarn2": 8, "kvarn3": 9, "kvarn4": 10, "kvarn5": 11, "kvarn6": 12, "kvarn8": 13,
    "q2_1": 14, "q3_1": 15, "q5_1": 16, "q6_1": 17,
}
KVQ_OK, KVQ_E_INVAL, KVQ_E_UNSUPPORTED, KVQ_E_CAPACITY = 0, -1, -2, -3
KVQ_E_ALIGN, KVQ_E_CUDA, KVQ_E_DEVICE, KVQ_E_SIZE = -4, -5, -6, -7
KVQ_DT_F32, KVQ_DT_BF16, KVQ_DT_F16 = 0, 1, 2


class kvq_params(C.Structure):
    _fields_ = [
        ("n_layers", C.c_int32), ("n_seqs", C.c_int32), ("n_kv_heads", C.c_int32),
        ("head_dim", C.c_int32), ("max_ctx", C.c_int64), ("type_k", C.c_int32),
        ("type_v", C.c_int32), ("tail", C.c_int32), ("group", C.c_int32),
        ("sinkhorn_iters", C.c_int32), ("page_tokens", C.c_int32), ("var_norm", C.c_int32), ("tail_f16", C.c_int32),
    ]


class kvq_rope_params(C.Structure):
    _fields_ = [
        ("rot_dim", C.c_int32), ("n_axes", C.c_int32), ("sections", C.c_int32 * 4), ("turns", C.c_int32),
        ("adjacent", C.c_int32), ("inverse", C.c_int32), ("theta", C.c_double),
    ]


class KVQError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {kvq_strerror(code)} ({code})")


_vp, _i32, _i64, _sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
_SIG = {
    "kvq_default_params": (None, [C.POINTER(kvq_params)]),
    "kvq_cache_bytes": (C.c_int, [C.POINTER(kvq_params), C.POINTER(_sz)]),
    "kvq_payload_bytes": (C.c_int, [_i32, _i32, _i64, _i64, _i64, _i64, C.POINTER(C.c_double)]),
    "kvq_cache_create": (C.c_int, [C.POINTER(kvq_params), _vp, _sz, C.POINTER(_vp)]),
    "kvq_cache_destroy": (None, [_vp]),
    "kvq_append": (C.c_int, [_vp, _i32, _i32, C.POINTER(_i32), C.POINTER(_i32), _vp, _vp, _vp]),
    "kvq_workspace_bytes": (C.c_int, [_vp, _i32, _i32, C.POINTER(_sz)]),
    "kvq_decode_attn": (C.c_int, [_vp, _i32, _i32, C.POINTER(_i32), _i32, _vp, C.c_float, _vp, _vp, _sz, _vp]),
    "kvq_prefill_attn": (C.c_int, [_vp, _i32, _i32, _i32, _i32, _vp, C.c_float, _vp, _vp, _sz, _vp]),
    "kvq_append_decode": (C.c_int, [_vp, _i32, _i32, C.POINTER(_i32), C.POINTER(_i32), _vp, _vp, _i32, _vp,
                                    C.c_float, _vp, _vp, _sz, _vp]),
    "kvq_dequant": (C.c_int, [_vp, _i32, _i32, _i32, _i64, _i64, _i32, _vp, _vp]),
    "kvq_seq_len": (C.c_int, [_vp, _i32, _i32, C.POINTER(_i64)]),
    "kvq_seq_reset": (C.c_int, [_vp, _i32]),
    "kvq_locate": (C.c_int, [_vp, _i32, _i32, _i32, _i64, _i32, _i32, _i64, C.POINTER(_sz), C.POINTER(_sz)]),
    "kvq_get_status": (C.c_int, [_vp, _vp]),
    "kvq_describe": (C.c_char_p, [_vp]),
    "kvq_strerror": (C.c_char_p, [C.c_int]),
    "kvq_launch_count": (C.c_int, [C.POINTER(C.c_uint64)]),
    "kvq_decode_attn_noalloc": (C.c_int, [_vp, _i32, _i32, C.POINTER(_i32), _i32, _vp, C.c_float, _vp, _vp]),
    "kvq_rope_default_params": (None, [C.POINTER(kvq_rope_params)]),
    "kvq_rope": (C.c_int, [C.POINTER(kvq_rope_params), C.POINTER(C.c_double), _i64, _vp, _i64, _i32, _vp, _i32, _i64,
                           _vp, _i32, _i64, _i32, _vp, _i64, _vp, _i64, _vp]),
    "kvq_batch_workspace_bytes": (C.c_int, [_vp, _i32, _i32, C.POINTER(_i32), C.POINTER(_i32), _i32, C.POINTER(_sz)]),
    "kvq_batch_attn": (C.c_int, [_vp, _i32, _i32, C.POINTER(_i32), C.POINTER(_i32), _i32, _i32, _vp, C.c_float, _vp,
                                 _vp, _vp, _sz, _vp]),
    "kvq_attn_mass": (C.c_int, [_vp, _i32, _i32, C.POINTER(_i32), C.POINTER(_i32), _i32, _i32, _vp, C.c_float, _vp,
                                C.c_float, _vp, _vp, _i64, _vp, _sz, _vp]),
    "kvq_evict_workspace_bytes": (C.c_int, [_vp, _vp, _i32, _i32, C.POINTER(_sz)]),
    "kvq_evict": (C.c_int, [_vp, _i32, _vp, _i32, _i32, C.POINTER(_i32), C.POINTER(_i32), _vp, _i64, _i32, _i32, _i32,
                            _vp, _vp, _i64, _vp, _sz, _vp]),
}
for _name, (_res, _args) in _SIG.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_SIG)


def _check(rc, where):
    if rc != KVQ_OK:
        raise KVQError(rc, where)


def _i32arr(xs):
    xs = [int(x) for x in xs]
    return (_i32 * max(1, len(xs)))(*xs)


def kvq_strerror(code):
    return _lib.kvq_strerror(code).decode()


def kvq_default_params(**overrides):
    p = kvq_params()
    _lib.kvq_default_params(C.byref(p))
    for k, v in overrides.items():
        if k in ("type_k", "type_v") and isinstance(v, str):
            v = TYPES[v]
        setattr(p, k, v)
    return p


def kvq_cache_bytes(p):
    n = _sz()
    _check(_lib.kvq_cache_bytes(C.byref(p), C.byref(n)), "kvq_cache_bytes")
    return n.value


def kvq_payload_bytes(type_, n_layers, n_kv_heads, n, tail, raw_bits=0):
    t = TYPES[type_] if isinstance(type_, str) else int(type_)
    out = C.c_double()
    _check(_lib.kvq_payload_bytes(t, raw_bits, n_layers, n_kv_heads, n, tail, C.byref(out)), "kvq_payload_bytes")
    return out.value


def kvq_cache_create(p, dev_ptr, nbytes):
    h = _vp()
    _check(_lib.kvq_cache_create(C.byref(p), _vp(dev_ptr), nbytes, C.byref(h)), "kvq_cache_create")
    return h


def kvq_cache_destroy(h):
    _lib.kvq_cache_destroy(h)


def kvq_append(h, layer, seq_ids, n_new, k_ptr, v_ptr, stream=0):
    rc = _lib.kvq_append(h, layer, len(seq_ids), _i32arr(seq_ids), _i32arr(n_new), _vp(k_ptr), _vp(v_ptr), _vp(stream))
    _check(rc, "kvq_append")


def kvq_workspace_bytes(h, n_seqs, n_q_heads):
    n = _sz()
    _check(_lib.kvq_workspace_bytes(h, n_seqs, n_q_heads, C.byref(n)), "kvq_workspace_bytes")
    return n.value


def kvq_decode_attn(h, layer, seq_ids, n_q_heads, q_ptr, softmax_scale, out_ptr, ws_ptr, ws_bytes, stream=0):
    rc = _lib.kvq_decode_attn(h, layer, len(seq_ids), _i32arr(seq_ids), n_q_heads, _vp(q_ptr), softmax_scale,
                              _vp(out_ptr), _vp(ws_ptr), ws_bytes, _vp(stream))
    _check(rc, "kvq_decode_attn")


def kvq_append_decode(h, layer, seq_ids, n_new, k_ptr, v_ptr, n_q_heads, q_ptr, softmax_scale, out_ptr, ws_ptr,
                      ws_bytes, stream=0):
    rc = _lib.kvq_append_decode(h, layer, len(seq_ids), _i32arr(seq_ids), _i32arr(n_new), _vp(k_ptr), _vp(v_ptr),
                                n_q_heads, _vp(q_ptr), softmax_scale, _vp(out_ptr), _vp(ws_ptr), ws_bytes, _vp(stream))
    _check(rc, "kvq_append_decode")


def kvq_prefill_attn(h, layer, seq, n_q_tokens, n_q_heads, q_ptr, softmax_scale, out_ptr, ws_ptr, ws_bytes, stream=0):
    rc = _lib.kvq_prefill_attn(h, layer, seq, n_q_tokens, n_q_heads, _vp(q_ptr), softmax_scale, _vp(out_ptr),
                               _vp(ws_ptr), ws_bytes, _vp(stream))
    _check(rc, "kvq_prefill_attn")


def kvq_decode_attn_noalloc(h, layer, seq_ids, n_q_heads, q_ptr, softmax_scale, out_ptr, stream=0):
    rc = _lib.kvq_decode_attn_noalloc(h, layer, len(seq_ids), _i32arr(seq_ids), n_q_heads, _vp(q_ptr), softmax_scale,
                                      _vp(out_ptr), _vp(stream))
    _check(rc, "kvq_decode_attn_noalloc")


def kvq_rope_default_params(**overrides):
    p = kvq_rope_params()
    _lib.kvq_rope_default_params(C.byref(p))
    for k, v in overrides.items():
        if k == "sections":
            v = (_i32 * 4)(*v)
        setattr(p, k, v)
    return p


def kvq_rope(p, inv_freq, n_tokens, pos_ptr, pos_ld, n_q_heads, q_ptr, q_type, q_ld, q_out_ptr, q_out_type, q_out_ld,
             n_k_heads, k_ptr, k_ld, k_out_ptr, k_out_ld, stream=0):
    """inv_freq: None or a ctypes array of rot_dim / 2 doubles"""
    rc = _lib.kvq_rope(C.byref(p), inv_freq, n_tokens, _vp(pos_ptr), pos_ld, n_q_heads, _vp(q_ptr), q_type, q_ld,
                       _vp(q_out_ptr), q_out_type, q_out_ld, n_k_heads, _vp(k_ptr), k_ld, _vp(k_out_ptr), k_out_ld,
                       _vp(stream))
    _check(rc, "kvq_rope")


def kvq_batch_workspace_bytes(h, layer, seq_ids, n_q, n_q_heads):
    n = _sz()
    rc = _lib.kvq_batch_workspace_bytes(h, layer, len(seq_ids), _i32arr(seq_ids), _i32arr(n_q), n_q_heads, C.byref(n))
    _check(rc, "kvq_batch_workspace_bytes")
    return n.value


def kvq_batch_attn(h, layer, seq_ids, n_q, n_q_heads, causal, q_ptr, softmax_scale, out_ptr, lse_ptr, ws_ptr, ws_bytes,
                   stream=0):
    rc = _lib.kvq_batch_attn(h, layer, len(seq_ids), _i32arr(seq_ids), _i32arr(n_q), n_q_heads, int(causal),
                             _vp(q_ptr), softmax_scale, _vp(out_ptr), _vp(lse_ptr), _vp(ws_ptr), ws_bytes, _vp(stream))
    _check(rc, "kvq_batch_attn")


def kvq_attn_mass(h, layer, seq_ids, n_q, n_q_heads, causal, q_ptr, softmax_scale, lse_ptr, decay, mass_in_ptr,
                  mass_out_ptr, mass_ld, ws_ptr, ws_bytes, stream=0):
    rc = _lib.kvq_attn_mass(h, layer, len(seq_ids), _i32arr(seq_ids), _i32arr(n_q), n_q_heads, int(causal), _vp(q_ptr),
                            softmax_scale, _vp(lse_ptr), decay, _vp(mass_in_ptr), _vp(mass_out_ptr), mass_ld,
                            _vp(ws_ptr), ws_bytes, _vp(stream))
    _check(rc, "kvq_attn_mass")


def kvq_evict_workspace_bytes(src, dst, n_seqs, budget):
    n = _sz()
    _check(_lib.kvq_evict_workspace_bytes(src, dst, n_seqs, budget, C.byref(n)), "kvq_evict_workspace_bytes")
    return n.value


def kvq_evict(src, src_layer, dst, dst_layer, src_ids, dst_ids, mass_ptr, mass_ld, budget, sink, recent, kept_ptr,
              mass_out_ptr, mass_out_ld, ws_ptr, ws_bytes, stream=0):
    rc = _lib.kvq_evict(src, src_layer, dst, dst_layer, len(src_ids), _i32arr(src_ids), _i32arr(dst_ids),
                        _vp(mass_ptr), mass_ld, budget, sink, recent, _vp(kept_ptr), _vp(mass_out_ptr), mass_out_ld,
                        _vp(ws_ptr), ws_bytes, _vp(stream))
    _check(rc, "kvq_evict")


def kvq_dequant(h, layer, seq, which, t0, t1, basis, out_ptr, stream=0):
    _check(_lib.kvq_dequant(h, layer, seq, which, t0, t1, basis, _vp(out_ptr), _vp(stream)), "kvq_dequant")


def kvq_seq_len(h, layer, seq):
    n = _i64()
    _check(_lib.kvq_seq_len(h, layer, seq, C.byref(n)), "kvq_seq_len")
    return n.value


def kvq_seq_reset(h, seq):
    _check(_lib.kvq_seq_reset(h, seq), "kvq_seq_reset")


def kvq_locate(h, kind, layer, seq, page, head, which, token=0):
    off, nb = _sz(), _sz()
    _check(_lib.kvq_locate(h, kind, layer, seq, page, head, which, token, C.byref(off), C.byref(nb)), "kvq_locate")
    return off.value, nb.value


def kvq_get_status(h, stream=0):
    return _lib.kvq_get_status(h, _vp(stream))


def kvq_launch_count():
    n = C.c_uint64()
    _check(_lib.kvq_launch_count(C.byref(n)), "kvq_launch_count")
    return n.value


def kvq_describe(h):
    return _lib.kvq_describe(h).decode()


def _refuse(where, why, code=KVQ_E_INVAL):
    raise KVQError(code, f"{where}: {why}")


def _raw_stream_of(torch):
    """device index -> the cudaStream_t current on it (the same number as
    torch.cuda.current_stream(index).cuda_stream, without building the stream object)"""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw if raw is not None else lambda index: torch.cuda.current_stream(index).cuda_stream


class _On:
    """Makes a device and a stream current: outputs and workspace then come from the caching
    allocator under the stream the kernels run on, so calls on several streams, and captured graphs,
    each have their own."""

    def __init__(self, torch, device, stream):
        if stream is not None and stream.device != device:
            _refuse("stream", f"a stream of {stream.device} for tensors on {device}")
        self.both = [torch.cuda.device(device)] + ([] if stream is None else [torch.cuda.stream(stream)])

    def __enter__(self):
        for c in self.both:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.both):
            c.__exit__(*exc)


class Rope:
    """Rotary positions with several axes (kvq_rope): what a model fixes once.

    sections: channel pairs of each axis, in the order of the rows of `pos`; `turns`: the axes take
    turns pair by pair instead of following one another; `adjacent`: pairs (2i, 2i+1) instead of
    (i, i + rot_dim/2); inv_freq: rot_dim/2 frequencies instead of theta's.
    """

    def __init__(self, sections=(64,), theta=10000.0, rot_dim=None, turns=False, adjacent=False, inv_freq=None):
        import torch

        self.torch = torch
        sections = [int(x) for x in sections]
        if not 1 <= len(sections) <= 4:
            _refuse("Rope", "1 to 4 sections")
        rot_dim = 2 * sum(sections) if rot_dim is None else int(rot_dim)
        self.n_axes = len(sections)
        self._p = [kvq_rope_default_params(rot_dim=rot_dim, n_axes=self.n_axes,
                                           sections=sections + [0] * (4 - len(sections)), turns=int(turns),
                                           adjacent=int(adjacent), inverse=i, theta=float(theta)) for i in (0, 1)]
        self._ref = [C.byref(p) for p in self._p]
        # the host checks of the parameters, once: a call over no tokens
        kvq_rope(self._p[0], None, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
        half = rot_dim // 2
        f = [theta ** (-2.0 * i / rot_dim) for i in range(half)] if inv_freq is None else [float(x) for x in inv_freq]
        if len(f) != half:
            _refuse("Rope", "inv_freq holds rot_dim / 2 values")
        self._freq = (C.c_double * half)(*f)
        self._raw_stream = _raw_stream_of(torch)
        self._types = {torch.float32: KVQ_DT_F32, torch.bfloat16: KVQ_DT_BF16, torch.float16: KVQ_DT_F16}

    @staticmethod
    def _rows(x, n, dev, name):
        """(heads, pointer, row stride) of a [tokens, heads, 128] tensor with contiguous heads"""
        s, st = x.shape, x.stride()
        if len(s) != 3 or s[0] != n or s[2] != 128 or st[2] != 1 or (s[1] > 1 and st[1] != 128):
            _refuse("Rope.apply", f"{name} is [tokens, heads, 128] with contiguous heads")
        if x.get_device() != dev:
            _refuse("Rope.apply", f"{name} is on another device than pos")
        # (the row stride of a single token says nothing)
        return s[1], x.data_ptr(), st[0] if n > 1 else max(st[0], s[1] * 128)

    def apply(self, pos, q=None, k=None, q_dtype=None, inverse=False, q_out=None, k_out=None, stream=None):
        """pos: int32 [n_axes, tokens] (or [tokens] for one axis; one row expanded over the axes is
        read as it is); q: [tokens, heads, 128] fp32, BF16
        or F16, a slice of a packed row allowed; k: BF16 likewise.  Returns (q_out, k_out), new
        contiguous tensors (q of q_dtype, its own type by default) unless given; an output may be its
        input."""
        torch = self.torch
        dev = pos.get_device()
        if dev < 0:
            _refuse("Rope.apply", "tensors are on a CUDA device")
        if stream is not None or torch.cuda.current_device() != dev:
            with _On(torch, pos.device, stream):
                return self.apply(pos, q, k, q_dtype, inverse, q_out, k_out)
        shape = pos.shape
        if len(shape) == 1:
            pos, shape = pos[None], (1, shape[0])
        n = shape[1]
        if pos.dtype is not torch.int32 or len(shape) != 2 or shape[0] != self.n_axes or (n > 1 and pos.stride(1) != 1):
            _refuse("Rope.apply", "pos is int32 [n_axes, tokens], the tokens contiguous")
        pos_ld = pos.stride(0) if self.n_axes > 1 else n  # (0: a row expanded over the axes)
        a, b = (0, 0, 0, 0, 0, 0, 0), (0, 0, 0, 0, 0)
        if q is not None:
            h, ptr, ld = self._rows(q, n, dev, "q")
            if q_out is None:
                q_out = torch.empty_like(q, dtype=q_dtype, memory_format=torch.contiguous_format)
                ho, ptr_o, ld_o = h, q_out.data_ptr(), h * 128
            else:
                ho, ptr_o, ld_o = self._rows(q_out, n, dev, "q_out")
            ti, to = self._types.get(q.dtype), self._types.get(q_out.dtype)
            if ti is None or to is None or (q_dtype is not None and q_out.dtype is not q_dtype):
                _refuse("Rope.apply", "type of q", KVQ_E_UNSUPPORTED)
            if ho != h:
                _refuse("Rope.apply", "q_out has q's heads")
            a = (h, ptr, ti, ld, ptr_o, to, ld_o)
        if k is not None:
            h, ptr, ld = self._rows(k, n, dev, "k")
            if k_out is None:
                k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
                ho, ptr_o, ld_o = h, k_out.data_ptr(), h * 128
            else:
                ho, ptr_o, ld_o = self._rows(k_out, n, dev, "k_out")
            if k.dtype is not torch.bfloat16 or k_out.dtype is not torch.bfloat16:
                _refuse("Rope.apply", "k is BF16", KVQ_E_UNSUPPORTED)
            if ho != h:
                _refuse("Rope.apply", "k_out has k's heads")
            b = (h, ptr, ld, ptr_o, ld_o)
        rc = _lib.kvq_rope(self._ref[1 if inverse else 0], self._freq, n, pos.data_ptr(), pos_ld, *a, *b,
                           self._raw_stream(dev))
        if rc:
            raise KVQError(rc, "kvq_rope")
        return q_out, k_out


class KVCache:
    """A cache whose storage and workspace are torch tensors on one CUDA device.

    PyTorch supplies the device memory and the stream; every call goes straight to the
    C ABI with the tensors' pointers.
    """

    def __init__(self, device=None, **params):
        import torch

        self.torch = torch
        self.params = kvq_default_params(**params)
        self.nbytes = kvq_cache_bytes(self.params)
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.storage = torch.empty(self.nbytes, dtype=torch.uint8, device=self.device)
        with torch.cuda.device(self.device):
            self.handle = kvq_cache_create(self.params, self.storage.data_ptr(), self.nbytes)
        self._index = self.storage.get_device()
        self._t16 = torch.float16 if self.params.tail_f16 else torch.bfloat16
        self._raw_stream = _raw_stream_of(torch)
        self._rows16 = {}  # layer -> view
        self._ws = None
        self._ws_bytes = {}  # (n_seqs, n_q_heads) -> kvq_workspace_bytes

    def __del__(self, destroy=_lib.kvq_cache_destroy):  # (this module's names are gone when the interpreter ends)
        h = getattr(self, "handle", None)
        if h:
            destroy(h)
            self.handle = None

    def _stream(self, stream):
        if stream is None:
            stream = self.torch.cuda.current_stream(self.device)
        return stream.cuda_stream

    def append(self, layer, seq_ids, n_new, k, v, stream=None):
        assert k.dtype == self.torch.bfloat16 and v.dtype == self.torch.bfloat16
        assert k.is_contiguous() and v.is_contiguous()
        kvq_append(self.handle, layer, list(seq_ids), list(n_new), k.data_ptr(), v.data_ptr(), self._stream(stream))

    def workspace(self, n_seqs, n_q_heads):
        key = (n_seqs, n_q_heads)
        nb = self._ws_bytes.get(key)
        if nb is None:
            nb = self._ws_bytes[key] = kvq_workspace_bytes(self.handle, n_seqs, n_q_heads)
        if self._ws is None or self._ws.numel() < nb:
            self._ws = self.torch.empty(max(nb, 256), dtype=self.torch.uint8, device=self.device)
        return self._ws

    def decode(self, layer, seq_ids, q, out=None, softmax_scale=0.0, stream=None):
        assert q.dtype == self.torch.float32 and q.is_contiguous()
        n_seqs, n_q_heads = q.shape[0], q.shape[1]
        if out is None:
            out = self.torch.empty_like(q)
        ws = self.workspace(n_seqs, n_q_heads)
        kvq_decode_attn(self.handle, layer, list(seq_ids), n_q_heads, q.data_ptr(), softmax_scale, out.data_ptr(),
                        ws.data_ptr(), ws.numel(), self._stream(stream))
        return out

    def append_decode(self, layer, seq_ids, n_new, k, v, q, out=None, softmax_scale=0.0, stream=None):
        """kvq_append_decode: append n_new[i] rows to seq_ids[i], then decode q (row i for
        seq_ids[i]) over the grown cache, the decode overlapping the append."""
        assert k.dtype == self.torch.bfloat16 and v.dtype == self.torch.bfloat16
        assert k.is_contiguous() and v.is_contiguous()
        assert q.dtype == self.torch.float32 and q.is_contiguous()
        n_seqs, n_q_heads = q.shape[0], q.shape[1]
        if out is None:
            out = self.torch.empty_like(q)
        ws = self.workspace(n_seqs, n_q_heads)
        kvq_append_decode(self.handle, layer, list(seq_ids), list(n_new), k.data_ptr(), v.data_ptr(), n_q_heads,
                          q.data_ptr(), softmax_scale, out.data_ptr(), ws.data_ptr(), ws.numel(), self._stream(stream))
        return out

    def prefill_attn(self, layer, seq, q, out=None, softmax_scale=0.0, stream=None):
        """kvq_prefill_attn: q [n_q_tokens, n_q_heads, 128] fp32, causal over the chunk of the
        sequence's newest n_q_tokens tokens."""
        assert q.dtype == self.torch.float32 and q.is_contiguous()
        n_q, n_q_heads = q.shape[0], q.shape[1]
        if out is None:
            out = self.torch.empty_like(q)
        ws = self.workspace(n_q, n_q_heads)
        kvq_prefill_attn(self.handle, layer, seq, n_q, n_q_heads, q.data_ptr(), softmax_scale, out.data_ptr(),
                         ws.data_ptr(), ws.numel(), self._stream(stream))
        return out

    def rows16(self, layer):
        """The 16-bit rows of a layer, a view of the storage [n_seqs, n_kv_heads, 2 (K, V), ring rows, 128]
        in the tail's type: token p of a sequence in row p mod the ring rows."""
        x = self._rows16.get(layer)
        if x is None:
            torch, p = self.torch, self.params
            kvarn = any(8 <= t <= 13 or (p.var_norm and t != 0) for t in (p.type_k, p.type_v))
            rows = p.max_ctx if p.type_k == 0 else p.tail + (256 if kvarn else 0)
            if rows == 0:
                _refuse("rows16", "a cache without a 16-bit tail")
            off, _ = kvq_locate(self.handle, 1, layer, 0, 0, 0, 0, 0)
            n = p.n_seqs * p.n_kv_heads * 2 * rows * 128
            x = self.storage[off:off + 2 * n].view(self._t16).view(p.n_seqs, p.n_kv_heads, 2, rows, 128)
            self._rows16[layer] = x
        return x

    def _elsewhere(self, stream):
        """Whether a stream or device other than the current one has to be made current (_on)."""
        return stream is not None or self.torch.cuda.current_device() != self._index

    def _on(self, stream):
        return _On(self.torch, self.storage.device, stream)

    def _queries(self, where, q, n_q):
        s = q.shape
        if q.dtype is not self._t16:
            _refuse(where, "q is in the cache's 16-bit type (BF16, or F16 with tail_f16)", KVQ_E_UNSUPPORTED)
        if len(s) != 3 or s[2] != 128 or s[0] != sum(n_q) or not q.is_contiguous():
            _refuse(where, "q is contiguous [sum(n_q), n_q_heads, 128]")
        if q.get_device() != self._index:
            _refuse(where, "q is on another device than the cache")
        return s[0], s[1]

    def _lse(self, where, lse, rows, hq):
        if lse.dtype is not self.torch.float32 or lse.shape != (rows, hq) or not lse.is_contiguous() or \
                lse.get_device() != self._index:
            _refuse(where, "lse is contiguous fp32 [sum(n_q), n_q_heads] on the cache's device")

    def _mass_rows(self, where, x, n, name):
        s = x.shape
        if x.dtype is not self.torch.float32 or len(s) != 3 or s[0] != n or s[1] != self.params.n_kv_heads or \
                not x.is_contiguous() or x.get_device() != self._index:
            _refuse(where, f"{name} is contiguous fp32 [sequences, n_kv_heads, tokens] on the cache's device")
        return s[2]

    def _batch_workspace(self, layer, n, ids, nq, hq):
        """(the tensor that owns it or None, pointer, bytes)"""
        size = _sz()  # of this call: the library runs without the interpreter's lock
        rc = _lib.kvq_batch_workspace_bytes(self.handle, layer, n, ids, nq, hq, C.byref(size))
        if rc:
            raise KVQError(rc, "kvq_batch_workspace_bytes")
        nb = size.value
        if nb == 0:
            return None, 0, 0
        ws = self.torch.empty(nb, dtype=self.torch.uint8, device=self.storage.device)
        return ws, ws.data_ptr(), nb

    def batch_attn(self, layer, seq_ids, n_q, q, causal=False, out=None, lse=None, return_lse=False, softmax_scale=0.0,
                   stream=None):
        """kvq_batch_attn: q [sum(n_q), n_q_heads, 128] in the cache's 16-bit type, n_q[i] query tokens
        over sequence seq_ids[i]; every token seen (cross attention), or causal over the newest n_q[i].
        Returns out, or (out, lse [sum(n_q), n_q_heads] fp32) with return_lse or a given lse."""
        torch = self.torch
        if self._elsewhere(stream):
            with self._on(stream):
                return self.batch_attn(layer, seq_ids, n_q, q, causal, out, lse, return_lse, softmax_scale)
        n = len(seq_ids)
        if n != len(n_q):
            _refuse("batch_attn", "one n_q for each sequence")
        rows, hq = self._queries("batch_attn", q, n_q)
        if out is None:
            out = torch.empty_like(q)
        elif out.shape != q.shape or out.dtype is not q.dtype or not out.is_contiguous() or \
                out.get_device() != self._index:
            _refuse("batch_attn", "out has q's shape, type and device")
        if lse is not None:
            self._lse("batch_attn", lse, rows, hq)
        elif return_lse:
            lse = q.new_empty((rows, hq), dtype=torch.float32)
        ids, nq = _i32arr(seq_ids), _i32arr(n_q)
        ws, ptr, nb = self._batch_workspace(layer, n, ids, nq, hq)
        rc = _lib.kvq_batch_attn(self.handle, layer, n, ids, nq, hq, 1 if causal else 0, q.data_ptr(), softmax_scale,
                                 out.data_ptr(), 0 if lse is None else lse.data_ptr(), ptr, nb,
                                 self._raw_stream(self._index))
        if rc:
            raise KVQError(rc, "kvq_batch_attn")
        return out if lse is None else (out, lse)

    def attn_mass(self, layer, seq_ids, n_q, q, lse, causal=False, decay=1.0, mass_in=None, mass_out=None,
                  softmax_scale=0.0, stream=None):
        """kvq_attn_mass: the weight each cached token gets from these query rows (lse as batch_attn
        returned it), summed over the query heads of its KV head, on top of decay * mass_in.
        mass_in, mass_out: fp32 [len(seq_ids), n_kv_heads, tokens >= the longest sequence]; mass_out
        defaults to a new tensor (zeros behind each sequence); both may be one tensor."""
        torch = self.torch
        if self._elsewhere(stream):
            with self._on(stream):
                return self.attn_mass(layer, seq_ids, n_q, q, lse, causal, decay, mass_in, mass_out, softmax_scale)
        n = len(seq_ids)
        if n != len(n_q):
            _refuse("attn_mass", "one n_q for each sequence")
        rows, hq = self._queries("attn_mass", q, n_q)
        self._lse("attn_mass", lse, rows, hq)
        if mass_in is None:
            decay = 0.0
        else:
            self._mass_rows("attn_mass", mass_in, n, "mass_in")
        if mass_out is None:
            most = max([self.seq_len(layer, s) for s in seq_ids] + [1])
            shape = (n, self.params.n_kv_heads, most) if mass_in is None else mass_in.shape
            mass_out = torch.zeros(shape, dtype=torch.float32, device=q.device)
        ld = self._mass_rows("attn_mass", mass_out, n, "mass_out")
        if mass_in is not None and mass_in.shape != mass_out.shape:
            _refuse("attn_mass", "mass_in has mass_out's shape")
        ids, nq = _i32arr(seq_ids), _i32arr(n_q)
        ws, ptr, nb = self._batch_workspace(layer, n, ids, nq, hq)
        rc = _lib.kvq_attn_mass(self.handle, layer, n, ids, nq, hq, 1 if causal else 0, q.data_ptr(), softmax_scale,
                                lse.data_ptr(), decay, 0 if mass_in is None else mass_in.data_ptr(),
                                mass_out.data_ptr(), ld, ptr, nb, self._raw_stream(self._index))
        if rc:
            raise KVQError(rc, "kvq_attn_mass")
        return mass_out

    def evict(self, dst, layer, dst_layer, seq_ids, dst_ids, mass, budget, sink=0, recent=0, kept=None, mass_out=None,
              stream=None):
        """kvq_evict: sequences dst_ids of the cache `dst` (any type) become the `budget` tokens that
        matter of this BF16 cache's seq_ids: per KV head the first `sink`, the last `recent` and those
        with the largest mass [len(seq_ids), n_kv_heads, tokens] of the others.  Returns (kept int32
        [len(seq_ids), n_kv_heads, budget], -1 behind the last; mass_out fp32 of the same shape, zeros
        behind the last)."""
        torch = self.torch
        if self._elsewhere(stream):
            with self._on(stream):
                return self.evict(dst, layer, dst_layer, seq_ids, dst_ids, mass, budget, sink, recent, kept, mass_out)
        n, hkv = len(seq_ids), self.params.n_kv_heads
        if len(dst_ids) != n:
            _refuse("evict", "one destination for each sequence")
        if budget < 0:
            _refuse("evict", "a budget below 0")
        ld = self._mass_rows("evict", mass, n, "mass")
        shape = (n, hkv, budget)
        if kept is None:
            kept = mass.new_empty(shape, dtype=torch.int32)
        elif kept.dtype is not torch.int32 or kept.shape != shape or not kept.is_contiguous() or \
                kept.get_device() != self._index:
            _refuse("evict", "kept is contiguous int32 [sequences, n_kv_heads, budget] on the cache's device")
        if mass_out is None:
            mass_out = mass.new_empty(shape)
            out_ld = budget
        else:
            out_ld = self._mass_rows("evict", mass_out, n, "mass_out")
        ptr = nb = 0
        if dst.params.type_k != 0:
            size = _sz()
            rc = _lib.kvq_evict_workspace_bytes(self.handle, dst.handle, n, budget, C.byref(size))
            if rc:
                raise KVQError(rc, "kvq_evict_workspace_bytes")
            nb = size.value
            ws = mass.new_empty(nb, dtype=torch.uint8)
            ptr = ws.data_ptr()
        rc = _lib.kvq_evict(self.handle, layer, dst.handle, dst_layer, n, _i32arr(seq_ids), _i32arr(dst_ids),
                            mass.data_ptr(), ld, budget, sink, recent, kept.data_ptr(), mass_out.data_ptr(), out_ld,
                            ptr, nb, self._raw_stream(self._index))
        if rc:
            raise KVQError(rc, "kvq_evict")
        return kept, mass_out

    def dequant(self, layer, seq, which, t0, t1, basis=0, out=None, stream=None):
        if out is None:
            out = self.torch.empty((t1 - t0, self.params.n_kv_heads, 128), dtype=self.torch.float32, device=self.device)
        kvq_dequant(self.handle, layer, seq, which, t0, t1, basis, out.data_ptr(), self._stream(stream))
        return out

    def seq_len(self, layer, seq):
        return kvq_seq_len(self.handle, layer, seq)

    def reset(self, seq):
        kvq_seq_reset(self.handle, seq)

    def locate(self, kind, layer, seq, page, head, which, token=0):
        return kvq_locate(self.handle, kind, layer, seq, page, head, which, token)

    def status(self, stream=None):
        return kvq_get_status(self.handle, self._stream(stream))

    def describe(self):
        return kvq_describe(self.handle)
