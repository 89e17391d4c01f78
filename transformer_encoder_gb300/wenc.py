"""Thin ctypes binding of libwenc.so (argument marshalling only).

Every step of the encoder runs in the library's CUDA kernels; this module only turns
PyTorch tensors (used here for device memory and streams) into the pointers and sizes
of the C ABI declared in include/wenc.h, and turns non-OK statuses into exceptions.
There is no fallback: if the library is missing or the device is not sm_103a, calls raise.

A call with ``stream=`` (a torch stream or a raw handle) runs there, and tensors that it makes come from that
stream's allocator: a caller that uses them on another stream orders the two streams and, before the tensor
is dropped, calls its ``record_stream``, as for any tensor made on another stream.
"""
from __future__ import annotations

import ctypes
import os
import struct

__all__ = [
    "WencError", "lib", "lib_path", "Encoder", "attention", "attention_tf32", "layernorm", "linear", "linear_tf32",
    "sync_status", "selftest_gemm_pair_abort", "EPI_BIAS_BF16", "EPI_BIAS_GELU_BF16", "EPI_BIAS_RESID_F32", "LN_OUT_F32", "LN_OUT_BF16",
    "LN_OUT_TF32", "PREC_BF16", "PREC_TF32", "EXPORTED_SYMBOLS", "prefix_attention", "kv_append", "quantize_rows",
    "linear_i8",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
# WENC_LIBRARY may name another library built in-tree into _lib/ (the index-checked
# libwenc_bounds.so); anything outside _lib/ is refused.
lib_path = os.path.join(_PKG, "_lib", os.path.basename(os.environ.get("WENC_LIBRARY") or "libwenc.so"))

EPI_BIAS_BF16, EPI_BIAS_GELU_BF16, EPI_BIAS_RESID_F32 = 0, 1, 2
LN_OUT_F32, LN_OUT_BF16, LN_OUT_TF32 = 0, 1, 2
PREC_BF16, PREC_TF32 = 0, 1
_STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "OOM", 4: "CUDA", 5: "DEVICE_TIMEOUT"}
LAUNCH_KINDS = {0: "layernorm", 1: "gemm_qkv", 2: "attention", 3: "gemm_out", 4: "gemm_fc1", 5: "gemm_fc2",
                6: "layernorm_final", 7: "copy", 8: "attention_combine", 9: "stem_unfold", 10: "gemm_conv1",
                11: "gemm_conv2", 12: "cross_kv_cast", 13: "gemm_cross_kv", 14: "row_stats"}

EXPORTED_SYMBOLS = (
    "wenc_create", "wenc_forward", "wenc_forward_layers", "wenc_forward_launches", "wenc_set_launch_events",
    "wenc_attention", "wenc_layernorm", "wenc_linear", "wenc_sync_status", "wenc_destroy", "wenc_last_error",
    "wenc_version", "wenc_selftest_wait_timeout", "wenc_attention_static", "wenc_attention_static_capacity",
    "wenc_linear_tf32", "wenc_attention_tf32", "wenc_set_stem", "wenc_stem", "wenc_encode", "wenc_encode_launches",
    "wenc_set_cross_kv", "wenc_cross_kv", "wenc_selftest_gemm_schedule", "wenc_selftest_gemm_pair_abort",
    "wenc_set_device_alloc_limit", "wenc_device_bytes_held", "wenc_selftest_attention_abort",
    "wenc_prefix_attention", "wenc_prefix_attention_workspace", "wenc_kv_append", "wenc_quantize_rows",
    "wenc_linear_i8", "wenc_linear_i8_workspace", "wenc_selftest_append_sequence", "wenc_selftest_append_angle",
    "wenc_selftest_attention_runs",
)


class WencError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"wenc {_STATUS.get(status, status)}: {message}")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("d_model", ctypes.c_int), ("n_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("ffn_dim", ctypes.c_int), ("seq_len", ctypes.c_int),
                ("max_batch", ctypes.c_int), ("final_ln", ctypes.c_int), ("ln_eps", ctypes.c_float),
                ("weight_dtype", ctypes.c_int), ("precision", ctypes.c_int)]


_LW_FIELDS = ("ln1_w", "ln1_b", "wq", "bq", "wk", "bk", "wv", "bv", "wo", "bo", "ln2_w", "ln2_b", "w1", "b1", "w2", "b2")


class LayerWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _LW_FIELDS]


STEM_KEYS = ("conv1_w", "conv1_b", "conv2_w", "conv2_b", "positions")


class StemWeights(ctypes.Structure):
    _fields_ = [("n_mels", ctypes.c_int)] + [(n, ctypes.c_void_p) for n in STEM_KEYS]


class KvAppendArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("n_tokens", ctypes.c_int), ("n_seqs", ctypes.c_int),
                ("n_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("k_page_stride", ctypes.c_int64), ("v_page_stride", ctypes.c_int64), ("n_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int64),
                ("max_pages", ctypes.c_int), ("lens", ctypes.c_void_p), ("seq_start", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int)]


class PrefixAttentionArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("n_seqs", ctypes.c_int), ("q_len", ctypes.c_int), ("n_heads", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("q", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
                ("n_groups", ctypes.c_int), ("max_group", ctypes.c_int), ("group_start", ctypes.c_void_p),
                ("k_prefix", ctypes.c_void_p), ("v_prefix", ctypes.c_void_p), ("k_group_stride", ctypes.c_int64),
                ("k_token_stride", ctypes.c_int64), ("v_group_stride", ctypes.c_int64),
                ("v_token_stride", ctypes.c_int64), ("prefix_max", ctypes.c_int), ("prefix_lens", ctypes.c_void_p),
                ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("k_page_stride", ctypes.c_int64),
                ("v_page_stride", ctypes.c_int64), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int64), ("max_pages", ctypes.c_int),
                ("lens", ctypes.c_void_p), ("scale", ctypes.c_float), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


# The same structures as one pack() each: a decode step makes these calls for every layer and token,
# and a ctypes field assignment each costs more there than everything else in the call.
_PREFIX_PACK = struct.Struct("@6i2P2q2i3P4qi3P2q2iPqiPfPN")
_APPEND_PACK = struct.Struct("@6i4P4q2P2q2iPqi4P2i")
assert _PREFIX_PACK.size == ctypes.sizeof(PrefixAttentionArgs) - ctypes.sizeof(PrefixAttentionArgs) % 8
assert _APPEND_PACK.size == ctypes.sizeof(KvAppendArgs)

_lib = None


def lib() -> ctypes.CDLL:
    """Load libwenc.so (built in-tree by transformer_encoder_gb300.build); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise RuntimeError(f"{lib_path} is missing: build it with `python -m transformer_encoder_gb300.build`")
        L = ctypes.CDLL(lib_path)
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        L.wenc_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(LayerWeights), vp, vp, vp, ctypes.POINTER(vp)]
        L.wenc_forward.argtypes = [vp, vp, vp, i, vp]
        L.wenc_forward_layers.argtypes = [vp, vp, vp, i, i, i, i, vp]
        L.wenc_forward_launches.argtypes = [vp, i, i, i]
        L.wenc_set_launch_events.argtypes = [vp, ctypes.POINTER(vp), i, ctypes.POINTER(i)]
        L.wenc_attention.argtypes = [vp, vp, vp, vp, i, i, i, i, vp]
        L.wenc_layernorm.argtypes = [vp, vp, vp, vp, i, i, f, i, vp]
        L.wenc_linear.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, vp]
        L.wenc_linear_tf32.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, vp]
        L.wenc_set_stem.argtypes = [vp, ctypes.POINTER(StemWeights), vp]
        L.wenc_stem.argtypes = [vp, vp, vp, i, vp]
        L.wenc_encode.argtypes = [vp, vp, vp, i, vp]
        L.wenc_encode_launches.argtypes = [vp]
        L.wenc_set_cross_kv.argtypes = [vp, i, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp), vp]
        L.wenc_cross_kv.argtypes = [vp, vp, vp, i, vp]
        L.wenc_attention_tf32.argtypes = [vp, vp, vp, vp, i, i, i, i, vp]
        L.wenc_sync_status.argtypes = [vp]
        L.wenc_selftest_wait_timeout.argtypes = [vp]
        L.wenc_selftest_gemm_pair_abort.argtypes = [vp, vp, vp, vp, i, i, i, i, vp]
        L.wenc_selftest_attention_abort.argtypes = [vp, vp, vp, vp, i, i, i, i, vp]
        L.wenc_set_device_alloc_limit.argtypes = [ctypes.c_size_t]
        L.wenc_set_device_alloc_limit.restype = None
        L.wenc_device_bytes_held.argtypes = []
        L.wenc_device_bytes_held.restype = ctypes.c_size_t
        ip = ctypes.POINTER(ctypes.c_int)
        L.wenc_selftest_gemm_schedule.argtypes = [i, i, i, i, ip, i, ip, ip, ip]
        L.wenc_attention_static.argtypes = [vp, vp, vp, vp, i, i, i, i, vp]
        L.wenc_attention_static.restype = ctypes.c_int
        L.wenc_attention_static_capacity.argtypes = []
        L.wenc_attention_static_capacity.restype = ctypes.c_size_t
        # (pointers to the argument structures: a byref() of one, or its packed bytes)
        L.wenc_prefix_attention.argtypes = [vp, vp]
        L.wenc_prefix_attention_workspace.argtypes = [vp]
        L.wenc_prefix_attention_workspace.restype = ctypes.c_size_t
        L.wenc_kv_append.argtypes = [vp, vp]
        L.wenc_quantize_rows.argtypes = [vp, i, vp, vp, i, i, vp]
        L.wenc_linear_i8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, vp, ctypes.c_size_t, vp]
        L.wenc_linear_i8_workspace.argtypes = [i, i, i]
        L.wenc_linear_i8_workspace.restype = ctypes.c_size_t
        L.wenc_selftest_append_sequence.argtypes = [vp, i, i, i, i, ip]
        L.wenc_selftest_append_sequence.restype = ctypes.c_int
        L.wenc_selftest_append_angle.argtypes = [ctypes.c_float, i, vp, vp]
        L.wenc_selftest_append_angle.restype = None
        L.wenc_selftest_attention_runs.argtypes = [i, vp, i, i, vp]
        L.wenc_selftest_attention_runs.restype = None
        L.wenc_destroy.argtypes = [vp]
        L.wenc_destroy.restype = None
        L.wenc_last_error.restype = ctypes.c_char_p
        L.wenc_version.restype = ctypes.c_char_p
        for name in ("wenc_create", "wenc_forward", "wenc_forward_layers", "wenc_set_launch_events", "wenc_attention",
                     "wenc_layernorm", "wenc_linear", "wenc_sync_status", "wenc_forward_launches",
                     "wenc_selftest_wait_timeout", "wenc_linear_tf32", "wenc_attention_tf32", "wenc_set_stem",
                     "wenc_stem", "wenc_encode", "wenc_encode_launches", "wenc_set_cross_kv", "wenc_cross_kv",
                     "wenc_selftest_gemm_schedule", "wenc_selftest_gemm_pair_abort", "wenc_selftest_attention_abort",
                     "wenc_prefix_attention", "wenc_kv_append", "wenc_quantize_rows", "wenc_linear_i8"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        raise WencError(status, lib().wenc_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _on(stream):
    """The given stream (a torch stream or a raw handle) as torch's current one."""
    import torch
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(
        stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)))


def _empty(shape, dtype, device, stream):
    """A new tensor (an output, a workspace) from the allocator of the stream the call runs on: its block was
    last used, and will be used again, in that stream's order, and is a graph's own while one is captured."""
    torch = _torch or _load_torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _require(t, dtype, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class Encoder:
    """A wenc handle: packed resident weights plus a workspace for `max_batch` windows.

    ``layers`` is a list of dicts with the keys of ``synth.LAYER_KEYS`` holding CUDA tensors
    (matrices float32 or bfloat16 [n_out, n_in], vectors float32). The library copies and
    packs them, so they may be freed after construction. ``precision`` is "bf16" (bf16
    tensor-core operands) or "tf32" (TF32 operands, fp32 activations).
    """

    def __init__(self, layers, n_heads: int, seq_len: int, max_batch: int, final=None, ln_eps: float = 1e-5,
                 stream=None, precision: str = "bf16"):
        import torch
        L = lib()
        d = layers[0]["wq"].shape[0]
        f = layers[0]["w1"].shape[0]
        mdtype = layers[0]["wq"].dtype
        if mdtype not in (torch.float32, torch.bfloat16):
            raise TypeError("weight matrices must be float32 or bfloat16")
        if precision not in ("bf16", "tf32"):
            raise ValueError(f"precision must be 'bf16' or 'tf32', got {precision!r}")
        cfg = Config(len(layers), d, n_heads, d // n_heads, f, seq_len, max_batch, 1 if final is not None else 0,
                     ln_eps, 1 if mdtype == torch.bfloat16 else 0, PREC_TF32 if precision == "tf32" else PREC_BF16)
        self.precision = precision
        self.n_dec = 0  # decoder layers of the cross K/V weights (set_cross_kv)
        arr = (LayerWeights * len(layers))()
        for i, p in enumerate(layers):
            for k in ("wq", "wk", "wv", "wo", "w1", "w2"):
                _require(p[k], mdtype, k)
            for k in ("ln1_w", "ln1_b", "bq", "bv", "bo", "ln2_w", "ln2_b", "b1", "b2"):
                _require(p[k], torch.float32, k)
            for k in _LW_FIELDS:
                setattr(arr[i], k, None if k == "bk" else p[k].data_ptr())
        lnf_w = lnf_b = None
        if final is not None:
            _require(final[0], torch.float32, "lnf_w")
            _require(final[1], torch.float32, "lnf_b")
            lnf_w, lnf_b = _ptr(final[0]), _ptr(final[1])
        h = ctypes.c_void_p()
        _check(L.wenc_create(ctypes.byref(cfg), arr, lnf_w, lnf_b, _stream(stream), ctypes.byref(h)))
        self._h = h
        self.cfg = cfg
        self.d_model, self.ffn_dim, self.n_layers, self.seq_len, self.max_batch = d, f, len(layers), seq_len, max_batch

    @property
    def handle(self):
        return self._h

    def forward(self, x, out=None, stream=None):
        """out = Encoder(x), x float32 CUDA [B, seq_len, d]; out may be x (in place)."""
        return self.forward_layers(x, out, 0, self.n_layers, True, stream)

    def forward_layers(self, x, out=None, first: int = 0, count: int | None = None, final_ln: bool = True,
                       stream=None):
        import torch
        _require(x, torch.float32, "x")
        if count is None:
            count = self.n_layers - first
        if out is None:
            out = _empty(x.shape, x.dtype, x.device, stream)
        _require(out, torch.float32, "out")
        B = x.shape[0]
        _check(lib().wenc_forward_layers(self._h, _ptr(x), _ptr(out), B, first, count, int(final_ln), _stream(stream)))
        return out

    def set_stem(self, stem: dict, stream=None):
        """Attach the convolutional stem: ``stem`` has the keys of ``STEM_KEYS`` as CUDA tensors
        (conv weights [d, C_in, 3] in the layers' matrix dtype, biases [d] and positions
        [seq_len, d] float32); n_mels is read from conv1_w."""
        import torch
        mdtype = torch.bfloat16 if self.cfg.weight_dtype == 1 else torch.float32
        _require(stem["conv1_w"], mdtype, "conv1_w")
        _require(stem["conv2_w"], mdtype, "conv2_w")
        for k in ("conv1_b", "conv2_b", "positions"):
            _require(stem[k], torch.float32, k)
        self.n_mels = int(stem["conv1_w"].shape[1])
        w = StemWeights(self.n_mels, *[stem[k].data_ptr() for k in STEM_KEYS])
        _check(lib().wenc_set_stem(self._h, ctypes.byref(w), _stream(stream)))

    def stem(self, mel, out=None, stream=None):
        """hidden [B, seq_len, d] = stem(mel), mel float32 CUDA [B, 2*seq_len, n_mels]."""
        import torch
        _require(mel, torch.float32, "mel")
        if out is None:
            out = _empty((mel.shape[0], self.seq_len, self.d_model), torch.float32, mel.device, stream)
        _require(out, torch.float32, "out")
        _check(lib().wenc_stem(self._h, _ptr(mel), _ptr(out), mel.shape[0], _stream(stream)))
        return out

    def encode(self, mel, out=None, stream=None):
        """The whole encoder from log-mel frames: stem, blocks and the final LayerNorm."""
        import torch
        _require(mel, torch.float32, "mel")
        if out is None:
            out = _empty((mel.shape[0], self.seq_len, self.d_model), torch.float32, mel.device, stream)
        _require(out, torch.float32, "out")
        _check(lib().wenc_encode(self._h, _ptr(mel), _ptr(out), mel.shape[0], _stream(stream)))
        return out

    def set_cross_kv(self, dec_layers, stream=None):
        """Attach the decoder's cross-attention K/V weights: a list (one per decoder layer) of
        dicts with wk, wv ([d, d], the layers' matrix dtype) and bv ([d] float32) CUDA tensors."""
        import torch
        mdtype = torch.bfloat16 if self.cfg.weight_dtype == 1 else torch.float32
        n = len(dec_layers)
        for p in dec_layers:
            _require(p["wk"], mdtype, "wk")
            _require(p["wv"], mdtype, "wv")
            _require(p["bv"], torch.float32, "bv")
        arr = lambda key: (ctypes.c_void_p * n)(*[p[key].data_ptr() for p in dec_layers])
        wk, wv, bv = arr("wk"), arr("wv"), arr("bv")
        _check(lib().wenc_set_cross_kv(self._h, n, wk, wv, bv, _stream(stream)))
        self.n_dec = n

    def cross_kv(self, enc_out, out=None, stream=None):
        """[2 n_dec, B * seq_len, d] cross K/V planes (K of layer l at 2l, V at 2l + 1) of an
        encoder output float32 [B, seq_len, d]; bf16 for the bf16 precision, float32 for TF32."""
        import torch
        _require(enc_out, torch.float32, "enc_out")
        B = enc_out.shape[0]
        dt = torch.float32 if self.precision == "tf32" else torch.bfloat16
        if self.n_dec == 0:  # the library reports the missing weights
            _check(lib().wenc_cross_kv(self._h, _ptr(enc_out), None, B, _stream(stream)))
        if out is None:
            out = _empty((2 * self.n_dec, B * self.seq_len, self.d_model), dt, enc_out.device, stream)
        _require(out, dt, "out")
        _check(lib().wenc_cross_kv(self._h, _ptr(enc_out), _ptr(out), B, _stream(stream)))
        return out

    def encode_launches(self) -> int:
        return lib().wenc_encode_launches(self._h)

    def launches(self, first: int = 0, count: int | None = None, final_ln: bool = True) -> int:
        count = self.n_layers - first if count is None else count
        return lib().wenc_forward_launches(self._h, first, count, int(final_ln))

    def set_launch_events(self, events, want_kinds: bool = True):
        """Arm the per-launch timing hook for the next forward call (torch.cuda.Event list)."""
        n = len(events)
        ev = (ctypes.c_void_p * n)(*[e.cuda_event for e in events])
        kinds = (ctypes.c_int * n)() if want_kinds else None
        self._ev_keep = (ev, kinds)
        _check(lib().wenc_set_launch_events(self._h, ev, n, kinds))
        return kinds

    def sync_status(self):
        _check(lib().wenc_sync_status(self._h))

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().wenc_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def attention(q, k, v, out=None, stream=None):
    """out = softmax(q k^T / 8) v per (window, head); q, k, v bf16 CUDA [B, T, H, 64]."""
    import torch
    for n, t in (("q", q), ("k", k), ("v", v)):
        _require(t, torch.bfloat16, n)
    B, T, H, hd = q.shape
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _require(out, torch.bfloat16, "out")
    _check(lib().wenc_attention(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, T, H, hd, _stream(stream)))
    return out


def layernorm(x, w, b, eps: float = 1e-5, out_bf16: bool = True, out=None, stream=None, out_format=None):
    """LayerNorm over the last axis of a float32 CUDA tensor.

    Output bf16 (``out_bf16``) or float32; ``out_format`` (LN_OUT_*) overrides it and also
    offers float32 rounded to TF32.
    """
    import torch
    _require(x, torch.float32, "x")
    fmt = (LN_OUT_BF16 if out_bf16 else LN_OUT_F32) if out_format is None else int(out_format)
    d = x.shape[-1]
    rows = x.numel() // d
    if out is None:
        out = _empty(x.shape, torch.bfloat16 if fmt == LN_OUT_BF16 else torch.float32, x.device, stream)
    _check(lib().wenc_layernorm(_ptr(x), _ptr(w), _ptr(b), _ptr(out), rows, d, eps, fmt, _stream(stream)))
    return out


def linear(a, w, bias, epilogue: int = EPI_BIAS_BF16, resid=None, out=None, stream=None):
    """out = epilogue(a w^T + bias); a bf16 [M, K], w bf16 [N, K], bias float32 [N]."""
    import torch
    _require(a, torch.bfloat16, "a")
    _require(w, torch.bfloat16, "w")
    _require(bias, torch.float32, "bias")
    M, K = a.shape
    N = w.shape[0]
    if out is None:
        dt = torch.float32 if epilogue == EPI_BIAS_RESID_F32 else torch.bfloat16
        out = _empty((M, N), dt, a.device, stream)
    _check(lib().wenc_linear(_ptr(a), _ptr(w), _ptr(bias), _ptr(resid), _ptr(out), M, N, K, epilogue, _stream(stream)))
    return out


def linear_tf32(a, w, bias, epilogue: int = EPI_BIAS_BF16, resid=None, out=None, stream=None):
    """out = epilogue(a w^T + bias) on TF32 tensor cores; a float32 [M, K], w float32 [N, K].

    Epilogues 0 and 1 write float32 rounded to TF32, epilogue 2 float32 (resid + product).
    """
    import torch
    _require(a, torch.float32, "a")
    _require(w, torch.float32, "w")
    _require(bias, torch.float32, "bias")
    M, K = a.shape
    N = w.shape[0]
    if out is None:
        out = _empty((M, N), torch.float32, a.device, stream)
    _require(out, torch.float32, "out")
    _check(lib().wenc_linear_tf32(_ptr(a), _ptr(w), _ptr(bias), _ptr(resid), _ptr(out), M, N, K, epilogue,
                                  _stream(stream)))
    return out


def attention_tf32(q, k, v, out=None, stream=None):
    """out = softmax(q k^T / 8) v per (window, head) with TF32 products; float32 [B, T, H, 64]."""
    import torch
    for n, t in (("q", q), ("k", k), ("v", v)):
        _require(t, torch.float32, n)
    B, T, H, hd = q.shape
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _require(out, torch.float32, "out")
    _check(lib().wenc_attention_tf32(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, T, H, hd, _stream(stream)))
    return out


# The decode-side calls below run once per layer and token, so what they cost on the host counts: the
# common case (packed tensors) is checked with few attribute reads, anything else more slowly.
_torch = None


def _load_torch():
    global _torch
    import torch
    _torch = torch
    lib()
    return torch


def _elsewhere(named):
    """The error for tensors that are not on the current CUDA device, where the library launches."""
    import torch
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
    for name, t in named:
        if t is not None and not t.is_cuda:
            return TypeError(f"{name} must be a CUDA tensor")
        if t is not None and t.get_device() != dev:
            return ValueError(f"{name} is on device {t.get_device()}, the current device is {dev}")
    return RuntimeError("tensors on several devices")


def _raw_stream(stream, dev):
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _bad_ints(t, name, n):
    return (TypeError(f"{name} must be torch.int32, got {t.dtype}") if t.dtype is not _torch.int32 else
            ValueError(f"{name} must be contiguous with shape ({n},), got {tuple(t.shape)}"))


def _token_stride(t, name):
    """Elements between the tokens of [..., heads, 64]: heads packed, leading axes evenly spaced."""
    shape, st = t.shape, t.stride()
    hd, heads = shape[-1], shape[-2]
    if shape[0] == 0:
        return heads * hd
    if hd > 1 and st[-1] != 1 or heads > 1 and st[-2] != hd:
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if len(shape) == 4:
        if shape[0] > 1 and shape[1] > 1 and st[0] != shape[1] * st[1]:
            raise ValueError(f"{name}: tokens must be evenly spaced over the first two axes")
        if shape[1] == 1:
            return st[0] if shape[0] > 1 else heads * hd
        return st[1]
    return st[0] if shape[0] > 1 else heads * hd


def _plane_strides(t, name):
    """(elements between groups, between tokens) of [groups, tokens, heads, 64], heads packed."""
    (G, T, heads, hd), st = t.shape, t.stride()
    if st[3] != 1 or heads > 1 and st[2] != hd:
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return (st[0] if G > 1 else 0), (st[1] if T > 1 else heads * hd)


def _page_stride(t, name):
    """Elements between the pages of [pages, page_size, heads, 64], each page packed."""
    (n, size, heads, hd), st = t.shape, t.stride()
    if st[3] != 1 or st[2] != hd and heads > 1 or st[1] != heads * hd and size > 1:
        raise ValueError(f"{name}: each page must be contiguous")
    return st[0] if n > 1 else size * heads * hd


def _pool(k_pages, v_pages, dtype, heads, hd):
    """(pages, page size, stride of K pages, of V pages) of a paged cache [pages, page_size, heads, hd]."""
    shape = k_pages.shape
    if k_pages.dtype is not dtype or v_pages.dtype is not dtype:
        raise TypeError(f"k_pages and v_pages must be {dtype}, got {k_pages.dtype} and {v_pages.dtype}")
    if len(shape) != 4 or shape[2] != heads or shape[3] != hd or v_pages.shape != shape:
        raise ValueError(f"k_pages and v_pages must be [pages, page_size, {heads}, {hd}], got {tuple(shape)} and "
                         f"{tuple(v_pages.shape)}")
    n, size = shape[:2]
    row = size * heads * hd
    return (n, size, row if k_pages.is_contiguous() else _page_stride(k_pages, "k_pages"),
            row if v_pages.is_contiguous() else _page_stride(v_pages, "v_pages"))


def _table(t, n_seqs):
    """(row stride, columns) of a block table."""
    shape = t.shape
    if t.dtype is not _torch.int32:
        raise TypeError(f"block_table must be torch.int32, got {t.dtype}")
    if len(shape) != 2 or shape[0] != n_seqs:
        raise ValueError(f"block_table must be [{n_seqs}, pages], got {tuple(shape)}")
    cols = shape[1]
    if t.is_contiguous():
        return cols, cols
    if cols > 1 and t.stride(1) != 1:
        raise ValueError("block_table: the entries of a sequence must be contiguous")
    return (t.stride(0) if n_seqs > 1 else cols), cols


def _room(workspace, dev):
    """(address, bytes) of a workspace tensor."""
    if workspace.get_device() != dev:
        raise _elsewhere((("workspace", workspace),))
    if not workspace.is_contiguous():  # its elements may be fewer bytes than they count
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _dtype_error(t, name):
    return TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def prefix_attention(q, k_prefix=None, v_prefix=None, *, prefix_lens=None, group_start=None, max_group=None,
                     k_pages=None, v_pages=None, block_table=None, lens=None, scale: float = 0.125, out=None,
                     workspace=None, stream=None):
    """Decode-step attention of sequences that share prefixes (see wenc_prefix_attention).

    ``q`` [n_seqs, q_len, H, 64] bf16 or float32 (the tokens may be slices of wider rows);
    ``k_prefix``, ``v_prefix`` [n_groups, prefix_max, Hkv, 64] with ``prefix_lens`` int32 [n_groups]
    (None: prefix_max each), for instance the planes of ``Encoder.cross_kv`` viewed as
    [windows, seq_len, H, 64]. The sequences are grouped in order: equal groups, or
    ``group_start`` int32 [n_groups + 1] with ``max_group`` at least the largest group (None: n_seqs).
    ``k_pages``, ``v_pages`` [pages, page_size, Hkv, 64] with ``block_table`` int32 [n_seqs, pages]
    and ``lens`` int32 [n_seqs]: each sequence's own keys, its q_len newest tokens included.
    ``workspace``: a uint8 tensor to use instead of an allocation where one is needed; it is busy
    until the call's work is done. A batch of no sequences gives an empty output, a prefix of no tokens counts as
    one of length zero.
    """
    torch = _torch or _load_torch()
    dtype = q.dtype
    dt = 1 if dtype is torch.bfloat16 else 0
    if not dt and dtype is not torch.float32:
        raise _dtype_error(q, "q")
    shape = q.shape
    if len(shape) != 4:
        raise ValueError(f"q must be [n_seqs, q_len, heads, 64], got {tuple(shape)}")
    if (k_prefix is None) != (v_prefix is None) or (k_pages is None) != (v_pages is None):
        raise ValueError("keys and values come together")
    if k_prefix is None and k_pages is None:
        raise ValueError("neither a prefix nor pages")
    n, t, H, hd = shape
    dev = q.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise _elsewhere((("q", q),))
    if out is None:
        out = _empty(shape, dtype, q.device, stream)
        out_stride = H * hd
    else:
        if out.dtype is not dtype or out.shape != shape:
            raise ValueError(f"out must be {dtype} {tuple(shape)}, got {out.dtype} {tuple(out.shape)}")
        out_stride = H * hd if out.is_contiguous() else _token_stride(out, "out")
        if out.get_device() != dev:
            raise _elsewhere((("out", out),))
    kv = G = S = T = kp = vp = kg = kt = vg = vt = p_lens = g_start = 0
    if k_prefix is not None:
        kshape = k_prefix.shape
        if k_prefix.dtype is not dtype or v_prefix.dtype is not dtype:
            raise TypeError(f"k_prefix and v_prefix must be {dtype}, got {k_prefix.dtype} and {v_prefix.dtype}")
        if len(kshape) != 4 or kshape[3] != hd or v_prefix.shape != kshape:
            raise ValueError(f"k_prefix and v_prefix must be [groups, tokens, heads, {hd}], got {tuple(kshape)} and "
                             f"{tuple(v_prefix.shape)}")
        G, T, kv, _ = kshape
        if T == 0:  # a prefix of no tokens: of one that is not counted
            T = 1
            k_prefix = v_prefix = _empty((G, 1, kv, hd), dtype, q.device, stream)
            if stream is None:
                prefix_lens = torch.zeros(G, dtype=torch.int32, device=q.device)
            else:
                with _on(stream):
                    prefix_lens = torch.zeros(G, dtype=torch.int32, device=q.device)
        kg = vg = T * kv * hd
        kt = vt = kv * hd
        if not k_prefix.is_contiguous():
            kg, kt = _plane_strides(k_prefix, "k_prefix")
        if not v_prefix.is_contiguous():
            vg, vt = _plane_strides(v_prefix, "v_prefix")
        if k_prefix.get_device() != dev or v_prefix.get_device() != dev:
            raise _elsewhere((("k_prefix", k_prefix), ("v_prefix", v_prefix)))
        kp, vp = k_prefix.data_ptr(), v_prefix.data_ptr()
        if group_start is not None:
            if (group_start.dtype is not torch.int32 or group_start.dim() != 1 or group_start.numel() != G + 1
                    or not group_start.is_contiguous()):
                raise _bad_ints(group_start, "group_start", G + 1)
            if group_start.get_device() != dev:
                raise _elsewhere((("group_start", group_start),))
            g_start = group_start.data_ptr()
            S = n if max_group is None else min(max_group, n)
        elif n == 0:
            S = 0
        elif G == 0 or n % G != 0:
            raise ValueError(f"{n} sequences are no multiple of {G} groups (pass group_start)")
        else:
            S = n // G
        if prefix_lens is not None:
            if (prefix_lens.dtype is not torch.int32 or prefix_lens.dim() != 1 or prefix_lens.numel() != G
                    or not prefix_lens.is_contiguous()):
                raise _bad_ints(prefix_lens, "prefix_lens", G)
            if prefix_lens.get_device() != dev:
                raise _elsewhere((("prefix_lens", prefix_lens),))
            p_lens = prefix_lens.data_ptr()
    elif prefix_lens is not None or group_start is not None:
        raise ValueError("prefix_lens and group_start go with a prefix")
    pages = size = kps = vps = kpg = vpg = tab = tab_stride = max_pages = own = 0
    if k_pages is not None:
        if block_table is None or lens is None:
            raise ValueError("pages need block_table and lens")
        if k_prefix is None and k_pages.dim() == 4:
            kv = k_pages.shape[2]
        pages, size, kps, vps = _pool(k_pages, v_pages, dtype, kv, hd)
        tab_stride, max_pages = _table(block_table, n)
        if lens.dtype is not torch.int32 or lens.dim() != 1 or lens.numel() != n or not lens.is_contiguous():
            raise _bad_ints(lens, "lens", n)
        if (k_pages.get_device() != dev or v_pages.get_device() != dev or block_table.get_device() != dev
                or lens.get_device() != dev):
            raise _elsewhere((("k_pages", k_pages), ("v_pages", v_pages), ("block_table", block_table), ("lens", lens)))
        kpg, vpg, tab, own = k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(), lens.data_ptr()
    elif block_table is not None or lens is not None:
        raise ValueError("block_table and lens go with pages")
    if n == 0 or t == 0:
        return out
    args = (dt, n, t, H, kv, hd, q.data_ptr(), out.data_ptr(),
            H * hd if q.is_contiguous() else _token_stride(q, "q"), out_stride, G, S, g_start, kp, vp, kg,
            kt, vg, vt, T, p_lens, kpg, vpg, kps, vps, pages, size, tab, tab_stride, max_pages, own, scale)
    ws = ws_bytes = 0
    # (up to 64 rows per key head never need a workspace)
    if workspace is not None or (S or 1) * t * H > 64 * kv:
        if workspace is None:
            need = _lib.wenc_prefix_attention_workspace(_PREFIX_PACK.pack(*args, 0, 0))
            workspace = _empty(need, torch.uint8, q.device, stream) if need else None
        if workspace is not None:
            ws, ws_bytes = _room(workspace, dev)
    status = _lib.wenc_prefix_attention(_PREFIX_PACK.pack(*args, ws, ws_bytes), _raw_stream(stream, dev))
    if status:
        _check(status)
    return out


def kv_append(k, v, k_pages, v_pages, block_table, lens, *, seq_start=None, q=None, q_out=None, positions=None,
              inv_freq=None, interleaved: bool = False, stream=None):
    """Write new tokens' keys and values into a paged cache, turning keys and queries by their
    positions on the way (see wenc_kv_append). Returns ``q_out`` (None without ``q``).

    ``k``, ``v`` [tokens, Hkv, 64] and ``q`` [tokens, H, 64], bf16 or float32 (slices of a fused
    projection's rows will do); ``k_pages``, ``v_pages`` [pages, page_size, Hkv, 64];
    ``block_table`` int32 [n_seqs, pages]; ``lens`` int32 [n_seqs], the call's tokens included;
    ``seq_start`` int32 [n_seqs + 1] (None: tokens / n_seqs each); ``positions`` int32 [tokens]
    (None: the cache positions); ``inv_freq`` float32 [rot_dim / 2] (None: no rotation). ``q_out``
    may be ``q``; without it the turned queries go to a new tensor, whose padding rows are zeros.
    """
    torch = _torch or _load_torch()
    dtype = k.dtype
    dt = 1 if dtype is torch.bfloat16 else 0
    if not dt and dtype is not torch.float32:
        raise _dtype_error(k, "k")
    shape = k.shape
    if len(shape) != 3 or v.shape != shape or v.dtype is not dtype:
        raise ValueError(f"k and v must be {dtype} [tokens, heads, 64], got {tuple(shape)} and {v.dtype} {tuple(v.shape)}")
    n, kv, hd = shape
    dev = k.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise _elsewhere((("k", k),))
    i32 = torch.int32
    H = qp = qo = qs = qos = 0
    if q is not None:
        qshape = q.shape
        if q.dtype is not dtype:
            raise TypeError(f"q must be {dtype}, got {q.dtype}")
        if len(qshape) != 3 or qshape[0] != n or qshape[2] != hd:
            raise ValueError(f"q must be [{n}, heads, {hd}], got {tuple(qshape)}")
        if q_out is None:
            q_out = _empty(qshape, dtype, q.device, stream)
            if stream is None:
                q_out.zero_()
            else:
                with _on(stream):  # in order with the kernel that writes over the zeros
                    q_out.zero_()
        elif q_out.dtype is not dtype or q_out.shape != qshape:
            raise ValueError(f"q_out must be {dtype} {tuple(qshape)}, got {q_out.dtype} {tuple(q_out.shape)}")
        if q.get_device() != dev or q_out.get_device() != dev:
            raise _elsewhere((("q", q), ("q_out", q_out)))
        H = qshape[1]
        qp, qo = q.data_ptr(), q_out.data_ptr()
        qs = H * hd if q.is_contiguous() else _token_stride(q, "q")
        qos = H * hd if q_out.is_contiguous() else _token_stride(q_out, "q_out")
    elif q_out is not None:
        raise ValueError("q_out goes with q")
    n_seqs = lens.numel()
    if lens.dtype is not i32 or lens.dim() != 1 or not lens.is_contiguous():
        raise _bad_ints(lens, "lens", n_seqs)
    pages, size, kps, vps = _pool(k_pages, v_pages, dtype, kv, hd)
    tab_stride, max_pages = _table(block_table, n_seqs)
    if (v.get_device() != dev or k_pages.get_device() != dev or v_pages.get_device() != dev
            or block_table.get_device() != dev or lens.get_device() != dev):
        raise _elsewhere((("v", v), ("k_pages", k_pages), ("v_pages", v_pages), ("block_table", block_table),
                          ("lens", lens)))
    start = pos = freq = rot = 0
    if seq_start is not None:
        if (seq_start.dtype is not i32 or seq_start.dim() != 1 or seq_start.numel() != n_seqs + 1
                or not seq_start.is_contiguous()):
            raise _bad_ints(seq_start, "seq_start", n_seqs + 1)
        if seq_start.get_device() != dev:
            raise _elsewhere((("seq_start", seq_start),))
        start = seq_start.data_ptr()
    if positions is not None:
        if positions.dtype is not i32 or positions.dim() != 1 or positions.numel() != n or not positions.is_contiguous():
            raise _bad_ints(positions, "positions", n)
        if positions.get_device() != dev:
            raise _elsewhere((("positions", positions),))
        pos = positions.data_ptr()
    if inv_freq is not None:
        if inv_freq.dtype is not torch.float32:
            raise TypeError(f"inv_freq must be torch.float32, got {inv_freq.dtype}")
        if inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError(f"inv_freq must be contiguous [rot_dim / 2], got {tuple(inv_freq.shape)}")
        if inv_freq.get_device() != dev:
            raise _elsewhere((("inv_freq", inv_freq),))
        freq, rot = inv_freq.data_ptr(), 2 * inv_freq.numel()
    if n == 0:
        return q_out
    status = _lib.wenc_kv_append(
        _APPEND_PACK.pack(dt, n, n_seqs, H, kv, hd, qp, qo, k.data_ptr(), v.data_ptr(), qs, qos,
                          kv * hd if k.is_contiguous() else _token_stride(k, "k"),
                          kv * hd if v.is_contiguous() else _token_stride(v, "v"), k_pages.data_ptr(), v_pages.data_ptr(),
                          kps, vps, pages, size, block_table.data_ptr(), tab_stride, max_pages, lens.data_ptr(), start, pos,
                          freq, rot, 1 if interleaved else 0),
        _raw_stream(stream, dev))
    if status:
        _check(status)
    return q_out


def quantize_rows(x, out=None, scale=None, stream=None):
    """(int8 rows, float32 scales) of x [..., d] bf16 or float32: scale = max|row| * (1 / 127) (see
    wenc_quantize_rows)."""
    torch = _torch or _load_torch()
    dt = 1 if x.dtype is torch.bfloat16 else 0
    if not dt and x.dtype is not torch.float32:
        raise _dtype_error(x, "x")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    dev = x.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise _elsewhere((("x", x),))
    shape = x.shape
    rows = shape[:-1]
    d = shape[-1]
    if out is None:
        out = _empty(shape, torch.int8, x.device, stream)
    elif out.dtype is not torch.int8 or out.shape != shape or not out.is_contiguous():
        raise ValueError(f"out must be contiguous int8 {tuple(shape)}, got {out.dtype} {tuple(out.shape)}")
    if scale is None:
        scale = _empty(rows, torch.float32, x.device, stream)
    elif scale.dtype is not torch.float32 or scale.shape != rows or not scale.is_contiguous():
        raise ValueError(f"scale must be contiguous float32 {tuple(rows)}, got {scale.dtype} {tuple(scale.shape)}")
    if out.get_device() != dev or scale.get_device() != dev:
        raise _elsewhere((("out", out), ("scale", scale)))
    if scale.numel() == 0:
        return out, scale
    status = _lib.wenc_quantize_rows(x.data_ptr(), dt, out.data_ptr(), scale.data_ptr(), scale.numel(), d,
                                     _raw_stream(stream, dev))
    if status:
        _check(status)
    return out, scale


def linear_i8(a, a_scale, w, w_scale, bias, epilogue: int = EPI_BIAS_BF16, resid=None, out=None, workspace=None,
              stream=None):
    """out = epilogue((a w^T) * a_scale[:, None] * w_scale + bias) on 8-bit integers: a int8 [M, K]
    with float32 scales [M] (``quantize_rows``), w int8 [N, K] with float32 scales [N]; epilogues
    and outputs as ``linear``. ``workspace``: a uint8 tensor to use instead of an allocation where
    one is needed."""
    torch = _torch or _load_torch()
    dev = a.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise _elsewhere((("a", a),))
    i8, f32 = torch.int8, torch.float32
    if a.dtype is not i8 or w.dtype is not i8:
        raise TypeError(f"a and w must be torch.int8, got {a.dtype} and {w.dtype}")
    if a_scale.dtype is not f32 or w_scale.dtype is not f32 or bias.dtype is not f32:
        raise TypeError("a_scale, w_scale and bias must be torch.float32")
    ash, wsh = a.shape, w.shape
    if len(ash) != 2 or len(wsh) != 2 or ash[1] != wsh[1]:
        raise ValueError(f"a {tuple(ash)} and w {tuple(wsh)} must be [M, K] and [N, K]")
    M, K = ash
    N = wsh[0]
    if a_scale.numel() != M or w_scale.numel() != N or bias.numel() != N:
        raise ValueError(f"a_scale must hold {M} scales, w_scale and bias {N}")
    if not (a.is_contiguous() and w.is_contiguous() and a_scale.is_contiguous() and w_scale.is_contiguous()
            and bias.is_contiguous()):
        raise ValueError("linear_i8 takes contiguous tensors")
    if (a_scale.get_device() != dev or w.get_device() != dev or w_scale.get_device() != dev
            or bias.get_device() != dev):
        raise _elsewhere((("a_scale", a_scale), ("w", w), ("w_scale", w_scale), ("bias", bias)))
    dt = f32 if epilogue == EPI_BIAS_RESID_F32 else torch.bfloat16
    if out is None:
        out = _empty((M, N), dt, a.device, stream)
    elif out.dtype is not dt or out.shape != (M, N) or not out.is_contiguous():
        raise ValueError(f"out must be contiguous {dt} {(M, N)}, got {out.dtype} {tuple(out.shape)}")
    elif out.get_device() != dev:
        raise _elsewhere((("out", out),))
    rp = 0
    if resid is not None:
        if resid.dtype is not f32 or resid.shape != (M, N) or not resid.is_contiguous():
            raise ValueError(f"resid must be contiguous float32 {(M, N)}, got {resid.dtype} {tuple(resid.shape)}")
        if resid.get_device() != dev:
            raise _elsewhere((("resid", resid),))
        rp = resid.data_ptr()
    if M == 0:
        return out
    ws = ws_bytes = 0
    if workspace is None and M > 16:
        need = _lib.wenc_linear_i8_workspace(M, N, K)
        if need:
            workspace = _empty(need, torch.uint8, a.device, stream)
    if workspace is not None:
        ws, ws_bytes = _room(workspace, dev)
    status = _lib.wenc_linear_i8(a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), bias.data_ptr(), rp,
                                 out.data_ptr(), M, N, K, epilogue, ws, ws_bytes, _raw_stream(stream, dev))
    if status:
        _check(status)
    return out


def selftest_gemm_pair_abort(a, w, bias, stop_after: int, out=None, stream=None):
    """Launch the CTA-pair GEMM self-test (the odd CTA of each pair stops after `stop_after`
    k-blocks); returns the (undefined) output tensor; read the outcome with sync_status()."""
    import torch
    _require(a, torch.bfloat16, "a")
    _require(w, torch.bfloat16, "w")
    _require(bias, torch.float32, "bias")
    M, K = a.shape
    N = w.shape[0]
    if out is None:
        out = _empty((M, N), torch.bfloat16, a.device, stream)
    _check(lib().wenc_selftest_gemm_pair_abort(_ptr(a), _ptr(w), _ptr(bias), _ptr(out), M, N, K, int(stop_after),
                                              _stream(stream)))
    return out


def selftest_attention_abort(q, k, v, stop_after: int, out=None, stream=None):
    """Launch the attention self-test (its producer stops after `stop_after` K tiles); returns the
    (undefined) output; read the outcome with sync_status()."""
    import torch
    for n, t in (("q", q), ("k", k), ("v", v)):
        _require(t, torch.bfloat16, n)
    B, T, H, hd = q.shape
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _check(lib().wenc_selftest_attention_abort(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, T, H, int(stop_after),
                                              _stream(stream)))
    return out


def selftest_wait_timeout(stream=None):
    """Launch the bounded-wait self-test (returns immediately; read it with sync_status())."""
    _check(lib().wenc_selftest_wait_timeout(_stream(stream)))


def gemm_schedule(M: int, N: int, pair: bool, max_units: int):
    """Host-only replay of a GEMM launch's tile schedule (see wenc_selftest_gemm_schedule).

    Returns (cover, unit_halves, units, halves): cover[t, h] = how often column half h of tile t
    is computed, unit_halves[u] = half tiles computed by unit u (u < units)."""
    import numpy as np
    rows = 256 if pair else 128
    bn = 256 if pair or N % 256 == 0 else 128
    tiles = -(-M // rows) * (N // bn)
    cover = (ctypes.c_int * max(2 * tiles, 2))()
    unit_halves = (ctypes.c_int * max_units)()
    units, halves = ctypes.c_int(), ctypes.c_int()
    _check(lib().wenc_selftest_gemm_schedule(M, N, int(pair), max_units, cover, len(cover), unit_halves,
                                             ctypes.byref(units), ctypes.byref(halves)))
    cov = np.frombuffer(cover, dtype=np.int32, count=2 * tiles).reshape(tiles, 2).copy()
    work = np.frombuffer(unit_halves, dtype=np.int32, count=units.value).copy()
    return cov, work, units.value, halves.value


def sync_status(encoder: Encoder | None = None):
    _check(lib().wenc_sync_status(encoder.handle if encoder is not None else None))
