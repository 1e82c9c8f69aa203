"""Thin Python binding of the C ABI in include/lsq.h (argument marshalling only).

Every function here has the name of the C entry point it calls, takes torch
tensors (or plain ints/floats), passes their data pointers and the current CUDA
stream, and raises LsqError on a non-zero status.  No computation happens here:
every step of the path runs in the CUDA library.  Importing this module loads
liblsq.so and fails loudly if it has not been built.
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liblsq.so")

LSQ_OK, LSQ_ERR_INVALID, LSQ_ERR_SHAPE, LSQ_ERR_CUDA = 0, 1, 2, 3
LSQ_ERR_TIMEOUT, LSQ_ERR_WORKSPACE, LSQ_ERR_ALIGN, LSQ_ERR_DEVICE = 4, 5, 6, 7

# device status word bits (lsq_device_status)
LSQ_DEV_ERR_WAIT, LSQ_DEV_ERR_NONFINITE, LSQ_DEV_ERR_INDEX = 1, 2, 4

# Every symbol include/lsq.h declares (checked by tests/test_abi.py).
EXPORTS = (
    "lsq_last_error", "lsq_version", "lsq_device_status", "lsq_nf4_codebook",
    "nf4_quantize", "nf4_dequantize", "nf4_lora_linear_workspace_bytes",
    "nf4_lora_linear_fwd", "nf4_lora_linear_bwd", "lsq_layer_layout_get",
    "lsq_lora_layout_get", "decoder_layer_workspace_bytes", "decoder_layer_fwd",
    "decoder_layer_bwd", "stream_stack_create", "stream_stack_destroy",
    "stream_stack_workspace_bytes", "stream_stack_step", "stream_stack_last_stats",
    "lora_adamw_step", "lsq_launch_counter", "lsq_profile_enable", "lsq_profile_read",
    "nf4_lora_linear_fwd_noalloc", "nf4_absmax_quantize8", "nf4_dequantize_dq",
    "stream_stack_dpo_workspace_bytes", "stream_stack_dpo_step", "lsq_bf16_from_f32",
    "lsq_shard_bytes", "lsq_nccl_unique_id", "stream_stack_shard", "lsq_stream_plan",
    "stream_stack_reduce_grads", "lsq_gemm_plan_get", "lsq_lora_plan_get",
    "packed_index_ints", "packed_index", "packed_targets", "packed_cross_entropy",
    "packed_attention_fwd", "packed_attention_bwd", "packed_attention_workspace_bytes",
    "adamw_scale_floats", "adamw_multi_step", "adamw_state_dequantize", "adamw_state_quantize",
    "decoder_layer_packed_fwd", "decoder_layer_packed_bwd",
    "stream_stack_packed_workspace_bytes", "stream_stack_packed_step",
)
LSQ_NCCL_ID_BYTES = 128


class LsqError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("lsq error %d: %s" % (code, msg))
        self.code = code


class lsq_cfg(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int64), ("ffn", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("n_layers", ctypes.c_int32),
                ("lora_r", ctypes.c_int32), ("block", ctypes.c_int32),
                ("lora_alpha", ctypes.c_float), ("rope_theta", ctypes.c_float),
                ("rms_eps", ctypes.c_float), ("absmax_bits", ctypes.c_int32),
                ("weight_bits", ctypes.c_int32)]


class lsq_layer_layout(ctypes.Structure):
    _fields_ = [("codes_off", ctypes.c_uint64 * 7), ("absmax_off", ctypes.c_uint64 * 7),
                ("g1_off", ctypes.c_uint64), ("g2_off", ctypes.c_uint64),
                ("rows", ctypes.c_int64 * 7), ("cols", ctypes.c_int64 * 7),
                ("bytes", ctypes.c_uint64), ("scale_off", ctypes.c_uint64 * 7),
                ("absmax_bits", ctypes.c_int32), ("weight_bits", ctypes.c_int32)]


class lsq_lora_layout(ctypes.Structure):
    _fields_ = [("a_off", ctypes.c_int64 * 7), ("b_off", ctypes.c_int64 * 7),
                ("floats_per_layer", ctypes.c_int64)]


class lsq_adamw(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("step", ctypes.c_int32), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class lsq_adamw_tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "g", "m", "v", "m_scale", "v_scale")] + [
        ("n", ctypes.c_int64), ("lr", ctypes.c_float), ("weight_decay", ctypes.c_float)]


class lsq_adamw_hyper(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_float), ("beta2", ctypes.c_float), ("eps", ctypes.c_float),
                ("step", ctypes.c_int32), ("state_bits", ctypes.c_int32),
                ("grad_bits", ctypes.c_int32), ("step_dev", ctypes.c_void_p)]


class lsq_prof_entry(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int64),
                ("total_ms", ctypes.c_double), ("flops", ctypes.c_double),
                ("bytes", ctypes.c_double)]


class lsq_step_stats(ctypes.Structure):
    _fields_ = [("layer_copies", ctypes.c_int32), ("h2d_bytes", ctypes.c_int64),
                ("step_ms", ctypes.c_float), ("copy_wait_ms", ctypes.c_float)]


class lsq_gemm_plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "pair", "bn", "nacc", "m_tiles", "t_tiles", "splits", "kt_total", "kt_per_split",
        "stages", "ring_stages", "x_stage_bytes", "w_stage_bytes", "ring_bytes",
        "absmax_ring_bytes", "smem_bytes", "smem_limit", "epilogue_bytes", "tmem_cols")] + [
        ("partial_bytes", ctypes.c_int64)]


class lsq_lora_plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_pad", "row_tiles", "col_tiles", "splits", "kt_total", "stages", "stage_bytes",
        "smem_bytes", "smem_limit", "ctas_per_sm", "tmem_cols", "reduce_bytes")]


# operand modes of lsq_gemm_plan_get
LSQ_GEMM_NF4_FWD, LSQ_GEMM_NF4_DX, LSQ_GEMM_BF16_FWD, LSQ_GEMM_BF16_DX = 0, 1, 2, 3
LSQ_GEMM_BF16_AS_F16_FWD = 4


_P = ctypes.c_void_p
_I32, _I64, _F, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_PROTOS = {
    "lsq_last_error": (ctypes.c_char_p, []),
    "lsq_version": (ctypes.c_int, []),
    "lsq_device_status": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int), ctypes.c_int]),
    "lsq_nf4_codebook": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float)]),
    "nf4_quantize": (ctypes.c_int, [_P, _I64, _I64, _I32, _P, _P, _P]),
    "nf4_dequantize": (ctypes.c_int, [_P, _P, _I64, _I64, _I32, _P, _P]),
    "nf4_absmax_quantize8": (ctypes.c_int, [_P, _I64, _P, _P, _P]),
    "lsq_bf16_from_f32": (ctypes.c_int, [_P, _I64, _P, _P]),
    "nf4_dequantize_dq": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I32, _P, _P]),
    "nf4_lora_linear_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I32]),
    "nf4_lora_linear_fwd": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _I32, _P, _P, _I32, _F,
                                           _P, _P, _I32, _P, _P, _SZ, _P]),
    "nf4_lora_linear_bwd": (ctypes.c_int, [_P, _P, _I64, _I64, _I64, _P, _P, _I32, _P, _P, _I32,
                                           _F, _P, _P, _P, _I32, _P, _SZ, _P]),
    "lsq_layer_layout_get": (ctypes.c_int, [ctypes.POINTER(lsq_cfg),
                                            ctypes.POINTER(lsq_layer_layout)]),
    "lsq_lora_layout_get": (ctypes.c_int, [ctypes.POINTER(lsq_cfg),
                                           ctypes.POINTER(lsq_lora_layout)]),
    "decoder_layer_workspace_bytes": (_SZ, [ctypes.POINTER(lsq_cfg), _I32, _I32]),
    "decoder_layer_fwd": (ctypes.c_int, [ctypes.POINTER(lsq_cfg), _P, _P, _P, _I32, _I32, _P, _P,
                                         _SZ, _P]),
    "decoder_layer_bwd": (ctypes.c_int, [ctypes.POINTER(lsq_cfg), _P, _P, _P, _P, _I32, _I32, _P,
                                         _P, _I32, _P, _SZ, _P]),
    "stream_stack_create": (ctypes.c_int, [ctypes.POINTER(lsq_cfg), ctypes.POINTER(_P), _I32, _P,
                                           _P, _I32, ctypes.POINTER(_P)]),
    "stream_stack_destroy": (ctypes.c_int, [_P]),
    "stream_stack_workspace_bytes": (_SZ, [ctypes.POINTER(lsq_cfg), _I32, _I32]),
    "stream_stack_step": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P,
                                         ctypes.POINTER(lsq_adamw), ctypes.POINTER(ctypes.c_float),
                                         _P, _P, _SZ, _P, _I64]),
    "stream_stack_last_stats": (ctypes.c_int, [_P, ctypes.POINTER(lsq_step_stats)]),
    "stream_stack_dpo_workspace_bytes": (_SZ, [ctypes.POINTER(lsq_cfg), _I32, _I32]),
    "stream_stack_dpo_step": (ctypes.c_int, [_P, _P, _I32, _I32, _F, _P, _P, _P, _P, _P,
                                             ctypes.POINTER(lsq_adamw),
                                             ctypes.POINTER(ctypes.c_float),
                                             ctypes.POINTER(ctypes.c_float), _P, _P, _SZ, _P,
                                             _I64]),
    "lora_adamw_step": (ctypes.c_int, [_P, _P, ctypes.POINTER(lsq_adamw), _I64, _P]),
    "lsq_shard_bytes": (_I64, [_I64, _I32]),
    "lsq_stream_plan": (ctypes.c_int, [_I32, _I32, _I32, _I32, _P, _P, _P, _I32,
                                       ctypes.POINTER(ctypes.c_int32)]),
    "lsq_nccl_unique_id": (ctypes.c_int, [_P, _I64]),
    "stream_stack_shard": (ctypes.c_int, [_P, _P, _I64, _I32, _I32, _I64]),
    "stream_stack_reduce_grads": (ctypes.c_int, [_P, _P, _I64, _I32, _I32]),
    "lsq_launch_counter": (ctypes.c_int64, []),
    "lsq_gemm_plan_get": (ctypes.c_int, [_I32, _I64, _I64, _I64, _I32, _I32,
                                         ctypes.POINTER(lsq_gemm_plan)]),
    "lsq_lora_plan_get": (ctypes.c_int, [_I64, _I64, _I64, _I32, ctypes.POINTER(lsq_lora_plan)]),
    "nf4_lora_linear_fwd_noalloc": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _I32, _P, _P, _I32,
                                                   _F, _P, _P, _I32, _P, _P]),
    "packed_index_ints": (_I64, [_I64, _I32]),
    "packed_index": (ctypes.c_int, [_P, _P, _I32, _I64, _P, _P]),
    "packed_attention_fwd": (ctypes.c_int, [_P, _P, _I32, _I64, _I32, _I32, _I32, _P, _P, _P]),
    "packed_attention_workspace_bytes": (_SZ, [_I64, _I32, _I32, _I32]),
    "packed_attention_bwd": (ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _I64, _I32, _I32, _I32, _P,
                                            _P, _SZ, _P]),
    "packed_targets": (ctypes.c_int, [_P, _P, _I32, _I64, _P, _P, _P, _I32, _P]),
    "packed_cross_entropy": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _P, _P, _P, _P, _I32, _P]),
    "decoder_layer_packed_fwd": (ctypes.c_int, [ctypes.POINTER(lsq_cfg), _P, _P, _P, _P, _I32, _I32,
                                                _P, _P, _SZ, _P]),
    "decoder_layer_packed_bwd": (ctypes.c_int, [ctypes.POINTER(lsq_cfg), _P, _P, _P, _P, _P, _I32,
                                                _I32, _P, _P, _I32, _P, _SZ, _P]),
    "stream_stack_packed_workspace_bytes": (_SZ, [ctypes.POINTER(lsq_cfg), _I32, _I32]),
    "stream_stack_packed_step": (ctypes.c_int, [_P, _P, _I32, _I32, _P, _P, _I32, _P, _P, _P, _P,
                                                _P, _P, ctypes.POINTER(lsq_adamw_tensor), _I32,
                                                ctypes.POINTER(lsq_adamw_hyper),
                                                ctypes.POINTER(ctypes.c_float), _P, _P, _SZ, _P,
                                                _I64]),
    "adamw_scale_floats": (_I64, [_I64]),
    "adamw_multi_step": (ctypes.c_int, [ctypes.POINTER(lsq_adamw_tensor), _I32,
                                        ctypes.POINTER(lsq_adamw_hyper), _P]),
    "adamw_state_dequantize": (ctypes.c_int, [_P, _P, _I64, _I32, _P, _P]),
    "adamw_state_quantize": (ctypes.c_int, [_P, _I64, _I32, _P, _P, _P]),
    "lsq_profile_enable": (ctypes.c_int, [ctypes.c_int]),
    "lsq_profile_read": (ctypes.c_int, [ctypes.POINTER(lsq_prof_entry), _I32,
                                        ctypes.POINTER(ctypes.c_int32)]),
}

_lib = None


def load():
    """Loads liblsq.so (once) and declares the prototypes; raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("liblsq.so is not built (run: python -m "
                               "layer_streamed_qlora_nf4_b200.build)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _PROTOS.items():
            if not hasattr(lib, name):
                continue   # tests/test_abi.py checks that every declared symbol exists
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
    return _lib


def _check(rc):
    if rc != LSQ_OK:
        raise LsqError(rc, load().lsq_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(stream)
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def cfg_struct(cfg):
    """A synth-style config dict -> lsq_cfg."""
    return lsq_cfg(hidden=cfg["hidden"], ffn=cfg["ffn"], vocab=cfg["vocab"],
                   n_heads=cfg["n_heads"], n_kv_heads=cfg["n_kv_heads"],
                   head_dim=cfg["head_dim"], n_layers=cfg["n_layers"], lora_r=cfg["lora_r"],
                   block=cfg["block"], lora_alpha=cfg["lora_alpha"],
                   rope_theta=cfg["rope_theta"], rms_eps=cfg["rms_eps"],
                   absmax_bits=cfg.get("absmax_bits", 32),
                   weight_bits=cfg.get("weight_bits", 4))


# ------------------------------------------------------------------ entry points
def lsq_version():
    return load().lsq_version()


def lsq_device_status(clear=False):
    v = ctypes.c_int(0)
    _check(load().lsq_device_status(ctypes.byref(v), 1 if clear else 0))
    return v.value


def lsq_nf4_codebook():
    out = (ctypes.c_float * 16)()
    _check(load().lsq_nf4_codebook(out))
    return list(out)


def nf4_quantize(W, codes, absmax, block=64, stream=None):
    N, K = W.shape
    _check(load().nf4_quantize(_ptr(W), N, K, block, _ptr(codes), _ptr(absmax), _stream(stream)))


def nf4_dequantize(codes, absmax, N, K, W_out, block=64, stream=None):
    _check(load().nf4_dequantize(_ptr(codes), _ptr(absmax), N, K, block, _ptr(W_out),
                                 _stream(stream)))


def lsq_bf16_from_f32(x, y, stream=None):
    _check(load().lsq_bf16_from_f32(_ptr(x), x.numel(), _ptr(y), _stream(stream)))


def nf4_absmax_quantize8(absmax, q, scale, stream=None):
    _check(load().nf4_absmax_quantize8(_ptr(absmax), absmax.numel(), _ptr(q), _ptr(scale),
                                       _stream(stream)))


def nf4_dequantize_dq(codes, q, scale, N, K, W_out, block=64, stream=None):
    _check(load().nf4_dequantize_dq(_ptr(codes), _ptr(q), _ptr(scale), N, K, block, _ptr(W_out),
                                    _stream(stream)))


def nf4_lora_linear_workspace_bytes(T, K, N, r):
    return load().nf4_lora_linear_workspace_bytes(T, K, N, r)


def _y_fp32(y):
    """1 for an fp32 output tensor, 0 for an fp16 one (the y_fp32 argument)."""
    import torch
    if y.dtype not in (torch.float32, torch.float16):
        raise TypeError("y must be float16 or float32")
    return 1 if y.dtype == torch.float32 else 0


def nf4_lora_linear_fwd(x, codes, absmax, A, B, scale, y, residual=None, u_out=None, ws=None,
                        block=64, stream=None):
    """x: fp16 [T, K]; y: fp16 [T, N], or fp32 [T, N] (required with an fp32 residual)."""
    T, K = x.shape
    N = y.shape[1]
    r = A.shape[0]
    _check(load().nf4_lora_linear_fwd(_ptr(x), T, K, N, _ptr(codes), _ptr(absmax), block,
                                      _ptr(A), _ptr(B), r, scale, _ptr(residual), _ptr(y),
                                      _y_fp32(y), _ptr(u_out), _ptr(ws),
                                      0 if ws is None else ws.numel(), _stream(stream)))


def nf4_lora_linear_bwd(dy, x, codes, absmax, A, B, scale, dx, dA, dB, accumulate=False,
                        ws=None, block=64, stream=None):
    """dy: bf16 [T, N]; x: fp16 [T, K] (the forward input); dx: bf16 [T, K]."""
    T, K = x.shape
    N = dy.shape[1]
    r = A.shape[0]
    _check(load().nf4_lora_linear_bwd(_ptr(dy), _ptr(x), T, K, N, _ptr(codes), _ptr(absmax),
                                      block, _ptr(A), _ptr(B), r, scale, _ptr(dx), _ptr(dA),
                                      _ptr(dB), 1 if accumulate else 0, _ptr(ws),
                                      0 if ws is None else ws.numel(), _stream(stream)))


def lsq_layer_layout_get(cfg):
    out = lsq_layer_layout()
    c = cfg_struct(cfg)
    _check(load().lsq_layer_layout_get(ctypes.byref(c), ctypes.byref(out)))
    return out


def lsq_lora_layout_get(cfg):
    out = lsq_lora_layout()
    c = cfg_struct(cfg)
    _check(load().lsq_lora_layout_get(ctypes.byref(c), ctypes.byref(out)))
    return out


def decoder_layer_workspace_bytes(cfg, batch, seq):
    c = cfg_struct(cfg)
    return load().decoder_layer_workspace_bytes(ctypes.byref(c), batch, seq)


def decoder_layer_fwd(cfg, blob, lora, x_in, batch, seq, x_out, ws, stream=None):
    """x_in, x_out: fp32 [batch * seq, D] (the residual stream)."""
    c = cfg_struct(cfg)
    _check(load().decoder_layer_fwd(ctypes.byref(c), _ptr(blob), _ptr(lora), _ptr(x_in), batch,
                                    seq, _ptr(x_out), _ptr(ws), ws.numel(), _stream(stream)))


def decoder_layer_bwd(cfg, blob, lora, x_in, dx_out, batch, seq, dx_in, lora_grad, ws,
                      accumulate=False, stream=None):
    c = cfg_struct(cfg)
    _check(load().decoder_layer_bwd(ctypes.byref(c), _ptr(blob), _ptr(lora), _ptr(x_in),
                                    _ptr(dx_out), batch, seq, _ptr(dx_in), _ptr(lora_grad),
                                    1 if accumulate else 0, _ptr(ws), ws.numel(),
                                    _stream(stream)))


class StreamStack:
    """Owns an lsq_stack handle (stream_stack_create / stream_stack_destroy)."""

    def __init__(self, cfg, layer_blobs, buf0, buf1, resident):
        self.cfg = cfg_struct(cfg)
        self._blobs = list(layer_blobs)   # keep the tensors alive
        arr = (ctypes.c_void_p * len(self._blobs))(*[b.data_ptr() for b in self._blobs])
        self.handle = ctypes.c_void_p()
        _check(load().stream_stack_create(ctypes.byref(self.cfg), arr, len(self._blobs),
                                          _ptr(buf0), _ptr(buf1), 1 if resident else 0,
                                          ctypes.byref(self.handle)))

    def shard(self, nccl_id, world, rank, buf_bytes):
        """stream_stack_shard: spread every layer copy over `world` ranks."""
        stream_stack_shard(self, nccl_id, world, rank, buf_bytes)

    def reduce_grads(self, nccl_id, world, rank):
        """stream_stack_reduce_grads: average the LoRA gradients over `world` ranks in each step."""
        stream_stack_reduce_grads(self, nccl_id, world, rank)

    def close(self):
        if self.handle:
            _check(load().stream_stack_destroy(self.handle))
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def lsq_stream_plan(n_layers, micro_batches, held0=-1, held1=-1):
    """-> list of (layer, buf, copy) per visit of one streamed step."""
    n = max(0, 2 * int(n_layers) * int(micro_batches))
    arrs = [(ctypes.c_int32 * max(n, 1))() for _ in range(3)]
    nv = ctypes.c_int32(0)
    _check(load().lsq_stream_plan(int(n_layers), int(micro_batches), int(held0), int(held1),
                                  arrs[0], arrs[1], arrs[2], n, ctypes.byref(nv)))
    return [(arrs[0][i], arrs[1][i], arrs[2][i]) for i in range(nv.value)]


def lsq_gemm_plan_get(mode, M, T, Kc, num_sms=148, allow_pair=True):
    """-> dict of the fused GEMM's launch plan for one product (host only)."""
    out = lsq_gemm_plan()
    _check(load().lsq_gemm_plan_get(int(mode), int(M), int(T), int(Kc), int(num_sms),
                                    1 if allow_pair else 0, ctypes.byref(out)))
    return {n: getattr(out, n) for n, _ in lsq_gemm_plan._fields_}


def lsq_lora_plan_get(M, N, K, num_sms=148):
    """-> dict of the rank-r product kernel's launch plan (host only)."""
    out = lsq_lora_plan()
    _check(load().lsq_lora_plan_get(int(M), int(N), int(K), int(num_sms), ctypes.byref(out)))
    return {n: getattr(out, n) for n, _ in lsq_lora_plan._fields_}


def lsq_shard_bytes(layer_bytes, world):
    return int(load().lsq_shard_bytes(int(layer_bytes), int(world)))


def lsq_nccl_unique_id():
    """-> bytes (LSQ_NCCL_ID_BYTES) of a new NCCL communicator id."""
    buf = ctypes.create_string_buffer(LSQ_NCCL_ID_BYTES)
    _check(load().lsq_nccl_unique_id(buf, LSQ_NCCL_ID_BYTES))
    return buf.raw


def stream_stack_shard(stack, nccl_id, world, rank, buf_bytes):
    nccl_id = bytes(nccl_id)
    if len(nccl_id) != LSQ_NCCL_ID_BYTES:
        raise ValueError("the NCCL id has %d bytes" % LSQ_NCCL_ID_BYTES)
    buf = ctypes.create_string_buffer(nccl_id, LSQ_NCCL_ID_BYTES)
    _check(load().stream_stack_shard(stack.handle, buf, LSQ_NCCL_ID_BYTES, int(world), int(rank),
                                     int(buf_bytes)))


def stream_stack_reduce_grads(stack, nccl_id, world, rank):
    nccl_id = bytes(nccl_id)
    if len(nccl_id) != LSQ_NCCL_ID_BYTES:
        raise ValueError("the NCCL id has %d bytes" % LSQ_NCCL_ID_BYTES)
    buf = ctypes.create_string_buffer(nccl_id, LSQ_NCCL_ID_BYTES)
    _check(load().stream_stack_reduce_grads(stack.handle, buf, LSQ_NCCL_ID_BYTES, int(world),
                                            int(rank)))


def stream_stack_workspace_bytes(cfg, batch, seq):
    c = cfg_struct(cfg)
    return load().stream_stack_workspace_bytes(ctypes.byref(c), batch, seq)


def stream_stack_step(stack, tokens, micro_batches, batch, seq, emb, lm_head, final_norm, lora,
                      lora_grad, opt, ws, logits_out=None, timeout_ms=600000, stream=None):
    """Returns the mean loss (host float).  opt: dict(lr, beta1, beta2, eps, weight_decay,
    step, m, v) or None."""
    loss = ctypes.c_float(0.0)
    o = _adamw_struct(opt) if opt is not None else None
    _check(load().stream_stack_step(stack.handle, _ptr(tokens), micro_batches, batch, seq,
                                    _ptr(emb), _ptr(lm_head), _ptr(final_norm), _ptr(lora),
                                    _ptr(lora_grad), ctypes.byref(o) if o is not None else None,
                                    ctypes.byref(loss), _ptr(logits_out), _ptr(ws), ws.numel(),
                                    _stream(stream), timeout_ms))
    return loss.value


def stream_stack_dpo_workspace_bytes(cfg, pairs, seq):
    c = cfg_struct(cfg)
    return load().stream_stack_dpo_workspace_bytes(ctypes.byref(c), pairs, seq)


def stream_stack_dpo_step(stack, tokens, pairs, seq, beta, emb, lm_head, final_norm, lora,
                          lora_grad, opt, ws, logits_out=None, timeout_ms=600000, stream=None):
    """tokens: int32 device [pairs, 2, seq] (chosen, rejected).  Returns (loss, logps) with
    logps a list of (policy chosen, policy rejected, reference chosen, reference rejected)
    per pair."""
    loss = ctypes.c_float(0.0)
    lp = (ctypes.c_float * (4 * pairs))()
    o = _adamw_struct(opt) if opt is not None else None
    _check(load().stream_stack_dpo_step(stack.handle, _ptr(tokens), pairs, seq, beta, _ptr(emb),
                                        _ptr(lm_head), _ptr(final_norm), _ptr(lora),
                                        _ptr(lora_grad),
                                        ctypes.byref(o) if o is not None else None,
                                        ctypes.byref(loss), lp, _ptr(logits_out), _ptr(ws),
                                        ws.numel(), _stream(stream), timeout_ms))
    return loss.value, [tuple(lp[4 * p: 4 * p + 4]) for p in range(pairs)]


def stream_stack_last_stats(stack):
    s = lsq_step_stats()
    _check(load().stream_stack_last_stats(stack.handle, ctypes.byref(s)))
    return dict(layer_copies=s.layer_copies, h2d_bytes=s.h2d_bytes, step_ms=s.step_ms,
                copy_wait_ms=s.copy_wait_ms)


def _adamw_struct(opt):
    return lsq_adamw(lr=opt["lr"], beta1=opt["beta1"], beta2=opt["beta2"], eps=opt["eps"],
                     weight_decay=opt["weight_decay"], step=opt["step"],
                     m=opt["m"].data_ptr(), v=opt["v"].data_ptr())


def lora_adamw_step(lora, grad, opt, stream=None):
    o = _adamw_struct(opt)
    _check(load().lora_adamw_step(_ptr(lora), _ptr(grad), ctypes.byref(o), lora.numel(),
                                  _stream(stream)))


def lsq_launch_counter():
    return load().lsq_launch_counter()


def lsq_profile_enable(enable=True):
    _check(load().lsq_profile_enable(1 if enable else 0))


def lsq_profile_read():
    """-> dict kernel class -> dict(launches, total_ms, flops, bytes)."""
    arr = (lsq_prof_entry * 64)()
    n = ctypes.c_int32(0)
    _check(load().lsq_profile_read(arr, 64, ctypes.byref(n)))
    return {arr[i].name.decode(): dict(launches=arr[i].launches, total_ms=arr[i].total_ms,
                                       flops=arr[i].flops, bytes=arr[i].bytes)
            for i in range(n.value)}


def nf4_lora_linear_fwd_noalloc(x, codes, absmax, A, B, scale, y, residual=None, u_out=None,
                                block=64, stream=None):
    """nf4_lora_linear_fwd with the library's built-in scratch instead of a workspace."""
    T, K = x.shape
    N = y.shape[1]
    r = A.shape[0]
    _check(load().nf4_lora_linear_fwd_noalloc(_ptr(x), T, K, N, _ptr(codes), _ptr(absmax), block,
                                              _ptr(A), _ptr(B), r, scale, _ptr(residual), _ptr(y),
                                              _y_fp32(y), _ptr(u_out), _stream(stream)))


# ------------------------------------------------------------ packed documents, AdamW
def _need(name, t, dtype, shape=None, numel=None):
    """Checks one tensor argument: its type, that it is contiguous, its shape or length."""
    if not isinstance(t, (_th or _torch()).Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, not %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    if numel is not None and t.numel() != numel:
        raise ValueError("%s must have %d elements, not %d" % (name, numel, t.numel()))


def _fits(t, dtype, shape):
    """Whether a tensor argument needs no closer look (_need says what is wrong with it)."""
    try:
        return t.dtype is dtype and t.shape == shape and t.is_contiguous()
    except AttributeError:
        return False


_th = _device = _raw_stream = None   # torch, its current device and stream: looked up once


def _torch():
    global _th, _device, _raw_stream
    if _th is None:
        import torch
        _device = torch.cuda.current_device
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
        _th = torch
    return _th


def _call(name, stream, tensors, *args, last=()):
    """Runs one entry point on the device that holds all the tensors (made current for
    the call) and on its current stream, or the given one.  args: those before the stream;
    last: those behind it."""
    th = _th or _torch()
    dev = -2
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if d < 0:
                    raise ValueError("%s: every tensor must be a CUDA tensor" % name)
                if dev != -2:
                    raise ValueError("%s: tensors on cuda:%d and cuda:%d" % (name, dev, d))
                dev = d
    fn = getattr(_lib or load(), name)
    if dev == _device():
        rc = fn(*args, _raw_stream(dev) if stream is None else stream, *last)
    else:
        with th.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev) if stream is None else stream, *last)
    if rc != LSQ_OK:
        _check(rc)


def _addr(t):
    return None if t is None else t.data_ptr()


def packed_index_ints(T, n_docs):
    return int(load().packed_index_ints(int(T), int(n_docs)))


class PackedIndex:
    """The buffer of a packed row's index: n_tokens tokens holding n_docs documents
    (filled by packed_index, once per batch; until then it is that of a row of padding)."""

    def __init__(self, n_tokens, n_docs, device="cuda"):
        import torch
        words = packed_index_ints(n_tokens, n_docs)
        if words <= 0:
            raise ValueError("a packed row has at least one token and one document")
        self.n_tokens, self.n_docs = int(n_tokens), int(n_docs)
        # (zeros: the operators take rows and places to write from it)
        self.buf = torch.zeros(words, dtype=torch.int32, device=device)


def packed_index(lengths, index, prefix=None, stream=None):
    """lengths, prefix: int32 [n_docs] on the device; index: PackedIndex (filled)."""
    i32, n = (_th or _torch()).int32, (index.n_docs,)
    if not _fits(lengths, i32, n):
        _need("lengths", lengths, i32, n)
    if prefix is not None and not _fits(prefix, i32, n):
        _need("prefix", prefix, i32, n)
    _call("packed_index", stream, (lengths, prefix, index.buf), lengths.data_ptr(), _addr(prefix),
          index.n_docs, index.n_tokens, index.buf.data_ptr())


def _packed_heads(qkv, index, n_heads, n_kv_heads):
    n = n_heads + 2 * n_kv_heads
    if n_heads <= 0 or n_kv_heads <= 0 or qkv.dim() != 2 or qkv.shape[1] % n:
        raise ValueError("qkv must be [T, (n_heads + 2 n_kv_heads) d]")
    return qkv.shape[1] // n


def packed_attention_fwd(qkv, index, n_heads, n_kv_heads, o, lse, stream=None):
    """qkv: fp16 [T, (H + 2 Hkv) d]; o: fp16 [T, H d]; lse: fp32 [H, T]."""
    th, T, buf = _th or _torch(), index.n_tokens, index.buf
    d = _packed_heads(qkv, index, n_heads, n_kv_heads)
    for name, t, dtype, shape in (
            ("qkv", qkv, th.float16, (T, (n_heads + 2 * n_kv_heads) * d)),
            ("o", o, th.float16, (T, n_heads * d)), ("lse", lse, th.float32, (n_heads, T))):
        if not _fits(t, dtype, shape):
            _need(name, t, dtype, shape)
    _call("packed_attention_fwd", stream, (qkv, buf, o, lse), qkv.data_ptr(), buf.data_ptr(),
          index.n_docs, T, n_heads, n_kv_heads, d, o.data_ptr(), lse.data_ptr())


def packed_attention_workspace_bytes(T, n_heads, n_kv_heads, d):
    return int(load().packed_attention_workspace_bytes(int(T), n_heads, n_kv_heads, d))


def packed_attention_bwd(qkv, index, o, lse, dout, n_heads, n_kv_heads, dqkv, ws, stream=None):
    """dout: bf16 [T, H d]; dqkv: bf16, the shape of qkv (overwritten); ws: uint8 of
    packed_attention_workspace_bytes."""
    th, T, buf = _th or _torch(), index.n_tokens, index.buf
    d = _packed_heads(qkv, index, n_heads, n_kv_heads)
    wide, hd = (T, (n_heads + 2 * n_kv_heads) * d), (T, n_heads * d)
    for name, t, dtype, shape in (
            ("qkv", qkv, th.float16, wide), ("o", o, th.float16, hd),
            ("lse", lse, th.float32, (n_heads, T)), ("dout", dout, th.bfloat16, hd),
            ("dqkv", dqkv, th.bfloat16, wide)):
        if not _fits(t, dtype, shape):
            _need(name, t, dtype, shape)
    _need("ws", ws, th.uint8)
    _call("packed_attention_bwd", stream, (qkv, buf, o, lse, dout, dqkv, ws), qkv.data_ptr(),
          buf.data_ptr(), index.n_docs, o.data_ptr(), lse.data_ptr(), dout.data_ptr(), T, n_heads,
          n_kv_heads, d, dqkv.data_ptr(), ws.data_ptr(), ws.numel())


def packed_targets(tokens, index, targets, count, loss_mask=None, accumulate=False, stream=None):
    """tokens, targets: int32 [T]; count: int32 [1]; loss_mask: uint8 or bool [T]."""
    import torch
    T = index.n_tokens
    _need("tokens", tokens, torch.int32, numel=T)
    _need("targets", targets, torch.int32, numel=T)
    _need("count", count, torch.int32, numel=1)
    if loss_mask is not None and loss_mask.dtype == torch.bool:
        loss_mask = loss_mask.view(torch.uint8)
    if loss_mask is not None:
        _need("loss_mask", loss_mask, torch.uint8, numel=T)
    _call("packed_targets", stream, (tokens, index.buf, targets, count, loss_mask),
          tokens.data_ptr(), index.buf.data_ptr(), index.n_docs, T, _addr(loss_mask),
          targets.data_ptr(), count.data_ptr(), 1 if accumulate else 0)


def packed_cross_entropy(logits, targets, row_loss, loss, dlogits=None, weight=None, count=None,
                         accumulate=False, stream=None):
    """logits: fp32 [T, V]; targets: int32 [T]; row_loss: fp32 [T]; loss: fp32 [1];
    dlogits: bf16 [T, V]; weight: fp32 [T]; count: int32 [1]."""
    th = _th or _torch()
    if logits.dim() != 2:
        raise ValueError("logits must be [T, V]")
    T, V = logits.shape
    # (targets, row losses and weights may be shaped as their batch is)
    for name, t, dtype, n, optional in (
            ("targets", targets, th.int32, T, False), ("row_loss", row_loss, th.float32, T, False),
            ("loss", loss, th.float32, 1, False), ("weight", weight, th.float32, T, True),
            ("count", count, th.int32, 1, True)):
        if not (t is None and optional) and not _fits(t, dtype, (n,)):
            _need(name, t, dtype, numel=n)
    if not _fits(logits, th.float32, (T, V)):
        _need("logits", logits, th.float32, (T, V))
    if dlogits is not None and not _fits(dlogits, th.bfloat16, (T, V)):
        _need("dlogits", dlogits, th.bfloat16, (T, V))
    _call("packed_cross_entropy", stream, (logits, targets, row_loss, loss, dlogits, weight, count),
          logits.data_ptr(), T, V, targets.data_ptr(), _addr(weight), _addr(count),
          _addr(dlogits), row_loss.data_ptr(), loss.data_ptr(), 1 if accumulate else 0)


def adamw_scale_floats(n):
    return int(load().adamw_scale_floats(int(n)))


def _state_signed(codes):
    th = _th or _torch()
    if codes.dtype is th.int8:
        return 1
    if codes.dtype is th.uint8:
        return 0
    raise TypeError("codes must be int8 (m) or uint8 (v)")


def adamw_state_dequantize(codes, scale, out, stream=None):
    """codes: int8 (m) or uint8 (v); scale: fp32 per 256 codes; out: fp32."""
    th = _th or _torch()
    signed, n = _state_signed(codes), codes.numel()
    _need("codes", codes, codes.dtype)
    _need("scale", scale, th.float32, numel=(n + 255) // 256)
    _need("out", out, th.float32, numel=n)
    _call("adamw_state_dequantize", stream, (codes, scale, out), codes.data_ptr(),
          scale.data_ptr(), n, signed, out.data_ptr())


def adamw_state_quantize(x, codes, scale, stream=None):
    """The inverse: x fp32 to int8 (m) or uint8 (v) codes and their scales."""
    import torch
    signed, n = _state_signed(codes), codes.numel()
    _need("codes", codes, codes.dtype)
    _need("x", x, torch.float32, numel=n)
    _need("scale", scale, torch.float32, numel=adamw_scale_floats(n))
    _call("adamw_state_quantize", stream, (x, codes, scale), x.data_ptr(), n, signed,
          codes.data_ptr(), scale.data_ptr())


class AdamWMulti:
    """AdamW over lists of tensors, one adamw_multi_step per step.

    params: fp32; grads: all fp32 or all bf16; m, v: fp32 (32-bit state), or int8 and
    uint8 with m_scale, v_scale (8-bit state, fp32 scales of adamw_scale_floats(numel)).
    lr, weight_decay: one number or one per tensor (set_rates changes them between steps).
    The tensors are checked and their addresses taken here; they must stay allocated while the
    object is used."""

    def __init__(self, params, grads, m, v, lr, weight_decay=0.0, m_scale=None, v_scale=None,
                 betas=(0.9, 0.999), eps=1e-8):
        import torch
        n = len(params)
        bits = 8 if n and m[0].dtype == torch.int8 else 32
        gdt = grads[0].dtype if n else torch.float32
        if gdt not in (torch.float32, torch.bfloat16):
            raise TypeError("gradients must be float32 or bfloat16")
        lists = [params, grads, m, v] + ([m_scale, v_scale] if bits == 8 else [])
        if any(x is None or len(x) != n for x in lists):
            raise ValueError("params, grads, m, v%s need one tensor each per parameter"
                             % (", m_scale, v_scale" if bits == 8 else ""))
        self._table = (lsq_adamw_tensor * max(n, 1))()
        self._n, self._keep = n, lists
        rates = self._per_tensor("lr", lr), self._per_tensor("weight_decay", weight_decay)
        self._dev = params[0] if n else None
        names = ("params", "grads", "m", "v", "m_scale", "v_scale")
        mdt, vdt = (torch.int8, torch.uint8) if bits == 8 else (torch.float32, torch.float32)
        dtypes = (torch.float32, gdt, mdt, vdt, torch.float32, torch.float32)
        for i in range(n):
            ts = [x[i] for x in lists]
            k = ts[0].numel() if isinstance(ts[0], torch.Tensor) else 0
            sizes = (k, k, k, k, (k + 255) // 256, (k + 255) // 256)
            for j, t in enumerate(ts):
                if not (isinstance(t, torch.Tensor) and t.dtype is dtypes[j] and
                        t.numel() == sizes[j] and t.is_contiguous()):
                    _need("%s[%d]" % (names[j], i), t, dtypes[j], numel=sizes[j])
                if not t.is_cuda:
                    raise ValueError("tensor %d is not on a CUDA device" % i)
                if t.get_device() != self._dev.get_device():
                    raise ValueError("tensor %d is on %s, the first on %s"
                                     % (i, t.device, self._dev.device))
            self._table[i] = lsq_adamw_tensor(*[t.data_ptr() for t in ts],
                                              *[None] * (6 - len(ts)), k)
        self._hyper = lsq_adamw_hyper(beta1=betas[0], beta2=betas[1], eps=eps, step=1,
                                      state_bits=bits,
                                      grad_bits=32 if gdt == torch.float32 else 16)
        self.set_rates(*rates)

    def _per_tensor(self, name, x):
        x = [float(v) for v in x] if hasattr(x, "__len__") else [float(x)] * self._n
        if len(x) != self._n:
            raise ValueError("%s needs one number per parameter" % name)
        return x

    def set_rates(self, lr, weight_decay=None):
        """The rates of the steps that follow (a schedule's): one number or one per tensor;
        weight_decay None: as it was.  A captured step keeps the rates it was captured with."""
        lr = self._per_tensor("lr", lr)
        if weight_decay is not None:
            for e, x in zip(self._table, self._per_tensor("weight_decay", weight_decay)):
                e.weight_decay = x
        for e, x in zip(self._table, lr):
            e.lr = x

    def at(self, step):
        """The arguments (tensors, n_tensors, opt) of an update; step as for step()."""
        import torch
        h = self._hyper
        if isinstance(step, torch.Tensor):
            _need("step", step, torch.int32, numel=1)
            h.step, h.step_dev = 1, step.data_ptr()
        else:
            h.step, h.step_dev = int(step), None
        return self._table, self._n, h

    def step(self, step, stream=None):
        """One update; step: the count from 1, or an int32 device tensor that holds it
        (for a captured update that is replayed as the count advances)."""
        import torch
        h = self.at(step)[2]
        if self._n == 0:
            return
        _call("adamw_multi_step", stream,
              (self._dev, step if isinstance(step, torch.Tensor) else None), self._table, self._n,
              ctypes.byref(h))


# ------------------------------------------------------------ packed layers and steps
def _need_layer(cfg, blob, loras, ws):
    """The arguments of a packed layer that are sized by the configuration: the blob (uint8, at
    least the layout's bytes), LoRA buffers (fp32, one layer's; None passes), the workspace."""
    import torch
    _need("ws", ws, torch.uint8)
    _need("blob", blob, torch.uint8)
    size = lsq_layer_layout_get(cfg).bytes
    if blob.numel() < size:
        raise ValueError("blob has %d bytes, the layer %d" % (blob.numel(), size))
    for name, t in loras:
        if t is not None:
            _need(name, t, torch.float32, numel=lsq_lora_layout_get(cfg).floats_per_layer)


def decoder_layer_packed_fwd(cfg, blob, lora, x_in, index, x_out, ws, stream=None):
    """x_in, x_out: fp32 [n_tokens, D] of one packed row; index: its PackedIndex; lora: fp32 of
    one layer, or None (adapter off); ws: uint8."""
    import torch
    T = index.n_tokens
    _need("x_in", x_in, torch.float32, (T, cfg["hidden"]))
    _need("x_out", x_out, torch.float32, (T, cfg["hidden"]))
    _need_layer(cfg, blob, (("lora", lora),), ws)
    c = cfg_struct(cfg)
    _call("decoder_layer_packed_fwd", stream, (blob, lora, x_in, index.buf, x_out, ws),
          ctypes.byref(c), blob.data_ptr(), _addr(lora), x_in.data_ptr(), index.buf.data_ptr(),
          index.n_docs, T, x_out.data_ptr(), ws.data_ptr(), ws.numel())


def decoder_layer_packed_bwd(cfg, blob, lora, x_in, dx_out, index, dx_in, lora_grad, ws,
                             accumulate=False, stream=None):
    import torch
    T = index.n_tokens
    for name, t in (("x_in", x_in), ("dx_out", dx_out), ("dx_in", dx_in)):
        _need(name, t, torch.float32, (T, cfg["hidden"]))
    if lora is None or lora_grad is None:
        raise TypeError("the backward needs lora and lora_grad")
    _need_layer(cfg, blob, (("lora", lora), ("lora_grad", lora_grad)), ws)
    c = cfg_struct(cfg)
    _call("decoder_layer_packed_bwd", stream, (blob, lora, x_in, dx_out, index.buf, dx_in,
                                               lora_grad, ws),
          ctypes.byref(c), blob.data_ptr(), lora.data_ptr(), x_in.data_ptr(), dx_out.data_ptr(),
          index.buf.data_ptr(), index.n_docs, T, dx_in.data_ptr(), lora_grad.data_ptr(),
          1 if accumulate else 0, ws.data_ptr(), ws.numel())


def stream_stack_packed_workspace_bytes(cfg, n_tokens, n_docs):
    c = cfg_struct(cfg)
    return load().stream_stack_packed_workspace_bytes(ctypes.byref(c), n_tokens, n_docs)


def stream_stack_packed_step(stack, tokens, lengths, emb, lm_head, final_norm, lora, lora_grad, ws,
                             prefix=None, loss_mask=None, opt=None, step=1, logits_out=None,
                             timeout_ms=600000, stream=None):
    """One SFT step on packed rows.  tokens: int32 [micro_batches, n_tokens]; lengths, prefix:
    int32 [micro_batches, n_docs]; loss_mask: uint8 or bool [micro_batches, n_tokens]; emb,
    lm_head: bf16 [V, D]; final_norm: bf16 [D]; lora, lora_grad: fp32 of all layers; ws: uint8;
    opt: an AdamWMulti over views of lora and lora_grad, updated with the count `step`, or None;
    logits_out: fp32 [n_tokens, V] or None.  Returns the mean loss over all targets (host float)."""
    import torch
    if tokens.dim() != 2 or lengths.dim() != 2 or lengths.shape[0] != tokens.shape[0]:
        raise ValueError("tokens must be [micro_batches, n_tokens], lengths [micro_batches, n_docs]")
    _need("tokens", tokens, torch.int32)
    _need("lengths", lengths, torch.int32)
    if prefix is not None:
        _need("prefix", prefix, torch.int32, lengths.shape)
    if loss_mask is not None:
        if loss_mask.dtype == torch.bool:
            loss_mask = loss_mask.view(torch.uint8)
        _need("loss_mask", loss_mask, torch.uint8, tokens.shape)
    c, bf16 = stack.cfg, torch.bfloat16
    layout = lsq_lora_layout()
    _check(load().lsq_lora_layout_get(ctypes.byref(c), ctypes.byref(layout)))
    _need("emb", emb, bf16, (c.vocab, c.hidden))
    _need("lm_head", lm_head, bf16, (c.vocab, c.hidden))
    _need("final_norm", final_norm, bf16, numel=c.hidden)
    _need("lora", lora, torch.float32, numel=layout.floats_per_layer * c.n_layers)
    _need("lora_grad", lora_grad, torch.float32, numel=lora.numel())
    if logits_out is not None:
        _need("logits_out", logits_out, torch.float32, (tokens.shape[1], c.vocab))
    _need("ws", ws, torch.uint8)
    loss = ctypes.c_float(0.0)
    table, n, hyper = opt.at(step) if opt is not None else (None, 0, None)
    _call("stream_stack_packed_step", stream,
          (tokens, lengths, prefix, loss_mask, emb, lm_head, final_norm, lora, lora_grad, logits_out,
           ws, opt._dev if opt is not None else None,
           step if opt is not None and isinstance(step, torch.Tensor) else None),
          stack.handle, tokens.data_ptr(), tokens.shape[0], tokens.shape[1], lengths.data_ptr(),
          _addr(prefix), lengths.shape[1], _addr(loss_mask), emb.data_ptr(), lm_head.data_ptr(),
          final_norm.data_ptr(), lora.data_ptr(), lora_grad.data_ptr(), table, n,
          ctypes.byref(hyper) if hyper is not None else None, ctypes.byref(loss),
          _addr(logits_out), ws.data_ptr(), ws.numel(), last=(timeout_ms,))
    return loss.value
