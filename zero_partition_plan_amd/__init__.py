"""Python binding of libzero_shard: one data-parallel rank's sharded ZeRO optimizer step on MI355X.

Argument marshalling only. Every step of the path runs in the HIP kernels of libzero_shard.so;
torch supplies device memory and the stream. The entry points carry the names of the C ABI in
``include/zero_shard.h``, where each one's arithmetic, layout, ownership and errors are stated.

The library must be built (``python -m zero_partition_plan_amd.build``); importing this package
without it raises, there is no fallback.
"""

from __future__ import annotations

import ctypes
import os

import torch  # noqa: F401  (loaded first so the library binds to the HIP runtime torch uses)

__all__ = [
    "ZeroError", "ZeroPlan", "ZeroAdamHParams", "ZeroAdamScalars", "ZeroStageChoice",
    "ZeroOffloadBuffers", "lib", "lib_path", "offload_buffers",
    "ZERO_MAX_REPLICAS", "ZERO_MAX_SHARDS", "ZERO_F32", "ZERO_F16", "ZERO_BF16",
    "ZERO_ADAMW", "ZERO_ADAM_L2", "ZERO_DEV_T_OUT_OF_TABLE", "adam_hparams",
    "zero_partition_plan", "zero_shard_range", "zero_stage_bytes", "zero_stage_comm_bytes",
    "zero_choose_stage",
    "zero_adam_derive", "ZeroArenaArray", "zero_arena_layout", "zero_arena_alloc", "zero_arena_free",
    "arena",
    "zero_sq_partials_len", "zero_reduce_shard", "zero_shard_sqnorm", "zero_reduce_shard_static",
    "ZERO_STATIC_SQ_PARTIALS", "ZERO_STATIC_MAX_ELEMS", "zero_adam_shard_step",
    "zero_adam_shard_step_dev_scale", "zero_clip_scale", "zero_adam_derive_table", "adam_table",
    "zero_adam_shard_step_dev_t",
    "AdamStep", "ReduceCall",
    "ZeroAdamTensor", "ZERO_STATE8_BLOCK", "ZERO_ADAM_MAX_TENSORS", "ZERO_ADAM_MAX_GROUPS", "adam_tensor",
    "adam_state", "zero_adam_tensors_step", "zero_adam_tensors_step_dev_t", "AdamTensorsStep",
    "zero_adam_state_values", "zero_adam_state_codes",
    "zero_gather_params", "zero_host_adam_step", "zero_offload_step",
    "ZeroLinearShape", "ZERO_ACT_NONE", "ZERO_ACT_RELU", "ZERO_ACT_GELU", "ZERO_ACT_GELU_TANH",
    "ZERO_ACT_SILU", "zero_linear_workspace_bytes", "zero_linear_forward", "zero_linear_backward",
    "ZeroDistillIn", "ZERO_DISTILL_MAX_TOPK", "ZERO_DISTILL_MAX_VOCAB", "zero_distill_forward",
    "zero_distill_backward", "zero_distill_step",
    "ZeroNormBlock", "ZERO_NORM_NONE", "ZERO_NORM_RMS", "ZERO_NORM_LAYER", "ZERO_NORM_MAX_FEATURES",
    "zero_norm_forward", "zero_norm_backward", "zero_norm_workspace_bytes",
    "ZeroTokenIn", "ZeroPolicy", "ZeroPreference", "ZERO_TOKEN_STATS", "zero_token_logp", "zero_policy_forward",
    "zero_policy_step", "zero_preference_forward", "zero_token_backward",
    "zero_status_str", "zero_last_error",
]

ZERO_MAX_REPLICAS = 64
ZERO_MAX_SHARDS = 64
ZERO_OK, ZERO_E_INVAL, ZERO_E_OVERFLOW, ZERO_E_UNSUPPORTED, ZERO_E_HIP = range(5)
ZERO_F32, ZERO_F16, ZERO_BF16 = 0, 1, 2
ZERO_ADAMW, ZERO_ADAM_L2 = 0, 1
ZERO_DEV_T_OUT_OF_TABLE = 1
ZERO_ACT_NONE, ZERO_ACT_RELU, ZERO_ACT_GELU, ZERO_ACT_GELU_TANH, ZERO_ACT_SILU = range(5)
ZERO_DISTILL_MAX_TOPK = 1024
ZERO_DISTILL_MAX_VOCAB = 393216
ZERO_STATIC_SQ_PARTIALS = 4 << 20
ZERO_STATIC_MAX_ELEMS = (ZERO_STATIC_SQ_PARTIALS - 1024) * 256

ZERO_NORM_NONE, ZERO_NORM_RMS, ZERO_NORM_LAYER = range(3)
ZERO_NORM_MAX_FEATURES = 16384
ZERO_STATE8_BLOCK = 256
ZERO_TOKEN_STATS = 8
ZERO_ADAM_MAX_TENSORS = 65536
ZERO_ADAM_MAX_GROUPS = 16

_TORCH_DT = {torch.float32: ZERO_F32, torch.float16: ZERO_F16, torch.bfloat16: ZERO_BF16}


class ZeroError(RuntimeError):
    def __init__(self, status: int, fn: str, detail: str):
        self.status = status
        super().__init__(f"{fn}: {zero_status_str(status)} ({detail})")


class ZeroPlan(ctypes.Structure):
    _fields_ = [("n", ctypes.c_uint64), ("padded_n", ctypes.c_uint64),
                ("shard_elems", ctypes.c_uint64), ("pad", ctypes.c_uint64),
                ("nd", ctypes.c_uint32), ("align_elems", ctypes.c_uint32)]

    def __repr__(self):
        return (f"ZeroPlan(n={self.n}, padded_n={self.padded_n}, shard_elems={self.shard_elems}, "
                f"pad={self.pad}, nd={self.nd}, align_elems={self.align_elems})")


class _GradSrc(ctypes.Structure):
    _fields_ = [("ptrs", ctypes.POINTER(ctypes.c_void_p)), ("count", ctypes.c_uint32),
                ("dtype", ctypes.c_int32)]


class ZeroAdamHParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("wd_mode", ctypes.c_int32), ("reserved", ctypes.c_int32), ("step", ctypes.c_int64)]


class ZeroStageChoice(ctypes.Structure):
    _fields_ = [("stage", ctypes.c_uint32), ("offload_advised", ctypes.c_uint32),
                ("bytes", ctypes.c_uint64 * 4)]


class ZeroOffloadBuffers(ctypes.Structure):
    _fields_ = [("d_grad", ctypes.c_void_p), ("h_grad", ctypes.c_void_p), ("h_param", ctypes.c_void_p),
                ("chunk_elems", ctypes.c_uint64), ("threads", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("h2d_stream", ctypes.c_void_p),
                ("events", ctypes.c_void_p * 4)]


class ZeroArenaArray(ctypes.Structure):
    _fields_ = [("bytes", ctypes.c_uint64), ("hot_offset", ctypes.c_uint64), ("group", ctypes.c_uint32),
                ("elem_bytes", ctypes.c_uint32)]


class ZeroAdamScalars(ctypes.Structure):
    _fields_ = [(k, ctypes.c_float) for k in ("b1", "b2", "c1", "c2", "ss", "bc", "e", "dec", "w")]


class ZeroAdamTensor(ctypes.Structure):
    _fields_ = [("n", ctypes.c_uint64)] + [(k, ctypes.c_void_p) for k in (
        "param", "grad", "out_param", "m", "v", "m_scale", "v_scale")] + [
        ("group", ctypes.c_uint32), ("state_bits", ctypes.c_uint32)]


class ZeroLinearShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_uint64), ("in_features", ctypes.c_uint64),
                ("out_features", ctypes.c_uint64), ("dtype", ctypes.c_int32), ("act", ctypes.c_int32)]


class ZeroDistillIn(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_uint64), ("vocab", ctypes.c_uint64), ("topk", ctypes.c_uint64),
                ("logit_dtype", ctypes.c_int32), ("teacher_dtype", ctypes.c_int32),
                ("index_bytes", ctypes.c_int32), ("temperature", ctypes.c_float),
                ("logits", ctypes.c_void_p), ("ld_logits", ctypes.c_uint64),
                ("top_index", ctypes.c_void_p), ("top_logits", ctypes.c_void_p),
                ("ld_top", ctypes.c_uint64), ("tail", ctypes.c_void_p), ("weight", ctypes.c_void_p)]


class ZeroNormBlock(ctypes.Structure):
    _fields_ = [(k, ctypes.c_uint64) for k in ("rows", "features", "gate_rows")] + [
        (k, ctypes.c_int32) for k in ("dtype", "stream_dtype", "post", "pre")] + [
        (k, ctypes.c_float) for k in ("eps", "residual_scale", "branch_scale")] + [
        ("reserved", ctypes.c_int32), ("branch", ctypes.c_void_p), ("ld_branch", ctypes.c_uint64),
        ("gate", ctypes.c_void_p), ("ld_gate", ctypes.c_uint64)] + [
        (k, ctypes.c_void_p) for k in ("post_weight", "post_bias", "pre_weight", "pre_bias")]


class ZeroTokenIn(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_uint64), ("vocab", ctypes.c_uint64), ("logit_dtype", ctypes.c_int32),
                ("label_bytes", ctypes.c_int32), ("temperature", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("logits", ctypes.c_void_p), ("ld_logits", ctypes.c_uint64), ("label", ctypes.c_void_p)]


class ZeroPolicy(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("old_logp", "advantage", "ref_logp", "weight")] + [
        (k, ctypes.c_float) for k in ("clip_low", "clip_high", "kl_coef")] + [("reserved", ctypes.c_int32)]


class ZeroPreference(ctypes.Structure):
    _fields_ = [("pairs", ctypes.c_uint64), ("seq_start", ctypes.c_void_p), ("start_bytes", ctypes.c_int32),
                ("average", ctypes.c_int32), ("ref_logp", ctypes.c_void_p), ("weight", ctypes.c_void_p)] + [
        (k, ctypes.c_float) for k in ("beta", "label_smoothing", "margin")] + [("reserved", ctypes.c_int32)]


def adam_hparams(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, wd_mode="adamw",
                 step=1) -> ZeroAdamHParams:
    mode = {"adamw": ZERO_ADAMW, "l2": ZERO_ADAM_L2}.get(wd_mode, wd_mode)
    return ZeroAdamHParams(lr, beta1, beta2, eps, weight_decay, int(mode), 0, int(step))


_lib = None


def lib_path() -> str:
    return os.environ.get("ZERO_SHARD_LIB") or os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                            "libzero_shard.so")


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is not built: run `python -m zero_partition_plan_amd.build`")
        L = ctypes.CDLL(path)
        u64, u32, i32, vp = ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int32, ctypes.c_void_p
        P = ctypes.POINTER
        sig = {
            "zero_partition_plan": [u64, u32, u32, P(ZeroPlan)],
            "zero_shard_range": [P(ZeroPlan), u32, P(u64), P(u64)],
            "zero_stage_bytes": [P(ZeroPlan), u32, u32, u32, u32, P(u64)],
            "zero_stage_comm_bytes": [P(ZeroPlan), u32, u32, u32, P(u64)],
            "zero_choose_stage": [P(ZeroPlan), u64, u32, u32, u32, P(ZeroStageChoice)],
            "zero_adam_derive": [P(ZeroAdamHParams), P(ZeroAdamScalars)],
            "zero_arena_layout": [P(ZeroArenaArray), u32, P(u64), P(u64)],
            "zero_arena_alloc": [u64, P(vp), P(i32)],
            "zero_arena_free": [vp],
            "zero_reduce_shard": [P(_GradSrc), u64, vp, vp, vp, ctypes.c_double, vp],
            "zero_shard_sqnorm": [vp, u64, ctypes.c_double, vp, vp, vp],
            "zero_reduce_shard_static": [P(_GradSrc), u64, vp, vp, ctypes.c_double, vp, vp],
            "zero_adam_shard_step": [P(_GradSrc), u64, ctypes.c_float, vp, vp, vp,
                                     P(ZeroAdamHParams), vp, i32, vp, vp],
            "zero_adam_shard_step_dev_scale": [P(_GradSrc), u64, vp, vp, vp, vp,
                                               P(ZeroAdamHParams), vp, i32, vp, vp],
            "zero_clip_scale": [vp, ctypes.c_double, ctypes.c_double, ctypes.c_double, vp, vp],
            "zero_adam_derive_table": [P(ZeroAdamHParams), u32, P(ZeroAdamScalars)],
            "zero_adam_shard_step_dev_t": [P(_GradSrc), u64, vp, vp, u32, vp, vp, i32, vp, vp, vp,
                                           vp, i32, vp, vp],
            "zero_adam_tensors_step": [P(ZeroAdamTensor), u32, i32, i32, P(ZeroAdamHParams), u32,
                                       ctypes.c_float, vp, vp, vp],
            "zero_adam_tensors_step_dev_t": [P(ZeroAdamTensor), u32, i32, i32, vp, vp, u32, u32, vp,
                                             vp, i32, vp, vp],
            "zero_adam_state_values": [vp, vp, u64, i32, vp, vp],
            "zero_adam_state_codes": [vp, u64, i32, vp, vp, vp],
            "zero_gather_params": [P(vp), u32, u64, u32, u64, u64, vp, vp],
            "zero_host_adam_step": [vp, u64, ctypes.c_float, vp, vp, vp, P(ZeroAdamHParams), vp, i32,
                                    u32],
            "zero_offload_step": [P(_GradSrc), u64, ctypes.c_float, vp, vp, vp, P(ZeroAdamHParams),
                                  vp, i32, P(ZeroOffloadBuffers), vp],
            "zero_linear_forward": [P(ZeroLinearShape), vp, u64, vp, vp, vp, u64, vp, u64, vp, u64,
                                    vp, u64, vp],
            "zero_linear_backward": [P(ZeroLinearShape), vp, u64, vp, u64, vp, vp, u64, vp, u64, vp,
                                     u64, vp, vp, i32, i32, vp, u64, vp],
            "zero_distill_forward": [P(ZeroDistillIn), vp, vp, vp],
            "zero_distill_backward": [P(ZeroDistillIn), vp, vp, ctypes.c_float, vp, u64, vp],
            "zero_distill_step": [P(ZeroDistillIn), vp, ctypes.c_float, vp, vp, u64, vp],
            "zero_norm_forward": [P(ZeroNormBlock), vp, u64, vp, u64, vp, u64, vp, vp],
            "zero_norm_backward": [P(ZeroNormBlock), vp, vp, u64, vp, u64, vp, u64, vp, u64, vp, u64, vp, u64,
                                   vp, vp, vp, vp, i32, i32, vp, u64, vp],
            "zero_token_logp": [P(ZeroTokenIn), vp, vp, vp],
            "zero_policy_forward": [P(ZeroTokenIn), P(ZeroPolicy), vp, vp, vp, vp],
            "zero_policy_step": [P(ZeroTokenIn), P(ZeroPolicy), vp, ctypes.c_float, vp, vp, vp, u64, vp],
            "zero_preference_forward": [P(ZeroTokenIn), P(ZeroPreference), vp, vp, vp, vp, vp],
            "zero_token_backward": [P(ZeroTokenIn), vp, vp, u64, ctypes.c_float, vp, u64, vp],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.zero_sq_partials_len.argtypes = [u64]
        L.zero_sq_partials_len.restype = u64
        L.zero_linear_workspace_bytes.argtypes = [u64, u64, u64, i32]
        L.zero_linear_workspace_bytes.restype = u64
        L.zero_norm_workspace_bytes.argtypes = [u64, u64, u64]
        L.zero_norm_workspace_bytes.restype = u64
        L.zero_status_str.argtypes = [ctypes.c_int]
        L.zero_status_str.restype = ctypes.c_char_p
        L.zero_last_error.argtypes = []
        L.zero_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def zero_status_str(status: int) -> str:
    return lib().zero_status_str(status).decode()


def zero_last_error() -> str:
    return lib().zero_last_error().decode()


def _check(status: int, fn: str):
    if status != ZERO_OK:
        raise ZeroError(status, fn, zero_last_error())


# ------------------------------------------------------------------------------ host-only calls

def zero_partition_plan(n: int, nd: int, align_elems: int = 1) -> ZeroPlan:
    p = ZeroPlan()
    _check(lib().zero_partition_plan(n, nd, align_elems, ctypes.byref(p)), "zero_partition_plan")
    return p


def zero_shard_range(plan: ZeroPlan, rank: int) -> tuple[int, int]:
    b, v = ctypes.c_uint64(), ctypes.c_uint64()
    _check(lib().zero_shard_range(ctypes.byref(plan), rank, ctypes.byref(b), ctypes.byref(v)),
           "zero_shard_range")
    return b.value, v.value


def zero_stage_bytes(plan: ZeroPlan, stage: int, param_b: int = 2, grad_b: int = 2,
                     opt_b: int = 12) -> tuple[int, int, int, int]:
    out = (ctypes.c_uint64 * 4)()
    _check(lib().zero_stage_bytes(ctypes.byref(plan), stage, param_b, grad_b, opt_b, out),
           "zero_stage_bytes")
    return tuple(int(x) for x in out)


def zero_stage_comm_bytes(plan: ZeroPlan, stage: int, param_b: int = 2,
                          grad_b: int = 2) -> tuple[int, int, int]:
    """(gradient, parameter, total) bytes one rank sends per step; stage 0 = DP, 1..3."""
    out = (ctypes.c_uint64 * 3)()
    _check(lib().zero_stage_comm_bytes(ctypes.byref(plan), stage, param_b, grad_b, out),
           "zero_stage_comm_bytes")
    return tuple(int(x) for x in out)


def zero_choose_stage(plan: ZeroPlan, usable_bytes: int, param_b: int = 2, grad_b: int = 2,
                      opt_b: int = 12) -> tuple[int, bool, tuple[int, int, int, int]]:
    """(stage 1..3, offload advised, the stage's per-rank bytes) for a usable byte budget."""
    out = ZeroStageChoice()
    _check(lib().zero_choose_stage(ctypes.byref(plan), usable_bytes, param_b, grad_b, opt_b,
                                   ctypes.byref(out)), "zero_choose_stage")
    return int(out.stage), bool(out.offload_advised), tuple(int(x) for x in out.bytes)


def zero_adam_derive(hp: ZeroAdamHParams) -> ZeroAdamScalars:
    out = ZeroAdamScalars()
    _check(lib().zero_adam_derive(ctypes.byref(hp), ctypes.byref(out)), "zero_adam_derive")
    return out


def zero_adam_derive_table(hp: ZeroAdamHParams, count: int):
    """The constants of steps 1..count (hp.step ignored) as a ctypes array of ZeroAdamScalars."""
    out = (ZeroAdamScalars * count)()
    _check(lib().zero_adam_derive_table(ctypes.byref(hp), count, out), "zero_adam_derive_table")
    return out


def adam_table(hp: ZeroAdamHParams, count: int, device="cuda") -> torch.Tensor:
    """zero_adam_derive_table's constants as a (count, 9) float32 tensor on ``device``, laid out
    as the device table of zero_adam_shard_step_dev_t expects (one zero_adam_scalars per row)."""
    tab = zero_adam_derive_table(hp, count)
    host = torch.frombuffer(bytearray(tab), dtype=torch.float32).view(count, 9)
    return host.to(device)


def zero_arena_layout(arrays) -> tuple[list[int], int]:
    """arrays: sequence of (bytes, hot_offset, group, elem_bytes) -> (byte offsets, total bytes)."""
    n = len(arrays)
    arr = (ZeroArenaArray * max(n, 1))(*[ZeroArenaArray(int(b), int(h), int(g), int(e))
                                         for b, h, g, e in arrays])
    offs = (ctypes.c_uint64 * max(n, 1))()
    total = ctypes.c_uint64()
    _check(lib().zero_arena_layout(arr, n, offs, ctypes.byref(total)), "zero_arena_layout")
    return [int(offs[i]) for i in range(n)], int(total.value)


def zero_arena_alloc(nbytes: int) -> tuple[int | None, bool]:
    """(device pointer, physically contiguous?) of a new allocation on the current device."""
    ptr, contig = ctypes.c_void_p(), ctypes.c_int32()
    _check(lib().zero_arena_alloc(nbytes, ctypes.byref(ptr), ctypes.byref(contig)), "zero_arena_alloc")
    return ptr.value, bool(contig.value)


def zero_arena_free(ptr: int | None):
    _check(lib().zero_arena_free(ptr), "zero_arena_free")


class _ArenaMemory:
    """Owner of one zero_arena_alloc allocation, handed to torch as a uint8 array. torch keeps this
    object alive while any tensor on the memory lives, and the memory is freed with it."""

    def __init__(self, nbytes: int):
        self.ptr, self.contiguous = zero_arena_alloc(nbytes)
        self.__cuda_array_interface__ = {"shape": (nbytes,), "typestr": "|u1", "strides": None,
                                         "data": (self.ptr, False), "version": 2}

    def __del__(self):
        # a destructor does not raise; hipFree waits for the device before releasing the memory
        ptr, self.ptr = getattr(self, "ptr", None), None
        if ptr and _lib is not None:
            _lib.zero_arena_free(ptr)


def arena(specs, device="cuda", contiguous: bool = True):
    """One device allocation holding every array of ``specs`` where zero_arena_layout places it.

    specs: sequence of (name, numel, dtype, group, hot_elem): hot_elem is the element at which the
    kernels' walk over the array starts (0, or r*S for rank r's slot in a gathered buffer). With
    ``contiguous`` (device memory only) the allocation comes from zero_arena_alloc, physically
    contiguous when the device can give it; otherwise from torch. Returns (storage, {name: 1-D
    view}); the views live as long as the storage, and ``storage.zero_arena_contiguous`` says
    whether the memory is physically contiguous.
    """
    specs = list(specs)
    es = [torch.empty(0, dtype=dt).element_size() for _, _, dt, _, _ in specs]
    offs, total = zero_arena_layout([(n * e, h * e, g, e) for (_, n, _, g, h), e in zip(specs, es)])
    dev = torch.device(device)
    if contiguous and dev.type == "cuda":
        with torch.cuda.device(dev):
            mem = _ArenaMemory(max(total, 1))
            storage = torch.as_tensor(mem, device=dev)
        if storage.data_ptr() != mem.ptr or storage.numel() != max(total, 1):
            raise RuntimeError("torch did not wrap the arena allocation in place")
        storage.zero_arena_contiguous = mem.contiguous
    else:
        storage = torch.empty(max(total, 1), dtype=torch.uint8, device=dev)
        storage.zero_arena_contiguous = False
    views = {name: storage[o:o + n * e].view(dt) for (name, n, dt, _, _), o, e in zip(specs, offs, es)}
    return storage, views


# ------------------------------------------------------------------------------ device calls

def _ptr(t, n: int, what: str, dtype=None, pinned_ok: bool = False) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not (t.is_cuda or (pinned_ok and t.is_pinned())):
        raise TypeError(f"{what} must be a device tensor" + (" or pinned host memory" if pinned_ok else ""))
    if dtype is not None and t.dtype not in dtype:
        raise TypeError(f"{what}: dtype {t.dtype} not in {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.numel() < n:
        raise ValueError(f"{what} holds {t.numel()} elements, {n} needed")
    return t.data_ptr()


def _src(reps, n: int):
    """Replica list (or a 2-D tensor whose rows are replicas) -> C gradient source."""
    rows = list(reps.unbind(0)) if isinstance(reps, torch.Tensor) and reps.dim() == 2 else list(reps)
    if not rows:
        raise ValueError("no gradient replicas")
    dt = rows[0].dtype
    if dt not in _TORCH_DT or any(r.dtype != dt for r in rows):
        raise TypeError("replicas must share one of float32, float16, bfloat16")
    arr = (ctypes.c_void_p * len(rows))(*[_ptr(r, n, f"replica {k}") for k, r in enumerate(rows)])
    return _GradSrc(ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)), len(rows), _TORCH_DT[dt]), arr


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def zero_sq_partials_len(n: int) -> int:
    """Doubles the squared-norm partials buffer needs for a shard of n elements."""
    return int(lib().zero_sq_partials_len(n))


def zero_reduce_shard(reps, n: int, out_grad=None, nonfinite=None, sq_partials=None,
                      sq_scale: float = 1.0, stream=None):
    """``out_grad`` may also be pinned host memory, which the kernel then writes over the host link."""
    src, keep = _src(reps, n)
    _check(lib().zero_reduce_shard(
        ctypes.byref(src), n, _ptr(out_grad, n, "out_grad", (torch.float32,), pinned_ok=True),
        _ptr(nonfinite, 1, "nonfinite", (torch.int32,)),
        _ptr(sq_partials, zero_sq_partials_len(n), "sq_partials", (torch.float64,)),
        float(sq_scale), _stream(stream)), "zero_reduce_shard")


def zero_shard_sqnorm(grad, n: int, sq_scale: float, partials, out, stream=None):
    _check(lib().zero_shard_sqnorm(
        _ptr(grad, n, "grad", (torch.float32,)), n, float(sq_scale),
        _ptr(partials, zero_sq_partials_len(n), "partials", (torch.float64,)),
        _ptr(out, 1, "out", (torch.float64,)), _stream(stream)), "zero_shard_sqnorm")


def zero_reduce_shard_static(reps, n: int, out_grad=None, nonfinite=None, sq=None,
                             sq_scale: float = 1.0, stream=None):
    """zero_reduce_shard then the squared-norm finish into ``sq`` (float64 device tensor), with the
    partials in the library's own device scratch: no workspace argument, nothing allocated."""
    src, keep = _src(reps, n)
    _check(lib().zero_reduce_shard_static(
        ctypes.byref(src), n, _ptr(out_grad, n, "out_grad", (torch.float32,)),
        _ptr(nonfinite, 1, "nonfinite", (torch.int32,)), float(sq_scale),
        _ptr(sq, 1, "sq", (torch.float64,)), _stream(stream)), "zero_reduce_shard_static")


def _out_dtype(out) -> int:
    if out is None:
        return ZERO_F32
    if out.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("out must be bfloat16 or float16")
    return _TORCH_DT[out.dtype]


def zero_adam_shard_step(reps, n: int, grad_scale: float, master, m, v, hp: ZeroAdamHParams,
                         out=None, skip=None, stream=None):
    """``out``: bf16/fp16 device tensor view starting at the rank's slot (or None)."""
    src, keep = _src(reps, n)
    f32 = (torch.float32,)
    out_dt = _out_dtype(out)
    _check(lib().zero_adam_shard_step(
        ctypes.byref(src), n, float(grad_scale), _ptr(master, n, "master", f32),
        _ptr(m, n, "m", f32), _ptr(v, n, "v", f32), ctypes.byref(hp),
        _ptr(out, n, "out"), out_dt, _ptr(skip, 1, "skip", (torch.int32,)), _stream(stream)),
        "zero_adam_shard_step")


def zero_adam_shard_step_dev_scale(reps, n: int, grad_scale, master, m, v, hp: ZeroAdamHParams,
                                   out=None, skip=None, stream=None):
    """zero_adam_shard_step with ``grad_scale`` a float32 device tensor, read on the device (as
    zero_clip_scale writes it)."""
    src, keep = _src(reps, n)
    f32 = (torch.float32,)
    out_dt = _out_dtype(out)
    _check(lib().zero_adam_shard_step_dev_scale(
        ctypes.byref(src), n, _ptr(grad_scale, 1, "grad_scale", f32), _ptr(master, n, "master", f32),
        _ptr(m, n, "m", f32), _ptr(v, n, "v", f32), ctypes.byref(hp),
        _ptr(out, n, "out"), out_dt, _ptr(skip, 1, "skip", (torch.int32,)), _stream(stream)),
        "zero_adam_shard_step_dev_scale")


def zero_adam_shard_step_dev_t(reps, n: int, grad_scale, table, step, status, master, m, v,
                               wd_mode="adamw", out=None, skip=None, stream=None):
    """The step with its grad scale (float32 device tensor), constants table ((len, 9) float32
    device tensor, e.g. adam_table) and step counter (int64 device tensor) all on the device; the
    counter advances on the device unless ``skip`` is set. A counter outside the table refuses the
    update (nothing written, no advance) and sets ``status`` (int32 device tensor, zeroed by the
    caller) to ZERO_DEV_T_OUT_OF_TABLE."""
    src, keep = _src(reps, n)
    f32 = (torch.float32,)
    out_dt = _out_dtype(out)
    mode = {"adamw": ZERO_ADAMW, "l2": ZERO_ADAM_L2}.get(wd_mode, wd_mode)
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.shape[1] != 9:
        raise ValueError("table must be a (len, 9) float32 device tensor")
    _check(lib().zero_adam_shard_step_dev_t(
        ctypes.byref(src), n, _ptr(grad_scale, 1, "grad_scale", f32),
        _ptr(table, table.numel(), "table", f32), table.shape[0],
        _ptr(step, 1, "step", (torch.int64,)), _ptr(status, 1, "status", (torch.int32,)), int(mode),
        _ptr(master, n, "master", f32), _ptr(m, n, "m", f32), _ptr(v, n, "v", f32),
        _ptr(out, n, "out"), out_dt, _ptr(skip, 1, "skip", (torch.int32,)), _stream(stream)),
        "zero_adam_shard_step_dev_t")


def zero_clip_scale(sq, max_norm: float, clip_eps: float, inv_loss_scale: float, grad_scale,
                    stream=None):
    """grad_scale[0] = fp32(min(1, max_norm / (sqrt(sq[0]) + clip_eps)) * inv_loss_scale), on the
    device: ``sq`` a float64 device tensor (zero_shard_sqnorm's output), ``grad_scale`` float32."""
    _check(lib().zero_clip_scale(
        _ptr(sq, 1, "sq", (torch.float64,)), float(max_norm), float(clip_eps), float(inv_loss_scale),
        _ptr(grad_scale, 1, "grad_scale", (torch.float32,)), _stream(stream)), "zero_clip_scale")


class AdamStep:
    """zero_adam_shard_step with its arrays and stream marshalled once; a call passes only the grad
    scale and the hyper-parameters (which change every step). For loops whose steps are short enough
    that per-call marshalling shows. The tensors must stay alive and in place while it is used."""

    def __init__(self, reps, n: int, master, m, v, out=None, skip=None, stream=None):
        self._src, self._keep = _src(reps, n)
        f32 = (torch.float32,)
        out_dt = _out_dtype(out)
        self._tensors = (reps, master, m, v, out, skip)
        self._fn = lib().zero_adam_shard_step
        self._args = (n, _ptr(master, n, "master", f32), _ptr(m, n, "m", f32), _ptr(v, n, "v", f32))
        self._tail = (_ptr(out, n, "out"), out_dt, _ptr(skip, 1, "skip", (torch.int32,)), _stream(stream))
        self._ref = ctypes.byref(self._src)

    def __call__(self, grad_scale: float, hp: ZeroAdamHParams):
        n, p, m, v = self._args
        _check(self._fn(self._ref, n, grad_scale, p, m, v, ctypes.byref(hp), *self._tail),
               "zero_adam_shard_step")


class ReduceCall:
    """zero_reduce_shard with its arrays and stream marshalled once; a call passes only sq_scale.
    For loops of launches short enough that per-call marshalling shows. The tensors must stay alive
    and in place while it is used."""

    def __init__(self, reps, n: int, out_grad=None, nonfinite=None, sq_partials=None, stream=None):
        self._src, self._keep = _src(reps, n)
        self._tensors = (reps, out_grad, nonfinite, sq_partials)
        self._fn = lib().zero_reduce_shard
        self._args = (ctypes.byref(self._src), n,
                      _ptr(out_grad, n, "out_grad", (torch.float32,), pinned_ok=True),
                      _ptr(nonfinite, 1, "nonfinite", (torch.int32,)),
                      _ptr(sq_partials, zero_sq_partials_len(n), "sq_partials", (torch.float64,)))
        self._stream = _stream(stream)

    def __call__(self, sq_scale: float = 1.0):
        _check(self._fn(*self._args, float(sq_scale), self._stream), "zero_reduce_shard")


def zero_gather_params(shards, begin: int, count: int, out, stream=None):
    """out[:count] = the rank shards laid end to end, elements [begin, begin + count).

    ``shards``: list of equally sized 1-D device tensors (one per rank; 16-bit or fp32), or a 2-D
    tensor whose rows are the shards. Shards the range does not touch may be None.
    """
    rows = list(shards.unbind(0)) if isinstance(shards, torch.Tensor) and shards.dim() == 2 else list(shards)
    if not rows or len(rows) > ZERO_MAX_SHARDS:
        raise ValueError(f"1..{ZERO_MAX_SHARDS} shards")
    ref = next((r for r in rows if r is not None), None)
    if ref is None:
        raise ValueError("every shard is None")
    S, dt = ref.numel(), ref.dtype
    eb = {torch.float16: 2, torch.bfloat16: 2, torch.int16: 2, torch.float32: 4, torch.int32: 4}.get(dt)
    if eb is None:
        raise TypeError(f"shard dtype {dt} is not a 2- or 4-byte type")
    ptrs = []
    for k, r in enumerate(rows):
        if r is None:
            ptrs.append(None)
            continue
        if r.dtype != dt or r.numel() != S:
            raise ValueError("shards must share one dtype and length")
        ptrs.append(_ptr(r, S, f"shard {k}"))
    if out is not None and out.element_size() != eb:
        raise TypeError("out must have the shards' element size")
    arr = (ctypes.c_void_p * len(rows))(*ptrs)
    _check(lib().zero_gather_params(ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)), len(rows), S, eb,
                                    begin, count, _ptr(out, count, "out"), _stream(stream)),
           "zero_gather_params")


# ------------------------------------------------------------------------------ layer and loss calls

_ACTS = {"none": ZERO_ACT_NONE, "relu": ZERO_ACT_RELU, "gelu": ZERO_ACT_GELU,
         "gelu_tanh": ZERO_ACT_GELU_TANH, "silu": ZERO_ACT_SILU}


# These calls are short enough that their marshalling shows (a one-row layer takes the GPU about as
# long), so every tensor is looked at once, by plain attribute reads.

def _here() -> int:
    """The device the library launches on: tensors elsewhere are refused."""
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -1


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(stream, here: int) -> int | None:
    if stream is None and _raw_stream is not None and here >= 0:
        return _raw_stream(here)
    return _stream(stream)


def _refuse(t, what: str, dtype, here: int):
    """The error for a tensor that _mat or _vec cannot take, whatever is wrong with it."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a device tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{what}: dtype {t.dtype}, {dtype} expected")
    if t.get_device() != here:
        raise ValueError(f"{what} is on {t.device}, the current device is cuda:{here}")
    raise TypeError(f"{what} cannot be used")


def _mat(t, rows: int, cols: int, what: str, dtype, here: int):
    """(address, leading dimension) of a row-major (rows, cols) device matrix, or (None, cols)."""
    if t is None:
        return None, cols
    if isinstance(t, torch.Tensor) and t.shape != (rows, cols):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, ({rows}, {cols}) expected")
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != here or here < 0:
        _refuse(t, what, dtype, here)
    ld, inner = t.stride()
    if inner != 1 and cols > 1 and rows:
        raise ValueError(f"{what}: the elements of a row must be adjacent")
    return t.data_ptr(), (ld if rows > 1 else cols)


def _vec(t, n: int, what: str, dtype, here: int):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != here or here < 0:
        _refuse(t, what, dtype, here)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: {n} contiguous elements expected")
    return t.data_ptr()


def _param(t, rows: int, cols: int, what: str, dtype, here: int):
    """A parameter or its gradient: (rows, cols), contiguous, as it lies in the flat space."""
    ptr, ld = _mat(t, rows, cols, what, dtype, here)
    if ld != cols and rows > 1 and cols:
        raise ValueError(f"{what} must be contiguous")
    return ptr


def _workspace(t, here: int):
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or not t.is_contiguous():
        raise TypeError("workspace must be a contiguous device tensor")
    if t.get_device() != here or here < 0:
        _refuse(t, "workspace", t.dtype, here)
    return t.data_ptr(), t.numel() * t.element_size()


def _linear_shape(dtype, rows: int, k: int, n: int, act) -> ZeroLinearShape:
    kind = _ACTS.get(act, act)
    if not isinstance(kind, int):
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(_ACTS)}")
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError("the linear layer takes bfloat16 or float16")
    return ZeroLinearShape(rows, k, n, _TORCH_DT[dtype], kind)


def zero_linear_workspace_bytes(rows: int, in_features: int, out_features: int,
                                backward: bool = False) -> int:
    """Bytes of device workspace the linear layer's forward or backward of this size needs."""
    return int(lib().zero_linear_workspace_bytes(rows, in_features, out_features, int(backward)))


def zero_linear_forward(x, weight, out, bias=None, residual=None, act="none", pre=None,
                        workspace=None, stream=None):
    """out = act(x @ weight.T + bias) + residual, and pre = the argument of act (both optional inputs
    and ``pre`` may be None). ``x`` (rows, in), ``weight`` (out, in) contiguous, e.g. a view of the
    gathered layer; ``workspace``: a device tensor of zero_linear_workspace_bytes."""
    if not isinstance(x, torch.Tensor) or not isinstance(weight, torch.Tensor) or x.dim() != 2 or weight.dim() != 2:
        raise TypeError("x and weight must be 2-D device tensors")
    if out is None:
        raise TypeError("out must be a device tensor")
    dt, here, M = weight.dtype, _here(), x.shape[0]
    N, K = weight.shape
    s = _linear_shape(dt, M, K, N, act)
    _check(lib().zero_linear_forward(
        ctypes.byref(s), *_mat(x, M, K, "x", dt, here), _param(weight, N, K, "weight", dt, here),
        _vec(bias, N, "bias", dt, here), *_mat(residual, M, N, "residual", dt, here),
        *_mat(pre, M, N, "pre", dt, here), *_mat(out, M, N, "out", dt, here), *_workspace(workspace, here),
        _stream_on(stream, here)), "zero_linear_forward")


def zero_linear_backward(dy, x, weight, act="none", pre=None, dz=None, dx=None, dweight=None,
                         dbias=None, accumulate: bool = False, workspace=None, stream=None):
    """The gradients of zero_linear_forward. With an activation ``dz`` receives dy * act'(pre) (it may
    be ``dy`` or ``pre`` itself); ``dx`` (rows, in), ``dweight`` (out, in) contiguous and ``dbias``
    (out), each optional; the last two of the layer's dtype or float32, e.g. views of a replica row,
    and added to with ``accumulate``. ``x`` is read for ``dweight`` only and ``weight`` for ``dx``
    only: where that is not asked for, either may be None (a layer already released)."""
    if not isinstance(dy, torch.Tensor) or dy.dim() != 2:
        raise TypeError("dy must be a 2-D device tensor")
    for t in (x, weight, dx, dweight):
        if t is not None and (not isinstance(t, torch.Tensor) or t.dim() != 2):
            raise TypeError("x, weight, dx and dweight must be 2-D device tensors or None")
    here, M = _here(), dy.shape[0]
    if weight is not None:
        dt, (N, K) = weight.dtype, weight.shape
    else:
        dt, N = dy.dtype, dy.shape[1]
        wide = x if x is not None else dx if dx is not None else dweight
        K = 0 if wide is None else wide.shape[1]
    s = _linear_shape(dt, M, K, N, act)
    g = dweight if dweight is not None else dbias
    gdt = dt if g is None else g.dtype
    if gdt not in _TORCH_DT:
        raise TypeError("dweight and dbias: the weight's dtype or float32")
    _check(lib().zero_linear_backward(
        ctypes.byref(s), *_mat(dy, M, N, "dy", dt, here), *_mat(x, M, K, "x", dt, here),
        _param(weight, N, K, "weight", dt, here), *_mat(pre, M, N, "pre", dt, here),
        *_mat(dz, M, N, "dz", dt, here), *_mat(dx, M, K, "dx", dt, here),
        _param(dweight, N, K, "dweight", gdt, here), _vec(dbias, N, "dbias", gdt, here), _TORCH_DT[gdt],
        int(bool(accumulate)), *_workspace(workspace, here), _stream_on(stream, here)), "zero_linear_backward")


def _distill_in(logits, top_index, top_logits, temperature, tail, weight, here: int) -> ZeroDistillIn:
    for t, what in ((logits, "logits"), (top_index, "top_index"), (top_logits, "top_logits")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise TypeError(f"{what} must be a 2-D device tensor")
    if logits.dtype not in _TORCH_DT or top_logits.dtype not in _TORCH_DT:
        raise TypeError("logits and top_logits must be float32, float16 or bfloat16")
    if top_index.dtype not in (torch.int32, torch.int64):
        raise TypeError("top_index must be int32 or int64")
    R, V = logits.shape
    K = top_index.shape[1]
    if top_index.shape != (R, K) or top_logits.shape != (R, K):
        raise ValueError("top_index and top_logits must be (rows, topk) alike")
    lp, ldl = _mat(logits, R, V, "logits", logits.dtype, here)
    ip, ldi = _mat(top_index, R, K, "top_index", top_index.dtype, here)
    tp, ldt = _mat(top_logits, R, K, "top_logits", top_logits.dtype, here)
    if ldi != ldt:
        raise ValueError("top_index and top_logits must have the same row stride")
    f32 = torch.float32
    return ZeroDistillIn(R, V, K, _TORCH_DT[logits.dtype], _TORCH_DT[top_logits.dtype],
                         top_index.element_size(), float(temperature), lp, ldl, ip, tp, ldt,
                         _vec(tail, R, "tail", f32, here), _vec(weight, R, "weight", f32, here))


def zero_distill_forward(logits, top_index, top_logits, temperature: float, loss, stats, tail=None,
                         weight=None, stream=None):
    """loss[r] = weight[r] * KL(teacher || student) over the teacher's top entries of row r (an entry
    of index -1 is none; ``tail``: the log of the teacher's remaining mass, float32). ``loss``:
    float32 (rows,); ``stats``: float32 (rows, 2), kept for zero_distill_backward."""
    here, f32 = _here(), torch.float32
    a = _distill_in(logits, top_index, top_logits, temperature, tail, weight, here)
    _check(lib().zero_distill_forward(ctypes.byref(a), _vec(loss, a.rows, "loss", f32, here),
                                      _vec(stats, 2 * a.rows, "stats", f32, here), _stream_on(stream, here)),
           "zero_distill_forward")


def zero_distill_backward(logits, top_index, top_logits, temperature: float, stats, dlogits, tail=None,
                          weight=None, upstream=None, scale: float = 1.0, stream=None):
    """dlogits = scale * upstream[r] * the gradient of loss[r] (``upstream``: float32 (rows,) or None);
    ``dlogits`` may be ``logits`` itself."""
    here, f32 = _here(), torch.float32
    a = _distill_in(logits, top_index, top_logits, temperature, tail, weight, here)
    _check(lib().zero_distill_backward(
        ctypes.byref(a), _vec(stats, 2 * a.rows, "stats", f32, here), _vec(upstream, a.rows, "upstream", f32, here),
        float(scale), *_mat(dlogits, a.rows, a.vocab, "dlogits", logits.dtype, here), _stream_on(stream, here)),
        "zero_distill_backward")


def zero_distill_step(logits, top_index, top_logits, temperature: float, loss, dlogits, tail=None,
                      weight=None, upstream=None, scale: float = 1.0, stream=None):
    """zero_distill_forward and zero_distill_backward in one pass over the logits."""
    here, f32 = _here(), torch.float32
    a = _distill_in(logits, top_index, top_logits, temperature, tail, weight, here)
    _check(lib().zero_distill_step(
        ctypes.byref(a), _vec(upstream, a.rows, "upstream", f32, here), float(scale),
        _vec(loss, a.rows, "loss", f32, here), *_mat(dlogits, a.rows, a.vocab, "dlogits", logits.dtype, here),
        _stream_on(stream, here)), "zero_distill_step")


# ------------------------------------------------------------------------------ the update of many tensors

class _Tensors:
    """A list of tensors marshalled for zero_adam_tensors_step: the entries, their common types, and what
    keeps their memory alive."""

    def __init__(self, tensors):
        tensors = list(tensors)
        self.count, self.keep = len(tensors), tensors
        self.array = (ZeroAdamTensor * max(1, self.count))(*[t[0] for t in tensors])
        gdts = {t[1]["grad"].dtype for t in tensors}
        odts = {t[1]["out"].dtype for t in tensors if t[1]["out"] is not None}
        if len(gdts) > 1 or len(odts) > 1:
            raise TypeError("the gradients of a call share one dtype, and so do its out tensors")
        self.grad_dtype = _TORCH_DT[gdts.pop()] if gdts else ZERO_F32
        self.out_dtype = _TORCH_DT[odts.pop()] if odts else ZERO_F32
        devices = {t[1]["param"].get_device() for t in tensors}
        if len(devices) > 1:
            raise ValueError("the tensors of a call must be on one device")
        self.device = devices.pop() if devices else None

    def check_device(self):
        if self.device is not None and self.device != _here():
            raise ValueError(f"the tensors are on cuda:{self.device}, the current device is cuda:{_here()}")


def adam_tensor(param, grad, m, v, out=None, m_scale=None, v_scale=None, group: int = 0):
    """One tensor of zero_adam_tensors_step: ``param`` float32, ``grad`` float32, bfloat16 or float16, ``m`` and
    ``v`` float32, or int8 and uint8 with their scales (as adam_state makes them), ``out`` the 16-bit copy or
    None. Contiguous device tensors of any shape with as many elements as ``param`` each."""
    if not isinstance(param, torch.Tensor):
        raise TypeError("param must be a device tensor")
    n, here = param.numel(), param.get_device()
    eight = isinstance(m, torch.Tensor) and m.dtype is torch.int8
    blocks = -(-n // ZERO_STATE8_BLOCK)
    if eight and (m_scale is None or v_scale is None):
        raise TypeError("8-bit states need m_scale and v_scale")
    if not eight and (m_scale is not None or v_scale is not None):
        raise TypeError("scales belong to 8-bit states")
    gdt = grad.dtype if isinstance(grad, torch.Tensor) and grad.dtype in _TORCH_DT else torch.float32
    odt = out.dtype if isinstance(out, torch.Tensor) and out.dtype in (torch.bfloat16, torch.float16) else torch.bfloat16
    f32 = torch.float32
    for t, what in ((grad, "grad"), (m, "m"), (v, "v")):
        if t is None:
            raise TypeError(f"{what} must be a device tensor")
    entry = ZeroAdamTensor(
        n, _vec(param, n, "param", f32, here), _vec(grad, n, "grad", gdt, here), _vec(out, n, "out", odt, here),
        _vec(m, n, "m", torch.int8 if eight else f32, here), _vec(v, n, "v", torch.uint8 if eight else f32, here),
        _vec(m_scale, blocks, "m_scale", f32, here), _vec(v_scale, blocks, "v_scale", f32, here), int(group),
        8 if eight else 32)
    return entry, {"param": param, "grad": grad, "out": out, "m": m, "v": v, "m_scale": m_scale, "v_scale": v_scale}


def adam_state(param, bits: int = 32) -> dict:
    """The state of a new parameter, as keyword arguments of adam_tensor. 8 bits suit tensors whose gradients stay of one
    size or change for 256 elements at once: nearest rounding keeps small shares of a block's largest moment (zero_shard.h)."""
    if bits == 32:
        return {"m": torch.zeros_like(param, dtype=torch.float32), "v": torch.zeros_like(param, dtype=torch.float32)}
    if bits != 8:
        raise ValueError("states have 32 or 8 bits")
    blocks = -(-param.numel() // ZERO_STATE8_BLOCK)
    scale = torch.zeros((2, blocks), dtype=torch.float32, device=param.device)
    return {"m": torch.zeros(param.shape, dtype=torch.int8, device=param.device),
            "v": torch.zeros(param.shape, dtype=torch.uint8, device=param.device),
            "m_scale": scale[0], "v_scale": scale[1]}


def _groups(groups):
    groups = [groups] if isinstance(groups, ZeroAdamHParams) else list(groups)
    return (ZeroAdamHParams * max(1, len(groups)))(*groups), len(groups)


def _tensors_step(t: _Tensors, groups, grad_scale, skip, stream):
    t.check_device()
    hp, count = _groups(groups)
    dev = grad_scale if isinstance(grad_scale, torch.Tensor) else None
    here = _here()
    _check(lib().zero_adam_tensors_step(
        t.array, t.count, t.grad_dtype, t.out_dtype, hp, count, 1.0 if dev is not None else float(grad_scale),
        _vec(dev, 1, "grad_scale", torch.float32, here), _vec(skip, 1, "skip", torch.int32, here),
        _stream_on(stream, here)), "zero_adam_tensors_step")


def zero_adam_tensors_step(tensors, groups, grad_scale=1.0, skip=None, stream=None):
    """One Adam/AdamW step of every tensor of ``tensors`` (of adam_tensor). ``groups``: the hyper-parameters
    of each group (adam_hparams), or one; ``grad_scale``: a number, or a float32 device tensor of one element."""
    _tensors_step(_Tensors(tensors), groups, grad_scale, skip, stream)


def zero_adam_tensors_step_dev_t(tensors, grad_scale, table, step, status, wd_mode="adamw", skip=None, stream=None):
    """The step with its counter, grad scale and constants on the device: ``table`` a (groups, len, 9) float32
    device tensor (adam_table's of each group, stacked), ``step`` int64, ``status`` int32 and ``grad_scale``
    float32 device tensors of one element. As zero_adam_shard_step_dev_t."""
    t = tensors if isinstance(tensors, _Tensors) else _Tensors(tensors)
    t.check_device()
    here, f32 = _here(), torch.float32
    mode = {"adamw": ZERO_ADAMW, "l2": ZERO_ADAM_L2}.get(wd_mode, wd_mode)
    if not isinstance(table, torch.Tensor) or table.dim() != 3 or table.shape[2] != 9:
        raise ValueError("table must be a (groups, len, 9) float32 device tensor")
    _check(lib().zero_adam_tensors_step_dev_t(
        t.array, t.count, t.grad_dtype, t.out_dtype, _vec(grad_scale, 1, "grad_scale", f32, here),
        _vec(table, table.numel(), "table", f32, here), table.shape[0], table.shape[1],
        _vec(step, 1, "step", torch.int64, here), _vec(status, 1, "status", torch.int32, here), int(mode),
        _vec(skip, 1, "skip", torch.int32, here), _stream_on(stream, here)), "zero_adam_tensors_step_dev_t")


class AdamTensorsStep:
    """zero_adam_tensors_step with its tensors marshalled once; a call passes the hyper-parameters of each
    group and the grad scale. Marshalling costs the host about 2.5 us a tensor for adam_tensor and 0.25 for the list; a call takes
    8 us for 48 tensors and 20 for 148 (with a list 20 and 59). It holds its tensors, gradients too, and steps on the memory that
    it was made with: a program whose gradients are allocated anew each step makes it anew as well, or copies them into place."""

    def __init__(self, tensors, skip=None):
        self._tensors, self._skip = _Tensors(tensors), skip

    def __call__(self, groups, grad_scale=1.0, stream=None):
        _tensors_step(self._tensors, groups, grad_scale, self._skip, stream)

    def dev_t(self, grad_scale, table, step, status, wd_mode="adamw", stream=None):
        """zero_adam_tensors_step_dev_t on the same tensors."""
        zero_adam_tensors_step_dev_t(self._tensors, grad_scale, table, step, status, wd_mode, self._skip, stream)


def _state_moment(codes) -> int:
    kinds = {torch.int8: 1, torch.uint8: 2}
    if not isinstance(codes, torch.Tensor) or codes.dtype not in kinds:
        raise TypeError("codes: int8 (first moment) or uint8 (second moment)")
    return kinds[codes.dtype]


def zero_adam_state_values(codes, scale, values, stream=None):
    """values = the numbers that an 8-bit moment stands for: ``codes`` int8 (m) or uint8 (v), ``scale`` float32 of
    one element for each 256, ``values`` float32 of as many elements as ``codes``."""
    moment, here, n = _state_moment(codes), _here(), codes.numel()
    _check(lib().zero_adam_state_values(
        _vec(codes, n, "codes", codes.dtype, here), _vec(scale, -(-n // ZERO_STATE8_BLOCK), "scale", torch.float32, here),
        n, moment, _vec(values, n, "values", torch.float32, here), _stream_on(stream, here)), "zero_adam_state_values")


def zero_adam_state_codes(values, codes, scale, stream=None):
    """codes, scale = the 8-bit moment of ``values``."""
    moment, here, n = _state_moment(codes), _here(), codes.numel()
    _check(lib().zero_adam_state_codes(
        _vec(values, n, "values", torch.float32, here), n, moment, _vec(codes, n, "codes", codes.dtype, here),
        _vec(scale, -(-n // ZERO_STATE8_BLOCK), "scale", torch.float32, here), _stream_on(stream, here)),
        "zero_adam_state_codes")


# ------------------------------------------------------------------------------ block boundaries

_NORMS = {"none": ZERO_NORM_NONE, "rms": ZERO_NORM_RMS, "layer": ZERO_NORM_LAYER}


def _norm_block(stream_like, what, dtype, branch, gate, gate_rows, post, post_weight, post_bias, pre, pre_weight, pre_bias,
                eps, residual_scale, branch_scale, here: int) -> ZeroNormBlock:
    """The block of a stream tensor (rows, features); ``dtype``: the block's 16-bit type."""
    if not isinstance(stream_like, torch.Tensor) or stream_like.dim() != 2:
        raise TypeError(f"{what} must be a 2-D device tensor")
    R, d = stream_like.shape
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError("the block's tensors must be bfloat16 or float16")
    if stream_like.dtype is not dtype and stream_like.dtype is not torch.float32:
        raise TypeError(f"{what}: {dtype} or float32 expected")
    kinds = []
    for k in (post, pre):
        kind = _NORMS.get(k, k)
        if not isinstance(kind, int):
            raise ValueError(f"unknown norm {k!r}: one of {', '.join(_NORMS)}")
        kinds.append(kind)
    if gate is not None and int(gate_rows) < 1:
        raise ValueError("gate_rows must be at least 1")
    per = int(gate_rows)
    bp, ldb = _mat(branch, R, d, "branch", dtype, here)
    gp, ldg = _mat(gate, -(-R // per), d, "gate", dtype, here) if gate is not None else (None, d)
    return ZeroNormBlock(R, d, max(per, 0), _TORCH_DT[dtype], _TORCH_DT[stream_like.dtype], *kinds, float(eps),
                         float(residual_scale), float(branch_scale), 0, bp, ldb, gp, ldg,
                         _vec(post_weight, d, "post_weight", dtype, here), _vec(post_bias, d, "post_bias", dtype, here),
                         _vec(pre_weight, d, "pre_weight", dtype, here), _vec(pre_bias, d, "pre_bias", dtype, here))


def _dtype_of(*tensors):
    for t in tensors:
        if isinstance(t, torch.Tensor):
            return t.dtype
    return None


def zero_norm_workspace_bytes(rows: int, features: int, gate_rows: int = 1) -> int:
    """Bytes of device workspace that zero_norm_backward of this size needs."""
    return int(lib().zero_norm_workspace_bytes(rows, features, gate_rows))


def zero_norm_forward(x, h=None, branch=None, y=None, gate=None, gate_rows: int = 1, post="none", post_weight=None,
                      post_bias=None, pre="rms", pre_weight=None, pre_bias=None, eps: float = 1e-5,
                      residual_scale: float = 1.0, branch_scale: float = 1.0, stats=None, stream=None):
    """y = residual_scale * x + branch_scale * gate * post_norm(branch) and h = pre_norm(y), in one pass. ``x`` and ``y``
    (rows, features) of the stream's type (the block's or float32; y may be x), ``branch``, ``h``, ``gate`` and the
    parameters bfloat16 or float16; ``gate`` has a row for every ``gate_rows`` rows (rows: one row for all). Without
    a branch y is x itself. Norms: "none", "rms", "layer". ``stats``: float32 (rows, 4), kept for the backward."""
    here, f32 = _here(), torch.float32
    dt = _dtype_of(branch, h)
    b = _norm_block(x, "x", dt, branch, gate, gate_rows, post, post_weight, post_bias, pre, pre_weight, pre_bias, eps,
                    residual_scale, branch_scale, here)
    R, d = x.shape
    _check(lib().zero_norm_forward(
        ctypes.byref(b), *_mat(x, R, d, "x", x.dtype, here), *_mat(y, R, d, "y", x.dtype, here),
        *_mat(h, R, d, "h", dt, here), _vec(stats, 4 * R, "stats", f32, here), _stream_on(stream, here)),
        "zero_norm_forward")


def zero_norm_backward(y, stats, dy=None, dh=None, branch=None, gate=None, gate_rows: int = 1, post="none",
                       post_weight=None, post_bias=None, pre="rms", pre_weight=None, pre_bias=None, eps: float = 1e-5,
                       residual_scale: float = 1.0, branch_scale: float = 1.0, dx=None, dbranch=None, dgate=None,
                       dpost_weight=None, dpost_bias=None, dpre_weight=None, dpre_bias=None, accumulate: bool = False,
                       workspace=None, stream=None):
    """The gradients of zero_norm_forward from ``dh`` and ``dy`` (or None: 0), with its ``y`` (without a branch: x) and
    ``stats``. ``dx`` of the stream's type (it may be dy), ``dbranch`` of the block's; ``dgate`` and the parameters'
    gradients of the block's type or float32, added to with ``accumulate``; each optional. ``workspace``: a device
    tensor of zero_norm_workspace_bytes (read and written only where a parameter's or a shared gate's gradient is
    asked for). Without a pre norm ``y`` may be None if ``dy`` or ``dx`` is given."""
    here, f32 = _here(), torch.float32
    like = y if y is not None else dy if dy is not None else dx
    dt = _dtype_of(branch, dh, dbranch)
    b = _norm_block(like, "y", dt, branch, gate, gate_rows, post, post_weight, post_bias, pre, pre_weight, pre_bias, eps,
                    residual_scale, branch_scale, here)
    R, d = like.shape
    sdt, gates = like.dtype, -(-R // max(1, int(gate_rows)))
    gdt = _dtype_of(dgate, dpost_weight, dpost_bias, dpre_weight, dpre_bias) or dt
    if gdt not in _TORCH_DT:
        raise TypeError("dgate and the parameters' gradients: the block's dtype or float32")
    _check(lib().zero_norm_backward(
        ctypes.byref(b), _vec(stats, 4 * R, "stats", f32, here), *_mat(y, R, d, "y", sdt, here),
        *_mat(dy, R, d, "dy", sdt, here), *_mat(dh, R, d, "dh", dt, here), *_mat(dx, R, d, "dx", sdt, here),
        *_mat(dbranch, R, d, "dbranch", dt, here), *_mat(dgate, gates, d, "dgate", gdt, here),
        _vec(dpost_weight, d, "dpost_weight", gdt, here), _vec(dpost_bias, d, "dpost_bias", gdt, here),
        _vec(dpre_weight, d, "dpre_weight", gdt, here), _vec(dpre_bias, d, "dpre_bias", gdt, here), _TORCH_DT[gdt],
        int(bool(accumulate)), *_workspace(workspace, here), _stream_on(stream, here)), "zero_norm_backward")


# ------------------------------------------------------------------------------ losses over tokens

def _token_in(logits, label, temperature, here: int) -> ZeroTokenIn:
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2 or not isinstance(label, torch.Tensor):
        raise TypeError("logits must be a 2-D and label a 1-D device tensor")
    if logits.dtype not in _TORCH_DT:
        raise TypeError("logits must be float32, float16 or bfloat16")
    if label.dtype is not torch.int64 and label.dtype is not torch.int32:
        raise TypeError("label must be int32 or int64")
    R, V = logits.shape
    lp, ld = _mat(logits, R, V, "logits", logits.dtype, here)
    return ZeroTokenIn(R, V, _TORCH_DT[logits.dtype], label.element_size(), float(temperature), 0, lp, ld,
                       _vec(label, R, "label", label.dtype, here))


def _policy(rows, old_logp, advantage, ref_logp, weight, clip, kl_coef, here: int) -> ZeroPolicy:
    f32 = torch.float32
    low, high = clip if isinstance(clip, (tuple, list)) else (clip, clip)
    return ZeroPolicy(_vec(old_logp, rows, "old_logp", f32, here), _vec(advantage, rows, "advantage", f32, here),
                      _vec(ref_logp, rows, "ref_logp", f32, here), _vec(weight, rows, "weight", f32, here),
                      float(low), float(high), float(kl_coef), 0)


def zero_token_logp(logits, label, logp, temperature: float = 1.0, stats=None, stream=None):
    """logp[r] = the log probability of row r's token under softmax(logits / temperature) (0 where label is -1).
    ``logits`` (rows, vocab), ``label`` int32 or int64 (rows,), ``logp`` float32 (rows,); ``stats``: float32
    (rows, ZERO_TOKEN_STATS), kept for zero_token_backward, or None."""
    here, f32 = _here(), torch.float32
    a = _token_in(logits, label, temperature, here)
    _check(lib().zero_token_logp(ctypes.byref(a), _vec(logp, a.rows, "logp", f32, here),
                                 _vec(stats, ZERO_TOKEN_STATS * a.rows, "stats", f32, here), _stream_on(stream, here)),
           "zero_token_logp")


def zero_policy_forward(logits, label, old_logp, advantage, loss, stats, ref_logp=None, weight=None, clip=0.2,
                        kl_coef: float = 0.0, temperature: float = 1.0, logp=None, stream=None):
    """loss[r] = weight[r] * (the clipped policy loss of row r's token + kl_coef * its KL estimate). float32
    (rows,) tensors but for ``logits``, ``label`` and ``stats`` (as zero_token_logp); ``clip``: one width or (low, high)."""
    here, f32 = _here(), torch.float32
    a = _token_in(logits, label, temperature, here)
    p = _policy(a.rows, old_logp, advantage, ref_logp, weight, clip, kl_coef, here)
    _check(lib().zero_policy_forward(
        ctypes.byref(a), ctypes.byref(p), _vec(loss, a.rows, "loss", f32, here), _vec(logp, a.rows, "logp", f32, here),
        _vec(stats, ZERO_TOKEN_STATS * a.rows, "stats", f32, here), _stream_on(stream, here)), "zero_policy_forward")


def zero_policy_step(logits, label, old_logp, advantage, loss, dlogits, ref_logp=None, weight=None, clip=0.2,
                     kl_coef: float = 0.0, temperature: float = 1.0, logp=None, upstream=None, scale: float = 1.0,
                     stream=None):
    """zero_policy_forward and zero_token_backward in one pass over the logits; ``dlogits`` may be ``logits``."""
    here, f32 = _here(), torch.float32
    a = _token_in(logits, label, temperature, here)
    p = _policy(a.rows, old_logp, advantage, ref_logp, weight, clip, kl_coef, here)
    _check(lib().zero_policy_step(
        ctypes.byref(a), ctypes.byref(p), _vec(upstream, a.rows, "upstream", f32, here), float(scale),
        _vec(loss, a.rows, "loss", f32, here), _vec(logp, a.rows, "logp", f32, here),
        *_mat(dlogits, a.rows, a.vocab, "dlogits", logits.dtype, here), _stream_on(stream, here)), "zero_policy_step")


def zero_preference_forward(logits, label, seq_start, loss, stats, ref_logp=None, weight=None, beta: float = 0.1,
                            label_smoothing: float = 0.0, margin: float = 0.0, average: bool = False,
                            temperature: float = 1.0, logp=None, seq_logp=None, stream=None):
    """loss[p] = weight[p] * the preference loss of pair p, whose answers are the rows seq_start[2p] to seq_start[2p+1]
    (preferred) and from there to seq_start[2p+2]. ``seq_start``: int32 or int64 (2 * pairs + 1,); ``loss`` and
    ``weight`` float32 (pairs,); ``ref_logp`` and ``seq_logp`` float32 (2 * pairs,); ``logp`` float32 (rows,);
    ``stats`` as zero_token_logp."""
    here, f32 = _here(), torch.float32
    a = _token_in(logits, label, temperature, here)
    if not isinstance(seq_start, torch.Tensor) or seq_start.dtype not in (torch.int32, torch.int64):
        raise TypeError("seq_start must be an int32 or int64 device tensor")
    n = seq_start.numel()
    if n % 2 != 1:
        raise ValueError("seq_start holds 2 * pairs + 1 rows")
    pairs = n // 2
    p = ZeroPreference(pairs, _vec(seq_start, n, "seq_start", seq_start.dtype, here), seq_start.element_size(),
                       int(bool(average)), _vec(ref_logp, 2 * pairs, "ref_logp", f32, here),
                       _vec(weight, pairs, "weight", f32, here), float(beta), float(label_smoothing), float(margin), 0)
    _check(lib().zero_preference_forward(
        ctypes.byref(a), ctypes.byref(p), _vec(loss, pairs, "loss", f32, here), _vec(logp, a.rows, "logp", f32, here),
        _vec(seq_logp, 2 * pairs, "seq_logp", f32, here), _vec(stats, ZERO_TOKEN_STATS * a.rows, "stats", f32, here),
        _stream_on(stream, here)), "zero_preference_forward")


def zero_token_backward(logits, label, stats, dlogits, upstream=None, scale: float = 1.0, temperature: float = 1.0,
                        stream=None):
    """dlogits = scale * upstream * the gradient of the loss whose forward left ``stats``; ``upstream``: float32 (rows,),
    after zero_preference_forward (pairs,), or None; ``dlogits`` may be ``logits`` itself."""
    here, f32 = _here(), torch.float32
    a = _token_in(logits, label, temperature, here)
    n = upstream.numel() if isinstance(upstream, torch.Tensor) else 0
    _check(lib().zero_token_backward(
        ctypes.byref(a), _vec(stats, ZERO_TOKEN_STATS * a.rows, "stats", f32, here),
        _vec(upstream, n, "upstream", f32, here), n, float(scale),
        *_mat(dlogits, a.rows, a.vocab, "dlogits", logits.dtype, here), _stream_on(stream, here)), "zero_token_backward")


# ------------------------------------------------------------------------------ host (offload) calls

def _hptr(a, n: int, what: str, itemsize: int):
    """Host array (numpy array or CPU torch tensor) -> address, checked for size and layout."""
    if a is None:
        return None
    if isinstance(a, torch.Tensor):
        if a.is_cuda:
            raise TypeError(f"{what} must be host memory")
        if not a.is_contiguous() or a.element_size() != itemsize:
            raise ValueError(f"{what}: contiguous {itemsize}-byte elements expected")
        if a.numel() < n:
            raise ValueError(f"{what} holds {a.numel()} elements, {n} needed")
        return a.data_ptr()
    import numpy as np
    if not isinstance(a, np.ndarray) or not a.flags["C_CONTIGUOUS"] or a.itemsize != itemsize:
        raise ValueError(f"{what}: contiguous numpy array of {itemsize}-byte elements expected")
    if a.size < n:
        raise ValueError(f"{what} holds {a.size} elements, {n} needed")
    return a.ctypes.data


def zero_host_adam_step(grad, n: int, grad_scale: float, master, m, v, hp: ZeroAdamHParams,
                        out=None, out_dtype: int = ZERO_BF16, threads: int = 0):
    """The host update on host arrays (numpy or CPU tensors); ``out`` holds 16-bit patterns."""
    _check(lib().zero_host_adam_step(
        _hptr(grad, n, "grad", 4), n, float(grad_scale), _hptr(master, n, "master", 4),
        _hptr(m, n, "m", 4), _hptr(v, n, "v", 4), ctypes.byref(hp), _hptr(out, n, "out", 2),
        out_dtype, threads), "zero_host_adam_step")


def offload_buffers(chunk_elems: int, device="cuda", threads: int = 0, h2d_stream=None,
                    direct: bool = False) -> dict:
    """Caller-side staging for zero_offload_step: device and pinned host chunk buffers (x2) and
    the four events the step records and waits on (torch events, created here by recording each
    once). ``direct``: no device staging; the reduce kernel writes each chunk into the pinned host
    buffer itself."""
    events = [torch.cuda.Event(enable_timing=False) for _ in range(4)]
    for ev in events:
        ev.record()                    # torch creates an event's handle on its first record
    bufs = {
        "d_grad": None if direct else torch.empty(2 * chunk_elems, dtype=torch.float32, device=device),
        "h_grad": torch.empty(2 * chunk_elems, dtype=torch.float32, pin_memory=True),
        "h_param": torch.empty(2 * chunk_elems, dtype=torch.int16, pin_memory=True),
        "chunk_elems": chunk_elems, "threads": threads, "h2d_stream": h2d_stream, "events": events,
    }
    return bufs


def zero_offload_step(reps, n: int, grad_scale: float, h_master, h_m, h_v, hp: ZeroAdamHParams,
                      out, buffers: dict, stream=None):
    """Offloaded step: device replicas -> host Adam on host state -> 16-bit params into ``out``."""
    src, keep = _src(reps, n)
    if out is None or out.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("out must be a bfloat16 or float16 device tensor")
    C = int(buffers["chunk_elems"])
    b = ZeroOffloadBuffers(_ptr(buffers["d_grad"], 2 * C, "d_grad", (torch.float32,)),
                           _hptr(buffers["h_grad"], 2 * C, "h_grad", 4),
                           _hptr(buffers["h_param"], 2 * C, "h_param", 2), C, int(buffers["threads"]), 0,
                           None if buffers.get("h2d_stream") is None else _stream(buffers["h2d_stream"]),
                           (ctypes.c_void_p * 4)(*[ev.cuda_event for ev in buffers["events"]]))
    _check(lib().zero_offload_step(
        ctypes.byref(src), n, float(grad_scale), _hptr(h_master, n, "master", 4), _hptr(h_m, n, "m", 4),
        _hptr(h_v, n, "v", 4), ctypes.byref(hp), _ptr(out, n, "out"), _TORCH_DT[out.dtype],
        ctypes.byref(b), _stream(stream)), "zero_offload_step")
