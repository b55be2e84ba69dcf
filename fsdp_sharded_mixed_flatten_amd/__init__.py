"""Python binding of ``libzs.so``, the MI355X shard-local step (ZeRO / FSDP).

Argument marshalling only: every step of the path runs in the library's HIP
kernels. Functions carry the C ABI's names (``include/zs.h``, ``include/zs_clip.h``, ``include/zs_lm.h``,
``include/zs_mx4.h``, ``include/zs_drafts.h``). Device buffers are PyTorch CUDA tensors (flat buffers of the step and the
quantized gather's payload may be raw integer device addresses; workspaces, matrices and scalars are tensors, since
their lengths and devices are looked at); the stream is
``torch.cuda.current_stream()`` unless one is given. Before each call the
binding checks that every tensor is a contiguous CUDA tensor of the right
dtype and at least as long as the kernels will touch, so a wrong shape is a
Python exception instead of an out-of-bounds access on the device.

If the library has not been built this module raises on import: there is no
fallback path.
"""

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzs.so")

ZS_OK, ZS_EINVAL, ZS_EALIGN, ZS_ERANGE, ZS_EHIP, ZS_ENOMEM = 0, -1, -2, -3, -4, -5
ZS_LAYOUT_FLAT, ZS_LAYOUT_PER_TENSOR = 0, 1
ZS_MAX_CONTRIBS = 256
ZS_MAX_GROUPS = 8
ZS_DTYPE_BF16, ZS_DTYPE_F32 = 0, 1
ZS_QUANT_MATVEC_MAX_ROWS = 64
ZS_LOGPROBS_MAX_TOP = 32
ZS_DISTILL_MAX_K = 1024
ZS_MX4_BLOCK = 32
ZS_VERIFY_MAX_DRAFTS = 64
GRAD_STATS_NOALLOC_MAX_ELEMS = 1431568384
FUSED_TWO_PASS_MIN_CONTRIBS = 52  # zs_fused_shard_step runs two passes from here when grad is given

_STATUS_NAMES = {0: "ZS_OK", -1: "ZS_EINVAL", -2: "ZS_EALIGN", -3: "ZS_ERANGE", -4: "ZS_EHIP",
                 -5: "ZS_ENOMEM"}


class ZsError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{_STATUS_NAMES.get(status, status)}: {message}")
        self.status = status
        self.message = message


class AdamWHParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("step", ctypes.c_int64)]

    def __init__(self, lr=1e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1):
        super().__init__(lr, beta1, beta2, eps, weight_decay, step)

    def at(self, step):
        return AdamWHParams(self.lr, self.beta1, self.beta2, self.eps, self.weight_decay, step)


class AdamWCoefs(ctypes.Structure):
    """The fp32 scalars of one AdamW step (zs_adamw_coefs)."""
    _fields_ = [(name, ctypes.c_float) for name in
                ("beta1", "one_minus_beta1", "beta2", "one_minus_beta2", "lr", "eps", "decay", "bias_correction1",
                 "bias_correction2")]

    def values(self):
        return [getattr(self, name) for name, _ in self._fields_]


class TensorInfo(ctypes.Structure):
    _fields_ = [("numel", ctypes.c_int64), ("flat_off", ctypes.c_int64),
                ("padded_numel", ctypes.c_int64), ("own_lo", ctypes.c_int64),
                ("own_hi", ctypes.c_int64), ("shard_off", ctypes.c_int64)]


class PlanOptions(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("tensor_align_elems", ctypes.c_int32),
                ("persist_below_elems", ctypes.c_int64), ("groups", ctypes.POINTER(ctypes.c_int32))]


class ReshardSlice(ctypes.Structure):
    _fields_ = [("group_size", ctypes.c_int32), ("slice_index", ctypes.c_int32), ("slice_off", ctypes.c_int64),
                ("slice_len", ctypes.c_int64), ("first_source", ctypes.c_int32), ("n_sources", ctypes.c_int32),
                ("owner_slice", ctypes.c_int32), ("reserved", ctypes.c_int32), ("own_off", ctypes.c_int64),
                ("retained_bytes", ctypes.c_int64)]


class PiecePtrs(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("master", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("param", ctypes.c_void_p), ("full", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built (run __graft_entry__.build() or "
                          f"python {os.path.join(_HERE, 'build.py')})")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    st = ctypes.c_int
    sigs = {
        "zs_shard_plan": (st, [ctypes.POINTER(i64), i32, i32, i32, i32, i32, ctypes.POINTER(vp)]),
        "zs_shard_plan_ex": (st, [ctypes.POINTER(i64), i32, i32, i32, ctypes.POINTER(PlanOptions),
                                  ctypes.POINTER(vp)]),
        "zs_plan_tensor_group": (i32, [vp, i32]),
        "zs_plan_tensor_replicated": (i32, [vp, i32]),
        "zs_plan_destroy": (None, [vp]),
        "zs_plan_padded_numel": (i64, [vp]),
        "zs_plan_shard_numel": (i64, [vp]),
        "zs_plan_persistent_bytes": (i64, [vp]),
        "zs_plan_num_tensors": (i32, [vp]),
        "zs_plan_world_size": (i32, [vp]),
        "zs_plan_rank": (i32, [vp]),
        "zs_plan_layout": (i32, [vp]),
        "zs_plan_tensor": (st, [vp, i32, ctypes.POINTER(TensorInfo)]),
        "zs_reduce_shard": (st, [vp, ctypes.POINTER(vp), i32, vp, i64, i64, vp]),
        "zs_adamw_shard_step": (st, [vp, ctypes.POINTER(AdamWHParams), vp, vp, vp, vp, vp, vp]),
        "zs_gather_params": (st, [vp, vp, vp, vp]),
        "zs_plan_reshard_slice": (st, [vp, i32, ctypes.POINTER(ReshardSlice)]),
        "zs_gather_params_to_slice": (st, [vp, i32, vp, vp, vp]),
        "zs_gather_slice": (st, [vp, i32, ctypes.POINTER(vp), i32, vp, vp]),
        "zs_fused_shard_step": (st, [vp, ctypes.POINTER(AdamWHParams), ctypes.POINTER(vp), i32, vp, vp,
                                     vp, vp, vp, vp, vp]),
        "zs_fused_shard_step_bucket": (st, [vp, ctypes.POINTER(AdamWHParams), ctypes.POINTER(vp), i32, vp, vp,
                                            vp, vp, vp, vp, i64, i64, vp]),
        "zs_multi_workspace_bytes": (i64, [vp, i32]),
        "zs_plan_workspace_bytes": (i64, [vp]),
        "zs_multi_bind": (st, [vp, ctypes.POINTER(PiecePtrs), ctypes.POINTER(vp), i32, vp, i64, vp]),
        "zs_multi_unbind": (st, [vp, vp]),
        "zs_reduce_shard_multi": (st, [vp, vp, vp]),
        "zs_adamw_shard_step_multi": (st, [vp, ctypes.POINTER(AdamWHParams), vp, vp]),
        "zs_gather_params_multi": (st, [vp, vp, vp]),
        "zs_fused_shard_step_multi": (st, [vp, ctypes.POINTER(AdamWHParams), vp, vp]),
        "zs_adamw_shard_step_multi_groups": (st, [vp, ctypes.POINTER(AdamWHParams), i32, vp, vp]),
        "zs_fused_shard_step_multi_groups": (st, [vp, ctypes.POINTER(AdamWHParams), i32, vp, vp]),
        "zs_quant_code_bytes": (i64, [vp, i32]),
        "zs_quant_num_scales": (i64, [vp, i32]),
        "zs_quantize_shard": (st, [vp, i32, i32, vp, vp, vp, vp]),
        "zs_fused_shard_step_quant": (st, [vp, ctypes.POINTER(AdamWHParams), ctypes.POINTER(vp), i32, vp, vp, vp,
                                           vp, vp, i32, i32, vp, vp, vp]),
        "zs_dequant_gather": (st, [vp, i32, i32, vp, vp, vp, vp]),
        "zs_host_adamw_step": (st, [ctypes.POINTER(AdamWHParams), vp, vp, vp, vp, vp, i64, i32]),
        "zs_offload_adamw_step": (st, [vp, ctypes.POINTER(AdamWHParams), vp, vp, vp, vp, vp, vp, vp, vp, i64, i32,
                                       vp]),
        "zs_accumulate_shard": (st, [vp, ctypes.POINTER(vp), i32, vp, i64, i64, i32, vp]),
        "zs_grad_stats_workspace_bytes": (i64, [vp]),
        "zs_grad_stats": (st, [vp, vp, ctypes.c_float, vp, vp, vp, i64, vp]),
        "zs_grad_stats_noalloc": (st, [vp, vp, ctypes.c_float, vp, vp, vp]),
        "zs_clip_scale": (st, [vp, vp, i32, ctypes.c_double, vp, vp, vp]),
        "zs_adamw_shard_step_accum": (st, [vp, ctypes.POINTER(AdamWHParams), vp, ctypes.c_float, vp, vp, vp, vp,
                                           vp, vp, vp, vp]),
        "zs_adamw_coefs_compute": (st, [ctypes.POINTER(AdamWHParams), ctypes.POINTER(AdamWCoefs)]),
        "zs_fused_shard_step_dc": (st, [vp, vp, ctypes.POINTER(vp), i32, vp, vp, vp, vp, vp, vp, vp]),
        "zs_adamw_shard_step_dc": (st, [vp, vp, vp, vp, vp, vp, vp, vp]),
        "zs_adamw_shard_step_accum_dc": (st, [vp, vp, vp, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, vp]),
        "zs_fused_shard_step_multi_dc": (st, [vp, vp, i32, vp, vp]),
        "zs_quant_matvec": (st, [vp, i32, i64, i64, i32, i32, vp, vp, vp, i64, i32, vp, i32, i64, vp]),
        "zs_token_logprobs": (st, [vp, i32, i64, i64, i64, vp, ctypes.c_float, vp, vp, vp, i32, vp, vp, vp]),
        "zs_token_logprobs_backward": (st, [vp, i32, i64, i64, i64, vp, ctypes.c_float, vp, vp, vp, vp, vp, i64, vp]),
        "zs_distill_topk": (st, [vp, i32, i64, i64, i64, vp, vp, i32, ctypes.c_float, vp, vp, vp, i64, vp]),
        "zs_mx4_quantize": (st, [vp, i32, i64, i64, i64, vp, i64, vp, i64, vp]),
        "zs_mx4_dequantize": (st, [vp, i64, vp, i64, i64, i64, vp, i32, i64, vp]),
        "zs_mx4_matmul": (st, [vp, i64, vp, i64, i64, vp, i64, vp, i64, i64, i64, vp, i32, i64, vp]),
        "zs_verify_drafts_workspace_bytes": (i64, [i64, i32, i64]),
        "zs_verify_drafts": (st, [vp, i32, i64, i32, i64, i64, vp, i64, vp, vp, vp, ctypes.c_double, vp, vp, vp, vp,
                                  i64, vp]),
        "zs_grad_stats_multi_workspace_bytes": (i64, [vp]),
        "zs_grad_stats_multi": (st, [vp, vp, vp, vp, vp, i64, vp]),
        "zs_adamw_shard_step_multi_clip": (st, [vp, ctypes.POINTER(AdamWHParams), i32, vp, vp, vp, vp]),
        "zs_last_error": (ctypes.c_char_p, []),
        "zs_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sigs.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


_lib = _load()
EXPORTED = ("zs_shard_plan", "zs_shard_plan_ex", "zs_plan_tensor_group", "zs_plan_tensor_replicated",
            "zs_plan_destroy", "zs_plan_padded_numel", "zs_plan_shard_numel",
            "zs_plan_persistent_bytes", "zs_plan_num_tensors", "zs_plan_world_size", "zs_plan_rank",
            "zs_plan_layout", "zs_plan_tensor", "zs_reduce_shard", "zs_adamw_shard_step",
            "zs_gather_params", "zs_plan_reshard_slice", "zs_gather_params_to_slice", "zs_gather_slice",
            "zs_fused_shard_step", "zs_fused_shard_step_bucket", "zs_multi_workspace_bytes",
            "zs_plan_workspace_bytes",
            "zs_multi_bind", "zs_multi_unbind",
            "zs_reduce_shard_multi", "zs_adamw_shard_step_multi", "zs_gather_params_multi",
            "zs_fused_shard_step_multi", "zs_adamw_shard_step_multi_groups",
            "zs_fused_shard_step_multi_groups", "zs_quant_code_bytes", "zs_quant_num_scales", "zs_quantize_shard",
            "zs_fused_shard_step_quant", "zs_dequant_gather", "zs_host_adamw_step", "zs_offload_adamw_step",
            "zs_accumulate_shard", "zs_grad_stats_workspace_bytes",
            "zs_grad_stats", "zs_grad_stats_noalloc", "zs_clip_scale", "zs_adamw_shard_step_accum",
            "zs_adamw_coefs_compute",
            "zs_fused_shard_step_dc", "zs_adamw_shard_step_dc", "zs_adamw_shard_step_accum_dc",
            "zs_fused_shard_step_multi_dc", "zs_last_error", "zs_version")
# the language-model operators (include/zs_lm.h)
EXPORTED_LM = ("zs_quant_matvec", "zs_token_logprobs", "zs_token_logprobs_backward", "zs_distill_topk")
# the microscaled 4-bit format, the verification of drafted tokens and the clipped multi-tensor step
EXPORTED_MX4 = ("zs_mx4_quantize", "zs_mx4_dequantize", "zs_mx4_matmul")
EXPORTED_DRAFTS = ("zs_verify_drafts_workspace_bytes", "zs_verify_drafts")
EXPORTED_CLIP = ("zs_grad_stats_multi_workspace_bytes", "zs_grad_stats_multi", "zs_adamw_shard_step_multi_clip")


def lib():
    return _lib


def _check(status):
    if status != ZS_OK:
        raise ZsError(status, _lib.zs_last_error().decode())


# ---------------------------------------------------------------- marshalling helpers


def _stream(stream):
    if stream is None:
        import torch
        if torch.cuda.is_initialized():  # what current_stream() gives, without its object
            return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


_BF16_NAMES = ("bfloat16", "int16", "uint16")


def _ptr(t, kind, need, what):
    """Device address of ``t`` after checking dtype, device, contiguity and length."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    import torch
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if kind == "bytes":
        if t.dtype not in (torch.uint8, torch.int8):
            raise ValueError(f"{what} must be a uint8 or int8 byte buffer, got {t.dtype}")
    elif kind == "bf16":
        if str(t.dtype).split(".")[-1] not in _BF16_NAMES:
            raise ValueError(f"{what} must hold bf16 (bfloat16 or 16-bit integer storage), got {t.dtype}")
    elif t.dtype != torch.float32:
        raise ValueError(f"{what} must be float32, got {t.dtype}")
    if t.numel() < need:
        raise ValueError(f"{what} holds {t.numel()} elements, the call touches {need}")
    return t.data_ptr()


def _ptr_array(ptrs):
    arr = (ctypes.c_void_p * max(len(ptrs), 1))()
    for i, p in enumerate(ptrs):
        arr[i] = p
    return arr


# ---------------------------------------------------------------- plan


class Plan:
    """Owns a ``zs_plan*``; destroyed with the object (or by ``close``)."""

    def __init__(self, handle):
        self._h = ctypes.c_void_p(handle)
        self._shape = None

    @property
    def shape(self):
        """(shard_numel, world_size), asked of the library once: a plan never changes."""
        if self._shape is None:
            self._shape = (self.shard_numel, self.world_size)
        return self._shape

    @property
    def handle(self):
        if not self._h:
            raise ValueError("plan is closed")
        return self._h

    def close(self):
        if self._h:
            _lib.zs_plan_destroy(self._h)
            self._h = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def padded_numel(self):
        return _lib.zs_plan_padded_numel(self.handle)

    @property
    def shard_numel(self):
        return _lib.zs_plan_shard_numel(self.handle)

    @property
    def persistent_bytes(self):
        return _lib.zs_plan_persistent_bytes(self.handle)

    @property
    def num_tensors(self):
        return _lib.zs_plan_num_tensors(self.handle)

    @property
    def world_size(self):
        return _lib.zs_plan_world_size(self.handle)

    @property
    def rank(self):
        return _lib.zs_plan_rank(self.handle)

    @property
    def layout(self):
        return _lib.zs_plan_layout(self.handle)

    @property
    def workspace_bytes(self):
        return _lib.zs_plan_workspace_bytes(self.handle)

    def tensor(self, i):
        info = TensorInfo()
        _check(_lib.zs_plan_tensor(self.handle, i, ctypes.byref(info)))
        return info

    def tensor_group(self, i):
        g = _lib.zs_plan_tensor_group(self.handle, i)
        if g < 0:
            raise IndexError(f"tensor {i} is not in the plan")
        return g

    def tensor_replicated(self, i):
        r = _lib.zs_plan_tensor_replicated(self.handle, i)
        if r < 0:
            raise IndexError(f"tensor {i} is not in the plan")
        return bool(r)


def zs_shard_plan(numels, world_size, rank, tensor_align_elems=1, layout=ZS_LAYOUT_FLAT):
    arr = (ctypes.c_int64 * max(len(numels), 1))(*numels)
    out = ctypes.c_void_p()
    _check(_lib.zs_shard_plan(arr, len(numels), world_size, rank, tensor_align_elems, layout,
                              ctypes.byref(out)))
    return Plan(out.value)


def zs_shard_plan_ex(numels, world_size, rank, layout=ZS_LAYOUT_PER_TENSOR, tensor_align_elems=1,
                     persist_below_elems=0, groups=None):
    arr = (ctypes.c_int64 * max(len(numels), 1))(*numels)
    opt = PlanOptions(layout, tensor_align_elems, persist_below_elems, None)
    if groups is not None:
        if len(groups) != len(numels):
            raise ValueError(f"groups has {len(groups)} entries for {len(numels)} tensors")
        garr = (ctypes.c_int32 * max(len(groups), 1))(*groups)
        opt.groups = ctypes.cast(garr, ctypes.POINTER(ctypes.c_int32))
    out = ctypes.c_void_p()
    _check(_lib.zs_shard_plan_ex(arr, len(numels), world_size, rank, ctypes.byref(opt), ctypes.byref(out)))
    return Plan(out.value)


# ---------------------------------------------------------------- flat step


def zs_reduce_shard(plan, contribs, grad, off=0, length=None, stream=None):
    S = plan.shard_numel
    length = S - off if length is None else length
    end = min(max(off + length, 0), S)  # a bucket outside the shard is the library's ZS_ERANGE
    ptrs = [_ptr(c, "bf16", end, f"contribs[{q}]") for q, c in enumerate(contribs)]
    g = _ptr(grad, "bf16", end, "grad")
    _check(_lib.zs_reduce_shard(plan.handle, _ptr_array(ptrs), len(ptrs), g, off, length,
                                _stream(stream)))


def zs_adamw_shard_step(plan, hp, grad, master, m, v, param, stream=None):
    S = plan.shard_numel
    _check(_lib.zs_adamw_shard_step(plan.handle, ctypes.byref(hp), _ptr(grad, "bf16", S, "grad"),
                                    _ptr(master, "f32", S, "master"), _ptr(m, "f32", S, "m"),
                                    _ptr(v, "f32", S, "v"), _ptr(param, "bf16", S, "param"),
                                    _stream(stream)))


def zs_gather_params(plan, param, full, stream=None):
    S, r = plan.shard_numel, plan.rank
    _check(_lib.zs_gather_params(plan.handle, _ptr(param, "bf16", S, "param"),
                                 _ptr(full, "bf16", (r + 1) * S, "full"), _stream(stream)))


def zs_plan_reshard_slice(plan, group_size):
    out = ReshardSlice()
    _check(_lib.zs_plan_reshard_slice(plan.handle, group_size, ctypes.byref(out)))
    return out


def zs_gather_params_to_slice(plan, group_size, param, slice_buf, stream=None):
    """param: the own updated bf16 shard (S); slice_buf: the buffer holding the
    k-way slice that contains it (T/k elements)."""
    sl = zs_plan_reshard_slice(plan, group_size)
    _check(_lib.zs_gather_params_to_slice(plan.handle, group_size, _ptr(param, "bf16", plan.shard_numel, "param"),
                                          _ptr(slice_buf, "bf16", sl.slice_len, "slice"), _stream(stream)))


def zs_gather_slice(plan, group_size, shards, slice_buf, stream=None):
    """shards[i]: the updated bf16 shard (S) of rank first_source + i;
    slice_buf: this rank's kept slice (T/k elements)."""
    sl = zs_plan_reshard_slice(plan, group_size)
    ptrs = [_ptr(t, "bf16", plan.shard_numel, f"shards[{i}]") for i, t in enumerate(shards)]
    _check(_lib.zs_gather_slice(plan.handle, group_size, _ptr_array(ptrs), len(ptrs),
                                _ptr(slice_buf, "bf16", sl.slice_len, "slice"), _stream(stream)))


def zs_fused_shard_step(plan, hp, contribs, master, m, v, grad=None, param=None, full=None,
                        stream=None):
    S, r = plan.shard_numel, plan.rank
    ptrs = [_ptr(c, "bf16", S, f"contribs[{q}]") for q, c in enumerate(contribs)]
    _check(_lib.zs_fused_shard_step(plan.handle, ctypes.byref(hp), _ptr_array(ptrs), len(ptrs),
                                    _ptr(master, "f32", S, "master"), _ptr(m, "f32", S, "m"),
                                    _ptr(v, "f32", S, "v"), _ptr(grad, "bf16", S, "grad"),
                                    _ptr(param, "bf16", S, "param"),
                                    _ptr(full, "bf16", (r + 1) * S, "full"), _stream(stream)))


def zs_fused_shard_step_bucket(plan, hp, contribs, master, m, v, off=0, length=None, grad=None, param=None,
                               full=None, stream=None):
    S, r = plan.shard_numel, plan.rank
    length = S - off if length is None else length
    end = min(max(off + length, 0), S)  # a bucket outside the shard is the library's ZS_ERANGE
    ptrs = [_ptr(c, "bf16", end, f"contribs[{q}]") for q, c in enumerate(contribs)]
    _check(_lib.zs_fused_shard_step_bucket(plan.handle, ctypes.byref(hp), _ptr_array(ptrs), len(ptrs),
                                           _ptr(master, "f32", end, "master"), _ptr(m, "f32", end, "m"),
                                           _ptr(v, "f32", end, "v"), _ptr(grad, "bf16", end, "grad"),
                                           _ptr(param, "bf16", end, "param"),
                                           _ptr(full, "bf16", r * S + end, "full"), off, length, _stream(stream)))


# ---------------------------------------------------------------- quantized parameter gather


def zs_quant_code_bytes(plan, bits):
    n = _lib.zs_quant_code_bytes(plan.handle, bits)
    if n < 0:
        raise ValueError(f"bits = {bits} must be 4 or 8")
    return n


def zs_quant_num_scales(plan, block):
    n = _lib.zs_quant_num_scales(plan.handle, block)
    if n < 0:
        raise ValueError(f"block = {block} must be a power of two in [8, 256]")
    return n


def zs_quantize_shard(plan, bits, block, param, codes, scales, stream=None):
    S = plan.shard_numel
    _check(_lib.zs_quantize_shard(plan.handle, bits, block, _ptr(param, "bf16", S, "param"),
                                  _ptr(codes, "bytes", S * bits // 8, "codes"),
                                  _ptr(scales, "f32", -(-S // max(block, 1)), "scales"), _stream(stream)))


def zs_fused_shard_step_quant(plan, hp, contribs, master, m, v, bits, block, codes, scales, grad=None, param=None,
                              stream=None):
    S = plan.shard_numel
    ptrs = [_ptr(c, "bf16", S, f"contribs[{q}]") for q, c in enumerate(contribs)]
    _check(_lib.zs_fused_shard_step_quant(plan.handle, ctypes.byref(hp), _ptr_array(ptrs), len(ptrs),
                                          _ptr(master, "f32", S, "master"), _ptr(m, "f32", S, "m"),
                                          _ptr(v, "f32", S, "v"), _ptr(grad, "bf16", S, "grad"),
                                          _ptr(param, "bf16", S, "param"), bits, block,
                                          _ptr(codes, "bytes", S * bits // 8, "codes"),
                                          _ptr(scales, "f32", -(-S // max(block, 1)), "scales"), _stream(stream)))


def zs_dequant_gather(plan, bits, block, codes_all, scales_all, full, stream=None):
    S, N = plan.shard_numel, plan.world_size
    _check(_lib.zs_dequant_gather(plan.handle, bits, block, _ptr(codes_all, "bytes", N * S * bits // 8, "codes_all"),
                                  _ptr(scales_all, "f32", N * -(-S // max(block, 1)), "scales_all"),
                                  _ptr(full, "bf16", N * S, "full"), _stream(stream)))


# ---------------------------------------------------------------- CPU-offloaded optimizer step

_HOST_KINDS = {"bf16": ("uint16", "int16", "bfloat16"), "f32": ("float32",)}


def _host_ptr(a, kind, need, what):
    """Host address of a numpy array or CPU tensor after checking dtype, contiguity and length."""
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if hasattr(a, "is_cuda"):  # torch tensor
        if a.is_cuda:
            raise ValueError(f"{what} must be host memory")
        if not a.is_contiguous():
            raise ValueError(f"{what} must be contiguous")
        dt, n, addr = str(a.dtype).split(".")[-1], a.numel(), a.data_ptr()
    else:
        if not a.flags.c_contiguous:
            raise ValueError(f"{what} must be contiguous")
        dt, n, addr = str(a.dtype), a.size, a.ctypes.data
    if dt not in _HOST_KINDS[kind]:
        raise ValueError(f"{what} must be {kind}, got {dt}")
    if n < need:
        raise ValueError(f"{what} holds {n} elements, the call touches {need}")
    return addr


def zs_host_adamw_step(hp, grad, master, m, v, param=None, n=None, n_threads=1):
    if n is None:
        n = master.numel() if hasattr(master, "numel") else master.size
    _check(_lib.zs_host_adamw_step(ctypes.byref(hp), _host_ptr(grad, "bf16", n, "grad"),
                                   _host_ptr(master, "f32", n, "master"), _host_ptr(m, "f32", n, "m"),
                                   _host_ptr(v, "f32", n, "v"), _host_ptr(param, "bf16", n, "param"), n, n_threads))


def zs_offload_adamw_step(plan, hp, grad_dev, master_host, m_host, v_host, grad_host, param_host, param_dev=None,
                          full_dev=None, chunk_elems=1 << 24, n_threads=8, stream=None):
    S, r = plan.shard_numel, plan.rank
    _check(_lib.zs_offload_adamw_step(plan.handle, ctypes.byref(hp), _ptr(grad_dev, "bf16", S, "grad_dev"),
                                      _host_ptr(master_host, "f32", S, "master_host"),
                                      _host_ptr(m_host, "f32", S, "m_host"), _host_ptr(v_host, "f32", S, "v_host"),
                                      _host_ptr(grad_host, "bf16", S, "grad_host"),
                                      _host_ptr(param_host, "bf16", S, "param_host"),
                                      _ptr(param_dev, "bf16", S, "param_dev"),
                                      _ptr(full_dev, "bf16", (r + 1) * S, "full_dev"), chunk_elems, n_threads,
                                      _stream(stream)))


# ---------------------------------------------------------------- multi-tensor


def zs_multi_workspace_bytes(plan, n_contribs):
    n = _lib.zs_multi_workspace_bytes(plan.handle, n_contribs)
    if n < 0:
        raise ZsError(ZS_EINVAL, "multi-tensor workspace needs a PER_TENSOR plan")
    return n


# Bound workspaces, keyed by device address: the workspace tensor and every
# tensor whose address its table holds. Keeping them referenced until
# zs_multi_unbind means no bound buffer can be freed (and its memory reused by
# the caching allocator) while a step may still write through the table.
_bindings = {}


def zs_multi_bind(plan, pieces, contribs, workspace, stream=None):
    """pieces[i]: dict with keys grad, master, m, v, param, full (tensors or
    None) for tensor i; contribs: None or contribs[q][i] = rank q's piece of
    tensor i. workspace: a CUDA uint8 tensor of zs_multi_workspace_bytes.
    The binding keeps references to the workspace and every bound tensor
    until zs_multi_unbind(workspace)."""
    n = plan.num_tensors
    if len(pieces) != n:
        raise ValueError(f"{len(pieces)} piece records for a plan of {n} tensors")
    recs = (PiecePtrs * max(n, 1))()
    for i, pc in enumerate(pieces):
        info = plan.tensor(i)
        Si = info.own_hi - info.own_lo
        recs[i] = PiecePtrs(_ptr(pc.get("grad"), "bf16", Si, f"pieces[{i}].grad"),
                            _ptr(pc.get("master"), "f32", Si, f"pieces[{i}].master"),
                            _ptr(pc.get("m"), "f32", Si, f"pieces[{i}].m"),
                            _ptr(pc.get("v"), "f32", Si, f"pieces[{i}].v"),
                            _ptr(pc.get("param"), "bf16", Si, f"pieces[{i}].param"),
                            _ptr(pc.get("full"), "bf16", info.padded_numel, f"pieces[{i}].full"))
    nq = 0 if contribs is None else len(contribs)
    flat = []
    for q in range(nq):
        if len(contribs[q]) != n:
            raise ValueError(f"contribs[{q}] has {len(contribs[q])} pieces, the plan has {n}")
        for i in range(n):
            info = plan.tensor(i)
            flat.append(_ptr(contribs[q][i], "bf16", info.own_hi - info.own_lo, f"contribs[{q}][{i}]"))
    import torch
    if not (isinstance(workspace, torch.Tensor) and workspace.is_cuda):
        raise ValueError("workspace must be a CUDA tensor")
    _check(_lib.zs_multi_bind(plan.handle, recs, _ptr_array(flat) if nq else None, nq,
                              workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                              _stream(stream)))
    refs = [t for pc in pieces for t in pc.values() if t is not None and not isinstance(t, int)]
    if nq:
        refs += [t for row in contribs for t in row if not isinstance(t, int)]
    _bindings[workspace.data_ptr()] = (workspace, refs)


def zs_multi_unbind(workspace, stream=None):
    _check(_lib.zs_multi_unbind(workspace.data_ptr(), _stream(stream)))
    _bindings.pop(workspace.data_ptr(), None)


def zs_reduce_shard_multi(plan, workspace, stream=None):
    _check(_lib.zs_reduce_shard_multi(plan.handle, workspace.data_ptr(), _stream(stream)))


def zs_adamw_shard_step_multi(plan, hp, workspace, stream=None):
    _check(_lib.zs_adamw_shard_step_multi(plan.handle, ctypes.byref(hp), workspace.data_ptr(),
                                          _stream(stream)))


def zs_gather_params_multi(plan, workspace, stream=None):
    _check(_lib.zs_gather_params_multi(plan.handle, workspace.data_ptr(), _stream(stream)))


def zs_fused_shard_step_multi(plan, hp, workspace, stream=None):
    _check(_lib.zs_fused_shard_step_multi(plan.handle, ctypes.byref(hp), workspace.data_ptr(),
                                          _stream(stream)))


def _hp_array(hps):
    if not hps:
        raise ValueError("at least one set of hyperparameters is needed")
    return (AdamWHParams * len(hps))(*hps), len(hps)


def zs_adamw_shard_step_multi_groups(plan, hps, workspace, stream=None):
    arr, n = _hp_array(hps)
    _check(_lib.zs_adamw_shard_step_multi_groups(plan.handle, arr, n, workspace.data_ptr(), _stream(stream)))


def zs_fused_shard_step_multi_groups(plan, hps, workspace, stream=None):
    arr, n = _hp_array(hps)
    _check(_lib.zs_fused_shard_step_multi_groups(plan.handle, arr, n, workspace.data_ptr(), _stream(stream)))


# ---------------------------------------------------------------- accumulation and clipping


def _scalar_ptr(t, dtype_name, what):
    if t is None:
        return None
    import torch
    if not (isinstance(t, torch.Tensor) and t.is_cuda and str(t.dtype).endswith(dtype_name) and t.numel() >= 1):
        raise ValueError(f"{what} must be a CUDA {dtype_name} tensor of at least one element")
    return t.data_ptr()


def zs_accumulate_shard(plan, contribs, acc, off=0, length=None, first=False, stream=None):
    S = plan.shard_numel
    length = S - off if length is None else length
    end = min(max(off + length, 0), S)
    ptrs = [_ptr(c, "bf16", end, f"contribs[{q}]") for q, c in enumerate(contribs)]
    _check(_lib.zs_accumulate_shard(plan.handle, _ptr_array(ptrs), len(ptrs), _ptr(acc, "f32", end, "acc"), off,
                                    length, 1 if first else 0, _stream(stream)))


def zs_grad_stats_workspace_bytes(plan):
    return _lib.zs_grad_stats_workspace_bytes(plan.handle)


def zs_grad_stats(plan, acc, grad_divisor, sumsq_out, nonfinite_out, workspace, stream=None):
    """sumsq_out: CUDA float64 tensor (>= 1 element); nonfinite_out: CUDA int32
    tensor; workspace: CUDA uint8 tensor of zs_grad_stats_workspace_bytes."""
    _check(_lib.zs_grad_stats(plan.handle, _ptr(acc, "f32", plan.shard_numel, "acc"), grad_divisor,
                              _scalar_ptr(sumsq_out, "float64", "sumsq_out"),
                              _scalar_ptr(nonfinite_out, "int32", "nonfinite_out"), workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), _stream(stream)))


def zs_grad_stats_noalloc(plan, acc, grad_divisor, sumsq_out, nonfinite_out, stream=None):
    """zs_grad_stats with the partials in the library's static device array
    (no workspace, no allocation); shards up to GRAD_STATS_NOALLOC_MAX_ELEMS."""
    _check(_lib.zs_grad_stats_noalloc(plan.handle, _ptr(acc, "f32", plan.shard_numel, "acc"),
                                      ctypes.c_float(grad_divisor), _scalar_ptr(sumsq_out, "float64", "sumsq_out"),
                                      _scalar_ptr(nonfinite_out, "int32", "nonfinite_out"), _stream(stream)))


def zs_clip_scale(sumsq, nonfinite, max_norm, scale_out, skip_out, stream=None):
    """sumsq: CUDA float64 tensor of the ranks' squared norms; nonfinite: CUDA
    int32 tensor of their flags (same length)."""
    n = sumsq.numel()
    if nonfinite.numel() != n:
        raise ValueError("sumsq and nonfinite must have one entry per rank")
    _check(_lib.zs_clip_scale(_scalar_ptr(sumsq, "float64", "sumsq"), _scalar_ptr(nonfinite, "int32", "nonfinite"),
                              n, max_norm, _scalar_ptr(scale_out, "float32", "scale_out"),
                              _scalar_ptr(skip_out, "int32", "skip_out"), _stream(stream)))


def zs_adamw_shard_step_accum(plan, hp, acc, grad_divisor, master, m, v, scale=None, skip=None, param=None,
                              full=None, stream=None):
    S, r = plan.shard_numel, plan.rank
    _check(_lib.zs_adamw_shard_step_accum(plan.handle, ctypes.byref(hp), _ptr(acc, "f32", S, "acc"), grad_divisor,
                                          _scalar_ptr(scale, "float32", "scale"), _scalar_ptr(skip, "int32", "skip"),
                                          _ptr(master, "f32", S, "master"), _ptr(m, "f32", S, "m"),
                                          _ptr(v, "f32", S, "v"), _ptr(param, "bf16", S, "param"),
                                          _ptr(full, "bf16", (r + 1) * S, "full"), _stream(stream)))


def zs_grad_stats_multi_workspace_bytes(plan):
    return _lib.zs_grad_stats_multi_workspace_bytes(plan.handle)


def _scalar_on(device, t, dtype_name, what):
    """_scalar_ptr of a tensor that has to be on the call's device."""
    p = _scalar_ptr(t, dtype_name, what)
    if t is not None and t.get_device() != device:
        raise _lm_elsewhere(t, device, what)
    return p


def zs_grad_stats_multi(plan, sumsq_out, nonfinite_out, workspace, stats_workspace, stream=None):
    """Squared norm and non-finite flag of the grad pieces bound to workspace.
    sumsq_out: CUDA float64 tensor (>= 1 element); nonfinite_out: CUDA int32
    tensor; stats_workspace: CUDA uint8 tensor of
    zs_grad_stats_multi_workspace_bytes."""
    device = _lm_device(workspace, "workspace")
    _lm_call(_lib.zs_grad_stats_multi, device, stream, plan.handle, workspace.data_ptr(),
             _scalar_on(device, sumsq_out, "float64", "sumsq_out"),
             _scalar_on(device, nonfinite_out, "int32", "nonfinite_out"),
             *_lm_workspace(stats_workspace, device, "stats_workspace"))


def zs_adamw_shard_step_multi_clip(plan, hps, workspace, scale=None, skip=None, stream=None):
    """The multi-tensor AdamW step from the gradient times *scale, left out
    where *skip is set. hps: one set of hyperparameters per group."""
    arr, n = _hp_array(hps)
    device = _lm_device(workspace, "workspace")
    _lm_call(_lib.zs_adamw_shard_step_multi_clip, device, stream, plan.handle, arr, n,
             _scalar_on(device, scale, "float32", "scale"), _scalar_on(device, skip, "int32", "skip"),
             workspace.data_ptr())


# ---------------------------------------------------------------- scalars in device memory


def zs_adamw_coefs_compute(hp):
    """The fp32 scalars of hp's step (an AdamWCoefs; .values() lists them in
    the order a device buffer holds them)."""
    out = AdamWCoefs()
    _check(_lib.zs_adamw_coefs_compute(ctypes.byref(hp), ctypes.byref(out)))
    return out


def _coefs_ptr(coefs, n_sets=1):
    return _ptr(coefs, "f32", 9 * n_sets, "coefs")


def zs_fused_shard_step_dc(plan, coefs, contribs, master, m, v, grad=None, param=None, full=None, stream=None):
    S, r = plan.shard_numel, plan.rank
    ptrs = [_ptr(c, "bf16", S, f"contribs[{q}]") for q, c in enumerate(contribs)]
    _check(_lib.zs_fused_shard_step_dc(plan.handle, _coefs_ptr(coefs), _ptr_array(ptrs), len(ptrs),
                                       _ptr(master, "f32", S, "master"), _ptr(m, "f32", S, "m"),
                                       _ptr(v, "f32", S, "v"), _ptr(grad, "bf16", S, "grad"),
                                       _ptr(param, "bf16", S, "param"), _ptr(full, "bf16", (r + 1) * S, "full"),
                                       _stream(stream)))


def zs_adamw_shard_step_dc(plan, coefs, grad, master, m, v, param, stream=None):
    S = plan.shard_numel
    _check(_lib.zs_adamw_shard_step_dc(plan.handle, _coefs_ptr(coefs), _ptr(grad, "bf16", S, "grad"),
                                       _ptr(master, "f32", S, "master"), _ptr(m, "f32", S, "m"),
                                       _ptr(v, "f32", S, "v"), _ptr(param, "bf16", S, "param"), _stream(stream)))


def zs_adamw_shard_step_accum_dc(plan, coefs, acc, grad_divisor, master, m, v, scale=None, skip=None, param=None,
                                 full=None, stream=None):
    S, r = plan.shard_numel, plan.rank
    _check(_lib.zs_adamw_shard_step_accum_dc(plan.handle, _coefs_ptr(coefs), _ptr(acc, "f32", S, "acc"),
                                             grad_divisor, _scalar_ptr(scale, "float32", "scale"),
                                             _scalar_ptr(skip, "int32", "skip"), _ptr(master, "f32", S, "master"),
                                             _ptr(m, "f32", S, "m"), _ptr(v, "f32", S, "v"),
                                             _ptr(param, "bf16", S, "param"), _ptr(full, "bf16", (r + 1) * S, "full"),
                                             _stream(stream)))


def zs_fused_shard_step_multi_dc(plan, coefs, n_groups, workspace, stream=None):
    _check(_lib.zs_fused_shard_step_multi_dc(plan.handle, _coefs_ptr(coefs, n_groups), n_groups,
                                             workspace.data_ptr(), _stream(stream)))


# ---------------------------------------------------------------- language-model operators
# A product for one token runs a few microseconds on the device, so what a call
# does in Python is kept short: integers instead of torch's shape and device
# objects, and error texts built only when a check fails.

_torch = None


def _lm_torch():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _lm_device(t, what):
    """Index of the call's device, that of its first tensor. The
    language-model calls run on this device's current stream, whichever device
    is current."""
    if not (isinstance(t, _lm_torch().Tensor) and t.is_cuda):
        raise ValueError(f"{what} must be a CUDA tensor")
    return t.get_device()


def _lm_elsewhere(t, device, what):
    return ValueError(f"{what} is on {t.device}, the call's first tensor on cuda:{device}")


def _lm_rows(t, rows, cols, device, what):
    """Row stride of a [rows, cols] matrix whose rows are contiguous (its dtype is the caller's to check)."""
    if t.get_device() != device:
        raise _lm_elsewhere(t, device, what)
    if t.shape != (rows, cols):
        raise ValueError(f"{what} must be [{rows}, {cols}], got {list(t.shape)}")
    row, col = t.stride()
    if cols > 1 and col != 1:
        raise ValueError(f"{what} must have contiguous rows, its strides are {t.stride()}")
    # the stride of a single row is free, and may be anything in torch
    return row if rows > 1 else max(cols, 1)


def _lm_array(t, dtype, numel, cols, device, what):
    """Address of a contiguous array of exactly [numel] (cols 0) or [numel / cols, cols], or None."""
    if t is None:
        return None
    if t.get_device() != device:
        raise _lm_elsewhere(t, device, what)
    if t.dtype is not dtype or t.numel() != numel or (t.dim() != 1 if cols == 0 else
                                                      t.dim() != 2 or t.size(1) != cols):
        shape = [numel] if cols == 0 else [numel // cols, cols]
        raise ValueError(f"{what} must be {dtype} of shape {shape}, got {t.dtype} of {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _lm_flat(t, dtypes, need, device, what):
    """Address of a contiguous buffer of at least `need` elements (an integer is taken as the address itself)."""
    if isinstance(t, int):
        return t
    if t.get_device() != device:
        raise _lm_elsewhere(t, device, what)
    if t.dtype not in dtypes or not t.is_contiguous() or t.numel() < need:
        raise ValueError(f"{what} must hold at least {need} contiguous elements of {dtypes[0]}, got {t.numel()} of "
                         f"{t.dtype}")
    return t.data_ptr()


def _lm_workspace(t, device, what):
    """(address, bytes) of a workspace, whose size the library checks: an address alone does not tell it."""
    if not isinstance(t, _torch.Tensor):
        raise ValueError(f"{what} must be a CUDA uint8 tensor, got {type(t).__name__}")
    return _lm_flat(t, (_torch.uint8,), 0, device, what), t.numel()


def _lm_call(fn, device, stream, *args):
    """Runs fn(*args, stream) with the call's device current."""
    torch = _torch
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device)
    elif not isinstance(stream, int):
        if stream.device.index != device:
            raise ValueError(f"stream is on {stream.device}, the call's tensors on cuda:{device}")
        stream = stream.cuda_stream
    if torch._C._cuda_getDevice() == device:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status != ZS_OK:
        _check(status)


def _lm_logits(logits):
    """(device, dtype code, rows, vocab, row stride) of a [rows, vocab] matrix of logits."""
    device = _lm_device(logits, "logits")
    dtype = logits.dtype
    if dtype is _torch.bfloat16:
        code = ZS_DTYPE_BF16
    elif dtype is _torch.float32:
        code = ZS_DTYPE_F32
    else:
        raise ValueError(f"logits must be bfloat16 or float32, got {dtype}")
    if logits.dim() != 2:
        raise ValueError(f"logits must be [rows, vocab], got {list(logits.shape)}")
    rows, vocab = logits.shape
    return device, code, rows, vocab, _lm_rows(logits, rows, vocab, device, "logits")


def _lm_grad(grad, logits, rows, vocab, device):
    if grad.dtype is not logits.dtype:
        raise ValueError(f"grad_logits must be {logits.dtype} like the logits, got {grad.dtype}")
    return grad.data_ptr(), _lm_rows(grad, rows, vocab, device, "grad_logits")


def zs_quant_matvec(plan, tensor, out_features, in_features, bits, block, codes_all, scales_all, x, y, stream=None):
    """y[r, o] = sum_i W[o, i] x[r, i] with W = tensor `tensor` of the plan (out_features x in_features) read from
    the quantized gather's payload. x: bfloat16 [rows, in_features]; y: bfloat16 or float32 [rows, out_features]."""
    device = _lm_device(x, "x")
    if x.dim() != 2 or x.dtype is not _torch.bfloat16:
        raise ValueError(f"x must be bfloat16 [rows, {in_features}], got {x.dtype} of {list(x.shape)}")
    rows = x.size(0)
    xs = _lm_rows(x, rows, in_features, device, "x")
    ys = _lm_rows(y, rows, out_features, device, "y")
    if y.dtype is _torch.bfloat16:
        y_dtype = ZS_DTYPE_BF16
    elif y.dtype is _torch.float32:
        y_dtype = ZS_DTYPE_F32
    else:
        raise ValueError(f"y must be bfloat16 or float32, got {y.dtype}")
    S, N = plan.shape
    _lm_call(_lib.zs_quant_matvec, device, stream, plan.handle, tensor, out_features, in_features, bits, block,
             _lm_flat(codes_all, (_torch.uint8, _torch.int8), N * S * bits // 8, device, "codes_all"),
             _lm_flat(scales_all, (_torch.float32,), N * -(-S // max(block, 1)), device, "scales_all"), x.data_ptr(),
             xs, rows, y.data_ptr(), y_dtype, ys)


def zs_token_logprobs(logits, tokens, temperature=1.0, logprob=None, entropy=None, stats=None, top_ids=None,
                      top_logprobs=None, stream=None):
    """logits: bfloat16 or float32 [rows, vocab]; tokens: int32 [rows]. Outputs, each optional: logprob and entropy
    float32 [rows]; stats float32 [rows, 2], which the gradient takes; top_ids int32 and top_logprobs float32
    [rows, top], together."""
    device, dtype, rows, vocab, stride = _lm_logits(logits)
    i32, f32 = _torch.int32, _torch.float32
    if (top_ids is None) != (top_logprobs is None):
        raise ValueError("top_ids and top_logprobs are given together")
    top = 0
    if top_ids is not None:
        if top_ids.dim() != 2:
            raise ValueError(f"top_ids must be [{rows}, top], got {list(top_ids.shape)}")
        top = top_ids.size(1)
        if top == 0:
            top_ids = top_logprobs = None
    _lm_call(_lib.zs_token_logprobs, device, stream, logits.data_ptr(), dtype, rows, vocab, stride,
             _lm_array(tokens, i32, rows, 0, device, "tokens"), temperature,
             _lm_array(logprob, f32, rows, 0, device, "logprob"),
             _lm_array(entropy, f32, rows, 0, device, "entropy"),
             _lm_array(stats, f32, 2 * rows, 2, device, "stats"), top,
             _lm_array(top_ids, i32, rows * top, top, device, "top_ids"),
             _lm_array(top_logprobs, f32, rows * top, top, device, "top_logprobs"))


def zs_token_logprobs_backward(logits, tokens, stats, grad_logprob, grad_logits, temperature=1.0, entropy=None,
                               grad_entropy=None, stream=None):
    """grad_logits (the logits' dtype; logits itself for in place) from the forward call's stats and the gradients of
    logprob and, with the forward call's entropy, of entropy."""
    device, dtype, rows, vocab, stride = _lm_logits(logits)
    f32 = _torch.float32
    gp, gs = _lm_grad(grad_logits, logits, rows, vocab, device)
    _lm_call(_lib.zs_token_logprobs_backward, device, stream, logits.data_ptr(), dtype, rows, vocab, stride,
             _lm_array(tokens, _torch.int32, rows, 0, device, "tokens"), temperature,
             _lm_array(stats, f32, 2 * rows, 2, device, "stats"),
             _lm_array(entropy, f32, rows, 0, device, "entropy"),
             _lm_array(grad_logprob, f32, rows, 0, device, "grad_logprob"),
             _lm_array(grad_entropy, f32, rows, 0, device, "grad_entropy"), gp, gs)


def zs_distill_topk(logits, teacher_ids, teacher_logits, loss, grad_logits=None, temperature=1.0, row_weight=None,
                    stream=None):
    """Distillation loss [rows] (float32) from the teacher's top entries (teacher_ids int32, teacher_logits float32,
    both [rows, k]; a negative id is unused) and, if given, its gradient grad_logits (the logits' dtype; logits itself
    for in place)."""
    device, dtype, rows, vocab, stride = _lm_logits(logits)
    f32 = _torch.float32
    if teacher_ids.dim() != 2:
        raise ValueError(f"teacher_ids must be [{rows}, k], got {list(teacher_ids.shape)}")
    k = teacher_ids.size(1)
    gp, gs = (None, vocab) if grad_logits is None else _lm_grad(grad_logits, logits, rows, vocab, device)
    _lm_call(_lib.zs_distill_topk, device, stream, logits.data_ptr(), dtype, rows, vocab, stride,
             _lm_array(teacher_ids, _torch.int32, rows * k, k, device, "teacher_ids"),
             _lm_array(teacher_logits, f32, rows * k, k, device, "teacher_logits"), k, temperature,
             _lm_array(row_weight, f32, rows, 0, device, "row_weight"),
             _lm_array(loss, f32, rows, 0, device, "loss"), gp, gs)


# ---------------------------------------------------------------- microscaled 4-bit floating point


def _float_code(t, what):
    if t.dtype is _torch.bfloat16:
        return ZS_DTYPE_BF16
    if t.dtype is _torch.float32:
        return ZS_DTYPE_F32
    raise ValueError(f"{what} must be bfloat16 or float32, got {t.dtype}")


def _mx4_matrix(codes, scales, rows, blocks, device, names):
    """(codes address, stride, scales address, stride) of a quantized [rows, 32 * blocks] matrix."""
    u8 = _torch.uint8
    if codes.dtype is not u8 or scales.dtype is not u8:
        raise ValueError(f"{names[0]} and {names[1]} must be uint8, got {codes.dtype} and {scales.dtype}")
    cs = _lm_rows(codes, rows, 16 * blocks, device, names[0])
    ss = _lm_rows(scales, rows, blocks, device, names[1])
    if rows <= 1 or blocks == 0:  # such a stride is free in torch, and the library takes whole blocks
        cs = 16 * blocks
    return codes.data_ptr(), cs, scales.data_ptr(), ss


def _mx4_conversion(x, codes, scales):
    device = _lm_device(x, "x")
    code = _float_code(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be [rows, cols], got {list(x.shape)}")
    rows, cols = x.shape
    return device, code, rows, cols, _lm_rows(x, rows, cols, device, "x"), \
        _mx4_matrix(codes, scales, rows, -(-cols // ZS_MX4_BLOCK), device, ("codes", "scales"))


def zs_mx4_quantize(x, codes, scales, stream=None):
    """Codes (uint8 [rows, 16 * blocks], two elements a byte) and scales (uint8 [rows, blocks]) of x, bfloat16 or
    float32 [rows, cols], in blocks = ceil(cols / 32) blocks a row."""
    device, code, rows, cols, xs, q = _mx4_conversion(x, codes, scales)
    _lm_call(_lib.zs_mx4_quantize, device, stream, x.data_ptr(), code, rows, cols, xs, *q)


def zs_mx4_dequantize(codes, scales, x, stream=None):
    """x (bfloat16 or float32 [rows, cols]) from its codes and scales."""
    device, code, rows, cols, xs, q = _mx4_conversion(x, codes, scales)
    _lm_call(_lib.zs_mx4_dequantize, device, stream, *q, rows, cols, x.data_ptr(), code, xs)


def zs_mx4_matmul(x_codes, x_scales, w_codes, w_scales, y, stream=None):
    """y = X W^T (bfloat16 or float32 [rows, out_features]) of two quantized matrices: codes uint8 [rows, 16 * blocks]
    and [out_features, 16 * blocks], scales uint8 [rows, blocks] and [out_features, blocks]."""
    device = _lm_device(x_codes, "x_codes")
    if x_scales.dim() != 2 or w_scales.dim() != 2:
        raise ValueError(f"x_scales and w_scales must be matrices, got {list(x_scales.shape)} and "
                         f"{list(w_scales.shape)}")
    rows, blocks = x_scales.shape
    out = w_scales.shape[0]
    x = _mx4_matrix(x_codes, x_scales, rows, blocks, device, ("x_codes", "x_scales"))
    w = _mx4_matrix(w_codes, w_scales, out, blocks, device, ("w_codes", "w_scales"))
    code = _float_code(y, "y")
    _lm_call(_lib.zs_mx4_matmul, device, stream, *x, rows, *w, out, ZS_MX4_BLOCK * blocks, y.data_ptr(), code,
             _lm_rows(y, rows, out, device, "y"))


# ---------------------------------------------------------------- verification of drafted tokens


def zs_verify_drafts_workspace_bytes(requests, drafts, vocab):
    n = _lib.zs_verify_drafts_workspace_bytes(requests, drafts, vocab)
    if n < 0:
        raise ZsError(ZS_EINVAL, zs_last_error())
    return n


def zs_verify_drafts(target_logits, draft_tokens, uniforms, accepted, tokens, workspace, draft_logits=None,
                     draft_lens=None, logprobs=None, temperature=1.0, stream=None):
    """How many drafted tokens of each request stand, and the token drawn behind them. target_logits: bfloat16 or
    float32 [requests * (drafts + 1), vocab]; draft_tokens: int32 [requests, drafts]; uniforms: float32
    [requests, drafts + 1]; draft_logits (None: the drafted token was certain): like target_logits
    [requests * drafts, vocab]; draft_lens (None: all have `drafts`): int32 [requests]. Outputs: accepted int32
    [requests], tokens int32 and logprobs (optional) float32 [requests, drafts + 1]. workspace: uint8, of
    zs_verify_drafts_workspace_bytes."""
    device, code, places, vocab, stride = _lm_logits(target_logits)
    if draft_tokens.dim() != 2:
        raise ValueError(f"draft_tokens must be [requests, drafts], got {list(draft_tokens.shape)}")
    requests, drafts = draft_tokens.shape
    if places != requests * (drafts + 1):
        raise ValueError(f"target_logits must have {requests * (drafts + 1)} rows, got {places}")
    i32, f32 = _torch.int32, _torch.float32
    dp, ds = None, vocab
    if draft_logits is not None:
        if draft_logits.dtype is not target_logits.dtype:
            raise ValueError(f"draft_logits must be {target_logits.dtype} like the target's, got {draft_logits.dtype}")
        dp, ds = draft_logits.data_ptr(), _lm_rows(draft_logits, requests * drafts, vocab, device, "draft_logits")
    _lm_call(_lib.zs_verify_drafts, device, stream, target_logits.data_ptr(), code, requests, drafts, vocab, stride,
             dp, ds, _lm_array(draft_tokens, i32, requests * drafts, drafts, device, "draft_tokens") if drafts else None,
             _lm_array(draft_lens, i32, requests, 0, device, "draft_lens"),
             _lm_array(uniforms, f32, places, drafts + 1, device, "uniforms"), temperature,
             _lm_array(accepted, i32, requests, 0, device, "accepted"),
             _lm_array(tokens, i32, places, drafts + 1, device, "tokens"),
             _lm_array(logprobs, f32, places, drafts + 1, device, "logprobs"),
             *_lm_workspace(workspace, device, "workspace"))


def zs_last_error():
    return _lib.zs_last_error().decode()


def zs_version():
    return _lib.zs_version().decode()
