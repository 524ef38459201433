"""GB300-native (sm_103a) Kimi Delta Attention serving hot path -- Python binding of ``libkda.so``.

Argument marshalling only: every step of the path runs in the CUDA kernels behind the C ABI declared in
``include/kda.h``.  PyTorch provides device memory and streams.  There is no fallback: if the library
is missing the import of an entry point raises.

Entry points (same names as the C ABI): ``kda_project_inputs``, ``kda_decode_step``, ``kda_decode_multi``,
``kda_prefill_chunked``,
``kda_resume_from_slot``, ``kda_prefill_workspace_bytes``, ``kda_checkpoint_count``,
``kda_status_string``; the host prefix index ``kda_prefix_*`` through :class:`PrefixIndex`; latent attention over
a paged cache (:class:`LatentCache`, :class:`PageTable`): ``kda_latent_append``, ``kda_latent_decode``,
``kda_latent_prefill`` and the page pool's ``kda_pages_reserve``, ``kda_pages_truncate``, ``kda_pages_fork``,
``kda_pages_compact``, ``kda_pages_copy``; grouped-query attention over the same pool (:class:`KvCache`):
``kda_kv_append``, ``kda_kv_decode``, ``kda_kv_evict``; rotary positions (:class:`Rope`): ``kda_rope_apply``.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkda.so")
_lib = None

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED_SHAPE, KDA_ERR_WORKSPACE, KDA_ERR_CUDA = 0, 1, 2, 3, 4
KDA_DEV_BAD_SLOT, KDA_DEV_BAD_SEQLENS, KDA_DEV_BAD_CKPT, KDA_DEV_TIMEOUT = 1, 2, 4, 16
KDA_DEV_BAD_PAGE, KDA_DEV_NO_PAGES = 8, 32


class KdaError(RuntimeError):
    def __init__(self, rc: int, what: str, detail: str = ""):
        super().__init__(f"{what}: {kda_status_string(rc)} (status {rc})" + (f": {detail}" if detail else ""))
        self.rc = rc
        self.detail = detail


KDA_STATE_FP32, KDA_STATE_BF16 = 0, 1
KDA_ELEM_BF16, KDA_ELEM_FP16 = 0, 1
LATENT_MAX_TOKENS, LATENT_MAX_HEADS = 64, 128  # KDA_LATENT_MAX_* in kda.h
KDA_ROPE_PLAIN, KDA_ROPE_LINEAR, KDA_ROPE_NTK, KDA_ROPE_PARTS = 0, 1, 2, 3
KV_MAX_TOKENS, KV_MAX_HEADS, KV_EVICT_MAX_LEN = 64, 256, 1 << 20  # KDA_KV_* in kda.h


class _Pool(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("conv_w", ctypes.c_int32),
                ("state_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32), ("num_slots", ctypes.c_int64),
                ("S", ctypes.c_void_p), ("conv", ctypes.c_void_p)]


class _Params(ctypes.Structure):
    _fields_ = [("conv_weight", ctypes.c_void_p), ("norm_weight", ctypes.c_void_p), ("l2_eps", ctypes.c_float),
                ("rms_eps", ctypes.c_float), ("scale", ctypes.c_float), ("conv_silu", ctypes.c_int32)]


class _LatentCache(ctypes.Structure):
    _fields_ = [("rank", ctypes.c_int32), ("rope", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("layers", ctypes.c_int32), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("layer_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("pages", ctypes.c_void_p)]


class _PageTable(ctypes.Structure):
    _fields_ = [("max_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("num_pages", ctypes.c_int64), ("table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("refcount", ctypes.c_void_p)]


class _KvCache(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("layers", ctypes.c_int32), ("dtype", ctypes.c_int32), ("stats", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("layer_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("pages", ctypes.c_void_p)]


class _Rope(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("offset", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scale", ctypes.c_float), ("turns", ctypes.c_void_p)]


class _PrefixPlan(ctypes.Structure):
    _fields_ = [("plan_id", ctypes.c_uint64), ("src_slot", ctypes.c_int32), ("private_slot", ctypes.c_int32),
                ("start_pos", ctypes.c_int64), ("num_ckpts", ctypes.c_int32), ("reserved", ctypes.c_int32)]


KDA_RETAIN_INTERVAL, KDA_RETAIN_SECOND_HIT = 0, 1


def load_library(path: str | None = None):
    """Load libkda.so (built in-tree by ``hybrid_linear_attention_decode_gb300/build.py``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libkda.so not built ({p}); run __graft_entry__.build() first")
    lib = ctypes.CDLL(p)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.kda_decode_step.argtypes = [ctypes.POINTER(_Pool), ctypes.POINTER(_Params), i32] + [vp] * 11
    lib.kda_decode_step.restype = ctypes.c_int
    lib.kda_decode_multi.argtypes = [ctypes.POINTER(_Pool), ctypes.POINTER(_Params), i32, i32] + [vp] * 11
    lib.kda_decode_multi.restype = ctypes.c_int
    lib.kda_project_inputs.argtypes = [i64, i32, i32, i32, i32] + [vp] * 10
    lib.kda_project_inputs.restype = ctypes.c_int
    lib.kda_checkpoint_count.argtypes = [i64, i64, i64]
    lib.kda_checkpoint_count.restype = i64
    lib.kda_prefill_workspace_bytes.argtypes = [ctypes.POINTER(_Pool), i32, i64, i32]
    lib.kda_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.kda_prefill_chunked.argtypes = [ctypes.POINTER(_Pool), ctypes.POINTER(_Params), i32, i64, vp, vp, vp, vp, i32,
                                        i64, vp, vp] + [vp] * 7 + [vp, ctypes.c_size_t, vp, vp]
    lib.kda_prefill_chunked.restype = ctypes.c_int
    lib.kda_prefill_chunked_noalloc.argtypes = [ctypes.POINTER(_Pool), ctypes.POINTER(_Params), i32, i64, vp, vp, vp,
                                                vp, i32, i64, vp, vp] + [vp] * 7 + [vp, vp]
    lib.kda_prefill_chunked_noalloc.restype = ctypes.c_int
    lib.kda_resume_from_slot.argtypes = [ctypes.POINTER(_Pool), i32, vp, vp, vp, vp]
    lib.kda_resume_from_slot.restype = ctypes.c_int
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_version.restype = ctypes.c_int
    lib.kda_last_error_string.argtypes = []
    lib.kda_last_error_string.restype = ctypes.c_char_p
    lib.kda_check_slots.argtypes = [i64, i32, vp, vp, i32, vp]
    lib.kda_check_slots.restype = ctypes.c_int
    pcache, ptable, f32 = ctypes.POINTER(_LatentCache), ctypes.POINTER(_PageTable), ctypes.c_float
    lib.kda_latent_append.argtypes = [pcache, i32, ptable, i32, vp, vp, i64, vp, i64, vp, i64, vp, vp]
    lib.kda_latent_append.restype = ctypes.c_int
    lib.kda_latent_decode_workspace_bytes.argtypes = [pcache, i32, i32, i32]
    lib.kda_latent_decode_workspace_bytes.restype = ctypes.c_size_t
    lib.kda_latent_decode.argtypes = [pcache, i32, ptable, i32, vp, vp, i64, i32, i32, vp, i64, i64, vp, f32, vp, vp,
                                      vp, ctypes.c_size_t, vp, vp]
    lib.kda_latent_decode.restype = ctypes.c_int
    lib.kda_latent_prefill.argtypes = [i32] * 6 + [vp, vp, i64, i64, i32, i32, vp, i64, i64, vp, i64, i64, vp, i64, vp,
                                                   i64, i64, f32, vp, vp, vp, vp]
    lib.kda_latent_prefill.restype = ctypes.c_int
    lib.kda_pages_workspace_bytes.argtypes = [ptable, i32]
    lib.kda_pages_workspace_bytes.restype = ctypes.c_size_t
    for name in ("kda_pages_reserve", "kda_pages_fork"):
        getattr(lib, name).argtypes = [ptable, pcache, i32, vp, vp, vp, ctypes.c_size_t, vp, vp]
        getattr(lib, name).restype = ctypes.c_int
    lib.kda_pages_truncate.argtypes = [ptable, i32, vp, vp, vp, ctypes.c_size_t, vp, vp]
    lib.kda_pages_truncate.restype = ctypes.c_int
    lib.kda_pages_compact.argtypes = [ptable, pcache, vp, ctypes.c_size_t, vp, vp]
    lib.kda_pages_compact.restype = ctypes.c_int
    lib.kda_pages_copy.argtypes = [pcache, i32, vp, vp, vp, vp]
    lib.kda_pages_copy.restype = ctypes.c_int
    pkv, prope, f64 = ctypes.POINTER(_KvCache), ctypes.POINTER(_Rope), ctypes.c_double
    lib.kda_kv_cache_pages.argtypes = [pkv, pcache]
    lib.kda_rope_turns.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp]
    lib.kda_rope_turns_of.argtypes = [i32, vp, vp]
    lib.kda_rope_apply.argtypes = [prope, i32, i64, i32, i32, vp, i32, vp, i64, i64, vp, i64, i64, vp]
    lib.kda_kv_append.argtypes = [pkv, i32, ptable, i32, vp, vp, i64, vp, i64, i64, vp, i64, i64, vp, prope, i32, vp, i64,
                                  i64, vp, vp, vp]
    lib.kda_kv_decode_workspace_bytes.argtypes = [pkv, i32, i32, i32, i64]
    lib.kda_kv_decode_workspace_bytes.restype = ctypes.c_size_t
    lib.kda_kv_decode.argtypes = [pkv, i32, ptable, i32, vp, vp, i64, i32, i32, vp, i64, i64, vp, f32, vp, vp, i32, f32,
                                  i64, vp, ctypes.c_size_t, vp, vp]
    lib.kda_kv_evict.argtypes = [pkv, ptable, i32, vp, vp, i32, vp, i32, vp, vp, vp]
    for name in ("kda_kv_cache_pages", "kda_rope_turns", "kda_rope_turns_of", "kda_rope_apply", "kda_kv_append",
                 "kda_kv_decode", "kda_kv_evict"):
        getattr(lib, name).restype = ctypes.c_int
    lib.kda_selftest_wait_timeout.argtypes = [i64, vp, vp]
    lib.kda_selftest_wait_timeout.restype = ctypes.c_int
    lib.kda_prefix_index_create.argtypes = [i32, i32, i32, i64]
    lib.kda_prefix_index_create.restype = vp
    lib.kda_prefix_index_destroy.argtypes = [vp]
    lib.kda_prefix_index_destroy.restype = None
    lib.kda_prefix_index_free_slots.argtypes = [vp]
    lib.kda_prefix_index_free_slots.restype = i32
    lib.kda_prefix_plan.argtypes = [vp, vp, i64, ctypes.POINTER(_PrefixPlan), vp, i32]
    lib.kda_prefix_plan.restype = ctypes.c_int
    lib.kda_prefix_commit.argtypes = [vp, ctypes.c_uint64]
    lib.kda_prefix_commit.restype = ctypes.c_int
    lib.kda_prefix_abort.argtypes = [vp, ctypes.c_uint64]
    lib.kda_prefix_abort.restype = ctypes.c_int
    lib.kda_prefix_release_slot.argtypes = [vp, i32]
    lib.kda_prefix_release_slot.restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libkda must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


@dataclass
class StatePool:
    """The state-slot pool: S [num_slots, H, dk, dv] fp32 or bf16, conv [num_slots, H, W-1, 2dk+dv] bf16."""
    S: torch.Tensor
    conv: torch.Tensor

    @staticmethod
    def empty(num_slots: int, H: int, dk: int, dv: int, W: int = 4, device="cuda",
              state_dtype=torch.float32) -> "StatePool":
        return StatePool(torch.zeros(num_slots, H, dk, dv, dtype=state_dtype, device=device),
                         torch.zeros(num_slots, H, W - 1, 2 * dk + dv, dtype=torch.bfloat16, device=device))

    @property
    def num_slots(self) -> int:
        return int(self.S.shape[0])

    def c(self) -> _Pool:
        ns, H, dk, dv = self.S.shape
        if self.S.dtype == torch.float32:
            sd = KDA_STATE_FP32
        elif self.S.dtype == torch.bfloat16:
            sd = KDA_STATE_BF16
        else:
            raise TypeError("state pool dtype must be float32 or bfloat16")
        return _Pool(H, dk, dv, self.conv.shape[2] + 1, sd, 0, ns, _ptr(self.S), _ptr(self.conv))


@dataclass
class LayerParams:
    """conv_weight [H, 2dk+dv, W] fp32, norm_weight [dv] fp32 and the layer's constants."""
    conv_weight: torch.Tensor
    norm_weight: torch.Tensor
    l2_eps: float = 1e-6
    rms_eps: float = 1e-6
    scale: float = 1.0
    conv_silu: bool = True

    def c(self) -> _Params:
        return _Params(_ptr(self.conv_weight), _ptr(self.norm_weight), self.l2_eps, self.rms_eps, self.scale,
                       int(bool(self.conv_silu)))


def kda_status_string(rc: int) -> str:
    return load_library().kda_status_string(int(rc)).decode()


def kda_checkpoint_count(start_pos: int, length: int, interval: int) -> int:
    return int(load_library().kda_checkpoint_count(int(start_pos), int(length), int(interval)))


def kda_prefill_workspace_bytes(pool: StatePool, nseq: int, total_tokens: int, chunk: int) -> int:
    pc = pool.c()
    return int(load_library().kda_prefill_workspace_bytes(ctypes.byref(pc), int(nseq), int(total_tokens), int(chunk)))


def kda_last_error_string() -> str:
    return load_library().kda_last_error_string().decode()


def _check(rc: int, what: str, detail: bool = True) -> None:
    if rc != KDA_OK:
        raise KdaError(rc, what, kda_last_error_string() if detail else "")


def _host_i32(x):
    import numpy as np
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        x = x.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(x, dtype=np.int32).reshape(-1))


def kda_check_slots(num_slots: int, src_slot, dst_slot, ckpt_slots=None) -> None:
    """Host check of one call's slot-aliasing contract (kda_check_slots in the C ABI); raises KdaError naming
    the first violation.  Arrays may be host or device tensors or sequences (device ones are copied)."""
    s, d, c = _host_i32(src_slot), _host_i32(dst_slot), _host_i32(ckpt_slots)
    if len(s) != len(d):
        raise ValueError("src_slot and dst_slot differ in length")
    vp = ctypes.c_void_p
    rc = load_library().kda_check_slots(int(num_slots), len(s), s.ctypes.data_as(vp), d.ctypes.data_as(vp),
                                        0 if c is None else len(c), None if c is None else c.ctypes.data_as(vp))
    _check(rc, "kda_check_slots")


def kda_selftest_wait_timeout(limit_ns: int, dev_status, stream=None) -> None:
    """Run the bounded-wait check: a wait that never completes gives up after limit_ns and sets
    KDA_DEV_TIMEOUT in dev_status (int32 [1] on the GPU)."""
    _check(load_library().kda_selftest_wait_timeout(int(limit_ns), _ptr(dev_status), _stream(stream)),
           "kda_selftest_wait_timeout")


# KDA_CHECK_SLOTS=1: every call checks its slot arrays on the host first (copies them from the device and
# synchronises; for debugging only).
_DEBUG_SLOTS = os.environ.get("KDA_CHECK_SLOTS", "0") not in ("", "0")


def kda_decode_step(pool: StatePool, params: LayerParams, q, k, v, a, b, z, y, src_slot, dst_slot, dev_status,
                    stream=None) -> None:
    """One fused decode token per request; see include/kda.h.  Tensors: q,k,a [n,H,dk] bf16, v,z,y
    [n,H,dv] bf16, b [n,H] bf16, src_slot/dst_slot [n] int32, dev_status [1] int32 (all on the GPU)."""
    n = int(src_slot.shape[0])
    if _DEBUG_SLOTS:
        kda_check_slots(pool.num_slots, src_slot, dst_slot)
    pc, pp = pool.c(), params.c()
    rc = load_library().kda_decode_step(ctypes.byref(pc), ctypes.byref(pp), n, _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                                        _ptr(b), _ptr(z), _ptr(y), _ptr(src_slot), _ptr(dst_slot),
                                        _ptr(dev_status), _stream(stream))
    _check(rc, "kda_decode_step")


def projection_width(H: int, dk: int, dv: int) -> int:
    """Rows of the packed projection weight: q, k, v, a, z and b."""
    return H * (3 * dk + 2 * dv) + H


def kda_project_inputs(x, w, H: int, dk: int, dv: int, q, k, v, a, b, z, dev_status, stream=None) -> None:
    """The six input projections in one GEMM (see include/kda.h): x [T, hidden] bf16, w [N, hidden] bf16 with
    the rows of q, k, v, a, z, b; outputs q, k, a [T, H, dk], v, z [T, H, dv], b [T, H] bf16 (z may be None)."""
    T, hidden = int(x.shape[0]), int(x.shape[1])
    rc = load_library().kda_project_inputs(T, hidden, int(H), int(dk), int(dv), _ptr(x), _ptr(w), _ptr(q), _ptr(k),
                                           _ptr(v), _ptr(a), _ptr(b), _ptr(z), _ptr(dev_status), _stream(stream))
    _check(rc, "kda_project_inputs")


DECODE_MULTI_MAX_L = 8  # KDA_DECODE_MULTI_MAX_L in kda.h


def kda_decode_multi(pool: StatePool, params: LayerParams, L: int, q, k, v, a, b, z, y, src_slot, dst_slots,
                     dev_status, stream=None) -> None:
    """L consecutive decode tokens per request with per-position state retention (speculative verification);
    see include/kda.h.  q,k,a [n*L,H,dk], v,z,y [n*L,H,dv], b [n*L,H] bf16 (row r*L+j = token j of request r);
    src_slot [n] int32; dst_slots [n*L] int32 (-1 = position not kept)."""
    n = int(src_slot.shape[0])
    if _DEBUG_SLOTS:
        kept = _host_i32(dst_slots)
        kda_check_slots(pool.num_slots, [], [], kept)
        src_h = _host_i32(src_slot)
        for r, s_ in enumerate(src_h):
            others = set(kept[:r * L].tolist()) | set(kept[(r + 1) * L:].tolist())
            if s_ >= 0 and int(s_) in others:
                raise KdaError(KDA_ERR_INVALID_ARG, "kda_decode_multi",
                               f"src_slot[{r}] = {s_} is kept by another request")
    pc, pp = pool.c(), params.c()
    rc = load_library().kda_decode_multi(ctypes.byref(pc), ctypes.byref(pp), n, int(L), _ptr(q), _ptr(k), _ptr(v),
                                         _ptr(a), _ptr(b), _ptr(z), _ptr(y), _ptr(src_slot), _ptr(dst_slots),
                                         _ptr(dev_status), _stream(stream))
    _check(rc, "kda_decode_multi")


def kda_prefill_chunked(pool: StatePool, params: LayerParams, cu_seqlens, start_pos, src_slot, dst_slot, chunk: int,
                        ckpt_interval: int, ckpt_offsets, ckpt_slots, q, k, v, a, b, z, y, workspace, dev_status,
                        stream=None) -> None:
    """Chunked prefill with checkpoint emission; see include/kda.h.  cu_seqlens/ckpt_offsets int32
    [nseq+1], start_pos int64 [nseq], slots int32, workspace a uint8 tensor of
    kda_prefill_workspace_bytes() bytes."""
    nseq = int(start_pos.shape[0])
    T = int(q.shape[0]) if q is not None else 0
    if _DEBUG_SLOTS:
        kda_check_slots(pool.num_slots, src_slot, dst_slot, ckpt_slots if ckpt_interval > 0 else None)
    pc, pp = pool.c(), params.c()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = load_library().kda_prefill_chunked(
        ctypes.byref(pc), ctypes.byref(pp), nseq, T, _ptr(cu_seqlens), _ptr(start_pos), _ptr(src_slot),
        _ptr(dst_slot), int(chunk), int(ckpt_interval), _ptr(ckpt_offsets), _ptr(ckpt_slots), _ptr(q), _ptr(k),
        _ptr(v), _ptr(a), _ptr(b), _ptr(z), _ptr(y), _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream))
    _check(rc, "kda_prefill_chunked")


# Size of the fixed scratch behind kda_prefill_chunked_noalloc (KDA_NOALLOC_SCRATCH_BYTES in kda.h).
NOALLOC_SCRATCH_BYTES = 64 << 20


def kda_prefill_chunked_noalloc(pool: StatePool, params: LayerParams, cu_seqlens, start_pos, src_slot, dst_slot,
                                chunk: int, ckpt_interval: int, ckpt_offsets, ckpt_slots, q, k, v, a, b, z, y,
                                dev_status, stream=None) -> None:
    """kda_prefill_chunked for callers that cannot allocate device memory: the workspace is the library's
    fixed scratch (NOALLOC_SCRATCH_BYTES per GPU).  Calls that overlap on the GPU race on that scratch;
    the first call on a device (nseq = 0 does only that set-up) should come at start-up, before any stream
    capture.  See include/kda.h."""
    nseq = int(start_pos.shape[0])
    T = int(q.shape[0]) if q is not None else 0
    if _DEBUG_SLOTS and nseq > 0:
        kda_check_slots(pool.num_slots, src_slot, dst_slot, ckpt_slots if ckpt_interval > 0 else None)
    pc, pp = pool.c(), params.c()
    rc = load_library().kda_prefill_chunked_noalloc(
        ctypes.byref(pc), ctypes.byref(pp), nseq, T, _ptr(cu_seqlens), _ptr(start_pos), _ptr(src_slot),
        _ptr(dst_slot), int(chunk), int(ckpt_interval), _ptr(ckpt_offsets), _ptr(ckpt_slots), _ptr(q), _ptr(k),
        _ptr(v), _ptr(a), _ptr(b), _ptr(z), _ptr(y), _ptr(dev_status), _stream(stream))
    _check(rc, "kda_prefill_chunked_noalloc")


def kda_resume_from_slot(pool: StatePool, src_slot, dst_slot, dev_status, stream=None) -> None:
    """Copy-on-write: slot dst_slot[i] receives a bit-exact copy of slot src_slot[i] (int32 [n])."""
    if _DEBUG_SLOTS:
        kda_check_slots(pool.num_slots, src_slot, dst_slot)
    pc = pool.c()
    rc = load_library().kda_resume_from_slot(ctypes.byref(pc), int(src_slot.shape[0]), _ptr(src_slot),
                                             _ptr(dst_slot), _ptr(dev_status), _stream(stream))
    _check(rc, "kda_resume_from_slot")


# ------------------------------------------------------------------------------------------ latent attention
_ELEM = {torch.bfloat16: KDA_ELEM_BF16, torch.float16: KDA_ELEM_FP16}


def _need(ok, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _raise(what: str):
    raise ValueError(what)


def _device_of(name: str, tensors) -> int:
    """The one CUDA device that the tensors (None among them skipped) live on."""
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if d < 0:
                    _raise(f"{name}: tensors must be on a CUDA device")
                if dev is not None:
                    _raise(f"{name}: tensors are on different devices")
                dev = d
    return dev


def _launch(fn, name: str, dev: int, stream, *args) -> None:
    """fn(*args, stream) on device `dev`, current or not, on its current stream unless one is given."""
    if stream is None:
        handle = _raw_stream(dev)
    elif stream.device.index == dev:
        handle = stream.cuda_stream
    else:
        _raise(f"{name}: the stream belongs to another device")
    if _get_device() == dev:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc:
        raise KdaError(rc, name, kda_last_error_string())


# Handle of a device's current stream, and the current device: torch.cuda's functions of these names make objects of them, at
# 1.0 and 0.25 us a call (0.1 both here); CUDA is running by then, because the call's tensors are on it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _int32(t, what: str, n: int | None = None):
    """The address of a contiguous int32 tensor of n elements (None for None)."""
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.dim() != 1 or (n is not None and t.shape[0] != n) or not t.is_contiguous():
        _raise(f"{what} must be a contiguous int32 vector" + ("" if n is None else f" of {n} elements"))
    return t.data_ptr()


def _rows_of(t, what: str, dtype, shape):
    """A tensor of that type and shape whose last axis is contiguous: its address and its other strides."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape:
        _raise(f"{what} must be a tensor of {dtype} and shape {tuple(shape)}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        _raise(f"{what}: the last axis must be contiguous")
    if 0 in shape or 1 in shape:  # the stride of an axis of one element is free in torch: give one that holds a row
        out, least = [], shape[-1]
        for k in range(len(shape) - 2, -1, -1):
            out.append(least if shape[k] <= 1 else st[k])
            least = max(least, out[-1] * shape[k])
        return (t.data_ptr(), *reversed(out))
    return (t.data_ptr(), *st[:-1])


def _out(t, what: str, dtype, shape):
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _raise(f"{what} must be a contiguous tensor of {dtype} and shape {tuple(shape)}")
    return t.data_ptr()


def _bytes(t):
    """Address and size of a workspace (0 for None)."""
    if t is None:
        return None, 0
    if not t.is_contiguous():
        _raise("the workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


@dataclass
class LatentCache:
    """Paged cache rows c | r of every layer: pages [layers, num_pages, page_size, rank + rope] bf16 or fp16.  The first
    two axes may be strided (a [num_pages, layers, ...] allocation transposed, for example)."""
    pages: torch.Tensor
    rank: int

    @staticmethod
    def empty(layers: int, num_pages: int, page_size: int, rank: int, rope: int, dtype=torch.bfloat16,
              device="cuda") -> "LatentCache":
        return LatentCache(torch.zeros(layers, num_pages, page_size, rank + rope, dtype=dtype, device=device), rank)

    @property
    def rope(self) -> int:
        return int(self.pages.shape[3]) - self.rank

    def c(self) -> _LatentCache:
        """The C struct of the pages as they are now (made again when anything that goes into it has changed)."""
        p = self.pages
        key = (p.data_ptr(), p.shape, p.stride(), p.dtype, self.rank)
        kept = self.__dict__.get("_kept")
        if kept is not None and kept[0] == key:
            return kept[1]
        if p.dtype not in _ELEM:
            raise TypeError("latent cache dtype must be bfloat16 or float16")
        layers, num, size, d = p.shape
        _need(p.stride(3) == 1 and (size == 1 or p.stride(2) == d), "latent cache: a page must be contiguous")
        c = _LatentCache(self.rank, d - self.rank, size, layers, _ELEM[p.dtype], 0, num, p.stride(0), p.stride(1),
                         ctypes.c_void_p(p.data_ptr()))
        self.__dict__["_kept"] = (key, c)
        return c


@dataclass
class PageTable:
    """table [max_seqs, max_pages], lens [max_seqs], refcount [num_pages], all int32, and the page size.  An empty
    pool has lens and refcount 0."""
    table: torch.Tensor
    lens: torch.Tensor
    refcount: torch.Tensor
    page_size: int

    @staticmethod
    def empty(max_seqs: int, max_pages: int, num_pages: int, page_size: int, device="cuda") -> "PageTable":
        i32 = dict(dtype=torch.int32, device=device)
        return PageTable(torch.full((max_seqs, max_pages), -1, **i32), torch.zeros(max_seqs, **i32),
                         torch.zeros(num_pages, **i32), page_size)

    def c(self) -> _PageTable:
        """The C struct of the tensors as they are now (made again when anything that goes into it has changed)."""
        t, n, r = self.table, self.lens, self.refcount
        key = (t.data_ptr(), t.shape, t.stride(), t.dtype, n.data_ptr(), n.shape, n.stride(), n.dtype, r.data_ptr(),
               r.shape, r.stride(), r.dtype, self.page_size)
        kept = self.__dict__.get("_kept")
        if kept is not None and kept[0] == key:
            return kept[1]
        _need(t.dtype == torch.int32 and t.dim() == 2 and t.is_contiguous(),
              "page table: table must be contiguous int32 [max_seqs, max_pages]")
        c = _PageTable(t.shape[0], t.shape[1], self.page_size, 0, r.shape[0], t.data_ptr(),
                       _int32(n, "page table: lens", int(t.shape[0])), _int32(r, "page table: refcount"))
        self.__dict__["_kept"] = (key, c)
        return c


def kda_latent_append(cache: LatentCache, layer: int, pt: PageTable, rows, cu_tokens, latent, rope, dev_status,
                      stream=None) -> None:
    """Cache rows of new tokens into one layer; see include/kda.h.  rows int32 [n] or None (row b for sequence b),
    cu_tokens int32 [n+1], latent [T, rank] and rope [T, rope] of the cache's type (rows may be strided; rope None
    when the cache has none).  The tokens become the last ones of their rows, which pt.lens already counts."""
    name = "kda_latent_append"
    dev = _device_of(name, (cache.pages, pt.table, pt.lens, rows, cu_tokens, latent, rope, dev_status))
    cc, dtype = cache.c(), cache.pages.dtype
    n, T = cu_tokens.shape[0] - 1, latent.shape[0]
    lp, ls = _rows_of(latent, "latent", dtype, (T, cc.rank))
    rp, rs = (None, 0) if cc.rope == 0 else _rows_of(rope, "rope", dtype, (T, cc.rope))
    _launch(load_library().kda_latent_append, name, dev, stream, cc, layer, pt.c(), n, _int32(rows, "rows", n),
            _int32(cu_tokens, "cu_tokens"), T, lp, ls, rp, rs, _int32(dev_status, "dev_status", 1))


def kda_latent_decode_workspace_bytes(cache: LatentCache, H: int, n: int, max_tokens: int) -> int:
    """Bytes of workspace kda_latent_decode needs on the cache's device (0 for unsupported sizes)."""
    with torch.cuda.device(cache.pages.device if cache.pages.is_cuda else -1):
        return int(load_library().kda_latent_decode_workspace_bytes(cache.c(), int(H), int(n), int(max_tokens)))


def kda_latent_decode(cache: LatentCache, layer: int, pt: PageTable, rows, cu_tokens, max_tokens: int, q, out, lse,
                      scale: float, workspace, dev_status, tree_mask=None, stream=None) -> None:
    """Absorbed latent attention of the newest tokens over the paged cache; see include/kda.h.  q [T, H, rank+rope]
    (token and head axes may be strided), out [T, H, rank], lse fp32 [T, H] or None; rows int32 [n] or None; cu_tokens int32
    [n+1], or None for max_tokens queries each of n = len(rows) (or all table rows); tree_mask int64 [T] (bit i: the query
    sees drafted token i of its sequence) or None; workspace uint8, kda_latent_decode_workspace_bytes() bytes."""
    name = "kda_latent_decode"
    dev = _device_of(name, (cache.pages, pt.table, pt.lens, rows, cu_tokens, q, out, lse, workspace, dev_status, tree_mask))
    cc, pc, dtype = cache.c(), pt.c(), cache.pages.dtype
    if q.dim() != 3:
        _raise("q must be [T, H, rank+rope]")
    T, H, d = q.shape
    n = (cu_tokens.shape[0] - 1 if cu_tokens is not None else rows.shape[0] if rows is not None else pc.max_seqs)
    if rows is None and n > pc.max_seqs:
        _raise(f"{name}: more sequences than table rows")
    qp, qt, qh = _rows_of(q, "q", dtype, (T, H, cc.rank + cc.rope))
    if tree_mask is not None and (tree_mask.dtype is not torch.int64 or tree_mask.shape != (T,)
                                  or not tree_mask.is_contiguous()):
        _raise(f"tree_mask must be a contiguous int64 vector of {T} elements")
    if out is None:
        _raise("out must be a tensor")
    ws, nbytes = _bytes(workspace)
    _launch(load_library().kda_latent_decode, name, dev, stream, cc, layer, pc, n, _int32(rows, "rows", n),
            _int32(cu_tokens, "cu_tokens", n + 1), T, max_tokens, H, qp, qt, qh,
            None if tree_mask is None else tree_mask.data_ptr(), scale, _out(out, "out", dtype, (T, H, cc.rank)),
            _out(lse, "lse", torch.float32, (T, H)), ws, nbytes, _int32(dev_status, "dev_status", 1))


def kda_latent_prefill(cu_q, cu_k, max_q: int, q, k_nope, k_rope, v, out, lse, scale: float, dev_status,
                       causal: bool = True, stream=None) -> None:
    """Expanded latent attention for prompts; see include/kda.h.  q [Tq, H, nope+rope], k_nope [Tk, H, nope],
    k_rope [Tk, rope], v [Tk, H, dv], one type, token and head axes may be strided (k_nope and v as halves of one
    tensor); out [Tq, H, dv], lse fp32 [Tq, H] or None; cu_q, cu_k int32 [nseq+1]."""
    name = "kda_latent_prefill"
    dev = _device_of(name, (cu_q, cu_k, q, k_nope, k_rope, v, out, lse, dev_status))
    dtype = q.dtype
    if dtype not in _ELEM:
        _raise("q must be bfloat16 or float16")
    if q.dim() != 3 or k_nope.dim() != 3 or k_rope.dim() != 2 or v.dim() != 3:
        _raise("q, k_nope and v must have three axes, k_rope two")
    n = cu_q.shape[0] - 1
    Tq, H, dq = q.shape
    Tk, _, nope = k_nope.shape
    rope, dv = k_rope.shape[1], v.shape[2]
    if dq != nope + rope:
        _raise("q's last axis must be that of k_nope and k_rope together")
    if out is None:
        _raise("out must be a tensor")
    _launch(load_library().kda_latent_prefill, name, dev, stream, _ELEM[dtype], H, nope, rope, dv, n,
            _int32(cu_q, "cu_q"), _int32(cu_k, "cu_k", n + 1), Tq, Tk, max_q, bool(causal),
            *_rows_of(q, "q", dtype, (Tq, H, dq)), *_rows_of(k_nope, "k_nope", dtype, (Tk, H, nope)),
            *_rows_of(k_rope, "k_rope", dtype, (Tk, rope)), *_rows_of(v, "v", dtype, (Tk, H, dv)), scale,
            _out(out, "out", dtype, (Tq, H, dv)), _out(lse, "lse", torch.float32, (Tq, H)),
            _int32(dev_status, "dev_status", 1))


def kda_pages_workspace_bytes(pt: PageTable, n: int) -> int:
    """Bytes of workspace a kda_pages_* call of n items needs."""
    return int(load_library().kda_pages_workspace_bytes(pt.c(), int(n)))


def _pages_call(name: str, pt: PageTable, cache, arrays, workspace, dev_status, stream) -> None:
    dev = _device_of(name, (pt.table, pt.lens, pt.refcount, workspace, dev_status, *arrays)
                     + ((cache.pages,) if cache is not None else ()))
    args = [pt.c()] if cache is None else [pt.c(), cache.c()]
    if arrays:
        n = arrays[0].shape[0]
        args += [n, _int32(arrays[0], f"{name}: items"), _int32(arrays[1], f"{name}: items", n)]
    _launch(getattr(load_library(), name), name, dev, stream, *args, *_bytes(workspace),
            _int32(dev_status, "dev_status", 1))


def kda_pages_reserve(pt: PageTable, cache: LatentCache, rows, new_lens, workspace, dev_status, stream=None) -> None:
    """Rows grow to new_lens tokens: pages from the lowest free ones, a shared partly filled last page copied first
    (rows, new_lens int32 [n]; row -1 = padding).  See include/kda.h."""
    _pages_call("kda_pages_reserve", pt, cache, (rows, new_lens), workspace, dev_status, stream)


def kda_pages_truncate(pt: PageTable, rows, keep_lens, workspace, dev_status, stream=None) -> None:
    """Rows keep their first keep_lens tokens (0 ends them); pages behind lose a reference.  See include/kda.h."""
    _pages_call("kda_pages_truncate", pt, None, (rows, keep_lens), workspace, dev_status, stream)


def kda_pages_fork(pt: PageTable, cache: LatentCache, parents, children, workspace, dev_status, stream=None) -> None:
    """The empty rows children become copies of rows parents: full pages shared, a partly filled last one copied (-1 as
    parent or child: padding, which names no row)."""
    _pages_call("kda_pages_fork", pt, cache, (parents, children), workspace, dev_status, stream)


def kda_pages_compact(pt: PageTable, cache: LatentCache, workspace, dev_status, stream=None) -> None:
    """Moves the used pages into the lowest places; tables and refcounts follow.  See include/kda.h."""
    _pages_call("kda_pages_compact", pt, cache, (), workspace, dev_status, stream)


def kda_pages_copy(cache: LatentCache, src, dst, dev_status, stream=None) -> None:
    """Contents of pages src into pages dst in every layer (int32 [n]; -1 = skip), no bookkeeping."""
    name = "kda_pages_copy"
    dev, n = _device_of(name, (cache.pages, src, dst, dev_status)), src.shape[0]
    _launch(load_library().kda_pages_copy, name, dev, stream, cache.c(), n, _int32(src, "src"), _int32(dst, "dst", n),
            _int32(dev_status, "dev_status", 1))


# ------------------------------------------------------------------------------- grouped-query attention, rotary positions
@dataclass
class KvCache:
    """Pages of keys and values of every layer: data [layers, num_pages, words] bf16 or fp16, a page of page_size tokens
    holding keys [heads, page_size, head_dim], values of the same shape and, with stats, fp32 sums of attention weights
    and int32 positions [heads, 2, page_size].  The first two axes of data may be strided.  The kda_pages_* calls take a
    KvCache as they take a :class:`LatentCache`."""
    data: torch.Tensor
    heads: int
    head_dim: int
    page_size: int
    stats: bool = False

    @staticmethod
    def words(page_size: int, heads: int, head_dim: int, stats: bool = False) -> int:
        """16-bit words of a page."""
        return page_size * heads * (2 * head_dim + (4 if stats else 0))

    @staticmethod
    def empty(layers: int, num_pages: int, page_size: int, heads: int, head_dim: int, stats: bool = False,
              dtype=torch.bfloat16, device="cuda") -> "KvCache":
        return KvCache(torch.zeros(layers, num_pages, KvCache.words(page_size, heads, head_dim, stats), dtype=dtype,
                                   device=device), heads, head_dim, page_size, stats)

    def _rows(self, part: int) -> torch.Tensor:
        size = self.heads * self.page_size * self.head_dim
        return self.data[..., part * size:(part + 1) * size].unflatten(-1, (self.heads, self.page_size, self.head_dim))

    @property
    def keys(self) -> torch.Tensor:
        """View [layers, num_pages, heads, page_size, head_dim]."""
        return self._rows(0)

    @property
    def values(self) -> torch.Tensor:
        """View [layers, num_pages, heads, page_size, head_dim]."""
        return self._rows(1)

    def _stats(self, part: int, dtype) -> torch.Tensor:
        _need(self.stats, "kv cache: it has no stats")
        at = self.heads * self.page_size * self.head_dim
        return self.data.view(dtype)[..., at:].unflatten(-1, (self.heads, 2, self.page_size))[..., part, :]

    @property
    def weights(self) -> torch.Tensor:
        """View [layers, num_pages, heads, page_size] fp32: each token's accumulated attention weight."""
        return self._stats(0, torch.float32)

    @property
    def positions(self) -> torch.Tensor:
        """View [layers, num_pages, heads, page_size] int32."""
        return self._stats(1, torch.int32)

    def _key(self):
        p = self.data
        return (p.data_ptr(), p.shape, p.stride(), p.dtype, self.heads, self.head_dim, self.page_size, self.stats)

    def kv(self) -> _KvCache:
        """The C struct of the pages as they are now (made again when anything that goes into it has changed)."""
        key, kept = self._key(), self.__dict__.get("_kept")
        if kept is not None and kept[0] == key:
            return kept[1]
        p = self.data
        if p.dtype not in _ELEM:
            raise TypeError("kv cache dtype must be bfloat16 or float16")
        _need(p.dim() == 3 and p.shape[2] == self.words(self.page_size, self.heads, self.head_dim, self.stats)
              and p.stride(2) == 1, "kv cache: data must be [layers, num_pages, words of a page], a page contiguous")
        c = _KvCache(self.heads, self.head_dim, self.page_size, p.shape[0], _ELEM[p.dtype], int(bool(self.stats)),
                     p.shape[1], p.stride(0), p.stride(1), ctypes.c_void_p(p.data_ptr()))
        self.__dict__["_kept"] = (key, c)
        return c

    def c(self) -> _LatentCache:
        """The C struct that the kda_pages_* calls take."""
        key, kept = self._key(), self.__dict__.get("_kept_pages")
        if kept is not None and kept[0] == key:
            return kept[1]
        c = _LatentCache()
        _check(load_library().kda_kv_cache_pages(self.kv(), c), "kda_kv_cache_pages")
        self.__dict__["_kept_pages"] = (key, c)
        return c

    @property
    def pages(self) -> torch.Tensor:
        return self.data


_SCALING = {"none": KDA_ROPE_PLAIN, "linear": KDA_ROPE_LINEAR, "ntk": KDA_ROPE_NTK, "parts": KDA_ROPE_PARTS}


@dataclass
class Rope:
    """Rotary positions of the channels offset .. offset + dim - 1 of a head: turns int64 [dim / 2] on the GPU (the bits
    of kda_rope.turns), pairs as halves or interleaved, rotated values times scale."""
    turns: torch.Tensor
    offset: int = 0
    interleaved: bool = False
    scale: float = 1.0

    @staticmethod
    def make(dim: int, base: float = 10000.0, offset: int = 0, interleaved: bool = False, scaling: str = "none",
             factor: float = 1.0, original: float = 0.0, low: float = 1.0, high: float = 32.0, scale: float = 1.0,
             device="cuda") -> "Rope":
        """theta_i = base^(-2i / dim), changed for long contexts as enum kda_rope_scaling in kda.h says: "none", "linear",
        "ntk" or "parts" (by `low` and `high` turns within the `original` length; for a ramp over the pairs' indices
        give the frequencies to :meth:`of`)."""
        if scaling not in _SCALING:
            _raise(f"scaling must be one of {', '.join(_SCALING)}")
        turns = torch.empty(max(dim // 2, 0), dtype=torch.int64)
        _check(load_library().kda_rope_turns(dim, base, _SCALING[scaling], factor, original, low, high, turns.data_ptr()),
               "kda_rope_turns")
        return Rope(turns.to(device), offset, interleaved, scale)

    @staticmethod
    def of(theta, offset: int = 0, interleaved: bool = False, scale: float = 1.0, device="cuda") -> "Rope":
        """Of dim / 2 frequencies in radians a position, given one by one."""
        theta = torch.as_tensor(theta, dtype=torch.float64, device="cpu").contiguous()
        turns = torch.empty(theta.shape, dtype=torch.int64)
        _check(load_library().kda_rope_turns_of(theta.numel(), theta.data_ptr(), turns.data_ptr()), "kda_rope_turns_of")
        return Rope(turns.to(device), offset, interleaved, scale)

    def c(self) -> _Rope:
        """The C struct of the tensor as it is now (made again when anything that goes into it has changed)."""
        t = self.turns
        key = (t.data_ptr(), t.shape, t.stride(), t.dtype, self.offset, self.interleaved, self.scale)
        kept = self.__dict__.get("_kept")
        if kept is not None and kept[0] == key:
            return kept[1]
        _need(t.dtype == torch.int64 and t.dim() == 1 and t.is_contiguous(),
              "rope: turns must be a contiguous int64 vector")
        c = _Rope(2 * t.shape[0], self.offset, int(bool(self.interleaved)), self.scale, ctypes.c_void_p(t.data_ptr()))
        self.__dict__["_kept"] = (key, c)
        return c


def kda_rope_apply(rope: Rope, x, positions, out, inverse: bool = False, stream=None) -> None:
    """x [T, H, D] with the channels that rope names rotated by positions (int32 [T]) into out; see include/kda.h.  Token and
    head axes may be strided; out may be x.  inverse: by minus the angle, the gradient of the rotation."""
    name = "kda_rope_apply"
    dev = _device_of(name, (rope.turns, x, positions, out))
    if x.dtype not in _ELEM:
        _raise("x must be bfloat16 or float16")
    if x.dim() != 3:
        _raise("x must be [T, H, D]")
    T, H, D = x.shape
    _launch(load_library().kda_rope_apply, name, dev, stream, rope.c(), _ELEM[x.dtype], T, H, D,
            _int32(positions, "positions", T), bool(inverse), *_rows_of(x, "x", x.dtype, x.shape),
            *_rows_of(out, "out", x.dtype, x.shape))


def kda_kv_append(cache: KvCache, layer: int, pt: PageTable, rows, cu_tokens, k, v, positions, dev_status,
                  rope: Rope | None = None, q=None, q_out=None, stream=None) -> None:
    """Keys and values of new tokens into one layer's pages; see include/kda.h.  rows int32 [n] or None (row b for
    sequence b), cu_tokens int32 [n+1], k and v [T, heads, head_dim] and q [T, H, head_dim] of the cache's type (token and
    head axes may be strided), positions int32 [T].  rope rotates the keys on their way and, into q_out [T, H, head_dim],
    the queries.  The tokens become the last ones of their rows, which pt.lens already counts."""
    name = "kda_kv_append"
    dev = _device_of(name, (cache.data, pt.table, pt.lens, rows, cu_tokens, k, v, positions, dev_status, q, q_out,
                            None if rope is None else rope.turns))
    cc, dtype = cache.kv(), cache.data.dtype
    n, T = cu_tokens.shape[0] - 1, k.shape[0]
    shape = (T, cc.heads, cc.head_dim)
    H, qa, qo = 0, (None, 0, 0), None
    if q is not None:
        if q.dim() != 3 or q_out is None:
            _raise("q must be [T, H, head_dim], and q_out given")
        H = q.shape[1]
        qa = _rows_of(q, "q", dtype, (T, H, cc.head_dim))
        qo = _out(q_out, "q_out", dtype, (T, H, cc.head_dim))
    _launch(load_library().kda_kv_append, name, dev, stream, cc, layer, pt.c(), n, _int32(rows, "rows", n),
            _int32(cu_tokens, "cu_tokens"), T, *_rows_of(k, "k", dtype, shape), *_rows_of(v, "v", dtype, shape),
            _int32(positions, "positions", T), None if rope is None else rope.c(), H, *qa, qo,
            _int32(dev_status, "dev_status", 1))


def kda_kv_decode_workspace_bytes(cache: KvCache, H: int, n: int, max_tokens: int, max_slots: int = 0) -> int:
    """Bytes of workspace kda_kv_decode needs on the cache's device (0 for unsupported sizes); max_slots: a bound on the sum
    of the call's lens, 1 or more, where weights are added up, else 0."""
    with torch.cuda.device(cache.data.device if cache.data.is_cuda else -1):
        return int(load_library().kda_kv_decode_workspace_bytes(cache.kv(), int(H), int(n), int(max_tokens),
                                                                int(max_slots)))


def kda_kv_decode(cache: KvCache, layer: int, pt: PageTable, rows, cu_tokens, max_tokens: int, q, out, lse, scale: float,
                  workspace, dev_status, tree_mask=None, weight_decay: float | None = None, max_slots: int | None = None,
                  stream=None) -> None:
    """Grouped-query attention of the newest tokens over the paged cache; see include/kda.h.  q [T, H, head_dim] (token and
    head axes may be strided), out [T, H, head_dim], lse fp32 [T, H] or None; rows, cu_tokens, tree_mask as for
    kda_latent_decode.  weight_decay: not None adds the call's weights to the cache's sums, after multiplying these
    with it; max_slots, 1 or more, then bounds the sum of the call's lens.  None stands for the pool's pages full once, which
    lens pass where sequences share many pages: sequences past the bound are flagged and keep their old sums, so such a program
    gives a bound of its own (and one with a large pool a closer one, as the workspace grows with it).  workspace uint8,
    kda_kv_decode_workspace_bytes() bytes for the same max_slots."""
    name = "kda_kv_decode"
    adds = weight_decay is not None
    dev = _device_of(name, (cache.data, pt.table, pt.lens, pt.refcount if adds else None, rows, cu_tokens, q, out, lse,
                            workspace, dev_status, tree_mask))
    cc, pc, dtype = cache.kv(), pt.c(), cache.data.dtype
    if q.dim() != 3:
        _raise("q must be [T, H, head_dim]")
    T, H, d = q.shape
    n = (cu_tokens.shape[0] - 1 if cu_tokens is not None else rows.shape[0] if rows is not None else pc.max_seqs)
    if rows is None and n > pc.max_seqs:
        _raise(f"{name}: more sequences than table rows")
    qp, qt, qh = _rows_of(q, "q", dtype, (T, H, cc.head_dim))
    if tree_mask is not None and (tree_mask.dtype is not torch.int64 or tree_mask.shape != (T,)
                                  or not tree_mask.is_contiguous()):
        _raise(f"tree_mask must be a contiguous int64 vector of {T} elements")
    if out is None:
        _raise("out must be a tensor")
    if max_slots is None:
        max_slots = cc.num_pages * cc.page_size if adds else 0
    ws, nbytes = _bytes(workspace)
    _launch(load_library().kda_kv_decode, name, dev, stream, cc, layer, pc, n, _int32(rows, "rows", n),
            _int32(cu_tokens, "cu_tokens", n + 1), T, max_tokens, H, qp, qt, qh,
            None if tree_mask is None else tree_mask.data_ptr(), scale, _out(out, "out", dtype, (T, H, d)),
            _out(lse, "lse", torch.float32, (T, H)), adds, weight_decay if adds else 1.0, max_slots, ws, nbytes,
            _int32(dev_status, "dev_status", 1))


def kda_kv_evict(cache: KvCache, pt: PageTable, rows, keep, new_lens, dev_status, first: int = 0, since=None,
                 max_len: int = 0, stream=None) -> None:
    """Each layer and head keeps keep[i] tokens of row rows[i], those with the largest sums, in the row's first slots; see
    include/kda.h.  rows, keep, new_lens, since int32 [n] (rows and since may be None), max_len a bound on the rows' lens (0:
    what the table has room for; a close one is faster); kda_pages_truncate(pt, rows, new_lens, ...) then gives the pages
    behind back."""
    name = "kda_kv_evict"
    dev = _device_of(name, (cache.data, pt.table, pt.lens, pt.refcount, rows, keep, new_lens, since, dev_status))
    n, pc = keep.shape[0], pt.c()
    if rows is None and n > pc.max_seqs:
        _raise(f"{name}: more sequences than table rows")
    _launch(load_library().kda_kv_evict, name, dev, stream, cache.kv(), pc, n, _int32(rows, "rows", n),
            _int32(keep, "keep"), first, _int32(since, "since", n), max_len, _int32(new_lens, "new_lens", n),
            _int32(dev_status, "dev_status", 1))


@dataclass
class PrefixPlan:
    """What one prompt needs: resume from ``src_slot`` (or start fresh when it is -1) into ``private_slot``,
    prefill tokens [start_pos, len) with checkpoint interval = the match unit and the ``ckpt_slots`` table
    (one entry per match-unit boundary in (start_pos, len]: a pool slot, or -1 to skip)."""
    plan_id: int
    src_slot: int
    private_slot: int
    start_pos: int
    ckpt_slots: list


class PrefixIndex:
    """Host prefix index over a state pool (``kda_prefix_index_*`` in the C ABI): chained match-unit hashes
    to checkpoint slots, copy-on-write private slots, LRU eviction, interval or second-hit retention."""

    def __init__(self, num_slots: int, match_unit: int = 128, policy: int = KDA_RETAIN_INTERVAL,
                 interval: int = 0):
        self._lib = load_library()
        self._h = self._lib.kda_prefix_index_create(int(num_slots), int(match_unit), int(policy), int(interval))
        if not self._h:
            raise KdaError(KDA_ERR_INVALID_ARG, "kda_prefix_index_create")
        self.match_unit = int(match_unit)

    def close(self) -> None:
        if self._h:
            self._lib.kda_prefix_index_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def free_slots(self) -> int:
        return int(self._lib.kda_prefix_index_free_slots(self._h))

    def plan(self, tokens) -> PrefixPlan:
        import numpy as np
        t = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
        cap = max(1, len(t) // self.match_unit)
        ck = np.empty(cap, dtype=np.int32)
        out = _PrefixPlan()
        rc = self._lib.kda_prefix_plan(self._h, t.ctypes.data_as(ctypes.c_void_p), len(t), ctypes.byref(out),
                                       ck.ctypes.data_as(ctypes.c_void_p), cap)
        _check(rc, "kda_prefix_plan", detail=False)
        return PrefixPlan(int(out.plan_id), int(out.src_slot), int(out.private_slot), int(out.start_pos),
                          [int(x) for x in ck[:out.num_ckpts]])

    def commit(self, plan: PrefixPlan) -> None:
        _check(self._lib.kda_prefix_commit(self._h, plan.plan_id), "kda_prefix_commit", detail=False)

    def abort(self, plan: PrefixPlan) -> None:
        _check(self._lib.kda_prefix_abort(self._h, plan.plan_id), "kda_prefix_abort", detail=False)

    def release_slot(self, slot: int) -> None:
        _check(self._lib.kda_prefix_release_slot(self._h, int(slot)), "kda_prefix_release_slot", detail=False)
