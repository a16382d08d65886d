"""ctypes binding of libdak.so: argument marshalling only, every step runs in the library.

Names match the C ABI in include/dak.h. Tensors are torch tensors (device memory and
streams come from PyTorch); host-side sources may also be numpy arrays of bf16 bits.
A missing library raises at import time: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdak.so")

DAK_OK = 0
STATUS_NAMES = {
    0: "DAK_OK", 1: "DAK_ERR_INVALID", 2: "DAK_ERR_ALIGN", 3: "DAK_ERR_HOST_ALLOC",
    4: "DAK_ERR_DEVICE_ALLOC", 5: "DAK_ERR_CUDA", 6: "DAK_ERR_TIMEOUT", 7: "DAK_ERR_UNSUPPORTED",
    8: "DAK_ERR_BOUNDS",
}

# every symbol include/dak.h declares
EXPORTS = [
    "dak_status_string", "dak_place_matrix", "dak_place_kv", "dak_free", "dak_placement_info",
    "dak_gemm", "dak_attn_workspace_bytes", "dak_attn", "dak_attn_default_split", "dak_plan_ratios",
    "dak_last_error", "dak_sm_count", "dak_probe_read_bw", "dak_probe_concurrent", "dak_prefetch",
    "dak_gemm_staged", "dak_attn_staged", "dak_attn_noalloc", "dak_selftest_wait",
    "dak_decoder_create", "dak_decoder_batch", "dak_decoder_step", "dak_decoder_capture",
    "dak_decoder_replay", "dak_decoder_launches", "dak_decoder_free", "dak_tune_gemm", "dak_tune_attn",
    "dak_place_matrix_glu", "dak_plan_units", "dak_gemm_workspace_bytes", "dak_gemm_ws", "dak_gemm_plan", "dak_gemm_launch_plan",
    "dak_attn_f32", "dak_inject_fault", "dak_fault_pending", "dak_alloc_counts", "dak_gemm_chain",
    "dak_gemm_chain_workspace_bytes", "dak_link_begin", "dak_link_timeouts", "dak_selftest_link",
    "dak_place_kv_heads", "dak_kv_append", "dak_gemm_chain_plan", "dak_placement_data", "dak_rope_make",
    "dak_rope_from_freqs", "dak_kv_append_rope", "dak_kv_append_rope_acc", "dak_kv_evict_workspace_bytes", "dak_kv_evict",
    "dak_attn_acc_workspace_bytes", "dak_attn_acc", "dak_attn_prefix_workspace_bytes", "dak_attn_prefix",
    "dak_rope_axes_make", "dak_kv_append_rope_axes", "dak_attn_tree_workspace_bytes", "dak_attn_tree", "dak_kv_commit",
    "dak_kv_fork",
]

# position scalings of dak_rope_make (DAK_ROPE_* in dak.h)
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}

# host-side fault injection kinds (DAK_FAULT_* in dak.h)
FAULT_HOST_ALLOC, FAULT_DEVICE_ALLOC, FAULT_TENSOR_MAP = 1, 2, 3

# size of the fixed device array dak_attn_noalloc uses (DAK_NOALLOC_SCRATCH_BYTES in dak.h)
NOALLOC_SCRATCH_BYTES = 4 << 20


class DakError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class dak_tuning(ctypes.Structure):
    _fields_ = [("host_ctas", ctypes.c_int), ("window", ctypes.c_int), ("hbm_window", ctypes.c_int),
                ("chunk_k", ctypes.c_int), ("n_split", ctypes.c_int), ("hbm_ctas", ctypes.c_int),
                ("split_k", ctypes.c_int), ("pdl", ctypes.c_int), ("ctas_per_sm", ctypes.c_int),
                ("no_wave_align", ctypes.c_int), ("column_blocks", ctypes.c_int), ("cluster_slots", ctypes.c_int),
                ("link", ctypes.c_int), ("chain_rr", ctypes.c_int)]


class dak_gemm_op(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("C", ctypes.c_void_p), ("c_fp32", ctypes.c_int),
                ("after_prev", ctypes.c_int)]


class dak_op(ctypes.Structure):
    _fields_ = [("bytes", ctypes.c_double), ("t_comp", ctypes.c_double), ("tile_bytes", ctypes.c_double)]


class dak_tune_result(ctypes.Structure):
    _fields_ = [("best", dak_tuning), ("best_us", ctypes.c_double), ("default_us", ctypes.c_double),
                ("cc_off_us", ctypes.c_double), ("no_align_us", ctypes.c_double), ("candidates", ctypes.c_int)]


class dak_gemm_chain_plan_info(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("grid", "units", "by_size", "busiest_per_op", "busiest_by_size")]


class dak_gemm_plan_info(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in (
        "tensor_cores", "launches", "cluster", "n_pad", "pieces", "piece_step", "chunk_k", "host_chunk_k",
        "hbm_stages", "host_stages", "host_ctas", "hbm_ctas", "host_window", "hbm_window", "smem_bytes",
        "tile_m", "cluster_slots")]


class dak_rope_config(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("scaling", ctypes.c_int),
                ("theta", ctypes.c_double), ("factor", ctypes.c_double), ("orig_len", ctypes.c_double),
                ("low_turns", ctypes.c_double), ("high_turns", ctypes.c_double), ("attn_scale", ctypes.c_double)]


class dak_rope_plan(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int), ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("scale", ctypes.c_float), ("turns", ctypes.c_uint64 * 64)]


class dak_rope_axes_plan(ctypes.Structure):
    _fields_ = [("rope", dak_rope_plan), ("n_axes", ctypes.c_int), ("axis", ctypes.c_ubyte * 64)]


class dak_decoder_config(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("hidden", ctypes.c_int), ("n_heads", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("ffn", ctypes.c_int),
                ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float), ("plain_launch", ctypes.c_int),
                ("op_tuning", dak_tuning * 5), ("no_link_handoff", ctypes.c_int)]


class dak_decoder_layer(ctypes.Structure):
    _fields_ = [("qkv", ctypes.c_void_p), ("o", ctypes.c_void_p), ("gate_up", ctypes.c_void_p),
                ("down", ctypes.c_void_p), ("kv", ctypes.c_void_p), ("attn_norm", ctypes.c_void_p),
                ("mlp_norm", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built (run __graft_entry__.build()); "
                          "the direct-access path has no fallback")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, dbl, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double, ctypes.c_size_t
    P = ctypes.POINTER
    sig = {
        "dak_status_string": (ctypes.c_char_p, [i32]),
        "dak_place_matrix": (i32, [vp, i32, i64, i64, i64, i32, i32, P(vp)]),
        "dak_place_kv": (i32, [vp, vp, i32, i32, i32, i32, i32, i32, P(vp)]),
        "dak_place_kv_heads": (i32, [vp, vp, i32, i32, i32, i32, i32, i32, P(vp)]),
        "dak_kv_append": (i32, [vp, vp, vp, vp, vp]),
        "dak_place_matrix_glu": (i32, [vp, i32, i64, i64, i64, i32, i32, P(vp)]),
        "dak_free": (i32, [vp]),
        "dak_placement_info": (i32, [vp, P(i64), P(i64), P(i64), P(i64)]),
        "dak_gemm": (i32, [vp, vp, vp, i32, i32, P(dak_tuning), vp]),
        "dak_gemm_staged": (i32, [vp, vp, vp, vp, i32, i32, P(dak_tuning), vp]),
        "dak_gemm_workspace_bytes": (sz, [vp, i32]),
        "dak_gemm_ws": (i32, [vp, vp, vp, i32, i32, P(dak_tuning), vp, sz, vp]),
        "dak_gemm_plan": (i32, [i64, i64, i32, i32, i32, i32, P(dak_tuning), sz, P(dak_gemm_plan_info)]),
        "dak_gemm_launch_plan": (i32, [vp, i32, P(dak_tuning), sz, P(dak_gemm_plan_info)]),
        "dak_gemm_chain_workspace_bytes": (sz, [P(dak_gemm_op), i32, i32, P(dak_tuning)]),
        "dak_gemm_chain": (i32, [P(dak_gemm_op), i32, i32, P(dak_tuning), vp, sz, vp]),
        "dak_gemm_chain_plan": (i32, [P(i64), P(i64), P(i32), P(i32), P(i32), i32, i32, i32, P(dak_tuning),
                                      P(dak_gemm_chain_plan_info)]),
        "dak_attn_workspace_bytes": (sz, [i32, i32, i32, i32]),
        "dak_attn": (i32, [vp, vp, vp, i32, ctypes.c_float, vp, vp, sz, P(dak_tuning), vp]),
        "dak_attn_staged": (i32, [vp, vp, vp, vp, i32, ctypes.c_float, vp, vp, sz, P(dak_tuning), vp]),
        "dak_attn_f32": (i32, [vp, vp, vp, i32, ctypes.c_float, vp, vp, sz, P(dak_tuning), vp]),
        "dak_attn_default_split": (i32, [vp]),
        "dak_placement_data": (i32, [vp, P(vp), P(vp)]),
        "dak_rope_make": (i32, [i32, P(dak_rope_config), P(dak_rope_plan)]),
        "dak_rope_from_freqs": (i32, [i32, P(dbl), i32, i32, dbl, P(dak_rope_plan)]),
        "dak_kv_append_rope": (i32, [vp, P(dak_rope_plan), vp, vp, vp, i32, i32, i32, i64, i64, i64, vp, vp, vp, vp,
                                     vp, vp]),
        "dak_kv_append_rope_acc": (i32, [vp, P(dak_rope_plan), vp, vp, vp, i32, i32, i32, i64, i64, i64, vp, vp, vp, vp,
                                         vp, vp, vp]),
        "dak_kv_evict_workspace_bytes": (sz, [vp]),
        "dak_kv_evict": (i32, [vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "dak_attn_acc_workspace_bytes": (sz, [vp, i32, i32]),
        "dak_attn_acc": (i32, [vp, vp, vp, i32, ctypes.c_float, vp, i32, vp, vp, vp, sz, P(dak_tuning), vp]),
        "dak_attn_prefix_workspace_bytes": (sz, [vp, vp, i32, i32, i32]),
        "dak_attn_prefix": (i32, [vp, vp, vp, vp, vp, vp, i32, ctypes.c_float, vp, i32, vp, vp, vp, sz, P(dak_tuning),
                                  vp]),
        "dak_rope_axes_make": (i32, [P(dak_rope_plan), i32, P(i32), P(dak_rope_axes_plan)]),
        "dak_kv_append_rope_axes": (i32, [vp, P(dak_rope_axes_plan), vp, vp, vp, i32, i32, i32, i64, i64, i64, vp, vp, vp,
                                          vp, vp, vp, vp]),
        "dak_attn_tree_workspace_bytes": (sz, [vp, i32, i32]),
        "dak_attn_tree": (i32, [vp, vp, vp, i32, vp, i64, vp, i32, ctypes.c_float, vp, i32, vp, sz, P(dak_tuning), vp]),
        "dak_kv_commit": (i32, [vp, vp, i32, vp, vp, i32, vp, vp, vp, vp, vp]),
        "dak_kv_fork": (i32, [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "dak_plan_ratios": (i32, [P(dak_op), i32, dbl, dbl, dbl, i32, P(dbl), P(dbl)]),
        "dak_plan_units": (i32, [P(dak_op), i32, dbl, dbl, dbl, P(i64), P(dbl)]),
        "dak_last_error": (i32, [vp, P(ctypes.c_uint64)]),
        "dak_sm_count": (i32, []),
        "dak_probe_read_bw": (i32, [i32, i64, i32, i32, i32, i32, i32, P(dbl), P(i32)]),
        "dak_probe_concurrent": (i32, [i64, i64, i32, i32, i32, i32, i32, i32, P(dbl), P(dbl)]),
        "dak_prefetch": (i32, [vp, vp, vp]),
        "dak_link_begin": (i32, [i32, vp]),
        "dak_link_timeouts": (i32, [vp, P(ctypes.c_uint32)]),
        "dak_selftest_link": (i32, [vp]),
        "dak_attn_noalloc": (i32, [vp, vp, vp, i32, ctypes.c_float, vp, P(dak_tuning), vp]),
        "dak_selftest_wait": (i32, [vp]),
        "dak_inject_fault": (i32, [i32, i32, i32]),
        "dak_fault_pending": (i32, [i32]),
        "dak_alloc_counts": (i32, [P(i64), P(i64)]),
        "dak_decoder_create": (i32, [P(dak_decoder_config), P(dak_decoder_layer), vp, P(vp)]),
        "dak_decoder_batch": (i32, [vp]),
        "dak_decoder_step": (i32, [vp, vp, vp, vp, i32, vp]),
        "dak_decoder_capture": (i32, [vp, vp, vp, vp, i32]),
        "dak_decoder_replay": (i32, [vp, vp]),
        "dak_decoder_launches": (i32, [vp, i32]),
        "dak_decoder_free": (i32, [vp]),
        "dak_tune_gemm": (i32, [vp, vp, vp, i32, i32, i32, P(dak_tuning), P(dak_tune_result)]),
        "dak_tune_attn": (i32, [vp, vp, vp, i32, vp, vp, sz, i32, P(dak_tuning), P(dak_tune_result)]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()


def _check(status: int, where: str):
    if status != DAK_OK:
        raise DakError(status, where)


def _stream_ptr(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _tuning(t):
    if t is None:
        return None
    if isinstance(t, dak_tuning):
        return ctypes.byref(t)
    tt = dak_tuning(**{k: int(v) for k, v in dict(t).items()})
    return ctypes.byref(tt)


def _ptr(x):
    """Data pointer of a torch tensor or numpy array."""
    if x is None:
        return None
    if isinstance(x, np.ndarray):
        if not x.flags["C_CONTIGUOUS"]:
            raise ValueError("numpy source must be C-contiguous")
        return ctypes.c_void_p(x.ctypes.data)
    return ctypes.c_void_p(x.data_ptr())


def _on_device(x) -> int:
    return 0 if isinstance(x, np.ndarray) else int(x.is_cuda)


class _DeviceMemory:
    """Device memory of a placement for torch.as_tensor (16-bit words; keeps the placement alive)."""

    def __init__(self, placement, ptr, shape):
        self._placement = placement
        self.__cuda_array_interface__ = {"shape": shape, "typestr": "<i2", "data": (ptr, False), "version": 2}


class Placement:
    """A library-owned placement (dak_placement*). Free with .free() or by dropping it."""

    def __init__(self, handle: ctypes.c_void_p, kind: str, **meta):
        self._h = handle
        self.kind = kind
        self.meta = meta
        self.shape = (meta["B"], meta["H_kv"], meta["D"], meta["L"]) if kind == "kv" else None
        self._cache = {}
        hb, gb, u, hu = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(lib.dak_placement_info(handle, ctypes.byref(hb), ctypes.byref(gb), ctypes.byref(u),
                                      ctypes.byref(hu)), "dak_placement_info")
        self.host_bytes, self.hbm_bytes = hb.value, gb.value
        self.units, self.host_units = u.value, hu.value

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("placement already freed")
        return self._h

    def cached(self, key, make):
        """make() once per key: sizes that depend on the placement and the key alone."""
        v = self._cache.get(key)
        if v is None:
            v = self._cache[key] = make()
        return v

    def slabs(self):
        """The parts of a placed KV cache as bf16 tensors that share its memory: (host, hbm), the
        pinned part on the CPU and the HBM part on the GPU, each [slabs of that tier][chunks of 64
        tokens][K, V][64][D] (dak_placement_data in dak.h says how a row is laid out), or None
        where the placement has none in that tier. The caller orders its reads after the work
        that writes the cache, and drops them before the placement is freed by .free()."""
        import torch
        if self.kind != "kv":
            raise ValueError("slabs() is for KV placements")
        host, hbm = ctypes.c_void_p(), ctypes.c_void_p()
        _check(lib.dak_placement_data(self.handle, ctypes.byref(host), ctypes.byref(hbm)), "dak_placement_data")
        tail = (-(-self.meta["L"] // 64), 2, 64, self.meta["D"])
        out = []
        for ptr, n, on_gpu in ((host.value, self.host_units, False), (hbm.value, self.units - self.host_units, True)):
            if not ptr or not n:
                out.append(None)
            elif on_gpu:
                mem = _DeviceMemory(self, ptr, (n,) + tail)
                out.append(torch.as_tensor(mem).view(torch.bfloat16))
            else:
                mem = (ctypes.c_int16 * (n * int(np.prod(tail)))).from_address(ptr)
                mem._placement = self
                out.append(torch.from_numpy(np.ctypeslib.as_array(mem)).view(torch.bfloat16).view((n,) + tail))
        return tuple(out)

    def free(self):
        if self._h is not None:
            lib.dak_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


# ------------------------------------------------------------------------------- placement

def host_tiles_for_ratio(x: float, M: int, tile_m: int = 64) -> int:
    """Tile rows to place on the host for offload ratio x: ceil(x * T), T = ceil(M / tile_m),
    so that at least the fraction x of the rows leaves HBM."""
    import math
    T = -(-int(M) // int(tile_m))
    return max(0, min(T, math.ceil(float(x) * T - 1e-12)))


def host_requests_for_ratio(x: float, batch: int) -> int:
    """Requests whose KV goes to the host for offload ratio x: ceil(x * B)."""
    import math
    return max(0, min(int(batch), math.ceil(float(x) * int(batch) - 1e-12)))


def host_heads_for_ratio(x: float, batch: int, h_kv: int) -> int:
    """(request, kv head) slabs whose KV goes to the host for offload ratio x: ceil(x * B * H_kv)."""
    return host_requests_for_ratio(x, int(batch) * int(h_kv))


def dak_place_matrix(A, n_host_tiles: int, tile_m: int = 64) -> Placement:
    """Place weights A [M][K] (bf16: torch tensor on host or device, or numpy uint16 bits)."""
    if A.ndim != 2:
        raise ValueError("A must be 2-D [M][K]")
    M, K = int(A.shape[0]), int(A.shape[1])
    out = ctypes.c_void_p()
    _check(lib.dak_place_matrix(_ptr(A), _on_device(A), M, K, K, tile_m, int(n_host_tiles),
                                ctypes.byref(out)), "dak_place_matrix")
    return Placement(out, "matrix", M=M, K=K, tile_m=tile_m)


def dak_place_matrix_glu(A, n_host_tiles: int, tile_m: int = 64) -> Placement:
    """Place a SwiGLU weight A [2f][K] (f gate rows, then f up rows) interleaved, so that
    dak_gemm over it returns silu(gate) * up [N][f]."""
    if A.ndim != 2 or int(A.shape[0]) % 2:
        raise ValueError("A must be 2-D [2f][K]")
    M, K = int(A.shape[0]), int(A.shape[1])
    out = ctypes.c_void_p()
    _check(lib.dak_place_matrix_glu(_ptr(A), _on_device(A), M // 2, K, K, tile_m, int(n_host_tiles),
                                    ctypes.byref(out)), "dak_place_matrix_glu")
    return Placement(out, "matrix", M=M, K=K, tile_m=tile_m, glu=True)


def dak_place_kv(K, V, n_host_requests: int) -> Placement:
    """Place a KV cache, K and V [B][H_kv][L][D] bf16 (torch or numpy uint16 bits)."""
    if K.shape != V.shape or K.ndim != 4:
        raise ValueError("K and V must both be [B][H_kv][L][D]")
    B, Hkv, L, D = (int(s) for s in K.shape)
    out = ctypes.c_void_p()
    _check(lib.dak_place_kv(_ptr(K), _ptr(V), _on_device(K), B, Hkv, L, D, int(n_host_requests),
                            ctypes.byref(out)), "dak_place_kv")
    return Placement(out, "kv", B=B, H_kv=Hkv, L=L, D=D)


def dak_place_kv_heads(K, V, n_host_heads: int) -> Placement:
    """dak_place_kv by (request, kv head) slab: the first n_host_heads slabs in request-major
    order (request b, head g is slab b * H_kv + g) go to the host."""
    if K.shape != V.shape or K.ndim != 4:
        raise ValueError("K and V must both be [B][H_kv][L][D]")
    B, Hkv, L, D = (int(s) for s in K.shape)
    out = ctypes.c_void_p()
    _check(lib.dak_place_kv_heads(_ptr(K), _ptr(V), _on_device(K), B, Hkv, L, D, int(n_host_heads),
                                  ctypes.byref(out)), "dak_place_kv_heads")
    return Placement(out, "kv", B=B, H_kv=Hkv, L=L, D=D)


def dak_kv_append(KV: Placement, k_new, v_new, positions, stream=None):
    """Write one new token per (request, kv head) into a placed cache: k_new and v_new bf16
    CUDA [B][H_kv][D], positions int32 CUDA [B] (the row each request's token goes to)."""
    import torch
    _check_bf16_cuda(k_new, "k_new")
    _check_bf16_cuda(v_new, "v_new")
    shape = (KV.meta["B"], KV.meta["H_kv"], KV.meta["D"])
    if tuple(k_new.shape) != shape or tuple(v_new.shape) != shape:
        raise ValueError(f"k_new / v_new must be {list(shape)}")
    if positions.dtype != torch.int32 or not positions.is_cuda or positions.numel() != shape[0]:
        raise ValueError("positions must be int32 CUDA [B]")
    _check(lib.dak_kv_append(KV.handle, _ptr(k_new), _ptr(v_new), _ptr(positions), _stream_ptr(stream)),
           "dak_kv_append")


def dak_free(p: Placement):
    p.free()


def dak_placement_info(p: Placement):
    return dict(host_bytes=p.host_bytes, hbm_bytes=p.hbm_bytes, units=p.units, host_units=p.host_units)


# ------------------------------------------------------------------------------- hot path

def _check_bf16_cuda(t, name):
    import torch
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")


def dak_gemm(A: Placement, B, C=None, c_fp32: bool = False, tuning=None, stream=None, workspace=None):
    """C [N][M] = B [N][K] . A^T over the tiered placement A (returns C). workspace: an optional
    split workspace of the caller's (a zeroed device tensor of dak_gemm_workspace_bytes(A, N)
    bytes or more), for launches that may overlap others on different streams."""
    import torch
    _check_bf16_cuda(B, "B")
    N = int(B.shape[0])
    if B.ndim != 2 or int(B.shape[1]) != A.meta["K"]:
        raise ValueError("B must be [N][K]")
    if C is None:
        cols = A.meta["M"] // 2 if A.meta.get("glu") else A.meta["M"]
        C = torch.empty((N, cols), dtype=torch.float32 if c_fp32 else torch.bfloat16, device=B.device)
    if workspace is None:
        _check(lib.dak_gemm(A.handle, _ptr(B), _ptr(C), N, int(bool(c_fp32)), _tuning(tuning), _stream_ptr(stream)),
               "dak_gemm")
    else:
        nbytes = workspace.numel() * workspace.element_size()
        _check(lib.dak_gemm_ws(A.handle, _ptr(B), _ptr(C), N, int(bool(c_fp32)), _tuning(tuning), _ptr(workspace),
                               ctypes.c_size_t(nbytes), _stream_ptr(stream)), "dak_gemm_ws")
    return C


def _chain_ops(ops):
    arr = (dak_gemm_op * len(ops))()
    for j, o in enumerate(ops):
        arr[j].A = o["A"].handle
        arr[j].B = o["B"].data_ptr() if o.get("B") is not None else None
        arr[j].C = o["C"].data_ptr() if o.get("C") is not None else None
        arr[j].c_fp32 = int(bool(o.get("c_fp32", False)))
        arr[j].after_prev = int(bool(o.get("after_prev", False)))
    return arr


def dak_gemm_chain_workspace_bytes(ops, N: int, tuning=None) -> int:
    """Bytes of the workspace dak_gemm_chain needs (ops: dicts with at least 'A')."""
    return int(lib.dak_gemm_chain_workspace_bytes(_chain_ops(ops), len(ops), int(N), _tuning(tuning)))


def dak_gemm_chain(ops, tuning=None, workspace=None, stream=None):
    """Several GEMMs in one persistent launch. ops: list of dicts with 'A' (Placement), 'B'
    (bf16 [N][K] CUDA tensor), optional 'C', 'c_fp32' and 'after_prev' (B comes from an
    earlier operation of the chain). workspace: a zeroed CUDA tensor of
    dak_gemm_chain_workspace_bytes bytes (allocated and zeroed here when None). Returns the
    list of C tensors."""
    import torch
    if not ops:
        raise ValueError("empty chain")
    N = int(ops[0]["B"].shape[0])
    ops = [dict(o) for o in ops]
    for o in ops:
        _check_bf16_cuda(o["B"], "B")
        if int(o["B"].shape[0]) != N or int(o["B"].shape[1]) != o["A"].meta["K"]:
            raise ValueError("every B must be [N][K] with the same N")
        if o.get("C") is None:
            cols = o["A"].meta["M"] // 2 if o["A"].meta.get("glu") else o["A"].meta["M"]
            o["C"] = torch.empty((N, cols), dtype=torch.float32 if o.get("c_fp32") else torch.bfloat16,
                                 device=o["B"].device)
    if workspace is None:
        nbytes = dak_gemm_chain_workspace_bytes(ops, N, tuning) if len(ops) <= 8 else 0
        if nbytes == 0:  # a chain the library rejects: let it say why
            _check(lib.dak_gemm_chain(_chain_ops(ops), len(ops), N, _tuning(tuning), None, 0, _stream_ptr(stream)),
                   "dak_gemm_chain")
        workspace = torch.zeros(nbytes, dtype=torch.uint8, device=ops[0]["B"].device)
    _check(lib.dak_gemm_chain(_chain_ops(ops), len(ops), N, _tuning(tuning), _ptr(workspace),
                              ctypes.c_size_t(workspace.numel() * workspace.element_size()), _stream_ptr(stream)),
           "dak_gemm_chain")
    return [o["C"] for o in ops]


def dak_gemm_chain_plan(shapes, N: int, n_host_tiles=None, tile_m=None, after_prev=None, sm_count: int = None,
                        tuning=None) -> dict:
    """How dak_gemm_chain would deal a chain's units over its CTAs, from host arithmetic alone:
    shapes [(M, K), ...], per operation n_host_tiles, tile_m (64 or 128) and after_prev;
    sm_count None = this process's GPU."""
    n = len(shapes)
    if sm_count is None:
        sm_count = dak_sm_count()

    def arr(t, vals):
        return (t * n)(*[int(v) for v in vals])
    out = dak_gemm_chain_plan_info()
    _check(lib.dak_gemm_chain_plan(arr(ctypes.c_int64, [m for m, _ in shapes]), arr(ctypes.c_int64, [k for _, k in shapes]),
                                   arr(ctypes.c_int, tile_m or [64] * n), arr(ctypes.c_int, n_host_tiles or [0] * n),
                                   arr(ctypes.c_int, after_prev or [0] * n), n, int(N), int(sm_count), _tuning(tuning),
                                   ctypes.byref(out)), "dak_gemm_chain_plan")
    return {f: int(getattr(out, f)) for f, _ in dak_gemm_chain_plan_info._fields_}


def dak_gemm_workspace_bytes(A: Placement, N: int) -> int:
    """Bytes of a caller's split workspace for dak_gemm over A with N hidden-state rows."""
    return int(lib.dak_gemm_workspace_bytes(A.handle, int(N)))


def dak_gemm_plan(M: int, K: int, n_host_tiles: int, N: int, sm_count: int = None, tuning=None,
                  ws_bytes: int = 0, tile_m: int = 64) -> dict:
    """The launch dak_gemm would make for an M x K matrix placed in tiles of tile_m rows with
    n_host_tiles of them on the host and N hidden-state rows (pieces, rings, CTAs of each
    role), from host arithmetic alone; sm_count None = this process's GPU."""
    if sm_count is None:
        sm_count = dak_sm_count()
    out = dak_gemm_plan_info()
    _check(lib.dak_gemm_plan(int(M), int(K), int(tile_m), int(n_host_tiles), int(N), int(sm_count), _tuning(tuning),
                             ctypes.c_size_t(int(ws_bytes)), ctypes.byref(out)), "dak_gemm_plan")
    return {f: int(getattr(out, f)) for f, _ in dak_gemm_plan_info._fields_}


def dak_gemm_launch_plan(A: Placement, N: int, tuning=None, ws_bytes: int = 0) -> dict:
    """The plan dak_gemm would use for placement A and N rows on this process's GPU."""
    out = dak_gemm_plan_info()
    _check(lib.dak_gemm_launch_plan(A.handle, int(N), _tuning(tuning), ctypes.c_size_t(int(ws_bytes)),
                                    ctypes.byref(out)), "dak_gemm_launch_plan")
    return {f: int(getattr(out, f)) for f, _ in dak_gemm_plan_info._fields_}


def dak_gemm_staged(A: Placement, staging, B, C=None, c_fp32: bool = False, tuning=None, stream=None):
    import torch
    _check_bf16_cuda(B, "B")
    N = int(B.shape[0])
    if C is None:
        C = torch.empty((N, A.meta["M"]), dtype=torch.float32 if c_fp32 else torch.bfloat16, device=B.device)
    _check(lib.dak_gemm_staged(A.handle, _ptr(staging), _ptr(B), _ptr(C), N, int(bool(c_fp32)), _tuning(tuning),
                               _stream_ptr(stream)), "dak_gemm_staged")
    return C


def dak_attn_workspace_bytes(B: int, H_q: int, D: int, n_split: int) -> int:
    return int(lib.dak_attn_workspace_bytes(B, H_q, D, n_split))


def dak_attn_default_split(KV: Placement) -> int:
    return int(lib.dak_attn_default_split(KV.handle))


def _attn_common(Q, KV, O, workspace, tuning):
    import torch
    _check_bf16_cuda(Q, "Q")
    B, Hq, D = (int(s) for s in Q.shape)
    if B != KV.meta["B"] or D != KV.meta["D"]:
        raise ValueError("Q does not match the KV placement")
    n_split = int(dict(tuning or {}).get("n_split", 0) or 0) if not isinstance(tuning, dak_tuning) else tuning.n_split
    if n_split <= 0:
        n_split = dak_attn_default_split(KV)
    ws_bytes = dak_attn_workspace_bytes(B, Hq, D, n_split)
    if workspace is None and ws_bytes:
        workspace = torch.empty(ws_bytes // 4, dtype=torch.float32, device=Q.device)
    if O is None:
        O = torch.empty_like(Q)
    tun = dict(tuning or {}) if not isinstance(tuning, dak_tuning) else tuning
    if not isinstance(tun, dak_tuning):
        tun["n_split"] = n_split
    ws_len = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return Hq, O, workspace, ws_len, tun


def dak_attn(Q, KV: Placement, seq_lens=None, scale: float = 0.0, O=None, workspace=None, tuning=None, stream=None):
    """Decode attention o [B][Hq][D] over the request-partitioned KV placement (returns O)."""
    Hq, O, workspace, ws_len, tun = _attn_common(Q, KV, O, workspace, tuning)
    _check(lib.dak_attn(_ptr(Q), KV.handle, _ptr(seq_lens), Hq, float(scale), _ptr(O), _ptr(workspace), ws_len,
                        _tuning(tun), _stream_ptr(stream)), "dak_attn")
    return O


def dak_attn_f32(Q, KV: Placement, seq_lens=None, scale: float = 0.0, O=None, workspace=None, tuning=None,
                 stream=None):
    """dak_attn with an fp32 output o [B][Hq][D] (the parity mode; returns O)."""
    import torch
    if O is None:
        O = torch.empty(tuple(Q.shape), dtype=torch.float32, device=Q.device)
    if not (O.dtype == torch.float32 and O.is_cuda and O.is_contiguous() and tuple(O.shape) == tuple(Q.shape)):
        raise ValueError("O must be a contiguous fp32 CUDA tensor shaped like Q")
    Hq, O, workspace, ws_len, tun = _attn_common(Q, KV, O, workspace, tuning)
    _check(lib.dak_attn_f32(_ptr(Q), KV.handle, _ptr(seq_lens), Hq, float(scale), _ptr(O), _ptr(workspace), ws_len,
                            _tuning(tun), _stream_ptr(stream)), "dak_attn_f32")
    return O


def dak_attn_staged(Q, KV: Placement, staging, seq_lens=None, scale: float = 0.0, O=None, workspace=None,
                    tuning=None, stream=None):
    Hq, O, workspace, ws_len, tun = _attn_common(Q, KV, O, workspace, tuning)
    _check(lib.dak_attn_staged(_ptr(Q), KV.handle, _ptr(staging), _ptr(seq_lens), Hq, float(scale), _ptr(O),
                               _ptr(workspace), ws_len, _tuning(tun), _stream_ptr(stream)), "dak_attn_staged")
    return O


def dak_attn_noalloc(Q, KV: Placement, O, seq_lens=None, scale: float = 0.0, tuning=None, stream=None):
    """dak_attn without a workspace argument, for callers that cannot allocate device memory
    (an engine whose pools already hold the device's memory, code without access to the
    process's allocator, a loop where an allocation would synchronise the device). The
    library takes the split workspace from its fixed NOALLOC_SCRATCH_BYTES device array,
    shared by all calls: calls that overlap on the GPU race on it. O must be preallocated."""
    _check_bf16_cuda(Q, "Q")
    _check_bf16_cuda(O, "O")
    B, Hq, D = (int(s) for s in Q.shape)
    if B != KV.meta["B"] or D != KV.meta["D"] or tuple(O.shape) != tuple(Q.shape):
        raise ValueError("Q / O do not match the KV placement")
    tun = tuning if isinstance(tuning, dak_tuning) else dict(tuning or {})
    n_split = tun.n_split if isinstance(tun, dak_tuning) else int(tun.get("n_split", 0) or 0)
    if n_split <= 0:
        n_split = dak_attn_default_split(KV)
    need = dak_attn_workspace_bytes(B, Hq, D, n_split)
    if need > NOALLOC_SCRATCH_BYTES:
        raise DakError(1, f"dak_attn_noalloc: needs {need} bytes of workspace, more than the fixed "
                          f"{NOALLOC_SCRATCH_BYTES}-byte array; use dak_attn with a workspace")
    _check(lib.dak_attn_noalloc(_ptr(Q), KV.handle, _ptr(seq_lens), Hq, float(scale), _ptr(O), _tuning(tuning),
                                _stream_ptr(stream)), "dak_attn_noalloc")
    return O


# ------------------------------------------------------------------------------- rotation, append, eviction

def dak_rope_make(head_dim: int, rot_dim: int = 0, theta: float = 0.0, interleaved: bool = False,
                  scaling: str = "none", factor: float = 1.0, orig_len: float = 0.0, low_turns: float = 0.0,
                  high_turns: float = 0.0, attn_scale: float = 1.0) -> dak_rope_plan:
    """The rotation of dak_kv_append_rope for heads of head_dim elements of which the first
    rot_dim (0 = all) turn, in halves or interleaved pairs, with scaling one of "none",
    "linear", "ntk", "by_parts" (dak_rope_config in dak.h)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    c = dak_rope_config(rot_dim=int(rot_dim), interleaved=int(bool(interleaved)), scaling=ROPE_SCALINGS[scaling],
                        theta=float(theta), factor=float(factor), orig_len=float(orig_len),
                        low_turns=float(low_turns), high_turns=float(high_turns), attn_scale=float(attn_scale))
    out = dak_rope_plan()
    _check(lib.dak_rope_make(int(head_dim), ctypes.byref(c), ctypes.byref(out)), "dak_rope_make")
    return out


def dak_rope_from_freqs(head_dim: int, inv_freq, interleaved: bool = False, attn_scale: float = 1.0) -> dak_rope_plan:
    """The same from given frequencies (radians per position, one per pair)."""
    f = [float(x) for x in inv_freq]
    out = dak_rope_plan()
    _check(lib.dak_rope_from_freqs(int(head_dim), (ctypes.c_double * max(1, len(f)))(*f), len(f),
                                   int(bool(interleaved)), float(attn_scale), ctypes.byref(out)), "dak_rope_from_freqs")
    return out


# The calls below are made once per layer and token, so that their host time counts: tensors are
# checked in one place each and handed over as plain addresses, results are made without a pass
# through torch's dispatcher (1.7 us instead of 3.3), and a workspace of the call's own is taken from
# torch's allocator for the call's stream and given back when the call is launched (1 us instead of
# 4): memory given back is handed out again in that stream's order, in a graph that is being captured
# from that graph's own pool.

def _t():
    global _torch, _get_device, _get_stream, _alloc, _free, _empty
    import torch
    _get_device, _get_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _alloc = torch._C._cuda_cudaCachingAllocator_raw_alloc
    _free = torch._C._cuda_cudaCachingAllocator_raw_delete
    try:
        from torch._C._dynamo.guards import _empty_strided_cuda as _empty
    except ImportError:
        def _empty(shape, strides, dtype):
            return torch.empty(shape, dtype=dtype, device="cuda")
    _torch = torch
    return torch


_torch = _get_device = _get_stream = _alloc = _free = _empty = None


def _current(stream):
    """The stream as the current one: a call that is given a stream makes its results and its
    workspace for that stream too."""
    return _torch.cuda.stream(_torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def _kv_shape(KV, name="KV"):
    """[B, H_kv, D, L] of a KV placement."""
    if KV.shape is None:
        raise ValueError(f"{name} must be a KV placement")
    return KV.shape


def _given(workspace, dev):
    """Address and bytes of the caller's workspace."""
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the current CUDA device")
    return workspace.data_ptr(), workspace.nbytes


def _arg(t, name, dtype, shape, dev):
    """Address of a contiguous tensor of this type and shape on the current device dev (None: none)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on the current CUDA device")
    return t.data_ptr()


def _token_rows(t, name, B, T, heads, D, dtype, dev):
    """Address of t [B][T][heads][D] (T = 1: also [B][heads][D]) and the pitch in elements between
    its tokens, which lie at one pitch with each token's heads contiguous, as in a slice of a
    packed projection."""
    if t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} tensor on the current CUDA device")
    shape, st = t.shape, t.stride()
    if T == 1 and shape == (B, heads, D):
        row, head, el = st
        ok = True
    elif shape == (B, T, heads, D):
        row, head, el = (st[1] if T > 1 else st[0]), st[2], st[3]
        ok = T == 1 or B == 1 or st[0] == T * st[1]
    else:
        raise ValueError(f"{name} must be [B={B}][T={T}][{heads}][{D}]")
    if not ok or el != 1 or (heads > 1 and head != D):
        raise ValueError(f"{name}: a token's heads must be contiguous and its tokens at one pitch")
    return t.data_ptr(), heads * D if B * T == 1 else row


def _append_rope(KV, rope, axes, q, k_new, v_new, slots, positions, n_new, q_out, slot_pos, acc):
    """dak_kv_append_rope_acc, or with axes (the axes of each token's own positions) dak_kv_append_rope_axes."""
    torch = _torch or _t()
    B, Hkv, D, L = _kv_shape(KV)
    T = k_new.shape[1] if k_new.ndim == 4 else 1
    dtype, dev = k_new.dtype, _get_device()
    fp32 = dtype is torch.float32
    if not fp32 and dtype is not torch.bfloat16:
        raise ValueError("k_new must be bf16 or fp32")
    ka, kp = _token_rows(k_new, "k_new", B, T, Hkv, D, dtype, dev)
    va, vp = _token_rows(v_new, "v_new", B, T, Hkv, D, dtype, dev)
    Hq = qp = 0
    qa = oa = None
    if q is not None:
        Hq = q.shape[-2]
        qa, qp = _token_rows(q, "q", B, T, Hq, D, dtype, dev)
        if q_out is None:
            if q.ndim == 4:
                q_out = _empty((B, T, Hq, D), (T * Hq * D, Hq * D, D, 1), torch.bfloat16)
            else:
                q_out = _empty((B, Hq, D), (Hq * D, D, 1), torch.bfloat16)
        oa = _arg(q_out, "q_out", torch.bfloat16, q.shape, dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    i32, per_request, table = torch.int32, (B,), (B, Hkv, L)
    fn, name = (lib.dak_kv_append_rope_axes, "dak_kv_append_rope_axes") if axes else (lib.dak_kv_append_rope_acc, "dak_kv_append_rope")
    _check(fn(KV.handle, rope, qa, ka, va, fp32, T, Hq, qp, kp, vp, _arg(slots, "slots", i32, per_request, dev),
              _arg(positions, "positions", i32, (B, T, axes) if axes else per_request, dev),
              _arg(n_new, "n_new", i32, per_request, dev), oa, _arg(slot_pos, "slot_pos", i32, table, dev),
              _arg(acc, "acc", torch.float32, table, dev), _get_stream(dev)), name)
    return q_out


def dak_kv_append_rope(KV: Placement, rope: dak_rope_plan, q, k_new, v_new, slots, positions=None, n_new=None,
                       q_out=None, slot_pos=None, stream=None, acc=None):
    """Rotate new tokens and append them to a placed cache (dak.h): q [B][T][H_q][D] (or None),
    k_new and v_new [B][T][H_kv][D], bf16 or fp32 CUDA, slices of one projection's output as
    they are (T = 1: the T axis may be absent); slots, positions, n_new int32 CUDA [B];
    slot_pos int32 and acc fp32 CUDA [B][H_kv][L], updated in place: a written row's position,
    and 0 for its accumulated weight (the table of dak_attn_acc). Returns q_out, bf16, shaped as q (None
    without q)."""
    if stream is not None:
        _torch or _t()
        with _current(stream):
            return _append_rope(KV, rope, 0, q, k_new, v_new, slots, positions, n_new, q_out, slot_pos, acc)
    return _append_rope(KV, rope, 0, q, k_new, v_new, slots, positions, n_new, q_out, slot_pos, acc)


def dak_rope_axes_make(rope: dak_rope_plan, axis=None, n_axes: int = None) -> dak_rope_axes_plan:
    """The rotation of dak_kv_append_rope_axes: the pairs and frequencies of rope, pair i turned by a
    token's position on axis[i] (one per pair of rope; None: axis 0 for all). n_axes: positions of
    a token, 1..4 (None: as many as axis names)."""
    a = None if axis is None else [int(x) for x in axis]
    if a is not None and len(a) != rope.rot_dim // 2:
        raise ValueError(f"axis must name one axis for each of the {rope.rot_dim // 2} pairs")
    n = int(n_axes) if n_axes is not None else 1 if a is None else max(a) + 1
    out = dak_rope_axes_plan()
    _check(lib.dak_rope_axes_make(ctypes.byref(rope), n, None if a is None else (ctypes.c_int * len(a))(*a),
                                  ctypes.byref(out)), "dak_rope_axes_make")
    return out


def dak_kv_append_rope_axes(KV: Placement, rope: dak_rope_axes_plan, q, k_new, v_new, slots, positions, n_new=None,
                            q_out=None, slot_pos=None, acc=None, stream=None):
    """dak_kv_append_rope for tokens with positions of their own (dak.h): positions int32 CUDA
    [B][T][rope.n_axes]. Rows are slots[b] + t; slot_pos takes a token's position on axis 0."""
    if positions is None:
        raise ValueError("positions int32 [B][T][n_axes] are required")
    if stream is not None:
        _torch or _t()
        with _current(stream):
            return _append_rope(KV, rope, rope.n_axes, q, k_new, v_new, slots, positions, n_new, q_out, slot_pos, acc)
    return _append_rope(KV, rope, rope.n_axes, q, k_new, v_new, slots, positions, n_new, q_out, slot_pos, acc)


def dak_kv_evict_workspace_bytes(KV: Placement) -> int:
    return int(lib.dak_kv_evict_workspace_bytes(KV.handle))


def dak_kv_evict(KV: Placement, seq_lens, n_keep: int, n_recent: int, acc, slot_pos, acc_out=None, slot_pos_out=None,
                 lens_out=None, src_out=None, workspace=None, stream=None):
    """Keep n_keep slots of every (request, kv head) of a placed cache that holds more: the
    n_recent newest positions, then the largest accumulated weights (dak.h). acc fp32 and
    slot_pos int32 CUDA [B][H_kv][L], updated in place unless acc_out / slot_pos_out are
    given; seq_lens int32 CUDA [B]. Returns (lens_out [B], src_out [B][H_kv][n_keep]), int32:
    the new lengths, and the slot each kept row came from (-1 past the length)."""
    torch = _torch or _t()
    if stream is not None:
        with _current(stream):
            return dak_kv_evict(KV, seq_lens, n_keep, n_recent, acc, slot_pos, acc_out, slot_pos_out, lens_out, src_out,
                                workspace)
    B, Hkv, _, L = _kv_shape(KV)
    n_keep = int(n_keep)
    if not 1 <= n_keep <= L:
        raise DakError(1, f"dak_kv_evict: n_keep {n_keep} outside 1..{L}")
    table, per_request, kept = (B, Hkv, L), (B,), (B, Hkv, n_keep)
    i32, f32, dev = torch.int32, torch.float32, _get_device()
    if lens_out is None:
        lens_out = _empty(per_request, (1,), i32)
    if src_out is None:
        src_out = _empty(kept, (Hkv * n_keep, n_keep, 1), i32)
    aa, pa = _arg(acc, "acc", f32, table, dev), _arg(slot_pos, "slot_pos", i32, table, dev)
    args = (_arg(seq_lens, "seq_lens", i32, per_request, dev), n_keep, int(n_recent), aa,
            aa if acc_out is None else _arg(acc_out, "acc_out", f32, table, dev), pa,
            pa if slot_pos_out is None else _arg(slot_pos_out, "slot_pos_out", i32, table, dev),
            _arg(lens_out, "lens_out", i32, per_request, dev), _arg(src_out, "src_out", i32, kept, dev))
    st = _get_stream(dev)
    if workspace is not None:
        _check(lib.dak_kv_evict(KV.handle, *args, *_given(workspace, dev), st), "dak_kv_evict")
        return lens_out, src_out
    n = KV.cached("evict", lambda: dak_kv_evict_workspace_bytes(KV))
    ws = _alloc(n, st)
    try:
        _check(lib.dak_kv_evict(KV.handle, *args, ws, n, st), "dak_kv_evict")
    finally:
        _free(ws)
    return lens_out, src_out


# ------------------------------------------------------------------------------- drafted trees, forked caches

MAX_TREE = 256  # DAK_MAX_TREE in dak.h


def dak_tree_mask(parents, device="cuda"):
    """The masks and depths of trees of drafted tokens: parents [B][T] (or [T]: one tree), each token's
    parent among the tokens before it, or -1 for one that continues the text itself. Returns (mask
    int64 [B][T][ceil(T / 64)], bit s % 64 of word s // 64 for draft s: a token's ancestors and
    itself; depths int32 [B][T], 0 for a token without parent: what to add to a request's length for
    its position). Host arithmetic, copied to device."""
    import torch
    p = np.asarray(parents.cpu() if isinstance(parents, torch.Tensor) else parents, dtype=np.int64)
    p = p[None] if p.ndim == 1 else p
    if p.ndim != 2 or p.shape[1] < 1:
        raise ValueError("parents must be [B][T] or [T]")
    B, T = p.shape
    if ((p < -1) | (p >= np.arange(T))).any():
        raise ValueError("a token's parent must be -1 or one of the tokens before it")
    mask, depth = np.zeros((B, T, -(-T // 64)), np.uint64), np.zeros((B, T), np.int32)
    b = np.arange(B)
    for t in range(T):
        has, at = p[:, t] >= 0, np.maximum(p[:, t], 0)
        mask[:, t] = np.where(has[:, None], mask[b, at], np.uint64(0))
        mask[:, t, t // 64] |= np.uint64(1) << np.uint64(t % 64)
        depth[:, t] = np.where(has, depth[b, at] + 1, 0)
    return torch.from_numpy(mask.view(np.int64)).to(device), torch.from_numpy(depth).to(device)


def dak_attn_tree_workspace_bytes(KV: Placement, T: int, H_q: int) -> int:
    return int(lib.dak_attn_tree_workspace_bytes(KV.handle, int(T), int(H_q)))


def dak_attn_tree(Q, KV: Placement, seq_lens, mask=None, n_new=None, scale: float = 0.0, O=None, o_fp32: bool = False,
                  workspace=None, tuning=None, stream=None):
    """Decode attention of T drafted tokens per request (dak.h): Q bf16 CUDA [B][T][H_q][D]; seq_lens
    int32 CUDA [B], the cached rows before the drafted ones, which lie behind them; mask int64 CUDA
    [B][T][ceil(T / 64)], or [1][T][ceil(T / 64)] for one tree for all (dak_tree_mask), None: a chain;
    n_new int32 CUDA [B], drafted tokens of each request (None: T). Returns O, shaped as Q; the
    rows of tokens t >= n_new[b] of a given O are left as they were (of a new one: anything)."""
    torch = _torch or _t()
    if stream is not None:
        with _current(stream):
            return dak_attn_tree(Q, KV, seq_lens, mask, n_new, scale, O, o_fp32, workspace, tuning)
    dev = _get_device()
    B, Hkv, D, L = _kv_shape(KV)
    shape = Q.shape
    if len(shape) != 4 or shape[0] != B or shape[3] != D:
        raise ValueError("Q must be [B][T][H_q][D] of the KV placement's B and D")
    _, T, Hq, _ = shape
    words = -(-T // 64)
    dtype = torch.float32 if o_fp32 else torch.bfloat16
    qa = _arg(Q, "Q", torch.bfloat16, shape, dev)
    pitch = 0
    if mask is not None and mask.shape[0] != 1:
        pitch = T * words
    ma = _arg(mask, "mask", torch.int64, (B if pitch else 1, T, words), dev)
    if O is None:
        O = _empty((B, T, Hq, D), (T * Hq * D, Hq * D, D, 1), dtype)
    la, na = _arg(seq_lens, "seq_lens", torch.int32, (B,), dev), _arg(n_new, "n_new", torch.int32, (B,), dev)
    args = (qa, KV.handle, la, T, ma, pitch, na, Hq, float(scale), _arg(O, "O", dtype, shape, dev), bool(o_fp32))
    st, tun = _get_stream(dev), _tuning(tuning)
    if workspace is not None:
        _check(lib.dak_attn_tree(*args, *_given(workspace, dev), tun, st), "dak_attn_tree")
        return O
    n = KV.cached(("tree", T, Hq), lambda: dak_attn_tree_workspace_bytes(KV, T, Hq))
    ws = _alloc(n, st)
    try:
        _check(lib.dak_attn_tree(*args, ws, n, tun, st), "dak_attn_tree")
    finally:
        _free(ws)
    return O


def dak_kv_commit(KV: Placement, seq_lens, path, n_path, T: int, n_new=None, lens_out=None, slot_pos=None, acc=None,
                  stream=None):
    """Keep the accepted drafts of a tree whose T rows lie behind each request's own (dak.h): row
    seq_lens[b] + path[b][i] becomes row seq_lens[b] + i for i < n_path[b]. path int32 CUDA [B][P], ascending
    draft numbers; seq_lens, n_path, n_new (None: T) int32 CUDA [B]; slot_pos int32 and acc fp32 CUDA
    [B][H_kv][L], updated in place. Returns lens_out int32 [B], the new lengths."""
    torch = _torch or _t()
    if stream is not None:
        with _current(stream):
            return dak_kv_commit(KV, seq_lens, path, n_path, T, n_new, lens_out, slot_pos, acc)
    B, Hkv, _, L = _kv_shape(KV)
    i32, per_request, table, dev = torch.int32, (B,), (B, Hkv, L), _get_device()
    if path.ndim != 2:
        raise ValueError("path must be [B][P]")
    P = path.shape[1]
    if lens_out is None:
        lens_out = _empty(per_request, (1,), i32)
    _check(lib.dak_kv_commit(KV.handle, _arg(seq_lens, "seq_lens", i32, per_request, dev), int(T),
                             _arg(n_new, "n_new", i32, per_request, dev), _arg(path, "path", i32, (B, P), dev), P,
                             _arg(n_path, "n_path", i32, per_request, dev), _arg(lens_out, "lens_out", i32, per_request, dev),
                             _arg(slot_pos, "slot_pos", i32, table, dev), _arg(acc, "acc", torch.float32, table, dev),
                             _get_stream(dev)), "dak_kv_commit")
    return lens_out


def dak_kv_fork(KV: Placement, src_of, seq_lens, first=None, source: Placement = None, lens_out=None, slot_pos=None,
                acc=None, source_slot_pos=None, source_acc=None, stream=None):
    """Let request b of a placed cache take over rows first[b] .. n - 1 of request src_of[b] (dak.h), of the
    same cache, all at once, or of another placement source; n is that request's seq_lens. src_of
    (negative: b stays) and first (None: 0) int32 CUDA [B], seq_lens int32 CUDA of the source's requests;
    slot_pos int32 and acc fp32 CUDA [B][H_kv][L], updated in place, with source_slot_pos and source_acc
    the source's (with source). Returns lens_out int32 [B], the new lengths; with source, the entries
    of requests that stay are left as they are, so that lens_out has to be given."""
    torch = _torch or _t()
    if stream is not None:
        with _current(stream):
            return dak_kv_fork(KV, src_of, seq_lens, first, source, lens_out, slot_pos, acc, source_slot_pos, source_acc)
    B, Hkv, _, L = _kv_shape(KV)
    i32, f32, per_request, table, dev = torch.int32, torch.float32, (B,), (B, Hkv, L), _get_device()
    if source is None:
        if source_slot_pos is not None or source_acc is not None:
            raise ValueError("source_slot_pos and source_acc need a source")
        source, source_slot_pos, source_acc, n, from_table = KV, slot_pos, acc, B, table
    else:
        n, shkv, _, sl = _kv_shape(source, "source")
        from_table = (n, shkv, sl)
        if lens_out is None:
            raise ValueError("a fork from another placement needs lens_out")
    if lens_out is None:
        lens_out = _empty(per_request, (1,), i32)
    _check(lib.dak_kv_fork(KV.handle, source.handle, _arg(src_of, "src_of", i32, per_request, dev),
                           _arg(seq_lens, "seq_lens", i32, (n,), dev), _arg(first, "first", i32, per_request, dev),
                           _arg(lens_out, "lens_out", i32, per_request, dev),
                           _arg(source_slot_pos, "source_slot_pos", i32, from_table, dev),
                           _arg(slot_pos, "slot_pos", i32, table, dev), _arg(source_acc, "source_acc", f32, from_table, dev),
                           _arg(acc, "acc", f32, table, dev), _get_stream(dev)), "dak_kv_fork")
    return lens_out


# ------------------------------------------------------------------------------- attention for serving

def _n_split_of(tuning) -> int:
    if isinstance(tuning, dak_tuning):
        return int(tuning.n_split)
    return int(dict(tuning or {}).get("n_split", 0) or 0)


def _serve_args(Q, KV, O, o_fp32, seq_lens, acc_in, acc_out, dev):
    """Addresses of Q, O, seq_lens, acc_in, acc_out, with O made where there is none."""
    torch = _torch or _t()
    B, Hkv, D, L = _kv_shape(KV)
    shape = Q.shape
    if len(shape) != 3 or shape[0] != B or shape[2] != D:
        raise ValueError("Q must be [B][H_q][D] of the KV placement's B and D")
    dtype = torch.float32 if o_fp32 else torch.bfloat16
    qa = _arg(Q, "Q", torch.bfloat16, shape, dev)
    if O is None:
        O = _empty((B, shape[1], D), (shape[1] * D, D, 1), dtype)
    table = (B, Hkv, L)
    return (O, qa, _arg(O, "O", dtype, shape, dev),
            _arg(seq_lens, "seq_lens", torch.int32, (B,), dev), _arg(acc_in, "acc_in", torch.float32, table, dev),
            _arg(acc_out, "acc_out", torch.float32, table, dev))


def dak_attn_acc_workspace_bytes(KV: Placement, H_q: int, n_split: int = 0) -> int:
    return int(lib.dak_attn_acc_workspace_bytes(KV.handle, int(H_q), int(n_split)))


def dak_attn_acc(Q, KV: Placement, acc_in=None, acc_out=None, seq_lens=None, scale: float = 0.0, O=None,
                 o_fp32: bool = False, workspace=None, tuning=None, stream=None):
    """dak_attn that adds every position's attention weight, summed over the query heads of its
    kv head, to acc_in fp32 [B][H_kv][L] (None = zeros). Returns (O, acc_out); acc_out may be
    acc_in; without one, a new tensor that is zero behind each request's tokens."""
    torch = _torch or _t()
    if stream is not None:
        with _current(stream):
            return dak_attn_acc(Q, KV, acc_in, acc_out, seq_lens, scale, O, o_fp32, workspace, tuning)
    dev = _get_device()
    if acc_out is None:
        B, Hkv, _, L = _kv_shape(KV)
        acc_out = torch.zeros((B, Hkv, L), dtype=torch.float32, device=Q.device)
    O, qa, oa, la, ia, aa = _serve_args(Q, KV, O, o_fp32, seq_lens, acc_in, acc_out, dev)
    Hq = Q.shape[1]
    st, tun = _get_stream(dev), _tuning(tuning)
    if workspace is not None:
        _check(lib.dak_attn_acc(qa, KV.handle, la, Hq, float(scale), oa, bool(o_fp32), ia, aa, *_given(workspace, dev), tun, st),
               "dak_attn_acc")
        return O, acc_out
    split = _n_split_of(tuning) if tuning else 0
    n = KV.cached(("acc", Hq, split), lambda: dak_attn_acc_workspace_bytes(KV, Hq, split))
    ws = _alloc(n, st)
    try:
        _check(lib.dak_attn_acc(qa, KV.handle, la, Hq, float(scale), oa, bool(o_fp32), ia, aa, ws, n, tun, st), "dak_attn_acc")
    finally:
        _free(ws)
    return O, acc_out


def dak_attn_prefix_workspace_bytes(KV: Placement, prefix: Placement, H_q: int, n_split: int = 0,
                                    with_acc: bool = False) -> int:
    return int(lib.dak_attn_prefix_workspace_bytes(KV.handle, prefix.handle, int(H_q), int(n_split), int(bool(with_acc))))


def dak_attn_prefix(Q, KV: Placement, prefix: Placement, prefix_of=None, prefix_lens=None, seq_lens=None, acc_in=None,
                    acc_out=None, scale: float = 0.0, O=None, o_fp32: bool = False, workspace=None, tuning=None,
                    stream=None):
    """Decode attention of requests that share prefixes: request b attends over the first
    prefix_lens[prefix_of[b]] rows of prefix placement slab prefix_of[b] (negative: none; None:
    prefix 0 for all) and over its own seq_lens[b] cached tokens. Each prefix is read once for
    all its requests. acc_out, if given, takes acc_in (None = zeros) plus the weights of the own
    cache's positions, as in dak_attn_acc. Returns O."""
    torch = _torch or _t()
    if stream is not None:
        with _current(stream):
            return dak_attn_prefix(Q, KV, prefix, prefix_of, prefix_lens, seq_lens, acc_in, acc_out, scale, O, o_fp32,
                                   workspace, tuning)
    dev = _get_device()
    if acc_in is not None and acc_out is None:
        raise ValueError("acc_in without acc_out")
    O, qa, oa, la, ia, aa = _serve_args(Q, KV, O, o_fp32, seq_lens, acc_in, acc_out, dev)
    Hq = Q.shape[1]
    pshape = _kv_shape(prefix, "prefix")
    args = (qa, KV.handle, la, prefix.handle, _arg(prefix_lens, "prefix_lens", torch.int32, (pshape[0],), dev),
            _arg(prefix_of, "prefix_of", torch.int32, (Q.shape[0],), dev), Hq, float(scale), oa, bool(o_fp32), ia, aa)
    st, tun = _get_stream(dev), _tuning(tuning)
    if workspace is not None:
        _check(lib.dak_attn_prefix(*args, *_given(workspace, dev), tun, st), "dak_attn_prefix")
        return O
    split = _n_split_of(tuning) if tuning else 0
    n = KV.cached(("prefix", pshape, Hq, split, aa is None),
                  lambda: dak_attn_prefix_workspace_bytes(KV, prefix, Hq, split, aa is not None))
    ws = _alloc(n, st)
    try:
        _check(lib.dak_attn_prefix(*args, ws, n, tun, st), "dak_attn_prefix")
    finally:
        _free(ws)
    return O


def dak_link_begin(slot: int, stream=None):
    """Start host-link handoff sequence `slot` (1..8) on `stream`: later dak_gemm / dak_attn
    calls with tuning link=slot stream their host tiles / requests only once the sequence's
    earlier launches have issued all of their host loads (paces the loads; results are
    unchanged)."""
    _check(lib.dak_link_begin(int(slot), _stream_ptr(stream)), "dak_link_begin")


def dak_link_timeouts(stream=None) -> int:
    """Handoff waits that gave up at their bound since the last call (0 when every launch of
    every sequence found its predecessors in time); the count restarts at zero."""
    c = ctypes.c_uint32()
    _check(lib.dak_link_timeouts(_stream_ptr(stream), ctypes.byref(c)), "dak_link_timeouts")
    return int(c.value)


def dak_selftest_link(stream=None):
    """One pacing wait that must give up (see dak_link_timeouts)."""
    _check(lib.dak_selftest_link(_stream_ptr(stream)), "dak_selftest_link")


def dak_prefetch(p: Placement, staging, stream=None):
    _check(lib.dak_prefetch(p.handle, _ptr(staging), _stream_ptr(stream)), "dak_prefetch")


# ------------------------------------------------------------------------------- planner

def dak_plan_ratios(ops, b_host: float, b_hbm: float, min_offload_bytes: float, mode: int = 0):
    """ops: iterable of (bytes, t_comp[, tile_bytes]). Returns (ratios ndarray, model time s)."""
    ops = list(ops)
    arr = (dak_op * max(1, len(ops)))()
    for i, o in enumerate(ops):
        arr[i].bytes = float(o[0])
        arr[i].t_comp = float(o[1])
        arr[i].tile_bytes = float(o[2]) if len(o) > 2 else 0.0
    ratios = (ctypes.c_double * max(1, len(ops)))()
    t = ctypes.c_double()
    _check(lib.dak_plan_ratios(arr, len(ops), float(b_host), float(b_hbm), float(min_offload_bytes), int(mode),
                               ratios, ctypes.byref(t)), "dak_plan_ratios")
    return np.array(ratios[:len(ops)], dtype=np.float64), t.value


def dak_plan_units(ops, b_host: float, b_hbm: float, min_offload_bytes: float):
    """ops: iterable of (bytes, t_comp, unit_bytes). Returns (host units ndarray int64, model time s)."""
    ops = list(ops)
    arr = (dak_op * max(1, len(ops)))()
    for i, o in enumerate(ops):
        arr[i].bytes, arr[i].t_comp, arr[i].tile_bytes = float(o[0]), float(o[1]), float(o[2])
    out = (ctypes.c_int64 * max(1, len(ops)))()
    t = ctypes.c_double()
    _check(lib.dak_plan_units(arr, len(ops), float(b_host), float(b_hbm), float(min_offload_bytes), out,
                              ctypes.byref(t)), "dak_plan_units")
    return np.array(out[:len(ops)], dtype=np.int64), t.value


# ------------------------------------------------------------------------------- errors / probes

def dak_last_error(stream=None):
    """Synchronise and return (status, info) of the device status word (cleared)."""
    info = ctypes.c_uint64()
    st = lib.dak_last_error(_stream_ptr(stream), ctypes.byref(info))
    return int(st), int(info.value)


def dak_selftest_wait(stream=None):
    """Launch the bounded-wait self-test kernel (its wait must time out after ~2 s)."""
    _check(lib.dak_selftest_wait(_stream_ptr(stream)), "dak_selftest_wait")


def dak_inject_fault(kind: int, count: int = 1, skip: int = 0):
    """Make the library's next `count` calls of this kind (FAULT_*) fail after `skip` more
    succeed (count -1: every call; count 0 clears). Host side only."""
    _check(lib.dak_inject_fault(int(kind), int(skip), int(count)), "dak_inject_fault")


def dak_fault_pending(kind: int) -> int:
    return int(lib.dak_fault_pending(int(kind)))


def dak_alloc_counts():
    """(pinned host buffers, device buffers) the library holds right now."""
    h, d = ctypes.c_int64(), ctypes.c_int64()
    _check(lib.dak_alloc_counts(ctypes.byref(h), ctypes.byref(d)), "dak_alloc_counts")
    return int(h.value), int(d.value)


def dak_sm_count() -> int:
    return int(lib.dak_sm_count())


def dak_probe_read_bw(tier: int, nbytes: int, method: int = 0, ctas: int = 16, window: int = 4,
                      chunk_bytes: int = 32768, iters: int = 5):
    g = ctypes.c_double()
    ok = ctypes.c_int()
    _check(lib.dak_probe_read_bw(tier, nbytes, method, ctas, window, chunk_bytes, iters, ctypes.byref(g),
                                 ctypes.byref(ok)), "dak_probe_read_bw")
    return g.value, bool(ok.value)


def dak_probe_concurrent(host_bytes: int, hbm_bytes: int, host_ctas: int, host_window: int, hbm_ctas: int,
                         hbm_window: int, chunk_bytes: int = 32768, iters: int = 5):
    h, g = ctypes.c_double(), ctypes.c_double()
    _check(lib.dak_probe_concurrent(host_bytes, hbm_bytes, host_ctas, host_window, hbm_ctas, hbm_window, chunk_bytes,
                                    iters, ctypes.byref(h), ctypes.byref(g)), "dak_probe_concurrent")
    return h.value, g.value


# ------------------------------------------------------------------------------- decode step

DECODER_OPS = ("qkv", "o", "gate_up", "down", "kv")
MODE_DIRECT, MODE_PREFETCH_SERIAL, MODE_PREFETCH_OVERLAP = 0, 1, 2


class Decoder:
    """A dak_decoder over placed layers. `layers` is a list of dicts with the placements
    'qkv', 'o', 'gate_up', 'down', 'kv' and the bf16 CUDA gains 'attn_norm', 'mlp_norm';
    the decoder keeps references to them (and frees the placements in .free())."""

    def __init__(self, cfg: dict, layers, final_norm, n_split: int = 0, plain_launch: bool = False,
                 op_tuning=None, link_handoff: bool = True):
        """op_tuning: optional dict mapping 'qkv', 'o', 'gate_up', 'down', 'attn' to dak_tuning
        fields (dicts); n_split sets the attention's context splits (0 = library default);
        link_handoff=False turns off the host-link handoff between the step's kernels."""
        c = dak_decoder_config(n_layers=len(layers), hidden=int(cfg["hidden"]), n_heads=int(cfg["n_heads"]),
                               n_kv_heads=int(cfg["n_kv_heads"]), head_dim=int(cfg["head_dim"]),
                               ffn=int(cfg["ffn"]), rms_eps=float(cfg.get("rms_eps", 1e-5)),
                               rope_theta=float(cfg.get("rope_theta", 500000.0)),
                               plain_launch=int(bool(plain_launch)), no_link_handoff=int(not link_handoff))
        for i, name in enumerate(("qkv", "o", "gate_up", "down", "attn")):
            for k, v in dict((op_tuning or {}).get(name, {})).items():
                setattr(c.op_tuning[i], k, int(v))
        if n_split:
            c.op_tuning[4].n_split = int(n_split)
        for L in layers:
            _check_bf16_cuda(L["attn_norm"], "attn_norm")
            _check_bf16_cuda(L["mlp_norm"], "mlp_norm")
        _check_bf16_cuda(final_norm, "final_norm")
        arr = (dak_decoder_layer * max(1, len(layers)))()
        for i, L in enumerate(layers):
            arr[i] = dak_decoder_layer(L["qkv"].handle, L["o"].handle, L["gate_up"].handle, L["down"].handle,
                                       L["kv"].handle, L["attn_norm"].data_ptr(), L["mlp_norm"].data_ptr())
        out = ctypes.c_void_p()
        _check(lib.dak_decoder_create(ctypes.byref(c), arr, _ptr(final_norm), ctypes.byref(out)),
               "dak_decoder_create")
        self._h = out
        self.cfg = dict(cfg)
        self.layers = list(layers)
        self.final_norm = final_norm
        self.batch = int(lib.dak_decoder_batch(out))

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("decoder already freed")
        return self._h

    def launches(self, mode: int = MODE_DIRECT) -> int:
        return int(lib.dak_decoder_launches(self.handle, int(mode)))

    def host_bytes(self) -> int:
        return sum(L[k].host_bytes for L in self.layers for k in DECODER_OPS)

    def step(self, x_in, positions, out=None, mode: int = MODE_DIRECT, stream=None):
        """One decode step: x_in bf16 [B][d], positions int32 [B] (CUDA) -> out bf16 [B][d]."""
        import torch
        _check_bf16_cuda(x_in, "x_in")
        if out is None:
            out = torch.empty_like(x_in)
        _check(lib.dak_decoder_step(self.handle, _ptr(x_in), _ptr(positions), _ptr(out), int(mode),
                                    _stream_ptr(stream)), "dak_decoder_step")
        return out

    def capture(self, x_in, positions, out, mode: int = MODE_DIRECT):
        """Capture one step with these buffers into the decoder's CUDA graph."""
        _check(lib.dak_decoder_capture(self.handle, _ptr(x_in), _ptr(positions), _ptr(out), int(mode)),
               "dak_decoder_capture")

    def replay(self, stream=None):
        _check(lib.dak_decoder_replay(self.handle, _stream_ptr(stream)), "dak_decoder_replay")

    def free(self, placements: bool = True):
        if self._h is not None:
            lib.dak_decoder_free(self._h)
            self._h = None
        if placements:
            for L in self.layers:
                for k in DECODER_OPS:
                    L[k].free()

    def __del__(self):
        try:
            self.free(placements=False)
        except Exception:
            pass


def place_decoder_layer(weights: dict, kv, host_units: dict, device=None, glu: bool = True) -> dict:
    """Place one layer: weights maps 'qkv', 'o', 'gate_up', 'down' to [out][in] bf16 sources
    (numpy bits or torch) and 'attn_norm', 'mlp_norm' to [d] gains; kv = (K, V) sources
    [B][H_kv][L][D]; host_units maps 'qkv', 'o', 'gate_up', 'down' to their host tile rows
    and either 'kv' to host requests or 'kv_heads' to host (request, kv head) slabs.
    glu places gate_up interleaved so that the SwiGLU runs in the GEMM's epilogue."""
    import torch
    dev = device or torch.device("cuda")
    L = {}
    for k in ("qkv", "o", "gate_up", "down"):
        if k == "gate_up" and glu:
            L[k] = dak_place_matrix_glu(weights[k], int(host_units[k]))
        else:
            L[k] = dak_place_matrix(weights[k], int(host_units[k]))
    if "kv_heads" in host_units:
        L["kv"] = dak_place_kv_heads(kv[0], kv[1], int(host_units["kv_heads"]))
    else:
        L["kv"] = dak_place_kv(kv[0], kv[1], int(host_units["kv"]))
    for k in ("attn_norm", "mlp_norm"):
        g = weights[k]
        if isinstance(g, np.ndarray):
            g = torch.from_numpy(g.view(np.int16)).view(torch.bfloat16)
        L[k] = g.to(dev).contiguous()
    return L


# ------------------------------------------------------------------------------- launch tuner

TUNING_FIELDS = [f for f, _ in dak_tuning._fields_]


def tuning_to_dict(t: dak_tuning, keep_zero: bool = False) -> dict:
    return {f: int(getattr(t, f)) for f in TUNING_FIELDS if keep_zero or getattr(t, f)}


def _tune_result(r: dak_tune_result) -> dict:
    return {"best": tuning_to_dict(r.best), "best_us": r.best_us, "default_us": r.default_us,
            "cc_off_us": r.cc_off_us, "no_align_us": r.no_align_us, "candidates": r.candidates}


def dak_tune_gemm(A: Placement, B, C, c_fp32: bool = False, reps: int = 5, base=None) -> dict:
    """Time dak_gemm over the tuner's candidates (host CTAs x window x chunk) and the
    congestion-control and wave-alignment ablations; returns the fastest tuning and times."""
    _check_bf16_cuda(B, "B")
    r = dak_tune_result()
    _check(lib.dak_tune_gemm(A.handle, _ptr(B), _ptr(C), int(B.shape[0]), int(bool(c_fp32)), int(reps),
                             _tuning(base), ctypes.byref(r)), "dak_tune_gemm")
    return _tune_result(r)


def dak_tune_attn(Q, KV: Placement, O, workspace=None, seq_lens=None, reps: int = 5, base=None) -> dict:
    """dak_tune_gemm for dak_attn (host CTAs x window; n_split from base or the default)."""
    Hq, O, workspace, ws_len, tun = _attn_common(Q, KV, O, workspace, base)
    r = dak_tune_result()
    _check(lib.dak_tune_attn(_ptr(Q), KV.handle, _ptr(seq_lens), Hq, _ptr(O), _ptr(workspace), ws_len, int(reps),
                             _tuning(tun), ctypes.byref(r)), "dak_tune_attn")
    return _tune_result(r)


def save_tuning(path: str, table: dict, meta: dict = None):
    """Persist a table {operation name: tuning fields} (e.g. the tuner's choices) as JSON."""
    import json
    doc = {"tuning": {k: {f: int(v) for f, v in dict(t).items() if f in TUNING_FIELDS} for k, t in table.items()}}
    if meta:
        doc["meta"] = meta
    with open(path, "w") as f:
        json.dump(doc, f, indent=1, sort_keys=True)


def load_tuning(path: str) -> dict:
    """Read a table written by save_tuning; unknown fields are rejected."""
    import json
    with open(path) as f:
        doc = json.load(f)
    table = {}
    for k, t in doc.get("tuning", {}).items():
        bad = set(t) - set(TUNING_FIELDS)
        if bad:
            raise ValueError(f"{path}: unknown tuning fields {sorted(bad)} for {k}")
        table[k] = {f: int(v) for f, v in t.items()}
    return table
