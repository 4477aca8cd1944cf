"""Certified sparse decode attention on GB300 -- Python binding of libcsa.

Thin ctypes layer over the C ABI in ``include/csa.h``: the functions below
carry the same names as the C entry points and only marshal arguments (torch
tensors -> device pointers, Python ints -> host arrays).  Every step of the
decode path runs in the library's CUDA kernels; there is no Python or CPU
fallback, and a missing library raises ``CsaLibraryMissing``.

PyTorch supplies device memory and streams only.

Paper: "Certified Sparse Attention via Perturbed Retrieval" (arXiv
2610.24991), picx.dev summary "Methodology" and "Algorithm Components" 1-4.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_lib", "libcsa.so")

CSA_OK = 0
CSA_BF16, CSA_F32 = 0, 1
CSA_MEASURE_VALUE, CSA_MEASURE_OUTPUT, CSA_MEASURE_DENOM, CSA_MEASURE_CLT = \
    0, 1, 2, 3
WINDOW = 64
BLOCK = 64

EXPORTED = ("csa_workspace_size", "csa_quantize_keys", "csa_decode_step",
            "csa_dense_workspace_size", "csa_dense_decode", "csa_check",
            "csa_status_string", "csa_workspace_layout",
            "csa_profile_enable", "csa_profile_read",
            "csa_dense_decode_static", "csa_decode_step_device",
            "csa_quantize_keys8", "csa_decode_step_refined",
            "csa_rope_turns", "csa_qk_norm_rope", "csa_kv4_append",
            "csa_kv4_unpack", "csa_kv4_workspace_size", "csa_kv4_decode")
# size of the fixed scratch array behind csa_dense_decode_static
DENSE_STATIC_SCRATCH_BYTES = 16 << 20
STATS_FIELDS = 10
STAT = {"level": 0, "keys_read": 1, "values_read": 2, "n_candidates": 3,
        "n_near_threshold": 4, "J": 5, "rounds": 6, "group_keys_read": 7,
        "group_values_read": 8, "rows8": 9}
PHASES = ("clear", "scan", "exact_max", "candidates", "rescore", "predict",
          "levels", "plan", "vgather", "certify", "fallback", "diagnostics",
          "refine8")


class CsaLibraryMissing(RuntimeError):
    pass


class CsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} (status {status})")
        self.status = status


class csa_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("d", ctypes.c_int),
                ("n_max", ctypes.c_int64), ("dtype", ctypes.c_int)]


class csa_params(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_float), ("delta", ctypes.c_float),
                ("r", ctypes.c_int), ("measure", ctypes.c_int),
                ("J_override", ctypes.c_int), ("sub_batches", ctypes.c_int),
                ("perturb", ctypes.c_int), ("qcode", ctypes.c_int),
                ("refine8", ctypes.c_int), ("dots", ctypes.c_int)]


class csa_head_stats(ctypes.Structure):
    _fields_ = [("level", ctypes.c_int32), ("keys_read", ctypes.c_int32),
                ("values_read", ctypes.c_int32),
                ("n_candidates", ctypes.c_int32),
                ("n_near_threshold", ctypes.c_int32), ("J", ctypes.c_int32),
                ("rounds", ctypes.c_int32),
                ("group_keys_read", ctypes.c_int32),
                ("group_values_read", ctypes.c_int32),
                ("rows8", ctypes.c_int32)]


class csa_workspace_map(ctypes.Structure):
    _fields_ = [("ubar", ctypes.c_size_t), ("cmax", ctypes.c_size_t),
                ("s32", ctypes.c_size_t), ("jr_hist", ctypes.c_size_t),
                ("bcnt", ctypes.c_size_t), ("total", ctypes.c_size_t),
                ("J1", ctypes.c_int32), ("sub_batches", ctypes.c_int32),
                ("sub_stride", ctypes.c_size_t), ("sub_B", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class csa_phase_times(ctypes.Structure):
    _fields_ = [("ms", ctypes.c_float * 13), ("steps", ctypes.c_int32),
                ("launches", ctypes.c_int64)]


class csa_strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("t", ctypes.c_int64),
                ("h", ctypes.c_int64)]


class csa_norm_rope(ctypes.Structure):
    _fields_ = [("wq", ctypes.c_void_p), ("wk", ctypes.c_void_p),
                ("norm_eps", ctypes.c_float), ("rot_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("turns", ctypes.c_void_p)]


class csa_kv4(ctypes.Structure):
    _fields_ = [("K4", ctypes.c_void_p), ("bounds", ctypes.c_void_p),
                ("V4", ctypes.c_void_p), ("vscale", ctypes.c_void_p),
                ("Kt", ctypes.c_void_p), ("Vt", ctypes.c_void_p),
                ("refused", ctypes.c_void_p)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libcsa.so (once).  Raises CsaLibraryMissing if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise CsaLibraryMissing(
            f"{path} is missing: build it with "
            "`python -m certified_sparse_attention_gb300.build`")
    lib = ctypes.CDLL(path)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    P = ctypes.POINTER
    lib.csa_workspace_size.argtypes = [P(csa_shape), P(csa_params)]
    lib.csa_workspace_size.restype = sz
    lib.csa_dense_workspace_size.argtypes = [P(csa_shape)]
    lib.csa_dense_workspace_size.restype = sz
    lib.csa_quantize_keys.argtypes = [P(csa_shape), vp, vp, P(ctypes.c_int64),
                                      ctypes.c_int64, vp, vp, vp, vp, vp]
    lib.csa_quantize_keys.restype = ctypes.c_int
    lib.csa_decode_step.argtypes = [P(csa_shape), P(csa_params), vp, vp, vp,
                                    vp, vp, vp, vp, P(ctypes.c_int64),
                                    P(ctypes.c_uint64), vp, vp, vp, vp, vp,
                                    vp, sz, vp]
    lib.csa_decode_step.restype = ctypes.c_int
    lib.csa_decode_step_device.argtypes = [P(csa_shape), P(csa_params), vp,
                                           vp, vp, vp, vp, vp, vp, vp, vp,
                                           ctypes.c_int, vp, vp, vp, vp, vp,
                                           vp, sz, vp]
    lib.csa_decode_step_device.restype = ctypes.c_int
    lib.csa_quantize_keys8.argtypes = [P(csa_shape), vp, P(ctypes.c_int64),
                                       ctypes.c_int64, vp, vp, vp]
    lib.csa_quantize_keys8.restype = ctypes.c_int
    lib.csa_decode_step_refined.argtypes = [P(csa_shape), P(csa_params), vp,
                                            vp, vp, vp, vp, vp, vp, vp, vp,
                                            P(ctypes.c_int64),
                                            P(ctypes.c_uint64), vp, vp, vp,
                                            vp, vp, vp, sz, vp]
    lib.csa_decode_step_refined.restype = ctypes.c_int
    lib.csa_dense_decode.argtypes = [P(csa_shape), vp, vp, vp,
                                     P(ctypes.c_int64), vp, vp, sz, vp]
    lib.csa_dense_decode.restype = ctypes.c_int
    lib.csa_dense_decode_static.argtypes = [P(csa_shape), vp, vp, vp,
                                            P(ctypes.c_int64), vp, vp]
    lib.csa_dense_decode_static.restype = ctypes.c_int
    lib.csa_rope_turns.argtypes = [P(ctypes.c_double), ctypes.c_int,
                                   P(ctypes.c_uint64)]
    lib.csa_rope_turns.restype = ctypes.c_int
    lib.csa_qk_norm_rope.argtypes = [P(csa_shape), ctypes.c_int,
                                     P(csa_norm_rope), vp, P(csa_strides), vp,
                                     P(csa_strides), vp, P(csa_strides), vp,
                                     vp, vp, vp, vp, ctypes.c_int, vp, vp]
    lib.csa_qk_norm_rope.restype = ctypes.c_int
    lib.csa_kv4_append.argtypes = [P(csa_shape), P(csa_kv4), ctypes.c_int, vp,
                                   P(csa_strides), vp, P(csa_strides), vp, vp,
                                   vp, vp]
    lib.csa_kv4_append.restype = ctypes.c_int
    lib.csa_kv4_unpack.argtypes = [P(csa_shape), P(csa_kv4), ctypes.c_int64,
                                   vp, vp, vp, vp, vp, vp]
    lib.csa_kv4_unpack.restype = ctypes.c_int
    lib.csa_kv4_workspace_size.argtypes = [P(csa_shape), ctypes.c_int]
    lib.csa_kv4_workspace_size.restype = sz
    lib.csa_kv4_decode.argtypes = [P(csa_shape), P(csa_kv4), ctypes.c_int, vp,
                                   P(csa_strides), vp, vp, vp, vp, vp, sz, vp]
    lib.csa_kv4_decode.restype = ctypes.c_int
    lib.csa_check.argtypes = [vp, vp]
    lib.csa_check.restype = ctypes.c_int
    lib.csa_workspace_layout.argtypes = [P(csa_shape), P(csa_params),
                                         P(csa_workspace_map)]
    lib.csa_workspace_layout.restype = ctypes.c_int
    lib.csa_profile_enable.argtypes = [ctypes.c_int]
    lib.csa_profile_enable.restype = ctypes.c_int
    lib.csa_profile_read.argtypes = [P(csa_phase_times)]
    lib.csa_profile_read.restype = ctypes.c_int
    lib.csa_status_string.argtypes = [ctypes.c_int]
    lib.csa_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(s: int) -> str:
    return load_library().csa_status_string(int(s)).decode()


# ------------------------------------------------------------ marshalling

def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _i64(xs: Sequence[int]):
    return (ctypes.c_int64 * len(xs))(*[int(x) for x in xs])


def _u64(xs: Sequence[int]):
    return (ctypes.c_uint64 * len(xs))(*[int(x) & 0xFFFFFFFFFFFFFFFF
                                         for x in xs])


def make_shape(B, Hq, Hkv, d, n_max, dtype) -> csa_shape:
    if not isinstance(dtype, int):
        dtype = CSA_F32 if str(dtype) in ("f32", "float32",
                                          "torch.float32") else CSA_BF16
    return csa_shape(int(B), int(Hq), int(Hkv), int(d), int(n_max), dtype)


def make_params(eps=0.05, delta=0.05, r=2, measure=CSA_MEASURE_VALUE,
                J_override=-1, sub_batches=0, perturb=0,
                qcode=0, refine8=0, dots=0) -> csa_params:
    return csa_params(float(eps), float(delta), int(r), int(measure),
                      int(J_override), int(sub_batches), int(perturb),
                      int(qcode), int(refine8), int(dots))


def csa_workspace_size(shape: csa_shape, params: csa_params) -> int:
    return int(load_library().csa_workspace_size(ctypes.byref(shape),
                                                 ctypes.byref(params)))


def csa_dense_workspace_size(shape: csa_shape) -> int:
    return int(load_library().csa_dense_workspace_size(ctypes.byref(shape)))


def csa_workspace_layout(shape: csa_shape, params: csa_params):
    m = csa_workspace_map()
    check(load_library().csa_workspace_layout(ctypes.byref(shape),
                                              ctypes.byref(params),
                                              ctypes.byref(m)),
          "csa_workspace_layout")
    return m


def decode_ordered(u):
    """Ordered-integer encoding of the maxima (csa_workspace_map.cmax) back
    to float32 values (numpy uint32 array in, float32 array out)."""
    import numpy as np
    u = np.asarray(u, dtype=np.uint32)
    bits = np.where(u >= np.uint32(0x80000000), u & np.uint32(0x7FFFFFFF),
                    ~u).astype(np.uint32)
    return bits.view(np.float32)


def csa_quantize_keys(shape, K, V, lens, from_token, K4, bounds, vmax,
                      vnorm2, stream=None) -> int:
    _check_batch(shape, lens)
    return load_library().csa_quantize_keys(
        ctypes.byref(shape), _ptr(K), _ptr(V), _i64(lens), int(from_token),
        _ptr(K4), _ptr(bounds), _ptr(vmax), _ptr(vnorm2), _stream(stream))


def csa_decode_step(shape, params, q, K, V, K4, bounds, vmax, vnorm2, lens,
                    seeds, o, beta, level, keys_read, stats, workspace,
                    workspace_bytes, stream=None) -> int:
    _check_batch(shape, lens, seeds)
    return load_library().csa_decode_step(
        ctypes.byref(shape), ctypes.byref(params), _ptr(q), _ptr(K), _ptr(V),
        _ptr(K4), _ptr(bounds), _ptr(vmax), _ptr(vnorm2), _i64(lens),
        _u64(seeds), _ptr(o),
        _ptr(beta), _ptr(level), _ptr(keys_read), _ptr(stats),
        _ptr(workspace), int(workspace_bytes), _stream(stream))


def csa_quantize_keys8(shape, K, lens, from_token, K8, delta8,
                       stream=None) -> int:
    _check_batch(shape, lens)
    return load_library().csa_quantize_keys8(
        ctypes.byref(shape), _ptr(K), _i64(lens), int(from_token), _ptr(K8),
        _ptr(delta8), _stream(stream))


def meta8_buffers(shape: csa_shape, device):
    """(K8, delta8) device tensors for csa_quantize_keys8 (the 8-bit tier)."""
    import torch
    nblk = (shape.n_max + BLOCK - 1) // BLOCK
    K8 = torch.zeros((shape.B, shape.Hkv, nblk * BLOCK, shape.d),
                     dtype=torch.uint8, device=device)
    d8 = torch.zeros((shape.B, shape.Hkv, nblk, shape.d), dtype=torch.float32,
                     device=device)
    return K8, d8


def csa_decode_step_refined(shape, params, q, K, V, K4, bounds, vmax, vnorm2,
                            K8, delta8, lens, seeds, o, beta, level,
                            keys_read, stats, workspace, workspace_bytes,
                            stream=None) -> int:
    _check_batch(shape, lens, seeds)
    return load_library().csa_decode_step_refined(
        ctypes.byref(shape), ctypes.byref(params), _ptr(q), _ptr(K), _ptr(V),
        _ptr(K4), _ptr(bounds), _ptr(vmax), _ptr(vnorm2), _ptr(K8),
        _ptr(delta8), _i64(lens), _u64(seeds), _ptr(o), _ptr(beta),
        _ptr(level), _ptr(keys_read), _ptr(stats), _ptr(workspace),
        int(workspace_bytes), _stream(stream))


def csa_decode_step_device(shape, params, q, K, V, K4, bounds, vmax, vnorm2,
                           lens_dev, seeds_dev, requantize_last, o, beta,
                           level, keys_read, stats, workspace,
                           workspace_bytes, stream=None) -> int:
    """lens_dev: device int64 [B]; seeds_dev: device uint64 (or int64) [B]."""
    return load_library().csa_decode_step_device(
        ctypes.byref(shape), ctypes.byref(params), _ptr(q), _ptr(K), _ptr(V),
        _ptr(K4), _ptr(bounds), _ptr(vmax), _ptr(vnorm2), _ptr(lens_dev),
        _ptr(seeds_dev), int(requantize_last), _ptr(o), _ptr(beta),
        _ptr(level), _ptr(keys_read), _ptr(stats), _ptr(workspace),
        int(workspace_bytes), _stream(stream))


def csa_dense_decode(shape, q, K, V, lens, o, workspace, workspace_bytes,
                     stream=None) -> int:
    _check_batch(shape, lens)
    return load_library().csa_dense_decode(
        ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(V), _i64(lens), _ptr(o),
        _ptr(workspace), int(workspace_bytes), _stream(stream))


def csa_dense_decode_static(shape, q, K, V, lens, o, stream=None) -> int:
    _check_batch(shape, lens)
    return load_library().csa_dense_decode_static(
        ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(V), _i64(lens), _ptr(o),
        _stream(stream))


def _strides(t) -> Optional[csa_strides]:
    """The (b, t, h) element strides of a [B][T][heads][d] tensor."""
    if t is None or isinstance(t, csa_strides):
        return t
    st = t.stride()
    return csa_strides(st[0], st[1], st[2])


def _ref(s):
    return None if s is None else ctypes.byref(s)


def csa_rope_turns(inv_freq) -> list:
    """The table csa_qk_norm_rope reads (host list of ints below 2^64) for
    the pairs' angles per position, in radians."""
    n = len(inv_freq)
    out = (ctypes.c_uint64 * n)()
    check(load_library().csa_rope_turns(
        (ctypes.c_double * n)(*[float(f) for f in inv_freq]), n, out),
        "csa_rope_turns")
    return list(out)


def csa_qk_norm_rope(shape, T, params, q, qs, k, ks, v, vs, lens_dev, n_new,
                     q_out, K, V, to_cache, status, stream=None) -> int:
    """params: csa_norm_rope; qs, ks, vs: csa_strides or the strided
    tensors; lens_dev, n_new: device int64 [B] (n_new None: T each)."""
    return load_library().csa_qk_norm_rope(
        ctypes.byref(shape), int(T), ctypes.byref(params), _ptr(q),
        _ref(_strides(qs)), _ptr(k), _ref(_strides(ks)), _ptr(v),
        _ref(_strides(vs)), _ptr(lens_dev), _ptr(n_new), _ptr(q_out),
        _ptr(K), _ptr(V), int(to_cache), _ptr(status), _stream(stream))


def csa_kv4_append(shape, cache, T, k, ks, v, vs, lens_dev, n_new, status,
                   stream=None) -> int:
    """cache: csa_kv4; the other arguments as csa_qk_norm_rope."""
    return load_library().csa_kv4_append(
        ctypes.byref(shape), ctypes.byref(cache), int(T), _ptr(k),
        _ref(_strides(ks)), _ptr(v), _ref(_strides(vs)), _ptr(lens_dev),
        _ptr(n_new), _ptr(status), _stream(stream))


def csa_kv4_unpack(shape, cache, rows, first, lens_dev, K, V, status,
                   stream=None) -> int:
    return load_library().csa_kv4_unpack(
        ctypes.byref(shape), ctypes.byref(cache), int(rows), _ptr(first),
        _ptr(lens_dev), _ptr(K), _ptr(V), _ptr(status), _stream(stream))


def csa_kv4_workspace_size(shape: csa_shape, T: int = 1) -> int:
    return int(load_library().csa_kv4_workspace_size(ctypes.byref(shape),
                                                     int(T)))


def csa_kv4_decode(shape, cache, T, q, qs, lens_dev, n_q, o, lse, workspace,
                   workspace_bytes, stream=None) -> int:
    return load_library().csa_kv4_decode(
        ctypes.byref(shape), ctypes.byref(cache), int(T), _ptr(q),
        _ref(_strides(qs)), _ptr(lens_dev), _ptr(n_q), _ptr(o), _ptr(lse),
        _ptr(workspace), int(workspace_bytes), _stream(stream))


def csa_profile_enable(on: bool) -> int:
    return load_library().csa_profile_enable(1 if on else 0)


def csa_profile_read() -> dict:
    """Accumulated ms per phase since the last read, steps, launches."""
    t = csa_phase_times()
    check(load_library().csa_profile_read(ctypes.byref(t)),
          "csa_profile_read")
    return {"ms": dict(zip(PHASES, list(t.ms))), "steps": int(t.steps),
            "launches": int(t.launches)}


def csa_check(workspace, stream=None) -> int:
    return load_library().csa_check(_ptr(workspace), _stream(stream))


def check(status: int, where: str = "csa") -> None:
    if status != CSA_OK:
        raise CsaError(status, where)


# ---------------------------------------------------- tensor conveniences

class KVMeta(NamedTuple):
    """Device metadata csa_quantize_keys writes and csa_decode_step reads."""
    K4: object
    bounds: object
    vmax: object
    vnorm2: object


def meta_buffers(shape: csa_shape, device) -> KVMeta:
    """Allocate K4, bounds, vmax, vnorm2 (torch, device) for a shape."""
    import torch
    nblk = (shape.n_max + BLOCK - 1) // BLOCK
    K4 = torch.zeros((shape.B, shape.Hkv, nblk * BLOCK, shape.d // 2),
                     dtype=torch.uint8, device=device)
    bounds = torch.zeros((shape.B, shape.Hkv, nblk, 2, shape.d),
                         dtype=torch.float32, device=device)
    vmax = torch.zeros((shape.B, shape.Hkv, nblk), dtype=torch.float32,
                       device=device)
    vnorm2 = torch.zeros((shape.B, shape.Hkv, shape.n_max),
                         dtype=torch.float32, device=device)
    return KVMeta(K4, bounds, vmax, vnorm2)


def _require(t, name: str, nbytes: int) -> None:
    """Refuse a tensor the kernels would read from host memory or past its
    end: it must be a contiguous CUDA tensor of at least ``nbytes``."""
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name}: a CUDA tensor is required")
    if not t.is_contiguous():
        raise ValueError(f"{name}: the tensor must be contiguous")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name}: {have} bytes, the shape needs {nbytes}")


def _check_batch(shape: csa_shape, lens, seeds=None) -> None:
    if len(lens) != shape.B:
        raise ValueError(f"lens: {len(lens)} entries for B = {shape.B}")
    if seeds is not None and len(seeds) != shape.B:
        raise ValueError(f"seeds: {len(seeds)} entries for B = {shape.B}")


def check_step_inputs(shape: csa_shape, q, K, V, meta=None, lens=(),
                      seeds=None) -> None:
    """Host-side checks of the tensors and host arrays a decode step (or,
    without ``meta``, a dense decode) reads: the layouts of include/csa.h,
    on the device, contiguous and large enough.  Raises ValueError."""
    B, Hq, Hkv, d, n = shape.B, shape.Hq, shape.Hkv, shape.d, shape.n_max
    esz = 4 if shape.dtype == CSA_F32 else 2
    nblk = (n + BLOCK - 1) // BLOCK
    _check_batch(shape, lens, seeds)
    _require(q, "q", B * Hq * d * esz)
    _require(K, "K", B * Hkv * n * d * esz)
    _require(V, "V", B * Hkv * n * d * esz)
    if meta is not None:
        _require(meta.K4, "K4", B * Hkv * nblk * BLOCK * (d // 2))
        _require(meta.bounds, "bounds", B * Hkv * nblk * 2 * d * 4)
        _require(meta.vmax, "vmax", B * Hkv * nblk * 4)
        _require(meta.vnorm2, "vnorm2", B * Hkv * n * 4)


class DecodeStep:
    """Owns the workspace and output buffers of csa_decode_step for one
    shape and parameter set; ``__call__`` runs one step on the current
    stream (asynchronously)."""

    def __init__(self, shape: csa_shape, params: csa_params, device,
                 with_stats: bool = False):
        import torch
        self.shape, self.params = shape, params
        nbytes = csa_workspace_size(shape, params)
        if nbytes == 0:
            raise CsaError(1, "csa_workspace_size")
        self.ws_bytes = nbytes
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        B, Hq, d = shape.B, shape.Hq, shape.d
        # the four outputs are views of one buffer (``outputs``), so that a
        # caller reads a step's results back with a single copy
        nh = B * Hq
        self.outputs = torch.empty((nh * (d + 3),), dtype=torch.float32,
                                   device=device)
        self.o = self.outputs[:nh * d].view(B, Hq, d)
        self.beta = self.outputs[nh * d:nh * (d + 1)].view(B, Hq)
        self.level = self.outputs[nh * (d + 1):nh * (d + 2)].view(
            torch.int32).view(B, Hq)
        self.keys_read = self.outputs[nh * (d + 2):].view(
            torch.int32).view(B, Hq)
        self.stats = (torch.zeros((B, Hq, STATS_FIELDS), dtype=torch.int32,
                                  device=device) if with_stats else None)

    def __call__(self, q, K, V, meta: KVMeta, lens, seeds, stream=None,
                 meta8=None):
        """meta8: (K8, delta8) of the 8-bit tier, required when the
        parameters ask for it (csa_decode_step_refined)."""
        check_step_inputs(self.shape, q, K, V, meta, lens, seeds)
        if self.params.refine8:
            if meta8 is None:
                raise ValueError("refine8: the 8-bit codes (meta8) are needed")
            nblk = (self.shape.n_max + BLOCK - 1) // BLOCK
            n8 = self.shape.B * self.shape.Hkv * nblk
            _require(meta8[0], "K8", n8 * BLOCK * self.shape.d)
            _require(meta8[1], "delta8", n8 * self.shape.d * 4)
            st = csa_decode_step_refined(
                self.shape, self.params, q, K, V, meta.K4, meta.bounds,
                meta.vmax, meta.vnorm2, meta8[0], meta8[1], lens, seeds,
                self.o, self.beta, self.level, self.keys_read, self.stats,
                self.ws, self.ws_bytes, stream)
            check(st, "csa_decode_step_refined")
        else:
            st = csa_decode_step(self.shape, self.params, q, K, V, meta.K4,
                                 meta.bounds, meta.vmax, meta.vnorm2, lens,
                                 seeds, self.o, self.beta, self.level,
                                 self.keys_read, self.stats, self.ws,
                                 self.ws_bytes, stream)
            check(st, "csa_decode_step")
        return self.o, self.beta, self.level, self.keys_read

    def device_step(self, q, K, V, meta: KVMeta, lens_dev, seeds_dev,
                    requantize_last: bool = True, stream=None):
        """The step with lengths and seeds read from device tensors (int64
        [B] each), optionally re-quantising the block of the token just
        appended; capturable into a CUDA graph that is replayed with new
        lengths and seeds written into the same tensors."""
        check_step_inputs(self.shape, q, K, V, meta, [1] * self.shape.B)
        for t, name in ((lens_dev, "lens_dev"), (seeds_dev, "seeds_dev")):
            _require(t, name, 8 * self.shape.B)
        st = csa_decode_step_device(self.shape, self.params, q, K, V,
                                    meta.K4, meta.bounds, meta.vmax,
                                    meta.vnorm2, lens_dev, seeds_dev,
                                    1 if requantize_last else 0, self.o,
                                    self.beta, self.level, self.keys_read,
                                    self.stats, self.ws, self.ws_bytes,
                                    stream)
        check(st, "csa_decode_step_device")
        return self.o, self.beta, self.level, self.keys_read


class DenseDecode:
    """Owns the workspace of csa_dense_decode for one shape."""

    def __init__(self, shape: csa_shape, device):
        import torch
        self.shape = shape
        self.ws_bytes = csa_dense_workspace_size(shape)
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8,
                              device=device)
        self.o = torch.empty((shape.B, shape.Hq, shape.d),
                             dtype=torch.float32, device=device)

    def __call__(self, q, K, V, lens, stream=None):
        check_step_inputs(self.shape, q, K, V, None, lens)
        check(csa_dense_decode(self.shape, q, K, V, lens, self.o, self.ws,
                               self.ws_bytes, stream), "csa_dense_decode")
        return self.o


# ------------------------------------- rows before the cache, 4-bit cache

# For inference: no gradient flows through these calls.

# The checks below run on every call of a decode loop, where the calls of a
# token take the device a few microseconds each: they look at each tensor's
# shape, strides, type, device and address once.

def _torch_type(shape: csa_shape):
    import torch
    return torch.float32 if shape.dtype == CSA_F32 else torch.bfloat16


def _call_stream(stream, device: int) -> Optional[int]:
    """The stream handle of a call on GPU ``device``, which must be the
    current one (the library launches there): the given stream, or the
    current one (asked for by its raw handle: torch.cuda.current_stream()
    makes an object, 3 us)."""
    import torch
    have = torch.cuda.current_device()
    if have != device:
        raise ValueError(f"the buffers lie on CUDA device {device}, the "
                         f"current device is {have}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return _stream(stream)


def _rows(t, name: str, B: int, T: int, heads: int, d: int, dtype,
          device: int):
    """Check a strided [B][T][heads][d] operand (T 0: any); its address and
    its (b, t, h) strides."""
    sz = t.shape
    if len(sz) != 4 or sz[0] != B or sz[2] != heads or sz[3] != d or \
            (sz[1] != T if T else sz[1] < 1):
        raise ValueError(f"{name}: shape {list(sz)}, [{B}][{T or 'T'}]"
                         f"[{heads}][{d}] is required")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {t.dtype}, {dtype} is required")
    if t.get_device() != device:
        raise ValueError(f"{name}: a tensor on CUDA device {device} is "
                         "required")
    sb, st, sh, sc = t.stride()
    p, esz = t.data_ptr(), t.element_size()
    if sc != 1 or ((sb | st | sh) * esz | p) & 15:
        # (the stride of an axis of length one is never used)
        if sc != 1 or p & 15 or any(n > 1 and s * esz & 15 for n, s in
                                    zip(sz, (sb, st, sh))):
            raise ValueError(f"{name}: channels must be contiguous and rows "
                             "start at multiples of 16 bytes")
    return p, sb, st, sh


def _whole(t, name: str, size: tuple, dtype, device: int) -> int:
    """Check a contiguous tensor of this size, aligned to 16 bytes; its
    address."""
    if t.shape != size or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name}: {t.dtype} {list(t.shape)}, a contiguous "
                         f"{dtype} tensor {list(size)} is required")
    if t.get_device() != device:
        raise ValueError(f"{name}: a tensor on CUDA device {device} is "
                         "required")
    p = t.data_ptr()
    if p & 15:
        raise ValueError(f"{name}: must start at a multiple of 16 bytes")
    return p


def _counts(t, name: str, B: int, device: int) -> Optional[int]:
    """Check a device int64 [B] (or None); its address."""
    if t is None:
        return None
    ty = t.dtype
    if ty.itemsize != 8 or ty.is_floating_point or ty.is_complex or \
            not ty.is_signed or t.shape != (B,) or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int64 tensor [{B}] is "
                         "required")
    if t.get_device() != device:
        raise ValueError(f"{name}: a tensor on CUDA device {device} is "
                         "required")
    return t.data_ptr()


def _settled(device: int) -> None:
    """Wait for what a constructor has sent to its device (buffers set to
    zero, tables): a first call on another stream would not."""
    import torch
    if device >= 0 and not torch.cuda.is_current_stream_capturing():
        torch.cuda.current_stream(device).synchronize()


class QKNormRope:
    """Per-head norms of queries and keys with the position rotation
    (csa_qk_norm_rope), for one shape and set of weights.

    wq, wk: norm weights [d] of the shape's type (None: no norm of that
    side); inv_freq: the rotated pairs' angles per position in radians (2 x
    their number = the rotated channels, a multiple of 8; None: no
    rotation); interleaved: pair i is channels (2i, 2i + 1) instead of (i,
    i + rot_dim / 2).  ``status`` is the device word csa_check reads; each
    call sets it anew."""

    def __init__(self, shape: csa_shape, device, wq=None, wk=None,
                 norm_eps: float = 1e-6, inv_freq=None,
                 interleaved: bool = False):
        import torch
        self.shape = shape
        self.dtype = _torch_type(shape)
        self.status = torch.zeros(4, dtype=torch.int32, device=device)
        self.device = self.status.get_device()
        table = [] if inv_freq is None else csa_rope_turns(inv_freq)
        if len(table) * 2 > shape.d or len(table) % 4:
            raise ValueError(f"inv_freq: {len(table)} pairs; a multiple of 4 "
                             f"up to {shape.d // 2} is required")
        self.turns = torch.tensor(
            [u - (1 << 64) if u >> 63 else u for u in table],
            dtype=torch.int64, device=device) if table else None
        pw = [None if w is None else
              _whole(w, name, (shape.d,), self.dtype, self.device)
              for name, w in (("wq", wq), ("wk", wk))]
        self.weights = (wq, wk)
        self.params = csa_norm_rope(
            pw[0], pw[1], float(norm_eps), 2 * len(table),
            1 if interleaved else 0, _ptr(self.turns))
        _settled(self.device)

    def __call__(self, q, k, v, K, V, lens_dev, n_new=None,
                 to_cache: bool = True, q_out=None, stream=None):
        """q [B][T][Hq][d], k and v [B][T][Hkv][d] (views with any strides
        of whole 16 bytes; v and V None: no values); K, V: the cache
        [B][Hkv][n_max][d], or with to_cache=False rows [B][T][Hkv][d].
        lens_dev: device int64 [B], the new tokens counted already; n_new:
        device int64 [B] (None: T each).  Returns q_out [B][T][Hq][d] (made
        when not given, on the current stream: needed with ``stream``, where
        that memory may still be in use)."""
        s, dev, dt = self.shape, self.device, self.dtype
        B, Hq, Hkv, d = s.B, s.Hq, s.Hkv, s.d
        pq, qb, qt, qh = _rows(q, "q", B, 0, Hq, d, dt, dev)
        T = q.shape[1]
        pk, kb, kt, kh = _rows(k, "k", B, T, Hkv, d, dt, dev)
        size = (B, Hkv, s.n_max, d) if to_cache else (B, T, Hkv, d)
        pK = _whole(K, "K", size, dt, dev)
        pv = pV = vs = None
        if v is not None:
            if V is None:
                raise ValueError("V: missing")
            pv, vb, vt, vh = _rows(v, "v", B, T, Hkv, d, dt, dev)
            pV = _whole(V, "V", size, dt, dev)
            vs = ctypes.byref(csa_strides(vb, vt, vh))
        elif V is not None:
            raise ValueError("V: given without v")
        pl = _counts(lens_dev, "lens_dev", B, dev)
        pn = _counts(n_new, "n_new", B, dev)
        if q_out is None:
            if stream is not None:
                raise ValueError("q_out: required when a stream is given")
            q_out = q.new_empty((B, T, Hq, d))
        po = _whole(q_out, "q_out", (B, T, Hq, d), dt, dev)
        st = load_library().csa_qk_norm_rope(
            ctypes.byref(s), T, ctypes.byref(self.params), pq,
            ctypes.byref(csa_strides(qb, qt, qh)), pk,
            ctypes.byref(csa_strides(kb, kt, kh)), pv, vs, pl, pn, po, pK,
            pV, 1 if to_cache else 0, self.status.data_ptr(),
            _call_stream(stream, dev))
        if st:
            raise CsaError(st, "csa_qk_norm_rope")
        return q_out


class KV4Cache:
    """Device buffers of a K/V cache held in 4 bits (csa_kv4), for one
    shape: K4, bounds, V4, vscale of the whole blocks of 64 tokens, Kt, Vt
    the rows of the incomplete last one.  buffers: those six tensors, in
    that order, instead of new ones.  ``status`` is the device word
    csa_check reads after append or unpack, which each set it anew;
    ``refused`` the one an append that had to leave a sequence out flags and
    nothing clears (``refused.zero_()`` does): checked at any later time,
    csa_check(cache.refused) tells whether every append went in."""

    def __init__(self, shape: csa_shape, device, buffers=None):
        import torch
        self.shape = shape
        if csa_kv4_workspace_size(shape, 1) == 0:
            raise CsaError(2, "KV4Cache")
        B, H, d = shape.B, shape.Hkv, shape.d
        nblk = (shape.n_max + BLOCK - 1) // BLOCK
        self.dtype = el = _torch_type(shape)
        layout = (("K4", (B, H, nblk * BLOCK, d // 2), torch.uint8),
                  ("bounds", (B, H, nblk, 2, d), torch.float32),
                  ("V4", (B, H, nblk, d, BLOCK // 2), torch.uint8),
                  ("vscale", (B, H, nblk * BLOCK, 2), torch.float32),
                  ("Kt", (B, H, BLOCK, d), el), ("Vt", (B, H, BLOCK, d), el))
        self.status = torch.zeros(4, dtype=torch.int32, device=device)
        self.refused = torch.zeros(4, dtype=torch.int32, device=device)
        self.device = self.status.get_device()
        if buffers is None:
            buffers = [torch.zeros(size, dtype=dt, device=device)
                       for _, size, dt in layout]
        if len(buffers) != len(layout):
            raise ValueError("buffers: K4, bounds, V4, vscale, Kt and Vt "
                             "are required")
        at = []
        for (name, size, dt), t in zip(layout, buffers):
            n = 1
            for x in size:
                n *= x
            if t.numel() != n or not t.is_contiguous():
                raise ValueError(f"{name}: a contiguous tensor {list(size)} "
                                 "is required")
            t = t.view(size)
            at.append(_whole(t, name, size, dt, self.device))
            setattr(self, name, t)
        self.desc = csa_kv4(*at, self.refused.data_ptr())
        _settled(self.device)

    def append(self, k, v, lens_dev, n_new=None, stream=None) -> None:
        """Append rows k, v [B][T][Hkv][d] (views with any strides of whole
        16 bytes): n_new[b] <= T of sequence b (None: T each), which
        lens_dev counts already (device int64 [B])."""
        s, dev, dt = self.shape, self.device, self.dtype
        B, H, d = s.B, s.Hkv, s.d
        pk, kb, kt, kh = _rows(k, "k", B, 0, H, d, dt, dev)
        T = k.shape[1]
        pv, vb, vt, vh = _rows(v, "v", B, T, H, d, dt, dev)
        pl = _counts(lens_dev, "lens_dev", B, dev)
        pn = _counts(n_new, "n_new", B, dev)
        st = load_library().csa_kv4_append(
            ctypes.byref(s), ctypes.byref(self.desc), T, pk,
            ctypes.byref(csa_strides(kb, kt, kh)), pv,
            ctypes.byref(csa_strides(vb, vt, vh)), pl, pn,
            self.status.data_ptr(), _call_stream(stream, dev))
        if st:
            raise CsaError(st, "csa_kv4_append")

    def unpack(self, K, V, lens_dev, first=None, stream=None):
        """Read positions first[b] + i (None: from 0) below lens_dev[b] back
        into row i of K, V (contiguous [B][Hkv][rows][d]); other rows are
        left as they are.  Returns (K, V)."""
        s, dev, dt = self.shape, self.device, self.dtype
        if len(K.shape) != 4 or K.shape[2] < 1:
            raise ValueError(f"K: [{s.B}][{s.Hkv}][rows][{s.d}] is required")
        size = (s.B, s.Hkv, K.shape[2], s.d)
        pK = _whole(K, "K", size, dt, dev)
        pV = _whole(V, "V", size, dt, dev)
        pl = _counts(lens_dev, "lens_dev", s.B, dev)
        pf = _counts(first, "first", s.B, dev)
        st = load_library().csa_kv4_unpack(
            ctypes.byref(s), ctypes.byref(self.desc), size[2], pf, pl, pK,
            pV, self.status.data_ptr(), _call_stream(stream, dev))
        if st:
            raise CsaError(st, "csa_kv4_unpack")
        return K, V


class KV4Decode:
    """Owns the workspace and outputs of csa_kv4_decode for one shape and up
    to T query tokens per sequence: o [B][T][Hq][d] (float32) and, with
    with_lse, lse [B][T][Hq].  One object serves one call at a time."""

    def __init__(self, shape: csa_shape, device, T: int = 1,
                 with_lse: bool = False):
        import torch
        self.shape, self.T = shape, int(T)
        self.dtype = _torch_type(shape)
        self.ws_bytes = csa_kv4_workspace_size(shape, self.T)
        if self.ws_bytes == 0:
            raise CsaError(2, "csa_kv4_workspace_size")
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.device = self.ws.get_device()
        self.o = torch.zeros((shape.B, self.T, shape.Hq, shape.d),
                             dtype=torch.float32, device=device)
        self.lse = (torch.zeros((shape.B, self.T, shape.Hq),
                                dtype=torch.float32, device=device)
                    if with_lse else None)
        _settled(self.device)

    def __call__(self, q, cache: KV4Cache, lens_dev, n_q=None, stream=None):
        """q [B][T][Hq][d] (a view with strides of whole 16 bytes); lens_dev
        and n_q: device int64 [B] (n_q None: T each).  Returns o."""
        s, c, dev = self.shape, cache.shape, self.device
        if c.B != s.B or c.Hkv != s.Hkv or c.d != s.d or \
                c.n_max != s.n_max or c.dtype != s.dtype or \
                cache.device != dev:
            raise ValueError("cache: made for another shape or device")
        pq, qb, qt, qh = _rows(q, "q", s.B, self.T, s.Hq, s.d, self.dtype,
                               dev)
        pl = _counts(lens_dev, "lens_dev", s.B, dev)
        pn = _counts(n_q, "n_q", s.B, dev)
        st = load_library().csa_kv4_decode(
            ctypes.byref(s), ctypes.byref(cache.desc), self.T, pq,
            ctypes.byref(csa_strides(qb, qt, qh)), pl, pn,
            self.o.data_ptr(), _ptr(self.lse), self.ws.data_ptr(),
            self.ws_bytes, _call_stream(stream, dev))
        if st:
            raise CsaError(st, "csa_kv4_decode")
        return self.o
