"""ctypes binding of libzha.so (include/zha.h): argument marshalling only.

Every step of the decode path runs in the library's CUDA kernels; this module
allocates the caller-owned device buffers with PyTorch, passes raw pointers
and the current CUDA stream, and turns error codes into exceptions.  There is
no fallback: if libzha.so is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libzha.so")

ZHA_OK, ZHA_ERR_INVALID, ZHA_ERR_CAPACITY, ZHA_ERR_UNSUPPORTED, ZHA_ERR_CUDA, ZHA_ERR_TIMEOUT = 0, -1, -2, -3, -4, -5
ZHA_F32, ZHA_BF16 = 0, 1
ZHA_PLANES_KEY, ZHA_PLANES_FP4 = 0, 1
PLANES_CODE = {"key": ZHA_PLANES_KEY, "fp4": ZHA_PLANES_FP4}
STAT_NODES_SCORED, STAT_LEAVES_KEPT, STAT_KEYS, STAT_STEPS, STAT_COUNT = 0, 1, 2, 3, 4

TORCH_DTYPE = {ZHA_F32: torch.float32, ZHA_BF16: torch.bfloat16}
DTYPE_CODE = {"f32": ZHA_F32, "bf16": ZHA_BF16, torch.float32: ZHA_F32, torch.bfloat16: ZHA_BF16}

# every function the header declares, with its ctypes signature
_c = ctypes
_SIGS = {
    "zha_tree_bytes": (_c.c_int, [_c.c_void_p, _c.POINTER(_c.c_size_t), _c.POINTER(_c.c_size_t)]),
    "zha_tree_layout": (_c.c_int, [_c.c_void_p, _c.c_int32, _c.POINTER(_c.c_size_t), _c.POINTER(_c.c_size_t),
                                   _c.POINTER(_c.c_int64), _c.POINTER(_c.c_size_t)]),
    "zha_tree_layout_fp4": (_c.c_int, [_c.c_void_p, _c.c_int32, _c.POINTER(_c.c_size_t), _c.POINTER(_c.c_size_t)]),
    "zha_tree_create": (_c.c_int, [_c.c_void_p] * 6 + [_c.POINTER(_c.c_void_p)]),
    "zha_tree_build": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_void_p]),
    "zha_tree_append": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_void_p]),
    "zha_tree_size": (_c.c_int64, [_c.c_void_p]),
    "zha_decode": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_void_p, _c.c_void_p,
                              _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_void_p]),
    "zha_route_multi": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_void_p, _c.c_void_p,
                                   _c.c_void_p]),
    "zha_decode_step_host": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                        _c.c_int32, _c.c_void_p]),
    "zha_dense_scratch_bytes": (_c.c_size_t, [_c.c_void_p, _c.c_int32, _c.c_int64]),
    "zha_dense_decode": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_void_p,
                                    _c.c_void_p, _c.c_int32, _c.c_void_p, _c.c_void_p]),
    "zha_dense_decode_noalloc": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64,
                                            _c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_void_p]),
    "zha_prefix_scratch_bytes": (_c.c_size_t, [_c.c_void_p, _c.c_int32, _c.c_int32, _c.c_int64, _c.c_int64]),
    "zha_prefix_decode": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_void_p,
                                     _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                     _c.c_int32, _c.c_int32, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "zha_weights_scratch_bytes": (_c.c_size_t, [_c.c_void_p, _c.c_int32, _c.c_int64]),
    "zha_dense_weights": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_void_p,
                                     _c.c_void_p, _c.c_int32, _c.c_int32, _c.c_void_p, _c.c_int64, _c.c_void_p,
                                     _c.c_int64, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "zha_cache_evict": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_void_p,
                                   _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_void_p,
                                   _c.c_int64, _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_size_t,
                                   _c.c_void_p]),
    "zha_evict_scratch_bytes": (_c.c_size_t, [_c.c_void_p, _c.c_int64]),
    "zha_tree_evict": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64,
                                  _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "zha_scratch_status": (_c.c_int, [_c.c_void_p, _c.c_void_p]),
    "zha_tree_status": (_c.c_int, [_c.c_void_p, _c.c_void_p]),
    "zha_tree_set_step_p": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int32]),
    "zha_tree_destroy": (None, [_c.c_void_p]),
    "zha_last_error": (_c.c_char_p, []),
    "zha_last_error_code": (_c.c_int, []),
    "zha_launch_count": (_c.c_uint64, []),
}

_lib = None


class ZhaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"zha error {code}: {msg}")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libzha.so (built in-tree); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m tree_indexed_sparse_03_b200.build_lib`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(rc: int) -> None:
    if rc != ZHA_OK:
        raise ZhaError(rc, lib().zha_last_error().decode())


class ZhaConfig(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("block", ctypes.c_int32), ("levels", ctypes.c_int32), ("n_refs", ctypes.c_int32),
                ("p", ctypes.c_float), ("dtype", ctypes.c_int32), ("capacity", ctypes.c_int64),
                ("max_batch", ctypes.c_int32), ("planes", ctypes.c_int32)]


def make_config(*, d: int, n_q_heads: int, n_kv_heads: int, block: int, levels: int, n_refs: int, p: float,
                dtype, capacity: int, max_batch: int = 1, planes: str = "key") -> ZhaConfig:
    return ZhaConfig(d, n_q_heads, n_kv_heads, block, levels, n_refs, p, DTYPE_CODE[dtype], capacity, max_batch,
                     PLANES_CODE[planes])


def _stream(stream: Optional[torch.cuda.Stream]) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def tree_bytes(cfg: ZhaConfig) -> Tuple[int, int]:
    nb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().zha_tree_bytes(ctypes.byref(cfg), ctypes.byref(nb), ctypes.byref(sb)))
    return nb.value, sb.value


@dataclass
class LevelLayout:
    rec_offset: int
    f_offset: int
    cap_nodes: int
    rec_bytes: int


def tree_layout(cfg: ZhaConfig, level: int) -> LevelLayout:
    ro, fo, rb = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    cap = ctypes.c_int64()
    _check(lib().zha_tree_layout(ctypes.byref(cfg), level, ctypes.byref(ro), ctypes.byref(fo), ctypes.byref(cap),
                                 ctypes.byref(rb)))
    return LevelLayout(ro.value, fo.value, cap.value, rb.value)


def tree_layout_fp4(cfg: ZhaConfig, level: int) -> Tuple[int, int]:
    """(byte offset, bytes per record) of the FP4 router records of a level."""
    ro, rb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().zha_tree_layout_fp4(ctypes.byref(cfg), level, ctypes.byref(ro), ctypes.byref(rb)))
    return ro.value, rb.value


class ZhaTree:
    """A tree over a caller-owned KV cache K, V [Hkv, capacity, d] (CUDA tensors)."""

    def __init__(self, cfg: ZhaConfig, K: torch.Tensor, V: torch.Tensor, refs: torch.Tensor):
        self.cfg = cfg
        dt = TORCH_DTYPE[cfg.dtype]
        shape = (cfg.n_kv_heads, cfg.capacity, cfg.d)
        for name, t in (("K", K), ("V", V)):
            if tuple(t.shape) != shape or t.dtype != dt or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor of shape {shape}")
        if (tuple(refs.shape) != (cfg.n_kv_heads, cfg.n_refs, cfg.d) or refs.dtype != dt or not refs.is_cuda
                or not refs.is_contiguous()):
            raise ValueError("refs must be a contiguous CUDA tensor [Hkv, R, d] of the cache dtype")
        self.K, self.V, self.refs = K, V, refs
        nb, sb = tree_bytes(cfg)
        self.nodes = torch.zeros(nb, dtype=torch.uint8, device=K.device)
        self.scratch = torch.zeros(sb, dtype=torch.uint8, device=K.device)
        h = ctypes.c_void_p()
        _check(lib().zha_tree_create(ctypes.byref(cfg), K.data_ptr(), V.data_ptr(), refs.data_ptr(),
                                     self.nodes.data_ptr(), self.scratch.data_ptr(), ctypes.byref(h)))
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib is not None:
            _lib.zha_tree_destroy(h)
            self._h = None

    @property
    def size(self) -> int:
        return int(lib().zha_tree_size(self._h))

    def build(self, n: int, stream=None) -> None:
        _check(lib().zha_tree_build(self._h, n, _stream(stream)))

    def append(self, K_new: torch.Tensor, V_new: torch.Tensor, stream=None) -> None:
        """Append tokens K_new, V_new [Hkv, m, d] (CUDA, cache dtype)."""
        c = self.cfg
        for name, t in (("K_new", K_new), ("V_new", V_new)):
            if (t.dim() != 3 or t.shape[0] != c.n_kv_heads or t.shape[2] != c.d or t.dtype != TORCH_DTYPE[c.dtype]
                    or not t.is_cuda):
                raise ValueError(f"{name} must be a CUDA {TORCH_DTYPE[c.dtype]} tensor [{c.n_kv_heads}, m, {c.d}]")
        if K_new.shape != V_new.shape:
            raise ValueError("K_new and V_new must have the same shape")
        m = K_new.shape[1]
        K_new = K_new.contiguous()
        V_new = V_new.contiguous()
        _check(lib().zha_tree_append(self._h, K_new.data_ptr(), V_new.data_ptr(), m, _stream(stream)))

    def decode(self, Q: torch.Tensor, *, want_kept: bool = False, want_stats: bool = False, out=None,
               scored_cap: int = 0, stream=None):
        """Decode queries Q [B, Hq, d].  Returns O [B, Hq, d] fp32 (and kept lists / stats when asked)."""
        c = self.cfg
        if Q.dim() != 3 or tuple(Q.shape[1:]) != (c.n_q_heads, c.d) or Q.dtype != TORCH_DTYPE[c.dtype] or not Q.is_cuda:
            raise ValueError(f"Q must be a CUDA {TORCH_DTYPE[c.dtype]} tensor [B, {c.n_q_heads}, {c.d}]")
        B = Q.shape[0]
        if out is not None and (tuple(out.shape) != (B, c.n_q_heads, c.d) or out.dtype != torch.float32
                                or not out.is_cuda or not out.is_contiguous()):
            raise ValueError(f"out must be a contiguous CUDA float32 tensor [{B}, {c.n_q_heads}, {c.d}]")
        Q = Q.contiguous()
        O = out if out is not None else torch.empty(B, self.cfg.n_q_heads, self.cfg.d, dtype=torch.float32,
                                                    device=Q.device)
        kept = cnt = stats = None
        if want_kept:
            kept = torch.full((B, self.cfg.n_q_heads, max(1, self.cfg.capacity // self.cfg.block)), -1,
                              dtype=torch.int32, device=Q.device)
            cnt = torch.zeros(B, self.cfg.n_q_heads, dtype=torch.int32, device=Q.device)
        if want_stats:
            stats = torch.zeros(B, self.cfg.n_q_heads, STAT_COUNT, dtype=torch.int64, device=Q.device)
        scored = None
        if scored_cap > 0:
            scored = torch.full((B, self.cfg.n_q_heads, scored_cap), -1, dtype=torch.int32, device=Q.device)
        _check(lib().zha_decode(self._h, Q.data_ptr(), O.data_ptr(), B, _ptr(kept), _ptr(cnt), _ptr(stats),
                                _ptr(scored), scored_cap, _stream(stream)))
        if not (want_kept or want_stats or scored is not None):
            return O
        res = [O]
        if want_kept:
            res.append((kept, cnt))
        if want_stats:
            res.append(stats)
        if scored is not None:
            res.append(scored)
        return tuple(res)

    def route_multi(self, Q: torch.Tensor, *, want_kept: bool = False, stream=None):
        """Route and attend m queries Q [m, Hq, d] of this context (zha_route_multi).  Returns O [m, Hq, d] fp32
        (and (kept, kept_cnt) when asked)."""
        c = self.cfg
        if Q.dim() != 3 or tuple(Q.shape[1:]) != (c.n_q_heads, c.d) or Q.dtype != TORCH_DTYPE[c.dtype] or not Q.is_cuda:
            raise ValueError(f"Q must be a CUDA {TORCH_DTYPE[c.dtype]} tensor [m, {c.n_q_heads}, {c.d}]")
        m = Q.shape[0]
        Q = Q.contiguous()
        O = torch.empty(m, c.n_q_heads, c.d, dtype=torch.float32, device=Q.device)
        kept = cnt = None
        if want_kept:
            kept = torch.full((m, c.n_q_heads, max(1, c.capacity // c.block)), -1, dtype=torch.int32, device=Q.device)
            cnt = torch.zeros(m, c.n_q_heads, dtype=torch.int32, device=Q.device)
        _check(lib().zha_route_multi(self._h, Q.data_ptr(), O.data_ptr(), m, _ptr(kept), _ptr(cnt), _stream(stream)))
        return (O, (kept, cnt)) if want_kept else O

    def decode_step_host(self, k_host: Optional[torch.Tensor], v_host: Optional[torch.Tensor], q_host: torch.Tensor,
                         o_host: torch.Tensor, stream=None) -> None:
        """One decode step from (pinned) host tensors; o_host [B, Hq, d] fp32 receives the output."""
        B = q_host.shape[0]
        _check(lib().zha_decode_step_host(self._h, _ptr(k_host), _ptr(v_host), q_host.data_ptr(), o_host.data_ptr(),
                                          B, _stream(stream)))

    def evict(self, acc: torch.Tensor, keep: int, *, first: int = 0, last: int = 0, stream=None) -> torch.Tensor:
        """Shorten the cache to `keep` tokens per KV head by the sums acc [Hkv, >= size] (fp32, shortened in place;
        see cache_evict) and rebuild the tree over them.  Returns the kept tokens' positions [Hkv, keep] int32."""
        c = self.cfg
        n = self.size
        if not 1 <= keep <= n:
            raise ValueError(f"keep must be in [1, {n}]")
        ld_acc = _sums_ld("acc", acc, c.n_kv_heads, n)
        dev = torch.cuda.current_device()
        if acc.get_device() != dev or self.K.get_device() != dev:
            _refuse_device("the cache and acc")
        idx = _empty(acc, (c.n_kv_heads, keep), torch.int32, stream)
        work, nbytes = _evict_scratch(c, acc, n, stream)
        _record(stream, dev, acc, self.K, self.V, self.refs, self.nodes, self.scratch)
        _check(lib().zha_tree_evict(self._h, acc.data_ptr(), ld_acc, keep, first, last, idx.data_ptr(), _ptr(work), nbytes,
                                    _stream(stream)))
        return idx

    def set_step_p(self, p) -> None:
        """Top-p threshold per routing step (p[s] for step s, the last value for later steps); [] or None
        returns to the configuration's p."""
        vals = [] if p is None else [float(x) for x in p]
        arr = (_c.c_float * max(len(vals), 1))(*vals)
        _check(lib().zha_tree_set_step_p(self._h, _c.cast(arr, _c.c_void_p) if vals else None, len(vals)))

    def status(self, stream=None) -> None:
        _check(lib().zha_tree_status(self._h, _stream(stream)))

    def level_planes(self, level: int):
        """Stored planes of one level: (mu [Hkv, cap, R, d], bias [Hkv, cap, R] fp32, f [Hkv, cap, R] fp32)."""
        c = self.cfg
        lay = tree_layout(c, level)
        es = 2 if c.dtype == ZHA_BF16 else 4
        n = c.n_kv_heads * lay.cap_nodes
        rec = self.nodes[lay.rec_offset: lay.rec_offset + n * lay.rec_bytes].view(c.n_kv_heads, lay.cap_nodes,
                                                                                lay.rec_bytes)
        mu_b = c.n_refs * c.d * es
        mu = rec[..., :mu_b].contiguous().view(TORCH_DTYPE[c.dtype]).view(c.n_kv_heads, lay.cap_nodes, c.n_refs, c.d)
        bias = rec[..., mu_b: mu_b + 4 * c.n_refs].contiguous().view(torch.float32)
        f = self.nodes[lay.f_offset: lay.f_offset + n * c.n_refs * 4].view(torch.float32).view(
            c.n_kv_heads, lay.cap_nodes, c.n_refs)
        return mu, bias, f

    def fp4_records(self, level: int):
        """FP4 router records of one level: (codes [Hkv, cap, R, d] uint8 (one code per dimension),
        scales [Hkv, cap, R, d/16] uint8 e4m3, bias [Hkv, cap, R] fp32)."""
        c = self.cfg
        off, rb = tree_layout_fp4(c, level)
        cap = tree_layout(c, level).cap_nodes
        rec = self.nodes[off: off + c.n_kv_heads * cap * rb].view(c.n_kv_heads, cap, rb)
        R, D = c.n_refs, c.d
        packed = rec[..., : R * D // 2].reshape(c.n_kv_heads, cap, R, D // 2)
        codes = torch.stack([packed & 15, packed >> 4], dim=-1).reshape(c.n_kv_heads, cap, R, D)
        scales = rec[..., R * D // 2: R * (D // 2 + D // 16)].reshape(c.n_kv_heads, cap, R, D // 16)
        b0 = R * (D // 2 + D // 16)
        bias = rec[..., b0: b0 + 4 * R].contiguous().view(torch.float32)
        return codes, scales, bias


def launch_count() -> int:
    """Kernels libzha.so has launched in this process."""
    return int(lib().zha_launch_count())


def dense_scratch_bytes(cfg: ZhaConfig, B: int, n: int) -> int:
    return int(lib().zha_dense_scratch_bytes(ctypes.byref(cfg), B, n))


class DenseDecoder:
    """Dense decode over tokens [0, n) of K, V [Hkv, ld, d] with a reusable zero-filled scratch."""

    def __init__(self, cfg: ZhaConfig, B: int, n_max: int, device="cuda"):
        self.cfg = cfg
        self.scratch = torch.zeros(max(256, dense_scratch_bytes(cfg, B, n_max)), dtype=torch.uint8, device=device)
        self.B = B

    def __call__(self, K: torch.Tensor, V: torch.Tensor, n: int, Q: torch.Tensor, out=None, stream=None):
        B = Q.shape[0]
        need = dense_scratch_bytes(self.cfg, B, n)
        if need > self.scratch.numel():
            self.scratch = torch.zeros(need, dtype=torch.uint8, device=Q.device)
        Q = Q.contiguous()
        O = out if out is not None else torch.empty(B, self.cfg.n_q_heads, self.cfg.d, dtype=torch.float32,
                                                    device=Q.device)
        _check(lib().zha_dense_decode(ctypes.byref(self.cfg), K.data_ptr(), V.data_ptr(), K.shape[1], n,
                                      Q.data_ptr(), O.data_ptr(), B, self.scratch.data_ptr(), _stream(stream)))
        return O


def dense_decode(cfg: ZhaConfig, K: torch.Tensor, V: torch.Tensor, n: int, Q: torch.Tensor, stream=None):
    return DenseDecoder(cfg, Q.shape[0], n, device=Q.device)(K, V, n, Q, stream=stream)


# ---------------------------------------------------------------- shared prefix, weights, eviction
# These entry points take tensors as they lie (row strides included) and never copy them; every tensor must be on
# the current CUDA device.  Outputs they allocate belong to the stream the call runs on; what else a call on another
# stream than the current one uses is recorded there, so that it may be dropped before that stream is done.  A short
# call takes the GPU about ten microseconds, so the checks read each tensor's attributes once.

_F32 = torch.float32


def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _empty(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _record(stream, dev: int, *tensors) -> None:
    """The memory of tensors that a call on `stream` uses is not handed out again before the call is done."""
    if stream is None or stream.cuda_stream == torch._C._cuda_getCurrentRawStream(dev):
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _refuse_device(name: str):
    raise ValueError(f"{name} must be on the current CUDA device (cuda:{torch.cuda.current_device()})")


def _cache_ld(name: str, t: torch.Tensor, hkv: int, d: int, dt, tokens: int) -> int:
    """Row stride in tokens of a cache tensor [hkv, >= tokens, d] whose heads may be slices of longer ones."""
    if t.dtype is not dt or t.dim() != 3 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA {dt} tensor [{hkv}, >= {tokens}, {d}]")
    h, have, dd = t.shape
    if h != hkv or dd != d or have < tokens:
        raise ValueError(f"{name} must be a CUDA {dt} tensor [{hkv}, >= {tokens}, {d}]")
    if t.is_contiguous():
        return have
    s0, s1, s2 = t.stride()
    if s2 != 1 or s1 != d or (h > 1 and (s0 % d or s0 < have * d)):
        raise ValueError(f"{name} must have contiguous rows, one after another, and heads a whole number of rows apart")
    return s0 // d if h > 1 else have


def _same_layout(a: str, x: torch.Tensor, b: str, y: torch.Tensor, ld: int, hkv: int, d: int, dt, tokens: int) -> None:
    if _cache_ld(b, y, hkv, d, dt, tokens) != ld or x.shape[1] != y.shape[1]:
        raise ValueError(f"{a} and {b} must have the same shape and strides")


def _sums_ld(name: str, t: torch.Tensor, hkv: int, n: int) -> int:
    """Row stride of per-token sums [hkv, >= n] fp32."""
    if t.dtype is not _F32 or t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA float32 tensor [{hkv}, >= {n}]")
    h, have = t.shape
    if h != hkv or have < n:
        raise ValueError(f"{name} must be a CUDA float32 tensor [{hkv}, >= {n}]")
    if t.is_contiguous():
        return have
    s0, s1 = t.stride()
    if s1 != 1 or (h > 1 and s0 < have):
        raise ValueError(f"{name} must have contiguous rows")
    return s0 if h > 1 else have


def _check_out(name: str, t: torch.Tensor, shape) -> None:
    if t.shape != shape or t.dtype is not _F32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA float32 tensor {list(shape)}")


def _new_scratch(nbytes: int, device) -> torch.Tensor:
    if nbytes == 0:
        _check(lib().zha_last_error_code())
    if torch.cuda.is_current_stream_capturing():
        raise ValueError("a workspace cannot be made while the stream is captured into a graph: make it before, call it inside")
    scratch = torch.zeros(nbytes, dtype=torch.uint8, device=device)
    torch.cuda.current_stream(scratch.device).synchronize()  # cleared before any stream uses it
    return scratch


class _Attend:
    """What PrefixDecoder and DenseWeights share: the configuration's fields, a workspace, its status."""

    def __init__(self, cfg: ZhaConfig, nbytes: int, device):
        self.cfg = cfg
        self._cfg = ctypes.byref(cfg)
        self._shape = (cfg.n_kv_heads, cfg.d, TORCH_DTYPE[cfg.dtype])
        self.scratch = _new_scratch(nbytes, device)
        self._device = self.scratch.get_device()
        self._scratch = (self.scratch.data_ptr(), self.scratch.numel())
        self._home = torch.cuda.current_stream(self.scratch.device).cuda_stream  # the stream its memory belongs to

    def _on(self, stream) -> int:
        """The raw stream of a call; the workspace lives until the call is done, whatever stream that is."""
        raw = _raw_stream(stream, self._device)
        if raw != self._home:
            self.scratch.record_stream(stream if stream is not None else torch.cuda.current_stream())
        return raw

    def _check_q(self, Q: torch.Tensor, dims, lead: str):
        c = self.cfg
        dt = TORCH_DTYPE[c.dtype]
        shape = Q.shape
        if (Q.dtype is not dt or not Q.is_cuda or not Q.is_contiguous() or len(shape) not in dims or shape[-1] != c.d
                or shape[-2] != c.n_q_heads):
            raise ValueError(f"Q must be a contiguous CUDA {dt} tensor {lead.format(c.n_q_heads, c.d)}")
        return shape

    def status(self, stream=None) -> None:
        """Waits for `stream` (the one the calls ran on) and raises if a wait of theirs ran out; looking clears it."""
        _check(lib().zha_scratch_status(self.scratch.data_ptr(), _stream(stream)))


class PrefixDecoder(_Attend):
    """Attention of up to B sequences x m query tokens over a shared prefix of up to n_max tokens and own caches of up
    to own_max tokens (zha_prefix_decode), with a workspace of its own.

    Calls of one PrefixDecoder must be issued in order on one stream, and graphs captured with one must not replay at
    the same time nor outlive it: they share its workspace.
    """

    def __init__(self, cfg: ZhaConfig, B: int, n_max: int, own_max: int = 0, m: int = 1, device="cuda"):
        super().__init__(cfg, int(lib().zha_prefix_scratch_bytes(ctypes.byref(cfg), B, m, n_max, own_max)), device)
        self.B, self.m, self.n_max, self.own_max = B, m, n_max, own_max

    def __call__(self, K: Optional[torch.Tensor], V: Optional[torch.Tensor], n: int, Q: torch.Tensor,
                 K_own: Optional[torch.Tensor] = None, V_own: Optional[torch.Tensor] = None,
                 own_len: Optional[torch.Tensor] = None, *, out=None, want_lse: bool = False, stream=None):
        """Q [B, m, Hq, d] (or [B, Hq, d]); K, V [Hkv, >= n, d] (None for n = 0); K_own, V_own [B, Hkv, >= own_len, d]
        with own_len [B] int32, or all three None.  Returns O fp32 of Q's shape, or (O, lse of Q's shape but d)."""
        shape = self._check_q(Q, (3, 4), "[B, m, {0}, {1}] or [B, {0}, {1}]")
        hkv, d, dt = self._shape
        dev = self._device
        if torch.cuda.current_device() != dev:
            _refuse_device("the workspace")
        if Q.get_device() != dev:
            _refuse_device("Q")
        B, m = shape[0], shape[1] if len(shape) == 4 else 1
        ld = ld_own = 0
        k = v = ko = vo = ln = None
        if n:
            if K is None or V is None:
                raise ValueError("n > 0 needs K and V")
            if n < 0:
                raise ValueError("n must be >= 0")
            ld = _cache_ld("K", K, hkv, d, dt, n)
            _same_layout("K", K, "V", V, ld, hkv, d, dt, n)
            if K.get_device() != dev or V.get_device() != dev:
                _refuse_device("K and V")
            k, v = K.data_ptr(), V.data_ptr()
        if K_own is not None:
            if V_own is None or own_len is None:
                raise ValueError("K_own, V_own and own_len go together")
            own_shape = K_own.shape
            if (len(own_shape) != 4 or own_shape[0] != B or own_shape[1] != hkv or own_shape[3] != d
                    or V_own.shape != own_shape or K_own.dtype is not dt or V_own.dtype is not dt
                    or not K_own.is_contiguous() or not V_own.is_contiguous()):
                raise ValueError(f"K_own and V_own must be contiguous CUDA {dt} tensors [{B}, {hkv}, tokens, {d}]")
            if own_len.dtype is not torch.int32 or own_len.shape != (B,) or not own_len.is_contiguous():
                raise ValueError(f"own_len must be a contiguous CUDA int32 tensor [{B}]")
            if K_own.get_device() != dev or V_own.get_device() != dev or own_len.get_device() != dev:
                _refuse_device("K_own, V_own and own_len")
            ld_own = own_shape[2]
            if ld_own:
                ko, vo, ln = K_own.data_ptr(), V_own.data_ptr(), own_len.data_ptr()
        elif V_own is not None or own_len is not None:
            raise ValueError("K_own, V_own and own_len go together")
        if B > self.B or m > self.m or n > self.n_max or ld_own > self.own_max:
            raise ValueError(f"the decoder was made for B <= {self.B}, m <= {self.m}, n <= {self.n_max} and own caches "
                             f"of at most {self.own_max} tokens")
        if out is None:
            out = _empty(Q, shape, _F32, stream)
        else:
            _check_out("out", out, shape)
            if out.get_device() != dev:
                _refuse_device("out")
        lse = _empty(Q, shape[:-1], _F32, stream) if want_lse else None
        if B and m:
            raw = self._on(stream)
            _record(stream, dev, Q, K, V, K_own, V_own, own_len, out)
            rc = lib().zha_prefix_decode(self._cfg, k, v, ld, n, ko, vo, ld_own, ln, Q.data_ptr(), out.data_ptr(),
                                         _ptr(lse), B, m, *self._scratch, raw)
            if rc:
                _check(rc)
        return (out, lse) if want_lse else out


def prefix_decode(cfg: ZhaConfig, K, V, n: int, Q: torch.Tensor, K_own=None, V_own=None, own_len=None, *,
                  want_lse: bool = False, stream=None):
    """One call of a PrefixDecoder made for it.  Making its workspace waits for the current stream: loops and graph
    captures (where it is refused) make a PrefixDecoder once."""
    dec = PrefixDecoder(cfg, max(1, Q.shape[0]), n, 0 if K_own is None else K_own.shape[-2],
                        max(1, Q.shape[1]) if Q.dim() == 4 else 1, device=Q.device)
    return dec(K, V, n, Q, K_own, V_own, own_len, want_lse=want_lse, stream=stream)


class DenseWeights(_Attend):
    """Dense attention of up to m query tokens over up to n_max tokens that adds up every token's attention weight
    (zha_dense_weights), with a workspace of its own (as for PrefixDecoder).  Sums in place are left as they were by a
    call whose status() is ZHA_ERR_TIMEOUT, and by later ones until it has been asked for."""

    def __init__(self, cfg: ZhaConfig, m: int, n_max: int, device="cuda"):
        super().__init__(cfg, int(lib().zha_weights_scratch_bytes(ctypes.byref(cfg), m, n_max)), device)
        self.m, self.n_max = m, n_max

    def __call__(self, K: torch.Tensor, V: Optional[torch.Tensor], n: int, Q: torch.Tensor,
                 acc: Optional[torch.Tensor] = None, *, causal: bool = False, acc_out: Optional[torch.Tensor] = None,
                 out=None, stream=None):
        """Q [m, Hq, d]; K, V [Hkv, >= n, d]; acc [Hkv, >= n] fp32 the sums so far (None: zeros).  Returns (O fp32 of
        Q's shape, acc_out [Hkv, n] = acc + the weights); V None leaves O out (None).  acc_out may be acc."""
        shape = self._check_q(Q, (3,), "[m, {0}, {1}]")
        hkv, d, dt = self._shape
        dev = self._device
        if torch.cuda.current_device() != dev:
            _refuse_device("the workspace")
        m = shape[0]
        if n < 1:
            raise ValueError("n must be >= 1")
        ld = _cache_ld("K", K, hkv, d, dt, n)
        if Q.get_device() != dev or K.get_device() != dev:
            _refuse_device("Q and K")
        if not 1 <= m <= self.m or n > self.n_max:
            raise ValueError(f"the workspace was made for 1 <= m <= {self.m} and n <= {self.n_max}")
        v = o = None
        if V is not None:
            _same_layout("K", K, "V", V, ld, hkv, d, dt, n)
            if out is None:
                out = _empty(Q, shape, _F32, stream)
            else:
                _check_out("out", out, shape)
            if V.get_device() != dev or out.get_device() != dev:
                _refuse_device("V and out")
            v, o = V.data_ptr(), out.data_ptr()
        elif out is not None:
            raise ValueError("out needs V")
        a, ld_in = None, 0
        if acc is not None:
            ld_in = _sums_ld("acc", acc, hkv, n)
            if acc.get_device() != dev:
                _refuse_device("acc")
            a = acc.data_ptr()
        if acc_out is None:
            acc_out, ld_out = _empty(Q, (hkv, n), _F32, stream), n
        else:
            ld_out = _sums_ld("acc_out", acc_out, hkv, n)
            if acc_out.get_device() != dev:
                _refuse_device("acc_out")
        raw = self._on(stream)
        _record(stream, dev, Q, K, V, acc, acc_out, out)
        rc = lib().zha_dense_weights(self._cfg, K.data_ptr(), v, ld, n, Q.data_ptr(), o, m, 1 if causal else 0, a, ld_in,
                                     acc_out.data_ptr(), ld_out, *self._scratch, raw)
        if rc:
            _check(rc)
        return out, acc_out


def _evict_scratch(cfg: ZhaConfig, acc: torch.Tensor, n: int, stream):
    nbytes = lib().zha_evict_scratch_bytes(ctypes.byref(cfg), n)
    return (_empty(acc, (nbytes,), torch.uint8, stream) if nbytes else None), nbytes


def cache_evict(cfg: ZhaConfig, K: torch.Tensor, V: torch.Tensor, n: int, acc: torch.Tensor, keep: int, *,
                first: int = 0, last: int = 0, K_out: Optional[torch.Tensor] = None,
                V_out: Optional[torch.Tensor] = None, acc_out: Optional[torch.Tensor] = None, stream=None):
    """Shorten a cache K, V [Hkv, >= n, d] to `keep` tokens per head: the first `first`, the last `last` and those with
    the largest sums acc [Hkv, >= n] between (zha_cache_evict).  K_out and V_out [Hkv, >= keep, d] both None: in
    place, the sums too unless acc_out is given.  Returns (kept positions [Hkv, keep] int32, acc_out)."""
    hkv, d, dt = cfg.n_kv_heads, cfg.d, TORCH_DTYPE[cfg.dtype]
    if n < 1:
        raise ValueError("n must be >= 1")
    if not 1 <= keep <= n:
        raise ValueError(f"keep must be in [1, {n}]")
    ld = _cache_ld("K", K, hkv, d, dt, n)
    _same_layout("K", K, "V", V, ld, hkv, d, dt, n)
    ld_acc = _sums_ld("acc", acc, hkv, n)
    dev = torch.cuda.current_device()
    if K.get_device() != dev or V.get_device() != dev or acc.get_device() != dev:
        _refuse_device("K, V and acc")
    if K_out is None:
        if V_out is not None:
            raise ValueError("K_out and V_out go together")
        K_out, V_out, ld_out = K, V, ld
        if acc_out is None:
            acc_out = acc
    else:
        if V_out is None:
            raise ValueError("K_out and V_out go together")
        ld_out = _cache_ld("K_out", K_out, hkv, d, dt, keep)
        _same_layout("K_out", K_out, "V_out", V_out, ld_out, hkv, d, dt, keep)
        if K_out.get_device() != dev or V_out.get_device() != dev:
            _refuse_device("K_out and V_out")
    if acc_out is None:
        acc_out, ld_acc_out = _empty(acc, (hkv, keep), _F32, stream), keep
    else:
        ld_acc_out = _sums_ld("acc_out", acc_out, hkv, keep)
        if acc_out.get_device() != dev:
            _refuse_device("acc_out")
    idx = _empty(acc, (hkv, keep), torch.int32, stream)
    work, nbytes = _evict_scratch(cfg, acc, n, stream)
    _record(stream, dev, K, V, acc, K_out, V_out, acc_out)
    rc = lib().zha_cache_evict(ctypes.byref(cfg), K.data_ptr(), V.data_ptr(), ld, n, acc.data_ptr(), ld_acc, keep, first,
                               last, K_out.data_ptr(), V_out.data_ptr(), ld_out, acc_out.data_ptr(), ld_acc_out,
                               idx.data_ptr(), _ptr(work), nbytes, _raw_stream(stream, dev))
    if rc:
        _check(rc)
    return idx, acc_out
