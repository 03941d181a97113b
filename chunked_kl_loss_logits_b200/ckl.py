"""Python binding of libckl.so (argument marshalling only).

Every step of the loss runs in the library's CUDA kernels; this module only
allocates outputs and the workspace with PyTorch, passes raw pointers and the
current CUDA stream, and turns status codes into exceptions. If the library has
not been built the import of `lib()` raises: there is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import importlib.machinery
import importlib.util
import os
import re
import threading

import torch
from torch.autograd.function import once_differentiable

_PKG = os.path.dirname(os.path.abspath(__file__))
# The in-tree build; CKL_LIBRARY names another build of the same library.
LIB_PATH = os.environ.get("CKL_LIBRARY") or os.path.join(_PKG, "lib", "libckl.so")
OPS_PATH = os.path.join(_PKG, "lib", "_ckl_ops.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "ckl.h")

F32, BF16 = 0, 1
_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported size", 3: "workspace",
           4: "top-K index out of range", 5: "CUDA error", 6: "device wait timed out",
           7: "pointer misaligned", 8: "internal consistency check failed",
           9: "a caller-supplied collective failed"}


class CKLError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {_STATUS.get(code, code)} (status {code})")
        self.code = code


_GatherFn = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                             ctypes.c_int64, ctypes.c_void_p)
_ReduceFn = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                             ctypes.c_void_p)


class _VocabGroupC(ctypes.Structure):
    """Mirror of ckl_vocab_group."""
    _fields_ = [("world", ctypes.c_int32), ("rank", ctypes.c_int32), ("V_total", ctypes.c_int64),
                ("v0", ctypes.c_int64), ("all_gather", _GatherFn), ("all_reduce_sum", _ReduceFn),
                ("user", ctypes.c_void_p)]


class KernelStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int64),
                ("total_ms", ctypes.c_double), ("flops", ctypes.c_double),
                ("bytes", ctypes.c_double)]


_lib = None
_P, _I64, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """Load libckl.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m chunked_kl_loss_logits_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    sig = {
        "ckl_create": ([ctypes.POINTER(_P), ctypes.c_int, ctypes.c_int, _I64, _I64, _I64, _I64],
                       ctypes.c_int),
        "ckl_destroy": ([_P], ctypes.c_int),
        "ckl_status_str": ([ctypes.c_int], ctypes.c_char_p),
        "ckl_workspace_bytes": ([_P, _I64, _I64, ctypes.POINTER(_SZ)], ctypes.c_int),
        "ckl_fwd_bwd": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P, _P],
                        ctypes.c_int),
        "ckl_forward": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _P, _P, _P, _P, _SZ, _P, _P],
                        ctypes.c_int),
        "ckl_fwd_bwd_from_host": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _P, _P, _P,
                                   _P, _SZ, _P, _P], ctypes.c_int),
        "ckl_sync_status": ([_P, _P], ctypes.c_int),
        "ckl_launch_count": ([_P], ctypes.c_int64),
        "ckl_set_recompute": ([_P, ctypes.c_int], ctypes.c_int),
        "ckl_topk_workspace_bytes": ([_P, _I64, _I64, ctypes.POINTER(_SZ)], ctypes.c_int),
        "ckl_topk_cache": ([_P, _P, _P, _I64, _I64, _P, _P, _P, _SZ, _P, ctypes.c_int], ctypes.c_int),
        "ckl_vp_workspace_bytes": ([_P, ctypes.c_int32, _I64, _I64, ctypes.POINTER(_SZ)],
                                   ctypes.c_int),
        "ckl_fwd_bwd_vocab_parallel": ([_P, ctypes.POINTER(_VocabGroupC), _P, _P, _P, _P, _P, _I64,
                                        _I64, _P, _P, _P, _P, _P, _P, _SZ, _P, _P], ctypes.c_int),
        "ckl_forward_vocab_parallel": ([_P, ctypes.POINTER(_VocabGroupC), _P, _P, _P, _P, _P, _I64,
                                        _I64, _P, _P, _P, _P, _SZ, _P, _P], ctypes.c_int),
        "ckl_selftest_wait_bound": ([_P, _P, ctypes.POINTER(_I64)], ctypes.c_int),
        "ckl_topk_vp_workspace_bytes": ([_P, ctypes.c_int32, _I64, _I64, ctypes.POINTER(_SZ)],
                                        ctypes.c_int),
        "ckl_topk_cache_vocab_parallel": ([_P, ctypes.POINTER(_VocabGroupC), _P, _P, _I64, _I64,
                                           _P, _P, _P, _SZ, _P, ctypes.c_int], ctypes.c_int),
        "ckl_embed": ([_P, _P, _P, _P, _I64, _I64, _I64, ctypes.c_float, _P, _P, ctypes.c_int],
                      ctypes.c_int),
        "ckl_embed_vp_workspace_bytes": ([_P, _I64, ctypes.POINTER(_SZ)], ctypes.c_int),
        "ckl_embed_vocab_parallel": ([_P, ctypes.POINTER(_VocabGroupC), _P, _P, _P, _I64,
                                      ctypes.c_float, _P, _P, _SZ, _P, ctypes.c_int], ctypes.c_int),
        "ckl_embed_grad_workspace_bytes": ([_P, _I64, ctypes.POINTER(_SZ)], ctypes.c_int),
        "ckl_embed_grad": ([_P, _P, _P, _P, _I64, _I64, _I64, ctypes.c_float, ctypes.c_int, _P, _P,
                            _SZ, _P, ctypes.c_int], ctypes.c_int),
        "ckl_act8_pack": ([_P, _P, _I64, _I64, ctypes.c_int, _P, _P, _P], ctypes.c_int),
        "ckl_act8_unpack": ([_P, _P, _P, _I64, _I64, ctypes.c_int, _P, _P], ctypes.c_int),
        "ckl_act8_weight_grad_workspace_bytes": ([_P, _I64, _I64, _I64, ctypes.POINTER(_SZ)],
                                                 ctypes.c_int),
        "ckl_act8_weight_grad": ([_P, _P, _I64, _I64, _P, _P, _I64, ctypes.c_int, ctypes.c_int, _P,
                                  _P, _SZ, _P, ctypes.c_int], ctypes.c_int),
        "ckl_norm": ([_P, _P, _P, _P, _I64, ctypes.c_float, ctypes.c_int, _P, _P, _P, _P, _P, _P],
                     ctypes.c_int),
        "ckl_norm_bwd_workspace_bytes": ([_P, _I64, ctypes.POINTER(_SZ)], ctypes.c_int),
        "ckl_norm_bwd": ([_P, _P, _P, _P, _P, _P, _P, _I64, ctypes.c_int, ctypes.c_int, _P, _P, _P,
                          _SZ, _P], ctypes.c_int),
        "ckl_profile_enable": ([_P, ctypes.c_int, ctypes.c_int], ctypes.c_int),
        "ckl_profile_collect": ([_P, ctypes.POINTER(KernelStat), ctypes.c_int,
                                 ctypes.POINTER(ctypes.c_int)], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name, None)
        if f is None:  # an older build: the calls that it has still work
            continue
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def header_functions() -> list:
    """Names of the functions include/ckl.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"\b(ckl_[a-z_0-9]+)\s*\(", text)))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(code: int, what: str):
    if code != 0:
        raise CKLError(code, what)


class _DevArray:
    """A raw device pointer seen as a float32 vector (CUDA array interface, no copy)."""

    def __init__(self, ptr: int, count: int):
        self.__cuda_array_interface__ = {"shape": (count,), "typestr": "<f4",
                                         "data": (ptr, False), "version": 3, "stream": None}


def vocab_shards(V_total: int, world: int, align: int = 256) -> list:
    """(v0, V_r) of each rank: contiguous row ranges of the LM head, as equal as
    possible in whole `align`-row blocks (the last rank takes the remainder)."""
    if world < 1 or V_total < world:
        raise ValueError("need 1 <= world <= V_total")
    blocks = (V_total + align - 1) // align
    out, v0 = [], 0
    for r in range(world):
        nb = blocks // world + (1 if r < blocks % world else 0)
        v1 = min(V_total, v0 + nb * align) if r < world - 1 else V_total
        out.append((v0, v1 - v0))
        v0 = v1
    if any(n <= 0 for _, n in out):
        raise ValueError("a rank would hold no rows")
    return out


class VocabGroup:
    """This rank's place in a vocabulary-parallel group and the group's two collectives.

    all_gather(send, recv): send is a float32 vector of n entries, recv one of
    world * n entries to fill rank-major; all_reduce_sum(buf): in place. Both
    get device tensors and must be ordered on the current CUDA stream (the
    library's stream is made current around each call) and return None.
    """

    def __init__(self, world: int, rank: int, V_total: int, v0: int, all_gather, all_reduce_sum):
        self.world, self.rank, self.V_total, self.v0 = world, rank, V_total, v0
        self.all_gather, self.all_reduce_sum = all_gather, all_reduce_sum
        self.error = None

    def _c(self, device):
        def as_stream(ptr):
            return torch.cuda.ExternalStream(ptr, device=device) if ptr else \
                torch.cuda.default_stream(device)

        def gather(_user, send, recv, count, stream):
            try:
                with torch.cuda.stream(as_stream(stream)):
                    a = torch.as_tensor(_DevArray(send, count), device=device)
                    b = torch.as_tensor(_DevArray(recv, count * self.world), device=device)
                    self.all_gather(a, b)
                return 0
            except Exception as e:  # reported as CKL_ERR_COLLECTIVE; kept for the caller
                self.error = e
                return 1

        def reduce(_user, buf, count, stream):
            try:
                with torch.cuda.stream(as_stream(stream)):
                    self.all_reduce_sum(torch.as_tensor(_DevArray(buf, count), device=device))
                return 0
            except Exception as e:
                self.error = e
                return 1

        fns = (_GatherFn(gather), _ReduceFn(reduce))  # kept alive by the caller for the call
        return _VocabGroupC(self.world, self.rank, self.V_total, self.v0, fns[0], fns[1], None), fns


def torch_vocab_group(V_total: int, group=None) -> VocabGroup:
    """A VocabGroup over a torch.distributed process group (NCCL on GPUs): this
    rank's rows come from vocab_shards(V_total, world)."""
    import torch.distributed as dist
    world, rank = dist.get_world_size(group), dist.get_rank(group)
    v0, _ = vocab_shards(V_total, world)[rank]
    return VocabGroup(world, rank, V_total, v0,
                      lambda send, recv: dist.all_gather_into_tensor(recv, send, group=group),
                      lambda buf: dist.all_reduce(buf, group=group))


ACT8_FORMATS = {"int8": 0, "e4m3": 1}
_ACT8_NAMES = ("int8", "e4m3")


def _act8_format(fmt, what="fmt") -> int:
    f = ACT8_FORMATS.get(fmt)
    if f is None:
        raise ValueError(f"{what} must be one of {sorted(ACT8_FORMATS)}")
    return f

_ops_module = None


def _ops():
    """The module that marshals the operators' calls, bound to the loaded library (raises if it
    was not built)."""
    global _ops_module
    if _ops_module is None:
        if not os.path.exists(OPS_PATH):
            raise RuntimeError(f"{OPS_PATH} is missing: build it with "
                               "`python -m chunked_kl_loss_logits_b200.build`")
        L = lib()
        try:
            calls = [getattr(L, "ckl_" + f) for f in (
                "embed", "embed_grad_workspace_bytes", "embed_grad", "act8_pack", "act8_unpack",
                "act8_weight_grad_workspace_bytes", "act8_weight_grad", "norm",
                "norm_bwd_workspace_bytes", "norm_bwd")]
        except AttributeError as e:
            raise RuntimeError(f"{LIB_PATH} is a build without these operators") from e
        loader = importlib.machinery.ExtensionFileLoader("_ckl_ops", OPS_PATH)
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_ckl_ops", loader))
        loader.exec_module(m)
        m.bind(CKLError, tuple(ctypes.cast(f, ctypes.c_void_p).value for f in calls))
        _ops_module = m
    return _ops_module


class Act8:
    """An 8-bit activation checkpoint: codes q (T x cols, uint8), one power-of-two scale per
    32 columns of a row (T x ceil(cols / 32), uint8: exponent + 127, 255 for a block that held
    an infinity or a NaN) and, from a norm, the rows' factors rstd (T, float32)."""

    def __init__(self, q, scale, fmt: str = "int8", rstd=None):
        _act8_format(fmt)
        if q.dtype != torch.uint8 or scale.dtype != torch.uint8:
            raise TypeError("q and scale must be uint8")
        if q.dim() != 2 or q.shape[1] == 0 or \
                tuple(scale.shape) != (q.shape[0], (q.shape[1] + 31) // 32):
            raise ValueError("q must be T x cols and scale T x ceil(cols / 32)")
        if rstd is not None and (rstd.dtype != torch.float32 or tuple(rstd.shape) != (q.shape[0],)):
            raise TypeError("rstd must be a float32 tensor of T entries")
        for t in (q, scale) + ((rstd,) if rstd is not None else ()):
            if not t.is_contiguous() or t.device != q.device:
                raise ValueError("q, scale and rstd must be contiguous tensors on one device")
        self._parts, self._buf = (q, scale, rstd), None
        self._desc = (q.data_ptr(), scale.data_ptr(), 0 if rstd is None else rstd.data_ptr(),
                      *q.shape, ACT8_FORMATS[fmt], q.get_device(), rstd is not None)

    __slots__ = ("_parts", "_buf", "_desc")

    @classmethod
    def _of(cls, buf, desc) -> "Act8":
        """The checkpoint that the library's calls wrote to `buf`, as they describe it: rstd, then q
        from a multiple of 16 on, then scale; desc = (addresses of q, scale and rstd, T, cols,
        format, device index, has rstd)."""
        self = cls.__new__(cls)
        self._parts, self._buf, self._desc = None, buf, desc
        return self

    def _views(self):
        if self._parts is None:
            q, e, r, T, cols, _, _, has_rstd = self._desc
            b, base = self._buf, self._buf.data_ptr()
            self._parts = (b[q - base:q - base + T * cols].view(T, cols),
                           b[e - base:].view(T, (cols + 31) // 32),
                           b[:4 * T].view(torch.float32) if has_rstd else None)
        return self._parts

    @property
    def q(self):
        return self._views()[0]

    @property
    def scale(self):
        return self._views()[1]

    @property
    def rstd(self):
        return self._views()[2]

    @property
    def fmt(self) -> str:
        return _ACT8_NAMES[self._desc[5]]

    @property
    def shape(self) -> tuple:
        return self._desc[3:5]

    @property
    def nbytes(self) -> int:
        T, cols = self.shape
        return T * (cols + (cols + 31) // 32 + (4 if self._desc[7] else 0))


class ChunkedKL:
    """A handle for one LM-head shape (V x d, K cached teacher entries) on one device."""

    def __init__(self, V: int, d: int, K: int, dtype=torch.bfloat16, max_chunk: int = 8192,
                 device=None):
        if dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("dtype must be torch.float32 or torch.bfloat16")
        self.V, self.d, self.K, self.dtype, self.max_chunk = V, d, K, dtype, max_chunk
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        self.device = dev
        h = _P()
        _check(lib().ckl_create(ctypes.byref(h), dev.index or 0,
                                F32 if dtype == torch.float32 else BF16, V, d, K, max_chunk),
               "ckl_create")
        self._h, self._index = h, dev.index or 0
        self._ctx = (h.value, V, d, dtype == torch.bfloat16, self._index)

    def close(self):
        if getattr(self, "_h", None):
            lib().ckl_destroy(self._h)
            self._h = None
            self._ctx = (0,) + self._ctx[1:]  # calls on a closed handle are refused

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------------ helpers
    def workspace_bytes(self, T: int, chunk: int) -> int:
        n = _SZ()
        _check(lib().ckl_workspace_bytes(self._h, T, chunk, ctypes.byref(n)), "ckl_workspace_bytes")
        return n.value

    def workspace(self, T: int, chunk: int) -> torch.Tensor:
        return torch.empty(max(1, self.workspace_bytes(T, chunk)), dtype=torch.uint8,
                           device=self.device)

    def set_recompute(self, on: bool):
        """bf16 only: form the logits again in the backward (True) or keep exp(z) (False)."""
        _check(lib().ckl_set_recompute(self._h, int(on)), "ckl_set_recompute")

    def launch_count(self) -> int:
        return int(lib().ckl_launch_count(self._h))

    def profile_enable(self, on: bool = True, max_launches: int = 8192):
        _check(lib().ckl_profile_enable(self._h, int(on), max_launches), "ckl_profile_enable")

    def profile_collect(self) -> list:
        arr = (KernelStat * 64)()
        n = ctypes.c_int()
        _check(lib().ckl_profile_collect(self._h, arr, 64, ctypes.byref(n)), "ckl_profile_collect")
        return [{"name": arr[i].name.decode(), "launches": arr[i].launches,
                 "total_ms": arr[i].total_ms, "flops": arr[i].flops, "bytes": arr[i].bytes}
                for i in range(min(n.value, 64))]

    def selftest_wait_bound(self, stream=None):
        """(status code, SM cycles waited) of the bounded-wait self-test; 6 (timeout) is a pass."""
        s = stream or torch.cuda.current_stream(self.device)
        cyc = _I64()
        code = lib().ckl_selftest_wait_bound(self._h, ctypes.c_void_p(s.cuda_stream),
                                             ctypes.byref(cyc))
        return code, cyc.value

    def sync_status(self, stream=None):
        s = stream or torch.cuda.current_stream(self.device)
        _check(lib().ckl_sync_status(self._h, ctypes.c_void_p(s.cuda_stream)), "ckl_sync_status")

    def _inputs(self, H, W, idx, logit, mask):
        T = H.shape[0]
        if H.dtype != self.dtype or W.dtype != self.dtype:
            raise TypeError(f"H and W must be {self.dtype}")
        if tuple(W.shape) != (self.V, self.d) or H.shape[1] != self.d:
            raise ValueError("H must be T x d and W must be V x d")
        if tuple(idx.shape) != (T, self.K) or tuple(logit.shape) != (T, self.K):
            raise ValueError("topk_idx and topk_logit must be T x K")
        if idx.dtype != torch.int32 or logit.dtype != torch.float32:
            raise TypeError("topk_idx must be int32 and topk_logit float32")
        if mask is not None and (mask.dtype != torch.uint8 or mask.numel() != T):
            raise TypeError("mask must be a uint8 tensor of T entries")
        for t in (H, W, idx, logit) + ((mask,) if mask is not None else ()):
            if not t.is_contiguous() or t.device != self.device:
                raise ValueError("inputs must be contiguous tensors on the handle's device")
        return T

    # ------------------------------------------------------------------ calls
    def fwd_bwd(self, H, W, idx, logit, mask=None, chunk: int | None = None, out=None,
                workspace=None, token_stats: bool = False, sync: bool = True, stream=None):
        """Loss (0-d float32 tensor), dH (T x d, dtype), dW (V x d, float32).

        With token_stats=True also returns per-token logsumexp and loss (float32, T).
        With sync=True the call waits and raises on a device-detected error.
        """
        T = self._inputs(H, W, idx, logit, mask)
        chunk = min(chunk or self.max_chunk, self.max_chunk)
        if out is None:
            out = (torch.empty((), dtype=torch.float32, device=self.device),
                   torch.empty_like(H), torch.empty((self.V, self.d), dtype=torch.float32,
                                                    device=self.device))
        loss, dH, dW = out
        ws = workspace if workspace is not None else self.workspace(T, chunk)
        lse = ell = None
        if token_stats:
            lse = torch.empty(T, dtype=torch.float32, device=self.device)
            ell = torch.empty(T, dtype=torch.float32, device=self.device)
        s = stream or torch.cuda.current_stream(self.device)
        host = ctypes.c_float() if sync else None
        code = lib().ckl_fwd_bwd(self._h, _ptr(H), _ptr(W), _ptr(idx), _ptr(logit), _ptr(mask), T,
                                 chunk, _ptr(loss), _ptr(dH), _ptr(dW), _ptr(lse), _ptr(ell),
                                 _ptr(ws), ws.numel(), ctypes.c_void_p(s.cuda_stream),
                                 ctypes.byref(host) if sync else None)
        _check(code, "ckl_fwd_bwd")
        return (loss, dH, dW, lse, ell) if token_stats else (loss, dH, dW)

    def forward(self, H, W, idx, logit, mask=None, chunk: int | None = None, workspace=None,
                token_stats: bool = False, sync: bool = True, stream=None):
        """Loss only (no gradients); optionally per-token logsumexp and loss."""
        T = self._inputs(H, W, idx, logit, mask)
        chunk = min(chunk or self.max_chunk, self.max_chunk)
        loss = torch.empty((), dtype=torch.float32, device=self.device)
        ws = workspace if workspace is not None else self.workspace(T, chunk)
        lse = ell = None
        if token_stats:
            lse = torch.empty(T, dtype=torch.float32, device=self.device)
            ell = torch.empty(T, dtype=torch.float32, device=self.device)
        s = stream or torch.cuda.current_stream(self.device)
        host = ctypes.c_float()
        _check(lib().ckl_forward(self._h, _ptr(H), _ptr(W), _ptr(idx), _ptr(logit), _ptr(mask), T,
                                 chunk, _ptr(loss), _ptr(lse), _ptr(ell), _ptr(ws), ws.numel(),
                                 ctypes.c_void_p(s.cuda_stream),
                                 ctypes.byref(host) if sync else None), "ckl_forward")
        return (loss, lse, ell) if token_stats else loss

    def fwd_bwd_vocab_parallel(self, group: VocabGroup, H, W_shard, idx, logit, mask=None,
                               chunk: int | None = None, token_stats: bool = False,
                               sync: bool = True, stream=None):
        """Loss, dH (full, identical on every rank) and dW_shard (this rank's V x d rows).

        The handle's V is this rank's row count; ids are global in [0, group.V_total).
        """
        T = self._inputs(H, W_shard, idx, logit, mask)
        chunk = min(chunk or self.max_chunk, self.max_chunk)
        n = _SZ()
        _check(lib().ckl_vp_workspace_bytes(self._h, group.world, T, chunk, ctypes.byref(n)),
               "ckl_vp_workspace_bytes")
        ws = torch.empty(max(1, n.value), dtype=torch.uint8, device=self.device)
        loss = torch.empty((), dtype=torch.float32, device=self.device)
        dH = torch.empty_like(H)
        dW = torch.empty((self.V, self.d), dtype=torch.float32, device=self.device)
        lse = ell = None
        if token_stats:
            lse = torch.empty(T, dtype=torch.float32, device=self.device)
            ell = torch.empty(T, dtype=torch.float32, device=self.device)
        s = stream or torch.cuda.current_stream(self.device)
        g, keep = group._c(self.device)
        host = ctypes.c_float() if sync else None
        group.error = None
        code = lib().ckl_fwd_bwd_vocab_parallel(
            self._h, ctypes.byref(g), _ptr(H), _ptr(W_shard), _ptr(idx), _ptr(logit), _ptr(mask),
            T, chunk, _ptr(loss), _ptr(dH), _ptr(dW), _ptr(lse), _ptr(ell), _ptr(ws), ws.numel(),
            ctypes.c_void_p(s.cuda_stream), ctypes.byref(host) if sync else None)
        del keep
        if code == 9 and group.error is not None:
            raise CKLError(code, "ckl_fwd_bwd_vocab_parallel") from group.error
        _check(code, "ckl_fwd_bwd_vocab_parallel")
        return (loss, dH, dW, lse, ell) if token_stats else (loss, dH, dW)

    def forward_vocab_parallel(self, group: VocabGroup, H, W_shard, idx, logit, mask=None,
                               chunk: int | None = None, token_stats: bool = False,
                               sync: bool = True, stream=None):
        """Loss only (identical on every rank); the handle's V is this rank's row count."""
        T = self._inputs(H, W_shard, idx, logit, mask)
        chunk = min(chunk or self.max_chunk, self.max_chunk)
        n = _SZ()
        _check(lib().ckl_vp_workspace_bytes(self._h, group.world, T, chunk, ctypes.byref(n)),
               "ckl_vp_workspace_bytes")
        ws = torch.empty(max(1, n.value), dtype=torch.uint8, device=self.device)
        loss = torch.empty((), dtype=torch.float32, device=self.device)
        lse = ell = None
        if token_stats:
            lse = torch.empty(T, dtype=torch.float32, device=self.device)
            ell = torch.empty(T, dtype=torch.float32, device=self.device)
        s = stream or torch.cuda.current_stream(self.device)
        g, keep = group._c(self.device)
        host = ctypes.c_float() if sync else None
        group.error = None
        code = lib().ckl_forward_vocab_parallel(
            self._h, ctypes.byref(g), _ptr(H), _ptr(W_shard), _ptr(idx), _ptr(logit), _ptr(mask),
            T, chunk, _ptr(loss), _ptr(lse), _ptr(ell), _ptr(ws), ws.numel(),
            ctypes.c_void_p(s.cuda_stream), ctypes.byref(host) if sync else None)
        del keep
        if code == 9 and group.error is not None:
            raise CKLError(code, "ckl_forward_vocab_parallel") from group.error
        _check(code, "ckl_forward_vocab_parallel")
        return (loss, lse, ell) if token_stats else loss

    def topk_cache(self, H, W, chunk: int | None = None, workspace=None, sync: bool = True,
                   stream=None):
        """Teacher top-K cache: (ids int32 T x K, logits float32 T x K), descending.

        The handle must have the teacher's shape (V, d = teacher hidden size, K).
        """
        T = H.shape[0]
        if H.dtype != self.dtype or W.dtype != self.dtype or H.shape[1] != self.d or \
                tuple(W.shape) != (self.V, self.d):
            raise ValueError("H must be T x d and W must be V x d, in the handle's dtype")
        chunk = min(chunk or self.max_chunk, self.max_chunk)
        idx = torch.empty((T, self.K), dtype=torch.int32, device=self.device)
        logit = torch.empty((T, self.K), dtype=torch.float32, device=self.device)
        if workspace is None:
            n = _SZ()
            _check(lib().ckl_topk_workspace_bytes(self._h, T, chunk, ctypes.byref(n)),
                   "ckl_topk_workspace_bytes")
            workspace = torch.empty(max(1, n.value), dtype=torch.uint8, device=self.device)
        s = stream or torch.cuda.current_stream(self.device)
        _check(lib().ckl_topk_cache(self._h, _ptr(H), _ptr(W), T, chunk, _ptr(idx), _ptr(logit),
                                    _ptr(workspace), workspace.numel(),
                                    ctypes.c_void_p(s.cuda_stream), int(sync)), "ckl_topk_cache")
        return idx, logit

    def topk_cache_vocab_parallel(self, group: VocabGroup, H, W_shard, chunk: int | None = None,
                                  sync: bool = True, stream=None):
        """Teacher top-K cache with the teacher's LM head split by vocabulary rows over
        `group`: (ids int32 T x K, global; logits float32 T x K), the same on every
        rank and the same as topk_cache with all of W on one rank."""
        T = H.shape[0]
        if H.dtype != self.dtype or W_shard.dtype != self.dtype or H.shape[1] != self.d or \
                tuple(W_shard.shape) != (self.V, self.d):
            raise ValueError("H must be T x d and W_shard V x d, in the handle's dtype")
        chunk = min(chunk or self.max_chunk, self.max_chunk)
        n = _SZ()
        _check(lib().ckl_topk_vp_workspace_bytes(self._h, group.world, T, chunk, ctypes.byref(n)),
               "ckl_topk_vp_workspace_bytes")
        ws = torch.empty(max(1, n.value), dtype=torch.uint8, device=self.device)
        idx = torch.empty((T, self.K), dtype=torch.int32, device=self.device)
        logit = torch.empty((T, self.K), dtype=torch.float32, device=self.device)
        s = stream or torch.cuda.current_stream(self.device)
        g, keep = group._c(self.device)
        group.error = None
        code = lib().ckl_topk_cache_vocab_parallel(
            self._h, ctypes.byref(g), _ptr(H), _ptr(W_shard), T, chunk, _ptr(idx), _ptr(logit),
            _ptr(ws), ws.numel(), ctypes.c_void_p(s.cuda_stream), int(sync))
        del keep
        if code == 9 and group.error is not None:
            raise CKLError(code, "ckl_topk_cache_vocab_parallel") from group.error
        _check(code, "ckl_topk_cache_vocab_parallel")
        return idx, logit

    # ------------------------------------------------------------------ operators around the loss
    # Checks, allocations and the call are made in csrc/torch_ops.cpp. Tensors must be dense, of the
    # handle's dtype and on its device; `stream` (by default the current one) is where the call
    # runs and what it allocates is allocated. A call captured in a CUDA graph takes sync=False.
    @functools.cached_property
    def _ops(self):  # at the first of these calls: the loss needs libckl.so alone
        return _ops()

    @contextlib.contextmanager
    def _on(self, stream):
        if stream.device.index != self._index:
            raise ValueError("stream must be one of the handle's device")
        with torch.cuda.stream(stream):
            yield

    def _workspace(self, query, *sizes) -> torch.Tensor:
        """A workspace of the size that the library's `query` gives for these sizes."""
        n = _SZ()
        _check(getattr(lib(), query)(self._h, *sizes, ctypes.byref(n)), query)
        return torch.empty(n.value, dtype=torch.uint8, device=self.device)

    def embed_grad_workspace(self, T: int) -> torch.Tensor:
        return self._workspace("ckl_embed_grad_workspace_bytes", T)

    def norm_bwd_workspace(self, T: int) -> torch.Tensor:
        return self._workspace("ckl_norm_bwd_workspace_bytes", T)

    def act8_weight_grad_workspace(self, T: int, n: int, cols: int) -> torch.Tensor:
        return self._workspace("ckl_act8_weight_grad_workspace_bytes", T, n, cols)

    def act8_empty(self, T: int, cols: int, fmt: str = "int8", rstd: bool = False) -> Act8:
        """Buffers for a checkpoint of T x cols (for a norm's with rstd=True), to write to later."""
        at, nb = (4 * T + 15) // 16 * 16 if rstd else 0, (cols + 31) // 32
        buf = torch.empty(at + T * (cols + nb), dtype=torch.uint8, device=self.device)
        return Act8(buf[at:at + T * cols].view(T, cols), buf[at + T * cols:].view(T, nb), fmt,
                    buf[:4 * T].view(torch.float32) if rstd else None)

    def embed(self, ids, W, mask=None, scale: float = 1.0, V_total: int | None = None, v0: int = 0,
              out=None, sync: bool = True, stream=None):
        """scale * W[ids - v0] in the handle's dtype (ids' shape, then d): zeros for tokens with
        mask 0 and for ids in [0, V_total) whose row is not among the handle's V (v0 ..)."""
        if stream is not None:
            with self._on(stream):
                return self.embed(ids, W, mask, scale, V_total, v0, out, sync)
        return self._ops.embed(self._ctx, ids, W, mask, scale, V_total, v0, out, sync)

    def embed_vocab_parallel(self, group: VocabGroup, ids, W_shard, mask=None, scale: float = 1.0,
                             sync: bool = True, stream=None):
        """As embed with W split by vocabulary rows over `group`: the full rows on every rank
        (one all-reduce)."""
        if stream is not None:
            with self._on(stream):
                return self.embed_vocab_parallel(group, ids, W_shard, mask, scale, sync)
        if ids.dtype != torch.int32 or W_shard.dtype != self.dtype:
            raise TypeError(f"ids must be int32 and W_shard {self.dtype}")
        if mask is not None and (mask.dtype != torch.uint8 or mask.numel() != ids.numel()):
            raise TypeError("mask must be a uint8 tensor with an entry for each id")
        if tuple(W_shard.shape) != (self.V, self.d):
            raise ValueError("W_shard must be V x d")
        for t in (ids, W_shard) + ((mask,) if mask is not None else ()):
            if not t.is_contiguous() or t.device != self.device:
                raise ValueError("inputs must be contiguous tensors on the handle's device")
        out = torch.empty(*ids.shape, self.d, dtype=self.dtype, device=self.device)
        ws = self._workspace("ckl_embed_vp_workspace_bytes", ids.numel())
        g, keep = group._c(self.device)
        group.error = None
        code = lib().ckl_embed_vocab_parallel(
            self._h, ctypes.byref(g), _ptr(ids), _ptr(mask), _ptr(W_shard), ids.numel(), scale,
            _ptr(out), _ptr(ws), ws.numel(),
            ctypes.c_void_p(torch.cuda.current_stream(self.device).cuda_stream), int(sync))
        del keep
        if code == 9 and group.error is not None:
            raise CKLError(code, "ckl_embed_vocab_parallel") from group.error
        _check(code, "ckl_embed_vocab_parallel")
        return out

    def embed_grad(self, ids, dX, mask=None, scale: float = 1.0, V_total: int | None = None,
                   v0: int = 0, dW=None, accumulate: bool = False, workspace=None,
                   sync: bool = True, stream=None):
        """dW (V x d, float32) of embed: the given buffer, added to with accumulate=True (a tied
        head's dW from fwd_bwd) and overwritten otherwise, or a new one."""
        if stream is not None:
            with self._on(stream):
                return self.embed_grad(ids, dX, mask, scale, V_total, v0, dW, accumulate,
                                       workspace, sync)
        return self._ops.embed_grad(self._ctx, ids, dX, mask, scale, V_total, v0, dW, accumulate,
                                    workspace, sync)

    def act8_pack(self, x, fmt: str = "int8", out: Act8 | None = None, stream=None) -> Act8:
        """The 8-bit checkpoint of x (T x cols, any cols that is a multiple of 8). With `out`, its
        buffers and format are used."""
        if stream is not None:
            with self._on(stream):
                return self.act8_pack(x, fmt, out)
        if out is not None:
            self._ops.act8_pack(self._ctx, x, 0, out._desc)
            return out
        return Act8._of(*self._ops.act8_pack(self._ctx, x, _act8_format(fmt), None))

    def act8_unpack(self, ckpt: Act8, out=None, stream=None):
        """The values of a checkpoint (T x cols, the handle's dtype)."""
        if stream is not None:
            with self._on(stream):
                return self.act8_unpack(ckpt, out)
        return self._ops.act8_unpack(self._ctx, ckpt._desc, out)

    def act8_weight_grad(self, dY, ckpt: Act8, dW=None, accumulate: bool = False, workspace=None,
                         sync: bool = True, stream=None):
        """dW = dY^T X' (n x cols, float32) of a linear layer Y = X W^T with X kept as the
        checkpoint; dY is T x n. dW is added to with accumulate=True."""
        if stream is not None:
            with self._on(stream):
                return self.act8_weight_grad(dY, ckpt, dW, accumulate, workspace, sync)
        return self._ops.act8_weight_grad(self._ctx, dY, ckpt._desc, dW, accumulate, workspace, sync)

    def norm(self, x, gain, residual=None, eps: float = 1e-5, checkpoint: str | None = "int8",
             out=None, stream=None):
        """(y, s, checkpoint): s = x + residual (x itself without one), y = s / rms(s) * gain and
        the 8-bit checkpoint of s with the rows' factors, all that norm_bwd needs (None for
        checkpoint=None). out = (y, s, checkpoint): buffers to write to instead of new ones
        (s only with a residual, and it may be x's or residual's)."""
        if stream is not None:
            with self._on(stream):
                return self.norm(x, gain, residual, eps, checkpoint, out)
        fmt = -1 if checkpoint is None else _act8_format(checkpoint, "checkpoint")
        if out is None:
            y, s, buf, desc = self._ops.norm(self._ctx, x, gain, residual, eps, fmt, None, None, None)
            return y, s, None if desc is None else Act8._of(buf, desc)
        y, s, ckpt = out
        if (ckpt is None) != (checkpoint is None):
            raise ValueError("out[2] must be an Act8 where a checkpoint is asked for")
        if ckpt is not None and (ckpt._desc[5] != fmt or not ckpt._desc[7]):
            raise ValueError("out[2] must be a checkpoint with rstd in that format")
        y, s, _, _ = self._ops.norm(self._ctx, x, gain, residual, eps, fmt, y, s,
                                    None if ckpt is None else ckpt._desc)
        return y, s, ckpt

    def norm_bwd(self, dY, ckpt: Act8, gain, d_residual=None, dX=None, dgain=None,
                 accumulate: bool = False, workspace=None, stream=None):
        """(dX, dgain) of norm from its checkpoint: dX (T x d) is the gradient of x and of
        residual, d_residual the gradient that reaches s other than through y; dgain (d,
        float32) is added to with accumulate=True."""
        if stream is not None:
            with self._on(stream):
                return self.norm_bwd(dY, ckpt, gain, d_residual, dX, dgain, accumulate, workspace)
        return self._ops.norm_bwd(self._ctx, dY, ckpt._desc, gain, d_residual, dX, dgain, accumulate,
                                  workspace)

    def fwd_bwd_from_host(self, H_host, idx_host, logit_host, mask_host, staging, W, chunk,
                          out, workspace, stream=None) -> float:
        """Fused loss with the per-step inputs in (pinned) host memory; returns the loss.

        `staging` = (H_dev, idx_dev, logit_dev, mask_dev or None): device buffers
        the inputs are copied into. `out` = (loss, dH, dW) device tensors.
        """
        H_dev, idx_dev, logit_dev, mask_dev = staging
        loss, dH, dW = out
        T = H_host.shape[0]
        s = stream or torch.cuda.current_stream(self.device)
        host = ctypes.c_float()
        _check(lib().ckl_fwd_bwd_from_host(
            self._h, _ptr(H_host), _ptr(idx_host), _ptr(logit_host), _ptr(mask_host),
            _ptr(H_dev), _ptr(idx_dev), _ptr(logit_dev), _ptr(mask_dev), _ptr(W), T, chunk,
            _ptr(loss), _ptr(dH), _ptr(dW), _ptr(workspace), workspace.numel(),
            ctypes.c_void_p(s.cuda_stream), ctypes.byref(host)), "ckl_fwd_bwd_from_host")
        return host.value


class _ChunkedKLFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, idx, logit, mask, handle, chunk, check):
        loss, dH, dW = handle.fwd_bwd(H.detach(), W.detach(), idx, logit, mask, chunk=chunk,
                                      sync=False)
        ctx.save_for_backward(dH, dW)
        ctx.w_dtype = W.dtype
        ctx.handle, ctx.check = handle, check
        return loss

    @staticmethod
    def backward(ctx, g):
        if ctx.check:
            ctx.handle.sync_status()  # raises CKLError on a device-detected error
        dH, dW = ctx.saved_tensors
        return (dH * g.to(dH.dtype), (dW * g).to(ctx.w_dtype), None, None, None, None, None, None)


class _VocabParallelKLFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W_shard, idx, logit, mask, handle, chunk, group, check):
        loss, dH, dW = handle.fwd_bwd_vocab_parallel(group, H.detach(), W_shard.detach(), idx,
                                                     logit, mask, chunk=chunk, sync=False)
        ctx.save_for_backward(dH, dW)
        ctx.w_dtype = W_shard.dtype
        ctx.handle, ctx.check = handle, check
        return loss

    @staticmethod
    def backward(ctx, g):
        if ctx.check:
            ctx.handle.sync_status()
        dH, dW = ctx.saved_tensors
        return (dH * g.to(dH.dtype), (dW * g).to(ctx.w_dtype), None, None, None, None, None, None,
                None)


_HANDLES = {}


def handle_for(W, K: int, chunk: int | None = None) -> ChunkedKL:
    """The cached handle for W's device, dtype and shape with K cached entries.

    chunked_kl_loss calls this when it is given no handle, so a training loop
    creates one handle per LM-head shape (ckl_create allocates and synchronises
    the device) instead of one per step. The handle is replaced by one with a
    larger max_chunk when a call asks for a chunk above the cached one's.
    """
    dev = W.device
    key = (dev.type, dev.index, W.dtype, W.shape[0], W.shape[1], K)
    h = _HANDLES.get(key)
    need = max(chunk or 4096, 1)
    if h is None or h.max_chunk < need:
        if h is not None:
            h.close()
        h = ChunkedKL(W.shape[0], W.shape[1], K, dtype=W.dtype, max_chunk=need, device=dev)
        _HANDLES[key] = h
    return h


def chunked_kl_loss(H, W, idx, logit, mask=None, chunk=None, handle: ChunkedKL | None = None,
                    group: VocabGroup | None = None, check: bool = True):
    """Autograd-friendly mean top-K forward KL; the gradients come from the fused call.

    With `group`, W is this rank's vocabulary rows (vocab_shards) and the loss is the
    full-vocabulary one, identical on every rank; H's gradient is the full dH on
    every rank and W's is this rank's rows. Without `handle` the handle cached for
    W's shape (handle_for) is used.

    check=True: backward() waits for the call's stream and raises CKLError if the
    device reported an error (a teacher id outside [0, V), a pipeline timeout);
    the outputs of such a call are undefined. check=False: nothing waits; the
    device status stays set in the handle (errors of later calls add to it) until
    the caller reads it with handle.sync_status() (handle_for(W, K) gives the
    cached handle), which raises and clears it.
    """
    if handle is None:
        handle = handle_for(W, idx.shape[1], chunk)
    if group is not None:
        return _VocabParallelKLFn.apply(H, W, idx, logit, mask, handle, chunk, group, check)
    return _ChunkedKLFn.apply(H, W, idx, logit, mask, handle, chunk, check)


_OP_HANDLES = threading.local()  # a handle must not be used by two calls at once


def operator_handle(t, V: int = 1) -> ChunkedKL:
    """The calling thread's cached handle for t's device and dtype, with d = t's last dimension
    and V rows of W: for the calls that need no teacher cache (embed, act8_*, norm*)."""
    index = t.get_device()
    if index < 0:
        raise ValueError("inputs must be CUDA tensors")
    d = t.shape[-1]
    key = (index, t.dtype, V, d)
    try:
        h = _OP_HANDLES.handles[key]
        if h._h:  # not closed by who had it before
            return h
    except AttributeError:
        _OP_HANDLES.handles = {}
    except KeyError:
        pass
    h = _OP_HANDLES.handles[key] = ChunkedKL(V, d, 1, dtype=t.dtype, max_chunk=1, device=t.device)
    return h


class _EmbeddingFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, W, ids, mask, scale, handle, check):
        ctx.save_for_backward(ids, mask)
        ctx.w_dtype, ctx.scale, ctx.handle, ctx.check = W.dtype, scale, handle, check
        return handle.embed(ids, W.detach(), mask, scale, sync=False)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        ids, mask = ctx.saved_tensors
        dW = ctx.handle.embed_grad(ids, g.contiguous(), mask, ctx.scale, sync=ctx.check)
        return dW.to(ctx.w_dtype), None, None, None, None, None


def embedding(ids, W, mask=None, scale: float = 1.0, handle: ChunkedKL | None = None,
              check: bool = True):
    """Autograd-friendly scale * W[ids] (zeros, and no gradient, for tokens with mask 0). W's
    gradient is formed in fp32 by sorted tokens and does not change from run to run.

    check=True: CKLError if an id was outside [0, V), raised by backward(), which waits, or by this
    call, which waits then, where W gets no gradient (grad mode off or a frozen W); only a call
    captured in a CUDA graph waits for nothing. Until a call has waited, the status of an id out of
    range stays in the handle (operator_handle(W, W.shape[0])), whose next waiting call raises it.
    check=False: nothing waits, as a step captured in a CUDA graph needs, and handle.sync_status()
    tells. Before that capture, as with any operator: run the step once on a side stream, and let go
    of whatever still holds an eager graph of the same leaves."""
    if handle is None:
        handle = operator_handle(W, W.shape[0])
    if check and not (torch.is_grad_enabled() and W.requires_grad):  # no backward pass to tell
        with torch.cuda.device(handle._index):
            capturing = torch.cuda.is_current_stream_capturing()
        return handle.embed(ids, W.detach(), mask, scale, sync=not capturing)
    return _EmbeddingFn.apply(W, ids, mask, scale, handle, check)


class _RmsNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gain, residual, eps, fmt, handle):
        flat = x.detach().view(-1, handle.d)
        res = None if residual is None else residual.detach().view(-1, handle.d)
        y, s, ckpt = handle.norm(flat, gain.detach(), res, eps, fmt)
        ctx.save_for_backward(ckpt._buf, gain)
        ctx.desc, ctx.handle, ctx.has_residual = ckpt._desc, handle, residual is not None
        ctx.base = ckpt._buf.data_ptr()
        ctx.set_materialize_grads(False)
        return y.view(x.shape) if residual is None else (y.view(x.shape), s.view(x.shape))

    @staticmethod
    @once_differentiable
    def backward(ctx, dY, d_sum=None):
        buf, gain = ctx.saved_tensors
        if dY is None:  # only s was used
            return d_sum, None, d_sum if ctx.has_residual else None, None, None, None
        h = ctx.handle
        flat = [None if g is None else g.contiguous().view(-1, h.d) for g in (dY, d_sum)]
        # what was saved may have been away (saved-tensor hooks) and be back at another address
        to = buf.data_ptr() - ctx.base
        ckpt = Act8._of(buf, tuple(p + to for p in ctx.desc[:3]) + ctx.desc[3:])
        dX, dgain = h.norm_bwd(flat[0], ckpt, gain.detach(), flat[1])
        dX = dX.view(dY.shape)
        return dX, dgain.to(gain.dtype), dX if ctx.has_residual else None, None, None, None


def rms_norm(x, gain, residual=None, eps: float = 1e-5, fmt: str = "int8",
             handle: ChunkedKL | None = None):
    """Autograd-friendly RMS norm over the last dimension; with `residual` returns (y, s) with
    s = x + residual. What is kept for the backward pass is the 8-bit checkpoint of s (fmt) and
    one float per row; the gradients are those of the norm at the checkpoint's values."""
    if handle is None:
        handle = operator_handle(x)
    if not x.is_contiguous() or (residual is not None and
                                 (not residual.is_contiguous() or residual.shape != x.shape)):
        raise ValueError("x and residual must be contiguous tensors of one shape")
    if x.dim() == 0 or x.shape[-1] != handle.d:
        raise ValueError("x's last dimension must be the handle's d")
    return _RmsNormFn.apply(x, gain, residual, eps, fmt, handle)


def forward_static(H, W, idx, logit, mask=None, chunk: int = 2048, stream=None,
                   token_stats: bool = False):
    """Forward-only loss through ckl_forward_static: no device allocation by the library.

    For callers that may not allocate device memory: the library's scratch is a
    fixed 32 MiB device array shared by all calls (overlapping calls race). The
    outputs here are allocated by torch on the caller's side; pass your own
    buffers to the C entry point if that is not allowed either. Returns the loss
    (0-d float32 tensor), plus per-token logsumexp and loss when token_stats.
    """
    f = lib().ckl_forward_static
    f.argtypes = [ctypes.c_int, ctypes.c_int, _I64, _I64, _I64, _P, _P, _P, _P, _P, _I64, _I64,
                  _P, _P, _P, _P, _P]
    f.restype = ctypes.c_int
    T, d = H.shape
    V, K = W.shape[0], idx.shape[1]
    dev = H.device
    loss = torch.empty((), dtype=torch.float32, device=dev)
    lse = ell = None
    if token_stats:
        lse = torch.empty(T, dtype=torch.float32, device=dev)
        ell = torch.empty(T, dtype=torch.float32, device=dev)
    s = stream or torch.cuda.current_stream(dev)
    host = ctypes.c_float()
    _check(f(dev.index or 0, F32 if H.dtype == torch.float32 else BF16, V, d, K, _ptr(H), _ptr(W),
             _ptr(idx), _ptr(logit), _ptr(mask), T, chunk, _ptr(loss), _ptr(lse), _ptr(ell),
             ctypes.c_void_p(s.cuda_stream), ctypes.byref(host)), "ckl_forward_static")
    return (loss, lse, ell) if token_stats else loss
