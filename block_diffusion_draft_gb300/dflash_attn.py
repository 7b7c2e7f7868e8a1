"""ctypes binding of libdflash_attn.so (include/dflash_attn.h).

Argument marshalling only: torch tensors in, their device pointers and the
current CUDA stream out to the C ABI.  Every step of the layer runs in the
library's CUDA kernels; if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from array import array
from ctypes import POINTER, byref, c_float, c_int, c_int32, c_int64, c_size_t, c_void_p
from typing import Dict, Optional, Sequence, Tuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libdflash_attn.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "dflash_attn.h")

DFLASH_BF16, DFLASH_FP32 = 0, 1
Q8_FORMATS = {"e4m3": 0, "int8": 1}
STATUS = {0: "OK", -1: "ERR_ARG", -2: "ERR_SHAPE", -3: "ERR_CAPACITY",
          -4: "ERR_RANGE", -5: "ERR_CUDA", -6: "ERR_DEVICE",
          -7: "ERR_UNSUPPORTED", -8: "ERR_MEMORY"}


class Config(ctypes.Structure):
    _fields_ = [("hidden", c_int32), ("n_heads", c_int32),
                ("n_kv_heads", c_int32), ("head_dim", c_int32),
                ("n_target_layers", c_int32), ("rms_eps", c_float),
                ("rope_theta", c_float), ("sliding_window", c_int32),
                ("max_position", c_int32), ("dtype", c_int32), ("causal", c_int32)]


class DFlashError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"{STATUS.get(code, code)}: {message}")
        self.code = code


_LIB = None

_SIGNATURES = {
    "dflash_last_error": ([], ctypes.c_char_p),
    "dflash_abi_version": ([], c_int),
    "dflash_attn_create": ([POINTER(Config)] + [c_void_p] * 8 + [POINTER(c_void_p)], c_int),
    "dflash_attn_destroy": ([c_void_p], c_int),
    "dflash_attn_reserve": ([c_void_p, c_int, c_int, c_int], c_int),
    "dflash_cache_create": ([c_void_p, c_int, c_int, POINTER(c_void_p)], c_int),
    "dflash_cache_destroy": ([c_void_p], c_int),
    "dflash_cache_lengths": ([c_void_p, POINTER(c_int32)], c_int),
    "dflash_cache_data": ([c_void_p, POINTER(c_void_p), POINTER(c_void_p)] +
                          [POINTER(c_int32)] * 4, c_int),
    "dflash_cache_read": ([c_void_p, c_void_p, c_void_p, c_void_p], c_int),
    "dflash_cache_crop": ([c_void_p, POINTER(c_int32)], c_int),
    "dflash_ctx_project": ([c_void_p, c_void_p, c_int, c_void_p, c_void_p], c_int),
    "dflash_ctx_project_noalloc": ([c_void_p, c_void_p, c_int, c_void_p, c_void_p], c_int),
    "dflash_attn_forward": ([c_void_p, c_void_p, c_int, c_int, c_void_p, c_void_p,
                             POINTER(c_int32), c_void_p, c_void_p, c_void_p], c_int),
    "dflash_attn_forward_packed": ([c_void_p, c_int, c_int, c_int, c_int, c_void_p,
                                    c_void_p, c_void_p, c_void_p, c_void_p], c_int),
    "dflash_paged_cache_create": ([c_void_p, c_int, c_int, POINTER(c_void_p)], c_int),
    "dflash_paged_cache_destroy": ([c_void_p], c_int),
    "dflash_paged_cache_data": ([c_void_p, POINTER(c_void_p), POINTER(c_void_p)] +
                                [POINTER(c_int32)] * 4, c_int),
    "dflash_paged_cache_read": ([c_void_p, c_void_p, c_void_p, c_void_p], c_int),
    "dflash_attn_forward_paged": ([c_void_p, c_void_p, c_int, c_int, c_void_p, c_void_p,
                                   POINTER(c_int32), POINTER(c_int32), c_void_p, c_void_p,
                                   c_void_p, c_int, c_void_p, c_void_p], c_int),
    "dflash_kv_group_create": ([POINTER(c_void_p), c_int, POINTER(c_void_p)], c_int),
    "dflash_kv_group_destroy": ([c_void_p], c_int),
    "dflash_kv_group_append": ([c_void_p, POINTER(c_void_p), c_int, c_void_p,
                                POINTER(c_int32), c_void_p, c_void_p], c_int),
    "dflash_mlp_create": ([c_int, c_int, c_float] + [c_void_p] * 5 + [POINTER(c_void_p)],
                          c_int),
    "dflash_mlp_destroy": ([c_void_p], c_int),
    "dflash_decoder_layer_forward": ([c_void_p, c_void_p, c_void_p, c_int, c_int, c_void_p,
                                      c_void_p, c_void_p, POINTER(c_int32), c_void_p,
                                      c_void_p, c_void_p, c_void_p], c_int),
    "dflash_q8_cache_create": ([c_void_p, c_int, c_int, c_int, POINTER(c_void_p)], c_int),
    "dflash_q8_cache_destroy": ([c_void_p], c_int),
    "dflash_q8_cache_lengths": ([c_void_p, POINTER(c_int32)], c_int),
    "dflash_q8_cache_crop": ([c_void_p, POINTER(c_int32)], c_int),
    "dflash_q8_cache_data": ([c_void_p] + [POINTER(c_void_p)] * 4 + [POINTER(c_int32)] * 4,
                             c_int),
    "dflash_q8_cache_reserve": ([c_void_p, c_int], c_int),
    "dflash_q8_cache_append": ([c_void_p, c_void_p, c_void_p, c_int64, c_int64,
                                POINTER(c_int32), c_void_p], c_int),
    "dflash_q8_cache_read": ([c_void_p, POINTER(c_int32), POINTER(c_int32), c_void_p, c_void_p,
                              c_void_p], c_int),
    "dflash_q8_attn_core": ([c_void_p, c_void_p, c_int, c_int] + [c_void_p] * 4, c_int),
    "dflash_attn_forward_q8": ([c_void_p, c_void_p, c_int, c_int, c_void_p, c_void_p,
                                POINTER(c_int32), c_void_p, c_void_p, c_void_p], c_int),
    "dflash_verify": ([c_int] * 4 + [c_void_p, c_void_p, c_int64, c_int64, c_void_p, c_int64,
                                     c_int64] + [c_void_p] * 6, c_int),
    "dflash_qk_norm_rope": ([c_void_p, c_int, c_int] + [c_void_p] * 8, c_int),
    "dflash_qk_norm_rope_workspace": ([c_void_p, POINTER(c_size_t)], c_int),
    "dflash_qk_norm_rope_backward": ([c_void_p, c_int, c_int] + [c_void_p] * 12 +
                                     [c_size_t, c_void_p], c_int),
    "dflash_linear_ce_workspace": ([c_int] * 4 + [POINTER(c_size_t)], c_int),
    "dflash_linear_ce": ([c_int] * 3 + [c_void_p, c_int64, c_void_p, c_int64] + [c_void_p] * 4 +
                         [c_size_t, c_void_p], c_int),
    "dflash_linear_ce_grad": ([c_int] * 3 + [c_void_p, c_int64, c_void_p, c_int64] +
                              [c_void_p] * 7 + [c_size_t, c_void_p], c_int),
    "dflash_grad_norm_workspace": ([c_int, POINTER(c_size_t)], c_int),
    "dflash_grad_norm": ([c_int] + [c_void_p] * 5 + [c_size_t, c_void_p], c_int),
    "dflash_clip_grad_norm": ([c_int] + [c_void_p] * 4 + [ctypes.c_double] + [c_void_p] * 2 +
                              [c_size_t, c_void_p], c_int),
    "dflash_device_error": ([c_void_p, POINTER(c_int32)], c_int),
    "dflash_wait_probe": ([c_void_p, ctypes.c_int64, c_int, c_void_p], c_int),
    "dflash_read_stream_probe": ([c_void_p, c_void_p, ctypes.c_int64, ctypes.c_int64, c_int,
                                  c_int, c_void_p], c_int),
    "dflash_kernel_launches": ([POINTER(ctypes.c_uint64)], c_int),
    "dflash_packed_attn_core": ([c_void_p, c_int, c_int, c_int, c_int] + [c_void_p] * 7, c_int),
    "dflash_packed_attn_core_backward": ([c_void_p, c_int, c_int, c_int, c_int] +
                                         [c_void_p] * 11, c_int),
    "dflash_trace_enable": ([c_void_p, c_int], c_int),
    "dflash_trace_read": ([c_void_p, c_int, POINTER(ctypes.c_double), POINTER(c_int32)],
                          c_int),
}

KERNEL_KINDS = {"fc": 0, "norm": 1, "qkv": 2, "attn": 3, "o_proj": 4, "misc": 5, "mlp": 6,
                "bwd": 7}


def declared_functions() -> list:
    """Names of the functions include/dflash_attn.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(dflash_\w+)\s*\(", text)))


def lib():
    """Load the library (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "block_diffusion_draft_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _LIB = L
    return _LIB


def check(rc: int) -> None:
    if rc != 0:
        raise DFlashError(rc, lib().dflash_last_error().decode())


def kernel_launches() -> int:
    """Kernels the library has launched in this process so far."""
    n = ctypes.c_uint64(0)
    check(lib().dflash_kernel_launches(ctypes.byref(n)))
    return n.value


def _p(t: Optional[torch.Tensor]):
    return None if t is None else c_void_p(t.data_ptr())


def _stream(dev: torch.device):
    return c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _int32_array(xs: Sequence[int]):
    if not isinstance(xs, (bytes, bytearray)):  # (an array would read those as machine words)
        try:
            return (c_int32 * len(xs)).from_buffer(array("i", xs))
        except (TypeError, OverflowError):
            pass
    return (c_int32 * len(xs))(*[int(x) for x in xs])  # as ctypes takes them: modulo 2^32


def _call(device: torch.device, f, *args) -> None:
    """f(*args, stream) with ``device`` current and its current stream, as under
    torch.cuda.device and torch.cuda.current_stream, in a tenth of their time:
    the small calls of a serving step take less of it than those two."""
    before = torch._C._cuda_getDevice()
    index = device.index
    if index is None or index == before:
        rc = f(*args, torch._C._cuda_getCurrentRawStream(before))
    else:
        torch._C._cuda_setDevice(index)
        try:
            rc = f(*args, torch._C._cuda_getCurrentRawStream(index))
        finally:
            torch._C._cuda_setDevice(before)
    if rc != 0:
        check(rc)


def _on(t: torch.Tensor, device: torch.device) -> bool:
    index = t.get_device()  # -1: not on a CUDA device
    return index == device.index or (device.index is None and index >= 0)


def _require(name: str, t: torch.Tensor, dtype: torch.dtype, device: torch.device,
             shape: Optional[tuple] = None) -> None:
    """A dense tensor of this type (and shape) on this device."""
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype is not dtype or not _on(t, device):
        raise ValueError(f"{name} must be {dtype} on {device}, got {t.dtype} on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _counts(name: str, n: Sequence[int], batch: int) -> Sequence[int]:
    if len(n) != batch:
        raise ValueError(f"{name} must hold one count for each of the {batch} sequences")
    return n


def _block_shape(noise: torch.Tensor, attn: "DFlashAttention") -> Tuple[int, int]:
    if noise.dim() != 3 or noise.shape[2] != attn.hidden:
        raise ValueError(f"noise must be [batch, q_len, {attn.hidden}], got {list(noise.shape)}")
    _require("noise", noise, torch.bfloat16, attn.device)
    return noise.shape[0], noise.shape[1]


def _rows_of(q: Optional[torch.Tensor], k: Optional[torch.Tensor]) -> Tuple[int, int]:
    x = q if q is not None else k
    if x is None or x.dim() != 4:
        raise ValueError("q or k must be given as [batch, rows, heads, head_dim]")
    return x.shape[0], x.shape[1]


def _like(x: Optional[torch.Tensor], out: Optional[torch.Tensor],
          name: str) -> Optional[torch.Tensor]:
    if x is None and out is not None:
        raise ValueError(f"{name} given without its input")
    if x is not None and out is None:
        return torch.empty(x.shape, device=x.device, dtype=x.dtype)
    return out


# Tells autograd that a call has written these tensors of the caller's: a backward
# pass that has saved one of them raises instead of using the new values.
_overwritten = torch.autograd.graph.increment_version


class DFlashAttention:
    """One draft attention layer held by the library.

    ``weights`` maps wq, wk, wv, wo, q_norm, k_norm and optionally fc,
    hidden_norm to tensors in nn.Linear [out, in] layout (any device; they are
    moved to ``device`` in ``dtype`` and copied into library memory).
    """

    def __init__(self, weights: Dict[str, torch.Tensor], *, hidden: int,
                 n_heads: int, n_kv_heads: int, head_dim: int = 0,
                 n_target_layers: int = 0, rms_eps: float = 1e-6,
                 rope_theta: float = 1e6, sliding_window: int = 0,
                 max_position: int = 0, dtype: torch.dtype = torch.bfloat16,
                 device: Optional[torch.device] = None, causal: bool = False):
        self.device = torch.device(device or "cuda")
        if self.device.type != "cuda":
            raise ValueError("the library runs on CUDA devices only")
        if dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("dtype must be bfloat16 or float32")
        self.dtype = dtype
        self.hidden, self.n_heads, self.n_kv_heads = hidden, n_heads, n_kv_heads
        self.head_dim = head_dim or hidden // n_heads
        self.cfg = Config(hidden, n_heads, n_kv_heads, self.head_dim,
                          n_target_layers, rms_eps, rope_theta, sliding_window,
                          max_position,
                          DFLASH_BF16 if dtype == torch.bfloat16 else DFLASH_FP32,
                          1 if causal else 0)
        dev_w = {k: v.to(self.device, dtype).contiguous() for k, v in weights.items()}
        fc = dev_w.get("fc") if n_target_layers > 0 else None
        hn = dev_w.get("hidden_norm") if n_target_layers > 0 else None
        h = c_void_p()
        with torch.cuda.device(self.device):
            check(lib().dflash_attn_create(
                ctypes.byref(self.cfg), _p(dev_w["wq"]), _p(dev_w["wk"]),
                _p(dev_w["wv"]), _p(dev_w["wo"]), _p(dev_w["q_norm"]),
                _p(dev_w["k_norm"]), _p(fc), _p(hn), ctypes.byref(h)))
        self.handle = h
        self._rope_ws: Optional[int] = None  # bytes of qk_norm_rope_backward's workspace

    # ---------------------------------------------------------------- calls
    def reserve(self, max_batch: int, max_rows: int, max_keys: int) -> None:
        with torch.cuda.device(self.device):
            check(lib().dflash_attn_reserve(self.handle, max_batch, max_rows, max_keys))

    def ctx_project(self, target_layers: torch.Tensor,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
        rows = target_layers.shape[0]
        if out is None:
            out = torch.empty(rows, self.hidden, device=self.device, dtype=self.dtype)
        with torch.cuda.device(self.device):
            check(lib().dflash_ctx_project(self.handle, _p(target_layers.contiguous()),
                                           rows, _p(out), _stream(self.device)))
        return out

    def forward(self, cache: "DraftCache", noise: torch.Tensor,
                target_hidden: Optional[torch.Tensor], n_ctx: Sequence[int],
                positions: torch.Tensor,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
        B, q_len, _ = noise.shape
        if out is None:
            out = torch.empty_like(noise)
        th = None if target_hidden is None or target_hidden.numel() == 0 else target_hidden
        with torch.cuda.device(self.device):
            check(lib().dflash_attn_forward(
                self.handle, cache.handle, B, q_len, _p(noise), _p(th),
                _int32_array(n_ctx), _p(positions), _p(out), _stream(self.device)))
        return out

    def forward_paged(self, cache: "PagedCache", noise: torch.Tensor,
                      target_hidden: Optional[torch.Tensor], n_ctx: Sequence[int],
                      len_before: Sequence[int], positions: torch.Tensor,
                      slot_mapping: torch.Tensor, block_table: torch.Tensor,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """forward() over a paged cache: new rows go to slot_mapping's slots
        (int32, in positions order), keys are read through block_table
        (int32 [batch, bt_stride])."""
        B, q_len, _ = noise.shape
        if out is None:
            out = torch.empty_like(noise)
        th = None if target_hidden is None or target_hidden.numel() == 0 else target_hidden
        bt = block_table.contiguous()
        with torch.cuda.device(self.device):
            check(lib().dflash_attn_forward_paged(
                self.handle, cache.handle, B, q_len, _p(noise), _p(th),
                _int32_array(n_ctx), _int32_array(len_before), _p(positions),
                _p(slot_mapping), _p(bt), bt.shape[1], _p(out), _stream(self.device)))
        return out

    def q8_core(self, cache: "Q8Cache", q: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
        """Attention of a block's queries q [B, q_len, n_heads, d] (bf16, dense,
        after norm and RoPE) over the rows an 8-bit cache holds.  Returns (out
        like q, lse [B, q_len, n_heads] fp32, natural log; a row that sees no
        key has out 0 and lse -inf)."""
        shape = q.shape
        if len(shape) != 4 or shape[0] != cache.batch or shape[2] != self.n_heads or (
                shape[3] != self.head_dim):
            raise ValueError(f"q must be [{cache.batch}, q_len, {self.n_heads}, "
                             f"{self.head_dim}], got {list(shape)}")
        _require("q", q, torch.bfloat16, self.device)
        out = torch.empty_like(q)
        lse = q.new_empty(shape[:3], dtype=torch.float32)
        _call(self.device, lib().dflash_q8_attn_core, self.handle, cache.handle, shape[0],
              shape[1], q.data_ptr(), out.data_ptr(), lse.data_ptr())
        return out, lse

    def forward_q8(self, cache: "Q8Cache", noise: torch.Tensor,
                   target_hidden: Optional[torch.Tensor], n_ctx: Sequence[int],
                   positions: torch.Tensor,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """forward() over an 8-bit cache: the new rows are encoded as they are
        appended, and the queries see the encoded rows."""
        B, q_len = _block_shape(noise, self)
        th = None if target_hidden is None or target_hidden.numel() == 0 else target_hidden
        rows = sum(_counts("n_ctx", n_ctx, B))
        if th is not None:
            if tuple(th.shape) != (rows, self.hidden):
                raise ValueError(f"target_hidden must be [{rows}, {self.hidden}], "
                                 f"got {list(th.shape)}")
            _require("target_hidden", th, torch.bfloat16, self.device)
        _require("positions", positions, torch.int32, self.device)
        if positions.numel() != rows + B * q_len:
            raise ValueError(f"positions must hold {rows + B * q_len} values, "
                             f"got {positions.numel()}")
        if out is None:
            out = torch.empty_like(noise)
        elif out.shape != noise.shape:
            raise ValueError("out must have the shape of noise")
        _require("out", out, torch.bfloat16, self.device)
        _call(self.device, lib().dflash_attn_forward_q8, self.handle, cache.handle, B, q_len,
              noise.data_ptr(), _p(th), _int32_array(n_ctx), positions.data_ptr(), out.data_ptr())
        return out

    def forward_packed(self, noise: torch.Tensor, target_hidden: torch.Tensor,
                       anchors: torch.Tensor, block_size: int,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
        B, q_total, _ = noise.shape
        seq = target_hidden.shape[1]
        nb = anchors.shape[1]
        if out is None:
            out = torch.empty_like(noise)
        with torch.cuda.device(self.device):
            check(lib().dflash_attn_forward_packed(
                self.handle, B, seq, nb, block_size, _p(noise), _p(target_hidden),
                _p(anchors), _p(out), _stream(self.device)))
        return out

    def packed_core(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    anchors: torch.Tensor, seq: int, block_size: int):
        """Packed-layout attention core: q [B, T, n_heads, d], k/v
        [B, n_kv, seq + T, d] bf16, anchors [B, n_blocks] int32.  Returns
        (out like q, lse [B, T, n_heads] fp32)."""
        B, T = q.shape[0], q.shape[1]
        out = torch.empty_like(q)
        lse = torch.empty(B, T, q.shape[2], device=q.device, dtype=torch.float32)
        with torch.cuda.device(self.device):
            check(lib().dflash_packed_attn_core(
                self.handle, B, seq, T // block_size, block_size, _p(q), _p(k), _p(v),
                _p(anchors), _p(out), _p(lse), _stream(self.device)))
        return out, lse

    def packed_core_backward(self, q, k, v, out, lse, d_out, anchors, seq: int,
                             block_size: int):
        """Gradients (dq, dk, dv) of packed_core's output given d_out."""
        B, T = q.shape[0], q.shape[1]
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        with torch.cuda.device(self.device):
            check(lib().dflash_packed_attn_core_backward(
                self.handle, B, seq, T // block_size, block_size, _p(q), _p(k), _p(v),
                _p(out), _p(lse), _p(d_out), _p(anchors), _p(dq), _p(dk), _p(dv),
                _stream(self.device)))
        return dq, dk, dv

    def qk_norm_rope(self, q: Optional[torch.Tensor], k: Optional[torch.Tensor],
                     positions: torch.Tensor, q_norm: Optional[torch.Tensor] = None,
                     k_norm: Optional[torch.Tensor] = None,
                     q_out: Optional[torch.Tensor] = None,
                     k_out: Optional[torch.Tensor] = None):
        """Per-head RMSNorm (gains q_norm, k_norm [d]; None: the layer's) and
        rotation of q [B, R, n_heads, d] and k [B, R, n_kv, d] at positions
        [B, R] (int32).  Channels are dense, other strides free; q or k may be
        None.  Results go to q_out and k_out (the inputs themselves, or any
        tensor of that shape, such as rows of packed_core's keys, transposed),
        by default dense tensors.  Returns (q_out, k_out), which carry no
        gradients: those are qk_norm_rope_backward's."""
        B, R = _rows_of(q, k)
        _require("positions", positions, torch.int32, self.device, (B, R))
        written = [t for t in (q_out, k_out) if t is not None]
        q_out, k_out = _like(q, q_out, "q_out"), _like(k, k_out, "k_out")
        v, at = self._views((B, R), q, k, q_out, k_out)
        _call(self.device, lib().dflash_qk_norm_rope, self.handle, B, R, at[0], at[1],
              self._gain("q_norm", q_norm), self._gain("k_norm", k_norm), positions.data_ptr(),
              at[2], at[3])
        if written:
            _overwritten(written)
        return q_out, k_out

    def qk_norm_rope_backward(self, q: Optional[torch.Tensor], k: Optional[torch.Tensor],
                              positions: torch.Tensor, q_norm: Optional[torch.Tensor],
                              k_norm: Optional[torch.Tensor], d_q: Optional[torch.Tensor],
                              d_k: Optional[torch.Tensor],
                              dq_out: Optional[torch.Tensor] = None,
                              dk_out: Optional[torch.Tensor] = None):
        """Gradients of qk_norm_rope's inputs: q, k, positions and gains as
        given there, d_q and d_k the gradients of its outputs.  Returns (dq, dk,
        d_q_norm, d_k_norm), the gains' in fp32, None for q or k None."""
        B, R = _rows_of(q, k)
        _require("positions", positions, torch.int32, self.device, (B, R))
        if (q is None) != (d_q is None) or (k is None) != (d_k is None):
            raise ValueError("d_q and d_k must be given exactly where q and k are")
        written = [t for t in (dq_out, dk_out) if t is not None]
        dq_out, dk_out = _like(q, dq_out, "dq_out"), _like(k, dk_out, "dk_out")
        v, at = self._views((B, R), q, k, d_q, d_k, dq_out, dk_out)
        if self._rope_ws is None:
            n = c_size_t(0)
            check(lib().dflash_qk_norm_rope_workspace(self.handle, byref(n)))
            self._rope_ws = n.value
        dev = self.device
        d_gain = [None if t is None else torch.empty(self.head_dim, device=dev,
                                                     dtype=torch.float32) for t in (q, k)]
        ws = torch.empty(self._rope_ws, device=dev, dtype=torch.uint8)
        _call(self.device, lib().dflash_qk_norm_rope_backward, self.handle, B, R, at[0], at[1],
              self._gain("q_norm", q_norm), self._gain("k_norm", k_norm), positions.data_ptr(),
              at[2], at[3], at[4], at[5], None if q is None else d_gain[0].data_ptr(),
              None if k is None else d_gain[1].data_ptr(), ws.data_ptr(), self._rope_ws)
        if written:
            _overwritten(written)
        return dq_out, dk_out, d_gain[0], d_gain[1]

    def _views(self, rows: Tuple[int, int], *tensors: Optional[torch.Tensor]):
        """dflash_heads of tensors of queries and keys in turn: an array of
        (address, batch, row and head stride) that has to outlive the call, and
        the addresses of its parts (None for None)."""
        flat, at, dt, d, dev = [], [], self.dtype, self.head_dim, self.device
        index = dev.index
        shape, other = (*rows, self.n_heads, d), (*rows, self.n_kv_heads, d)
        for t in tensors:
            if t is None:
                flat += (0, 0, 0, 0)
                at.append(None)
            else:
                s = t.stride()
                on = t.get_device()  # (as _on, without its calls)
                if t.shape != shape or t.dtype is not dt or on < 0 or (
                        on != index and index is not None):
                    raise ValueError(f"queries must be {[*rows, self.n_heads, d]} and keys "
                                     f"{[*rows, self.n_kv_heads, d]}, {dt} on {dev}, got "
                                     f"{list(t.shape)}, {t.dtype} on {t.device}")
                if s[3] != 1 and t.numel():
                    raise ValueError("a head's channels must be dense")
                at.append(8 * len(flat))
                flat += (t.data_ptr() or 16, s[0], s[1], s[2])  # (no data: no rows)
            shape, other = other, shape
        v = array("q", flat)
        base = v.buffer_info()[0]
        return v, [x if x is None else base + x for x in at]

    def _gain(self, name: str, t: Optional[torch.Tensor]) -> Optional[int]:
        if t is None:
            return None
        _require(name, t, self.dtype, self.device, (self.head_dim,))
        return t.data_ptr()

    def trace(self, enable: bool) -> None:
        """Start (fresh) or stop recording CUDA events around each launch."""
        with torch.cuda.device(self.device):
            check(lib().dflash_trace_enable(self.handle, 1 if enable else 0))

    def trace_read(self) -> dict:
        """{kernel kind: (total ms, launches)} of the current trace."""
        res = {}
        for name, kind in KERNEL_KINDS.items():
            ms, n = ctypes.c_double(0), c_int32(0)
            with torch.cuda.device(self.device):
                check(lib().dflash_trace_read(self.handle, kind, ctypes.byref(ms),
                                              ctypes.byref(n)))
            if n.value:
                res[name] = (ms.value, n.value)
        return res

    def device_error(self) -> int:
        code = c_int32(0)
        with torch.cuda.device(self.device):
            rc = lib().dflash_device_error(self.handle, ctypes.byref(code))
        if rc not in (0, -6):
            check(rc)
        return code.value

    def wait_probe(self, limit_ns: int, arrive: bool) -> None:
        """One bounded device wait of at most limit_ns on the current stream
        (arrive=False: a barrier nothing completes, so the wait runs out and
        records DFLASH_DEV_WAIT_TIMEOUT; read it with device_error())."""
        with torch.cuda.device(self.device):
            check(lib().dflash_wait_probe(self.handle, int(limit_ns), int(bool(arrive)),
                                          _stream(self.device)))

    def read_stream_probe(self, matrix: torch.Tensor, ctas: int, stages: int) -> None:
        """Enqueue one TMA read pass over a bf16 [rows, cols] matrix on the
        current stream (measurement aid: the weight boxes of the GEMMs,
        `stages` boxes in flight per CTA, data discarded)."""
        if matrix.dtype != torch.bfloat16 or matrix.dim() != 2 or not matrix.is_contiguous():
            raise ValueError("matrix must be a contiguous 2-D bf16 tensor")
        with torch.cuda.device(self.device):
            check(lib().dflash_read_stream_probe(self.handle, _p(matrix), matrix.shape[0],
                                                 matrix.shape[1], int(ctas), int(stages),
                                                 _stream(self.device)))

    def close(self) -> None:
        if getattr(self, "handle", None):
            with torch.cuda.device(self.device):
                lib().dflash_attn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class DraftCache:
    """Draft KV cache held by the library ([batch][n_kv][capacity][head_dim])."""

    def __init__(self, attn: DFlashAttention, batch: int, capacity: int):
        self.attn = attn
        self.batch, self.capacity = batch, capacity
        h = c_void_p()
        with torch.cuda.device(attn.device):
            check(lib().dflash_cache_create(attn.handle, batch, capacity, ctypes.byref(h)))
        self.handle = h

    def lengths(self) -> list:
        arr = (c_int32 * self.batch)()
        check(lib().dflash_cache_lengths(self.handle, arr))
        return list(arr)

    def crop(self, keep: Sequence[int]) -> None:
        check(lib().dflash_cache_crop(self.handle, _int32_array(keep)))

    def read(self):
        """Copies of the K and V storage as [batch, n_kv, capacity, head_dim]."""
        a = self.attn
        shape = (self.batch, a.n_kv_heads, self.capacity, a.head_dim)
        k = torch.empty(shape, device=a.device, dtype=a.dtype)
        v = torch.empty(shape, device=a.device, dtype=a.dtype)
        with torch.cuda.device(a.device):
            check(lib().dflash_cache_read(self.handle, _p(k), _p(v), _stream(a.device)))
        return k, v

    def close(self) -> None:
        if getattr(self, "handle", None):
            lib().dflash_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagedCache:
    """Paged KV storage held by the library ([n_pages][n_kv][page_size]
    [head_dim] for K and for V); lengths and page tables are the caller's."""

    def __init__(self, attn: DFlashAttention, n_pages: int, page_size: int):
        self.attn = attn
        self.n_pages, self.page_size = n_pages, page_size
        h = c_void_p()
        with torch.cuda.device(attn.device):
            check(lib().dflash_paged_cache_create(attn.handle, n_pages, page_size,
                                                  ctypes.byref(h)))
        self.handle = h

    def read(self):
        """Copies of the K and V storage as [n_pages, n_kv, page_size, head_dim]."""
        a = self.attn
        shape = (self.n_pages, a.n_kv_heads, self.page_size, a.head_dim)
        k = torch.empty(shape, device=a.device, dtype=a.dtype)
        v = torch.empty(shape, device=a.device, dtype=a.dtype)
        with torch.cuda.device(a.device):
            check(lib().dflash_paged_cache_read(self.handle, _p(k), _p(v), _stream(a.device)))
        return k, v

    def close(self) -> None:
        if getattr(self, "handle", None):
            lib().dflash_paged_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Q8Cache:
    """Draft KV cache in 8 bits held by the library: one code byte per channel
    and a power-of-two scale per 32 channels (``fmt`` "int8" or "e4m3"; see
    dflash_q8_cache_* in include/dflash_attn.h)."""

    def __init__(self, attn: DFlashAttention, batch: int, capacity: int, fmt: str = "int8"):
        if fmt not in Q8_FORMATS:
            raise ValueError(f"fmt must be one of {sorted(Q8_FORMATS)}")
        self.attn = attn
        self.batch, self.capacity, self.fmt = batch, capacity, fmt
        h = c_void_p()
        with torch.cuda.device(attn.device):
            check(lib().dflash_q8_cache_create(attn.handle, batch, capacity, Q8_FORMATS[fmt],
                                               ctypes.byref(h)))
        self.handle = h

    def lengths(self) -> list:
        arr = (c_int32 * self.batch)()
        check(lib().dflash_q8_cache_lengths(self.handle, arr))
        return list(arr)

    def crop(self, keep: Sequence[int]) -> None:
        check(lib().dflash_q8_cache_crop(self.handle, _int32_array(
            _counts("keep", keep, self.batch))))

    def reserve(self, max_new_rows: int) -> None:
        """Size the scratch of forward_q8 calls that append at most this many
        rows to a sequence."""
        with torch.cuda.device(self.attn.device):
            check(lib().dflash_q8_cache_reserve(self.handle, max_new_rows))

    def append(self, k: torch.Tensor, v: torch.Tensor, n: Sequence[int]) -> None:
        """Encode n[b] rows behind those of sequence b, from k and v [sum n,
        n_kv, d] bf16: the sequences' rows one after another.  A row's heads
        are dense; rows may be slices of a wider tensor."""
        a = self.attn
        rows = sum(_counts("n", n, self.batch))
        shape = (rows, a.n_kv_heads, a.head_dim)
        strides = []
        for name, t in (("k", k), ("v", v)):
            if t.shape != shape:
                raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
            if t.dtype is not torch.bfloat16 or not _on(t, a.device):
                raise ValueError(f"{name} must be bfloat16 on {a.device}, "
                                 f"got {t.dtype} on {t.device}")
            s = t.stride()
            dense = s[2] == 1 and (s[1] == a.head_dim or a.n_kv_heads == 1)
            if rows > 0 and not dense:
                raise ValueError(f"{name}: a row's heads must be dense")
            strides.append(s[0] if rows > 1 else a.n_kv_heads * a.head_dim)
        _call(a.device, lib().dflash_q8_cache_append, self.handle, k.data_ptr(), v.data_ptr(),
              strides[0], strides[1], _int32_array(n))

    def read(self, first: Optional[Sequence[int]] = None, n: Optional[Sequence[int]] = None):
        """K and V [sum n, n_kv, d] bf16 of rows first[b] .. first[b] + n[b] - 1
        of every sequence, one sequence after another (default: every row)."""
        a = self.attn
        first = [0] * self.batch if first is None else _counts("first", first, self.batch)
        if n is None:
            n = [length - f for length, f in zip(self.lengths(), first)]
        shape = (max(0, sum(_counts("n", n, self.batch))), a.n_kv_heads, a.head_dim)
        k = torch.empty(shape, device=a.device, dtype=torch.bfloat16)
        v = torch.empty_like(k)
        _call(a.device, lib().dflash_q8_cache_read, self.handle, _int32_array(first),
              _int32_array(n), k.data_ptr(), v.data_ptr())
        return k, v

    def close(self) -> None:
        if getattr(self, "handle", None):
            lib().dflash_q8_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def verify_draft(draft_tokens: torch.Tensor, draft_probs: Optional[torch.Tensor],
                 target_probs: torch.Tensor, u_accept: torch.Tensor, u_sample: torch.Tensor,
                 n_draft: Optional[torch.Tensor] = None):
    """Verify drafted tokens [B, D] (int32) against the target's probabilities
    [B, D + 1, V] (fp32 or bf16, a row's values dense, other strides free) from
    uniform numbers u_accept [B, D] and u_sample [B] (fp32).  draft_probs [B, D,
    V] are the distributions the drafts were drawn from, None if they were
    chosen without sampling; n_draft [B] (int32) are the drafts of each
    sequence where they differ.  Returns (accepted [B], tokens [B, D + 1])
    int32: the number of accepted drafts, and those followed by one drawn token
    and -1s.  See dflash_verify in include/dflash_attn.h."""
    if draft_tokens.dim() != 2 or target_probs.dim() != 3:
        raise ValueError("draft_tokens must be [B, D] and target_probs [B, D + 1, V]")
    B, D = draft_tokens.shape
    V, dev, dt = target_probs.shape[2], target_probs.device, target_probs.dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise ValueError("probabilities must be float32 or bfloat16")
    if not target_probs.is_cuda:
        raise ValueError("the library runs on CUDA devices only")
    _require("draft_tokens", draft_tokens, torch.int32, dev)
    _require("u_accept", u_accept, torch.float32, dev, (B, D))
    _require("u_sample", u_sample, torch.float32, dev, (B,))
    if n_draft is not None:
        _require("n_draft", n_draft, torch.int32, dev, (B,))
    q, q_strides = None, (0, 0)
    if draft_probs is not None:
        q_strides = _probabilities("draft_probs", draft_probs, dt, dev, (B, D, V))
        q = draft_probs.data_ptr()
    p_strides = _probabilities("target_probs", target_probs, dt, dev, (B, D + 1, V))
    accepted = u_sample.new_empty((B,), dtype=torch.int32)
    tokens = u_sample.new_empty((B, D + 1), dtype=torch.int32)
    _call(dev, lib().dflash_verify, B, D, V, DFLASH_BF16 if dt == torch.bfloat16 else DFLASH_FP32,
          draft_tokens.data_ptr(), q, q_strides[0], q_strides[1], target_probs.data_ptr(),
          p_strides[0], p_strides[1], u_accept.data_ptr(), u_sample.data_ptr(), _p(n_draft),
          accepted.data_ptr(), tokens.data_ptr())
    return accepted, tokens


def _probabilities(name: str, t: torch.Tensor, dtype: torch.dtype, device: torch.device,
                   shape: Tuple[int, int, int]) -> Tuple[int, ...]:
    """The strides of a tensor of rows of probabilities, each row dense."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype is not dtype or not _on(t, device):
        raise ValueError(f"{name} must be {dtype} on {device}, got {t.dtype} on {t.device}")
    strides = t.stride()
    if strides[2] != 1 and shape[2] > 1 and t.numel():
        raise ValueError(f"{name}: a row's values must be dense")
    return strides


def linear_cross_entropy(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor):
    """Cross entropy of a linear head: x [N, H] and w [V, H] bf16 (rows dense,
    H a multiple of 8), targets [N] int32, one outside [0, V) for a row that does
    not count.  Returns (nll, lse) [N] fp32: logsumexp(x w^T) - (x w^T)[target]
    and logsumexp(x w^T), 0 for rows that do not count.  The logits are never
    held.  Neither result carries gradients, whatever x and w require: in a sum
    of losses this one's part comes from linear_cross_entropy_grad.  See
    dflash_linear_ce in include/dflash_attn.h."""
    nll, lse, _, _ = _linear_ce(x, w, targets, None, 0)
    return nll, lse


def linear_cross_entropy_grad(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor,
                              d_nll: torch.Tensor, need_dw: bool = True):
    """linear_cross_entropy and the gradients of sum(d_nll * nll) (d_nll [N]
    fp32, the rows' weights in the loss) in one call.  Returns (nll, lse, dx [N,
    H] bf16, dw [V, H] bf16 or None: a head that is not trained needs none), which
    the caller passes on (``x.backward(dx)``, ``w.grad = dw``): autograd knows
    nothing of them."""
    return _linear_ce(x, w, targets, d_nll, 2 if need_dw else 1)


@functools.lru_cache(maxsize=64)
def _linear_ce_workspace(rows: int, vocab: int, hidden: int, grads: int) -> int:
    size = c_size_t(0)
    check(lib().dflash_linear_ce_workspace(rows, vocab, hidden, grads, byref(size)))
    return size.value


def _linear_ce(x, w, targets, d_nll, grads: int):
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError(f"x must be [N, H] and w [V, H], got {list(x.shape)} and "
                         f"{list(w.shape)}")
    (N, H), V, dev = x.shape, w.shape[0], w.device
    if dev.type != "cuda":
        raise ValueError("the library runs on CUDA devices only")
    if x.dtype is not torch.bfloat16 or w.dtype is not torch.bfloat16 or x.device != dev:
        raise ValueError(f"x and w must be bfloat16 on {dev}, got {x.dtype} on {x.device} and "
                         f"{w.dtype}")
    xs, ws = x.stride(), w.stride()
    if (xs[1] != 1 and H > 1 and x.numel()) or (ws[1] != 1 and H > 1 and w.numel()):
        raise ValueError("x, w: a row's values must be dense")
    _require("targets", targets, torch.int32, dev, (N,))
    if grads:
        _require("d_nll", d_nll, torch.float32, dev, (N,))
    size = _linear_ce_workspace(N, V, H, grads)
    space = torch.empty(size, device=dev, dtype=torch.uint8)
    nll = torch.empty(N, device=dev, dtype=torch.float32)
    lse = torch.empty(N, device=dev, dtype=torch.float32)
    if not grads:
        _call(dev, lib().dflash_linear_ce, N, V, H, x.data_ptr(), xs[0], w.data_ptr(), ws[0],
              targets.data_ptr(), nll.data_ptr(), lse.data_ptr(), space.data_ptr(), size)
        return nll, lse, None, None
    dx = torch.empty((N, H), device=dev, dtype=torch.bfloat16)
    dw = torch.empty((V, H), device=dev, dtype=torch.bfloat16) if grads == 2 else None
    _call(dev, lib().dflash_linear_ce_grad, N, V, H, x.data_ptr(), xs[0], w.data_ptr(), ws[0],
          targets.data_ptr(), d_nll.data_ptr(), nll.data_ptr(), lse.data_ptr(), dx.data_ptr(),
          None if dw is None else dw.data_ptr(), space.data_ptr(), size)
    return nll, lse, dx, dw


def grad_norm(grads: Sequence[torch.Tensor]) -> torch.Tensor:
    """The norm of all values of the tensors (fp32 or bf16, dense, one device)
    as an fp32 scalar on their device; see dflash_grad_norm."""
    return _grad_norm(grads, None, None)


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float,
                   out: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
    """Scale the tensors by max_norm / norm where their norm (as grad_norm) is
    above max_norm, in place or into ``out`` (as grads).  Gradients with an
    infinity or NaN among them stay as they are.  Returns the norm before
    clipping, on the device.  See dflash_clip_grad_norm in
    include/dflash_attn.h."""
    return _grad_norm(grads, float(max_norm), out)


_GRAD_TYPES = {torch.bfloat16: DFLASH_BF16, torch.float32: DFLASH_FP32}


@functools.lru_cache(maxsize=64)
def _grad_norm_workspace(n: int) -> int:
    size = c_size_t(0)
    check(lib().dflash_grad_norm_workspace(n, byref(size)))
    return size.value


def _grad_norm(grads, max_norm, out) -> torch.Tensor:
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    dev, n = grads[0].device, len(grads)
    index = dev.index
    if dev.type != "cuda":
        raise ValueError("the library runs on CUDA devices only")
    # (whole lists at a time: a training step has hundreds of tensors)
    types = [_GRAD_TYPES.get(g.dtype) for g in grads]
    if None in types or any([g.get_device() != index for g in grads]):
        raise ValueError(f"gradients must be float32 or bfloat16 on {dev}")
    dense = [g.is_contiguous() for g in grads]
    if not all(dense) and not all([c or _dense(g) for c, g in zip(dense, grads)]):
        raise ValueError("gradients must be dense")
    ptrs = array("Q", [g.data_ptr() for g in grads])
    outs = None
    if out is not None:
        out = list(out)
        if len(out) != n:
            raise ValueError(f"out must hold {n} tensors, got {len(out)}")
        for g, o, c in zip(grads, out, dense):
            if o.dtype is not g.dtype or o.get_device() != index or o.shape != g.shape or not (
                    c and o.is_contiguous() or o.stride() == g.stride() or g.numel() <= 1):
                raise ValueError("out must have the gradients' shapes, strides, types and device")
        outs = array("Q", [o.data_ptr() for o in out])
    counts, types = array("q", [g.numel() for g in grads]), array("i", types)
    size = _grad_norm_workspace(n)
    ws = torch.empty(size, device=dev, dtype=torch.uint8)
    norm = torch.empty((), device=dev, dtype=torch.float32)
    lists = [a if a is None else a.buffer_info()[0] for a in (ptrs, outs, counts, types)]
    if max_norm is None:
        _call(dev, lib().dflash_grad_norm, n, lists[0], lists[2], lists[3], norm.data_ptr(),
              ws.data_ptr(), size)
    else:
        _call(dev, lib().dflash_clip_grad_norm, n, *lists, max_norm, norm.data_ptr(),
              ws.data_ptr(), size)
        _overwritten(grads if out is None else out)
    return norm


def _dense(t: torch.Tensor) -> bool:
    """Whether a tensor's values fill one run of memory, in any order of axes."""
    if t.is_contiguous():
        return True
    run = 1
    for stride, size in sorted(zip(t.stride(), t.shape)):
        if size == 1:
            continue
        if stride != run:
            return False
        run *= size
    return True


class KVGroup:
    """Context K/V of several layers from one projection (the layers' K and V
    weights stacked); see dflash_kv_group_* in include/dflash_attn.h."""

    def __init__(self, layers: Sequence[DFlashAttention]):
        self.layers = list(layers)
        self.device = self.layers[0].device
        arr = (c_void_p * len(self.layers))(*[l.handle.value for l in self.layers])
        h = c_void_p()
        with torch.cuda.device(self.device):
            check(lib().dflash_kv_group_create(arr, len(self.layers), ctypes.byref(h)))
        self.handle = h

    def append(self, caches: Sequence["DraftCache"], target_hidden: Optional[torch.Tensor],
               n_ctx: Sequence[int], positions: Optional[torch.Tensor]) -> None:
        """Append the new context rows' K/V of every layer to its cache."""
        arr = (c_void_p * len(caches))(*[c.handle.value for c in caches])
        th = None if target_hidden is None or target_hidden.numel() == 0 else target_hidden
        with torch.cuda.device(self.device):
            check(lib().dflash_kv_group_append(self.handle, arr, len(n_ctx), _p(th),
                                               _int32_array(n_ctx), _p(positions),
                                               _stream(self.device)))

    def close(self) -> None:
        if getattr(self, "handle", None):
            with torch.cuda.device(self.device):
                lib().dflash_kv_group_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class DecoderMLP:
    """Norms and Qwen3 MLP of a draft decoder layer (dflash_mlp_*): weights
    ``gate``, ``up`` [intermediate, hidden], ``down`` [hidden, intermediate],
    ``input_norm``, ``post_norm`` [hidden], all bf16."""

    def __init__(self, w: dict, hidden: int, intermediate: int, rms_eps: float = 1e-6,
                 device="cuda"):
        self.device = torch.device(device)
        self.hidden, self.intermediate = hidden, intermediate
        with torch.cuda.device(self.device):
            self._w = {k: w[k].to(self.device, torch.bfloat16).contiguous()
                       for k in ("gate", "up", "down", "input_norm", "post_norm")}
            h = c_void_p()
            check(lib().dflash_mlp_create(hidden, intermediate, rms_eps,
                                          *[_p(self._w[k]) for k in ("gate", "up", "down",
                                                                      "input_norm", "post_norm")],
                                          ctypes.byref(h)))
        self._w = None  # the library holds copies
        self.handle = h

    def layer_forward(self, attn: DFlashAttention, cache: "DraftCache", hidden: torch.Tensor,
                      residual: Optional[torch.Tensor], target_hidden: Optional[torch.Tensor],
                      n_ctx: Sequence[int], positions: torch.Tensor):
        """One decoder layer; returns (hidden_out, residual_out)."""
        B, q_len, _ = hidden.shape
        out = torch.empty_like(hidden)
        res = torch.empty_like(hidden)
        th = None if target_hidden is None or target_hidden.numel() == 0 else target_hidden
        with torch.cuda.device(self.device):
            check(lib().dflash_decoder_layer_forward(
                attn.handle, self.handle, cache.handle, B, q_len, _p(hidden), _p(residual),
                _p(th), _int32_array(n_ctx), _p(positions), _p(out), _p(res),
                _stream(self.device)))
        return out, res

    def layer_forward_into(self, attn: DFlashAttention, cache: "DraftCache",
                           hidden: torch.Tensor, residual: Optional[torch.Tensor],
                           target_hidden: Optional[torch.Tensor], n_ctx: Sequence[int],
                           positions: torch.Tensor, out: torch.Tensor,
                           residual_out: torch.Tensor) -> None:
        """layer_forward writing into caller-owned output tensors."""
        B, q_len, _ = hidden.shape
        th = None if target_hidden is None or target_hidden.numel() == 0 else target_hidden
        with torch.cuda.device(self.device):
            check(lib().dflash_decoder_layer_forward(
                attn.handle, self.handle, cache.handle, B, q_len, _p(hidden), _p(residual),
                _p(th), _int32_array(n_ctx), _p(positions), _p(out), _p(residual_out),
                _stream(self.device)))

    def close(self) -> None:
        if getattr(self, "handle", None):
            with torch.cuda.device(self.device):
                lib().dflash_mlp_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
