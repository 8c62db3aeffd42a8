"""GB300-native fused attention over an FP8 E4M3 KV cache.

Python binding of the C ABI in include/fp8kv.h.  The functions below carry
the C names and do argument marshalling only (torch tensors -> device
pointers, the current torch stream -> cudaStream_t); every step of the path
runs in the library's CUDA kernels.  torch provides device memory and streams.

    cache = Fp8KVCache.contiguous(batch, kv_heads, head_dim, max_tokens, "k8v8")
    fp8kv_append(cache, k_new, v_new, seq_idx, pos)
    out = fp8kv_decode_attention(q, cache, seq_lens)
    out = fp8kv_prefill_attention(q, cache, q_pos0)
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional

import torch

from ._lib import EXPORTS, CacheStruct, get_lib

K8V8, K16V8, K16V16, K8V16, MXK8V8 = 0, 1, 2, 3, 4
DTYPES = {"k8v8": K8V8, "k16v8": K16V8, "k16v16": K16V16, "k8v16": K8V16, "mxk8v8": MXK8V8}
LAYOUT_CONTIGUOUS, LAYOUT_PAGED = 0, 1
OUT_BF16, OUT_F32 = 0, 1

DEVERR_SEQ_TOO_LONG, DEVERR_BAD_PAGE, DEVERR_TIMEOUT, DEVERR_NO_PAGES, DEVERR_BAD_TREE = 0x1, 0x2, 0x4, 0x8, 0x10
STEP_EARLY_CACHE_READ = 0x1
KERNEL_AUTO, KERNEL_CUDA_CORES, KERNEL_TENSOR_CORES = 0, 1, 2
KERNEL_TENSOR_CORES_K_F16, KERNEL_TENSOR_CORES_K_F16_PRODUCER, KERNEL_WARP_MMA = 3, 4, 5
KERNELS = {"auto": KERNEL_AUTO, "cuda_cores": KERNEL_CUDA_CORES, "tensor_cores": KERNEL_TENSOR_CORES,
           "tensor_cores_k_f16": KERNEL_TENSOR_CORES_K_F16,
           "tensor_cores_k_f16_producer": KERNEL_TENSOR_CORES_K_F16_PRODUCER, "warp_mma": KERNEL_WARP_MMA}

STATUS_NAMES = {0: "FP8KV_OK", 1: "FP8KV_ERR_INVALID_ARG", 2: "FP8KV_ERR_UNSUPPORTED",
                3: "FP8KV_ERR_WORKSPACE", 4: "FP8KV_ERR_CUDA", 5: "FP8KV_ERR_TIMEOUT",
                6: "FP8KV_ERR_DEVICE_CHECK"}


class Fp8KVError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = get_lib().fp8kv_status_string(status).decode()
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({msg})")


def _check(status: int, where: str):
    if status != 0:
        raise Fp8KVError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t: torch.Tensor, dtype, name, host_ok=False):
    """A contiguous CUDA tensor of `dtype` (or, where host_ok, a contiguous
    page-locked host tensor, which the kernels address directly)."""
    where_ok = t.is_cuda or (host_ok and t.is_pinned())
    if t.dtype != dtype or not where_ok or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor"
                         f"{' (or pinned host tensor)' if host_ok else ''}, got "
                         f"{t.dtype} on {t.device} (contiguous={t.is_contiguous()})")


class Fp8KVCache:
    """Device tensors of one KV cache (allocated with torch) and the C struct
    that describes them.  Layouts are those of include/fp8kv.h."""

    def __init__(self, *, dtype, layout, batch, kv_heads, head_dim, k, v, k_scale, v_scale,
                 max_tokens=0, page_size=0, num_pages=0, page_table=None, k_bias=None, rope_cos=None,
                 rope_sin=None):
        self.dtype = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
        self.layout = layout
        self.batch, self.kv_heads, self.head_dim = batch, kv_heads, head_dim
        self.max_tokens, self.page_size, self.num_pages = max_tokens, page_size, num_pages
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.page_table = page_table
        if k_bias is not None:
            _need(k_bias, torch.float32, "k_bias")
        self.k_bias = k_bias
        if (rope_cos is None) != (rope_sin is None):
            raise ValueError("rope_cos and rope_sin come together")
        if rope_cos is not None:
            for t, name in ((rope_cos, "rope_cos"), (rope_sin, "rope_sin")):
                _need(t, torch.float32, name)
                if t.dim() != 2 or t.shape[1] != head_dim // 2 or t.shape != rope_cos.shape:
                    raise ValueError(f"{name}: want [positions, head_dim / 2] fp32, got {tuple(t.shape)}")
        self.rope_cos, self.rope_sin = rope_cos, rope_sin
        self._struct = CacheStruct(
            dtype=self.dtype, layout=layout, batch=batch, kv_heads=kv_heads, head_dim=head_dim,
            max_tokens=max_tokens, page_size=page_size, num_pages=num_pages,
            max_pages_per_seq=0 if page_table is None else page_table.shape[1],
            rope_positions=0 if rope_cos is None else rope_cos.shape[0],
            k=k.data_ptr(), v=v.data_ptr(),
            k_scale=None if k_scale is None else k_scale.data_ptr(),
            v_scale=None if v_scale is None else v_scale.data_ptr(),
            page_table=None if page_table is None else page_table.data_ptr(),
            k_bias=None if k_bias is None else k_bias.data_ptr(),
            rope_cos=None if rope_cos is None else rope_cos.data_ptr(),
            rope_sin=None if rope_sin is None else rope_sin.data_ptr())

    @property
    def struct_ref(self):
        return ctypes.byref(self._struct)

    @property
    def capacity(self) -> int:
        if self.layout == LAYOUT_PAGED:
            return self.page_table.shape[1] * self.page_size
        return self.max_tokens

    @staticmethod
    def _alloc(dtype, lead, head_dim, device):
        dt = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
        k8, v8 = dt in (K8V8, K8V16, MXK8V8), dt in (K8V8, K16V8, MXK8V8)
        kel = torch.uint8 if k8 else torch.bfloat16
        vel = torch.uint8 if v8 else torch.bfloat16
        k = torch.zeros(lead + (head_dim,), dtype=kel, device=device)
        v = torch.zeros(lead + (head_dim,), dtype=vel, device=device)
        if dt == MXK8V8:    # the four E8M0 block bytes of each row in its 4-byte slot
            ks = torch.zeros(lead + (4,), dtype=torch.uint8, device=device)
        else:
            ks = torch.zeros(lead, dtype=torch.float32, device=device) if k8 else None
        vs = torch.zeros(lead, dtype=torch.float32, device=device) if v8 else None
        return k, v, ks, vs

    @classmethod
    def contiguous(cls, batch, kv_heads, head_dim, max_tokens, dtype="k8v8", device="cuda", k_bias=None,
                   rope_cos=None, rope_sin=None):
        """k_bias: optional [kv_heads, head_dim] fp32 key bias; the cache then
        holds pre-bias residual keys (include/fp8kv.h, fp8kv_cache.k_bias).
        rope_cos, rope_sin: optional [positions, head_dim / 2] fp32 rotary
        tables; the bias then turns with the key's position (rope_cos)."""
        k, v, ks, vs = cls._alloc(dtype, (batch, kv_heads, max_tokens), head_dim, device)
        return cls(dtype=dtype, layout=LAYOUT_CONTIGUOUS, batch=batch, kv_heads=kv_heads, k_bias=k_bias,
                   head_dim=head_dim, k=k, v=v, k_scale=ks, v_scale=vs, max_tokens=max_tokens,
                   rope_cos=rope_cos, rope_sin=rope_sin)

    @classmethod
    def paged(cls, page_table: torch.Tensor, num_pages, kv_heads, head_dim, page_size=16,
              dtype="k8v8", device="cuda", k_bias=None, rope_cos=None, rope_sin=None):
        pt = page_table.to(device=device, dtype=torch.int32).contiguous()
        k, v, ks, vs = cls._alloc(dtype, (num_pages, kv_heads, page_size), head_dim, device)
        return cls(dtype=dtype, layout=LAYOUT_PAGED, batch=pt.shape[0], kv_heads=kv_heads, k_bias=k_bias,
                   head_dim=head_dim, k=k, v=v, k_scale=ks, v_scale=vs, page_size=page_size,
                   num_pages=num_pages, page_table=pt, rope_cos=rope_cos, rope_sin=rope_sin)


# ------------------------------------------------------------ C-ABI calls --

def fp8kv_quantize(x: torch.Tensor, codes: Optional[torch.Tensor] = None,
                   scales: Optional[torch.Tensor] = None, stream=None):
    """bf16 rows [..., D] -> (uint8 codes [..., D], fp32 scales [...])."""
    _need(x, torch.bfloat16, "x")
    D = x.shape[-1]
    rows = x.numel() // D if D else 0
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _check(get_lib().fp8kv_quantize(_ptr(x), rows, D, _ptr(codes), _ptr(scales), _stream(stream)),
           "fp8kv_quantize")
    return codes, scales


def fp8kv_quantize_mx(x: torch.Tensor, codes: Optional[torch.Tensor] = None,
                      scales: Optional[torch.Tensor] = None, stream=None):
    """bf16 rows [..., D] (D 64 or 128) -> (uint8 codes [..., D], uint8 E8M0
    block scales [..., D/32]): MXFP8, one power-of-two scale per 32 elements."""
    _need(x, torch.bfloat16, "x")
    D = x.shape[-1]
    rows = x.numel() // D if D else 0
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(x.shape[:-1] + (max(D // 32, 1),), dtype=torch.uint8, device=x.device)
    _check(get_lib().fp8kv_quantize_mx(_ptr(x), rows, D, _ptr(codes), _ptr(scales), _stream(stream)),
           "fp8kv_quantize_mx")
    return codes, scales


def fp8kv_append(cache: Fp8KVCache, k_new: torch.Tensor, v_new: torch.Tensor,
                 seq_idx: torch.Tensor, pos: torch.Tensor, stream=None):
    """Quantise and write K/V rows [n, kv_heads, D] (bf16) for tokens
    (seq_idx[i], pos[i])."""
    _need(k_new, torch.bfloat16, "k_new")
    _need(v_new, torch.bfloat16, "v_new")
    _need(seq_idx, torch.int32, "seq_idx")
    _need(pos, torch.int32, "pos")
    n = k_new.shape[0]
    _check(get_lib().fp8kv_append(cache.struct_ref, _ptr(k_new), _ptr(v_new), _ptr(seq_idx),
                                  _ptr(pos), n, _stream(stream)), "fp8kv_append")


def _kernel(kernel) -> int:
    return KERNELS[kernel] if isinstance(kernel, str) else int(kernel)


def fp8kv_decode_num_splits(cache: Fp8KVCache, q_heads: int, num_splits: int = 0, kernel=0) -> int:
    return int(get_lib().fp8kv_decode_num_splits(cache.struct_ref, q_heads, num_splits, _kernel(kernel)))


def fp8kv_decode_workspace_bytes(cache: Fp8KVCache, q_heads: int, num_splits: int = 0, kernel=0) -> int:
    return int(get_lib().fp8kv_decode_workspace_bytes(cache.struct_ref, q_heads, num_splits,
                                                      _kernel(kernel)))


def fp8kv_decode_attention(q: torch.Tensor, cache: Fp8KVCache, seq_lens: torch.Tensor,
                           sm_scale: Optional[float] = None, num_splits: int = 0,
                           out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                           workspace: Optional[torch.Tensor] = None, kernel=0, stream=None):
    """q [B, Hq, D] bf16, seq_lens [B] int32 -> out [B, Hq, D] (bf16 or fp32).
    kernel: "auto" / "cuda_cores" / "tensor_cores" / "tensor_cores_k_f16" /
    "tensor_cores_k_f16_producer" (or 0 .. 4)."""
    _need(q, torch.bfloat16, "q")
    _need(seq_lens, torch.int32, "seq_lens")
    B, Hq, D = q.shape
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=out_dtype, device=q.device)
    odt = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    k = _kernel(kernel)
    need = fp8kv_decode_workspace_bytes(cache, Hq, num_splits, k)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check(get_lib().fp8kv_decode_attention(
        _ptr(q), cache.struct_ref, _ptr(seq_lens), Hq, float(sm_scale), num_splits, k,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out), odt,
        _stream(stream)), "fp8kv_decode_attention")
    return out


def fp8kv_decode_split(q: torch.Tensor, cache: Fp8KVCache, seq_lens: torch.Tensor,
                       workspace: torch.Tensor, sm_scale: Optional[float] = None,
                       num_splits: int = 0, kernel=0, stream=None):
    """Kernel 1 of decode: fp32 partials of every split into `workspace`."""
    _need(q, torch.bfloat16, "q")
    _need(seq_lens, torch.int32, "seq_lens")
    B, Hq, D = q.shape
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    _check(get_lib().fp8kv_decode_split(
        _ptr(q), cache.struct_ref, _ptr(seq_lens), Hq, float(sm_scale), num_splits, _kernel(kernel),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)),
        "fp8kv_decode_split")


def fp8kv_decode_merge(cache: Fp8KVCache, q_heads: int, workspace: torch.Tensor,
                       out: torch.Tensor, num_splits: int = 0, kernel=0, stream=None):
    """Kernel 2 of decode: merge the partials in `workspace` into `out`."""
    odt = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    _check(get_lib().fp8kv_decode_merge(
        cache.struct_ref, q_heads, num_splits, _kernel(kernel), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), odt, _stream(stream)),
        "fp8kv_decode_merge")
    return out


def fp8kv_decode_step_workspace_bytes(cache: Fp8KVCache, q_heads: int, num_splits: int = 0,
                                      kernel=0) -> int:
    return int(get_lib().fp8kv_decode_step_workspace_bytes(cache.struct_ref, q_heads, num_splits,
                                                           _kernel(kernel)))


def fp8kv_decode_step(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, cache: Fp8KVCache,
                      seq_lens: torch.Tensor, sm_scale: Optional[float] = None, num_splits: int = 0,
                      out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                      workspace: Optional[torch.Tensor] = None, kernel=0, early_cache_read=False,
                      stream=None):
    """Append k_new/v_new [B, Hkv, D] at position seq_lens[b]-1 and decode
    q [B, Hq, D] over seq_lens[b] tokens.  `workspace` must start zero-filled
    (a fresh one is allocated that way when not given).  early_cache_read:
    FP8KV_STEP_EARLY_CACHE_READ (the kernel issued just before on the stream
    must not write this cache or seq_lens)."""
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new")):
        _need(t, torch.bfloat16, n, host_ok=True)
    _need(seq_lens, torch.int32, "seq_lens", host_ok=True)
    B, Hq, D = q.shape
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    dev = cache.k.device                   # (q and the others may be pinned host tensors)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=out_dtype, device=dev)
    _need(out, out.dtype, "out", host_ok=True)
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"out: expected bf16 or fp32, got {out.dtype}")
    odt = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    k = _kernel(kernel)
    if workspace is None:
        need = fp8kv_decode_step_workspace_bytes(cache, Hq, num_splits, k)
        workspace = torch.zeros(max(need, 16), dtype=torch.uint8, device=dev)
    _need(workspace, torch.uint8, "workspace")
    _check(get_lib().fp8kv_decode_step(
        _ptr(q), _ptr(k_new), _ptr(v_new), cache.struct_ref, _ptr(seq_lens), Hq, float(sm_scale),
        num_splits, k, _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out), odt,
        STEP_EARLY_CACHE_READ if early_cache_read else 0, _stream(stream)), "fp8kv_decode_step")
    return out


def fp8kv_prefill_attention(q: torch.Tensor, cache: Fp8KVCache, q_pos0: torch.Tensor,
                            sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                            out_dtype=torch.bfloat16, kernel="auto", stream=None):
    """q [B, n_q, Hq, D] bf16, q_pos0 [B] int32 -> out [B, n_q, Hq, D].
    kernel: "auto", "tensor_cores" (K8V8, head_dim 128) or "cuda_cores"."""
    _need(q, torch.bfloat16, "q")
    _need(q_pos0, torch.int32, "q_pos0")
    B, n_q, Hq, D = q.shape
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((B, n_q, Hq, D), dtype=out_dtype, device=q.device)
    odt = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    _check(get_lib().fp8kv_prefill_attention(
        _ptr(q), cache.struct_ref, _ptr(q_pos0), n_q, Hq, float(sm_scale), _kernel(kernel), _ptr(out),
        odt, _stream(stream)), "fp8kv_prefill_attention")
    return out


# ----------------------------------------------------- serving-step calls --

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}


def _refuse(t, dtype, name, shape, contiguous):
    if t.dtype is not dtype or not t.is_cuda or (contiguous and not t.is_contiguous()):
        raise ValueError(f"{name}: expected a {'contiguous ' if contiguous else ''}CUDA {dtype} tensor, got "
                         f"{t.dtype} on {t.device} (contiguous={t.is_contiguous()})")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: on {t.device}, but the call runs on cuda:{torch.cuda.current_device()}, the current device")


def _here(t: torch.Tensor, dtype, name, dev, shape=None):
    """Address of a contiguous CUDA tensor of `dtype` on device `dev` (the
    current one: the launch goes to that device's stream)."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or (shape is not None and t.shape != shape):
        _refuse(t, dtype, name, shape, True)
    return t.data_ptr()


def _current(cache: Fp8KVCache) -> int:
    """The current device, which has to be the cache's."""
    dev = cache.k.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError(f"cache: on {cache.k.device}, but the current device is "
                         f"{torch.cuda.current_device() if torch.cuda.is_available() else 'none'}")
    return dev


def _on(stream):
    """Allocations of a call that launches on `stream` belong to that stream."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _raw_stream(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def fp8kv_build_tables(cache: Fp8KVCache, cached_lens: torch.Tensor, new_lens: torch.Tensor, n_rows: int,
                       free_pages: Optional[torch.Tensor] = None, free_head: Optional[torch.Tensor] = None,
                       cu_new=None, seq_lens=None, seq_idx=None, pos=None, slots=None, free_head_out=None,
                       stream=None):
    """Page tables and slot maps of one step: sequence b holds cached_lens[b]
    tokens and gets new_lens[b] more ([B] int32 each).  Fresh pages come from
    free_pages[free_head:] ([F], [1] int32; paged caches only) and go into
    cache.page_table in place.  Returns a dict of cu_new [B + 1], seq_lens [B],
    seq_idx and pos [n_rows] (int32), slots [n_rows] (int64) and free_head [1]
    (None for a contiguous cache); rows behind the last sequence hold -1.
    Output tensors may be passed in and may not be input tensors."""
    B, N = cache.batch, int(n_rows)
    paged = cache.layout == LAYOUT_PAGED
    if paged != (free_pages is not None) or paged != (free_head is not None):
        raise ValueError("free_pages and free_head come with a paged cache, and only with one")
    dev, i32 = _current(cache), torch.int32
    F, a_free, a_head, a_out = 0, None, None, None
    if paged:
        F = free_pages.numel()
        a_free, a_head = _here(free_pages, i32, "free_pages", dev, (F,)), _here(free_head, i32, "free_head", dev, (1,))
    if cu_new is None or seq_lens is None or seq_idx is None or pos is None or slots is None or \
            (paged and free_head_out is None):
        with _on(stream):
            def new(t, shape, dtype=torch.int32):
                return torch.empty(shape, dtype=dtype, device=cache.k.device) if t is None else t
            cu_new, seq_lens, seq_idx, pos = new(cu_new, B + 1), new(seq_lens, B), new(seq_idx, N), new(pos, N)
            slots = new(slots, N, torch.int64)
            free_head_out = new(free_head_out, 1) if paged else free_head_out
    if paged:
        a_out = _here(free_head_out, i32, "free_head_out", dev, (1,))
    elif free_head_out is not None:
        raise ValueError("free_head_out comes with a paged cache")
    _check(get_lib().fp8kv_build_tables(
        cache.struct_ref, _here(cached_lens, i32, "cached_lens", dev, (B,)), _here(new_lens, i32, "new_lens", dev, (B,)), a_free, F,
        a_head, N, _here(cu_new, i32, "cu_new", dev, (B + 1,)), _here(seq_lens, i32, "seq_lens", dev, (B,)),
        _here(seq_idx, i32, "seq_idx", dev, (N,)), _here(pos, i32, "pos", dev, (N,)), _here(slots, torch.int64, "slots", dev, (N,)),
        a_out, _raw_stream(stream, dev)), "fp8kv_build_tables")
    return {"cu_new": cu_new, "seq_lens": seq_lens, "seq_idx": seq_idx, "pos": pos, "slots": slots,
            "free_head": free_head_out}


def fp8kv_rope_tables(positions: int, rot_dim: int, base: float = 10000.0, factor: float = 1.0,
                      original_positions: int = 0, ramp=(1.0, 4.0), amplitude: float = 1.0,
                      cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, stream=None):
    """cos and sin [positions, rot_dim / 2] fp32 of t * base^(-2 i / rot_dim).
    factor > 1 stretches the context: every pair, or (original_positions > 0)
    those that turn fewer than ramp[1] times within original_positions, fully
    below ramp[0] turns.  amplitude scales both tables."""
    if cos is None or sin is None:
        with _on(stream):
            shape = (int(positions), int(rot_dim) // 2)
            cos = torch.empty(shape, device="cuda") if cos is None else cos
            sin = torch.empty(shape, device="cuda") if sin is None else sin
    shape, dev = (positions, rot_dim // 2), torch.cuda.current_device()
    _check(get_lib().fp8kv_rope_tables(
        positions, rot_dim, base, factor, original_positions, ramp[0], ramp[1], amplitude,
        _here(cos, torch.float32, "cos", dev, shape), _here(sin, torch.float32, "sin", dev, shape), _raw_stream(stream, dev)),
        "fp8kv_rope_tables")
    return cos, sin


def _rows(t, heads, dim, n, name, dev):
    """[n, heads, dim] bf16 whose tokens may lie apart (a slice of a fused
    projection): address and token stride."""
    if t.dtype is not torch.bfloat16 or t.get_device() != dev or t.shape != (n, heads, dim):
        _refuse(t, torch.bfloat16, name, (n, heads, dim), False)
    s0, s1, s2 = t.stride()
    if s2 != 1 or (heads > 1 and s1 != dim):
        raise ValueError(f"{name}: heads of a token must lie side by side, got strides {t.stride()}")
    return t.data_ptr(), (s0 if n > 1 else heads * dim)


def fp8kv_rope_append(cache: Fp8KVCache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor,
                      slots: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor, layout="half",
                      q_out: Optional[torch.Tensor] = None, stream=None):
    """Rotate q [n, Hq, D] and k [n, Hkv, D] (bf16; token strides as in a
    slice of a fused projection) at positions pos [n] int32 with the tables
    cos, sin [positions, R / 2], write k and v quantised into the cache at
    slots [n] int64 (negative: padding, row skipped) and return the rotated
    queries [n, Hq, D] bf16 (q_out; may be q)."""
    n, Hq, D = q.shape
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout: expected one of {tuple(ROPE_LAYOUTS)}, got {layout!r}")
    if cos.dim() != 2:
        raise ValueError(f"cos: expected [positions, rot_dim / 2], got {tuple(cos.shape)}")
    if D != cache.head_dim:
        raise ValueError(f"q: head dim {D}, but the cache's is {cache.head_dim}")
    dev = _current(cache)
    a_q, s_q = _rows(q, Hq, D, n, "q", dev)
    a_k, s_k = _rows(k, cache.kv_heads, D, n, "k", dev)
    a_v, s_v = _rows(v, cache.kv_heads, D, n, "v", dev)
    if q_out is None:
        with _on(stream):
            q_out = torch.empty((n, Hq, D), dtype=torch.bfloat16, device=q.device)
    T, half = cos.shape
    _check(get_lib().fp8kv_rope_append(
        cache.struct_ref, a_q, s_q, a_k, s_k, a_v, s_v, Hq, _here(pos, torch.int32, "pos", dev, (n,)),
        _here(slots, torch.int64, "slots", dev, (n,)), n, _here(cos, torch.float32, "cos", dev),
        _here(sin, torch.float32, "sin", dev, (T, half)), T, 2 * half, ROPE_LAYOUTS[layout],
        _here(q_out, torch.bfloat16, "q_out", dev, (n, Hq, D)), _raw_stream(stream, dev)), "fp8kv_rope_append")
    return q_out


def fp8kv_chunk_num_splits(cache: Fp8KVCache, total_q: int, q_heads: int, window: int = 0, sinks: int = 0,
                           num_splits: int = 0, kernel=0) -> int:
    return int(get_lib().fp8kv_chunk_num_splits(cache.struct_ref, total_q, q_heads, window, sinks, num_splits, _kernel(kernel)))


def fp8kv_chunk_workspace_bytes(cache: Fp8KVCache, total_q: int, q_heads: int, window: int = 0, sinks: int = 0,
                                num_splits: int = 0, kernel=0) -> int:
    return int(get_lib().fp8kv_chunk_workspace_bytes(cache.struct_ref, total_q, q_heads, window, sinks, num_splits,
                                                     _kernel(kernel)))


def fp8kv_chunk_attention(q: torch.Tensor, cache: Fp8KVCache, cu_q: Optional[torch.Tensor], seq_lens: torch.Tensor,
                          sm_scale: Optional[float] = None, window: int = 0, sinks: int = 0, num_splits: int = 0,
                          out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                          workspace: Optional[torch.Tensor] = None, kernel="auto", stream=None):
    """Ragged chunk attention: q [total_q, Hq, D] bf16, sequence b's queries in
    rows cu_q[b]..cu_q[b+1]-1 (cu_q [B + 1] int32, or None: one query per
    sequence), the last at position seq_lens[b] - 1 of its cached tokens.
    window > 0: a query sees the last `window` tokens, its own among them, and
    the first `sinks`.  Returns out [total_q, Hq, D]; rows outside every
    sequence stay as they were (an `out` made here holds anything there).
    kernel: "auto", "warp_mma" or "tensor_cores" (head dim 128, not block-scaled
    keys)."""
    total_q, Hq, D = q.shape
    if D != cache.head_dim:
        raise ValueError(f"q: head dim {D}, but the cache's is {cache.head_dim}")
    dev = _current(cache)
    k = _kernel(kernel)
    if out is None or workspace is None:
        with _on(stream):
            if out is None:
                out = torch.empty((total_q, Hq, D), dtype=out_dtype, device=q.device)
            if workspace is None:
                need = fp8kv_chunk_workspace_bytes(cache, total_q, Hq, window, sinks, num_splits, k)
                workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    odt = out.dtype
    if odt is not torch.bfloat16 and odt is not torch.float32:
        raise ValueError(f"out: expected bf16 or fp32, got {odt}")
    _check(get_lib().fp8kv_chunk_attention(
        _here(q, torch.bfloat16, "q", dev), cache.struct_ref,
        None if cu_q is None else _here(cu_q, torch.int32, "cu_q", dev, (cache.batch + 1,)),
        _here(seq_lens, torch.int32, "seq_lens", dev, (cache.batch,)), total_q, Hq,
        1.0 / math.sqrt(D) if sm_scale is None else sm_scale, window, sinks, num_splits, k,
        _here(workspace, torch.uint8, "workspace", dev), workspace.numel(), _here(out, odt, "out", dev, (total_q, Hq, D)),
        OUT_F32 if odt is torch.float32 else OUT_BF16, _raw_stream(stream, dev)), "fp8kv_chunk_attention")
    return out


def fp8kv_tree_tables(parents: torch.Tensor, cu_new: torch.Tensor, seq_lens: torch.Tensor, max_nodes: int,
                      masks: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None, stream=None, window: int = 0,
                      sinks: int = 0):
    """Masks and positions of trees of drafted tokens: parents [n] int32 (of
    row cu_new[b] + i: index of node i's parent within its tree, -1: none),
    cu_new [B + 1], seq_lens [B] int32 (nodes counted).  max_nodes: nodes that a
    row of bits has room for.  Returns masks [n, ceil(max_nodes / 32)] int32 (bit
    i: node i, the node itself or an ancestor) and pos [n] int32 (context length +
    depth); rows of no tree get no bits and -1.  window > 0: ancestors `window` or
    more positions above a node have no bit, unless they are among the first `sinks`
    tokens (fp8kv_tree_attention itself hides no node under a window)."""
    n, B, words, dev, i32 = parents.numel(), seq_lens.numel(), (int(max_nodes) + 31) // 32, torch.cuda.current_device(), torch.int32
    if masks is None or pos is None:
        with _on(stream):
            masks = torch.empty((n, words), dtype=i32, device=parents.device) if masks is None else masks
            pos = torch.empty(n, dtype=i32, device=parents.device) if pos is None else pos
    args = (_here(parents, i32, "parents", dev, (n,)), _here(cu_new, i32, "cu_new", dev, (B + 1,)), _here(seq_lens, i32, "seq_lens", dev, (B,)),
            B, n, words)
    outs = (_here(masks, i32, "masks", dev, (n, words)), _here(pos, i32, "pos", dev, (n,)), _raw_stream(stream, dev))
    if window or sinks:
        _check(get_lib().fp8kv_tree_tables_window(*args, window, sinks, *outs), "fp8kv_tree_tables_window")
    else:
        _check(get_lib().fp8kv_tree_tables(*args, *outs), "fp8kv_tree_tables")
    return masks, pos


def fp8kv_tree_workspace_bytes(cache: Fp8KVCache, total_q: int, q_heads: int, window: int = 0, sinks: int = 0,
                               num_splits: int = 0, kernel=0) -> int:
    return int(get_lib().fp8kv_tree_workspace_bytes(cache.struct_ref, total_q, q_heads, window, sinks, num_splits,
                                                    _kernel(kernel)))


def fp8kv_tree_attention(q: torch.Tensor, cache: Fp8KVCache, cu_q: torch.Tensor, seq_lens: torch.Tensor, masks: torch.Tensor,
                         pos: Optional[torch.Tensor] = None, sm_scale: Optional[float] = None, window: int = 0, sinks: int = 0,
                         num_splits: int = 0, out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                         workspace: Optional[torch.Tensor] = None, kernel="auto", stream=None):
    """Attention of trees of drafted tokens: q [total_q, Hq, D] bf16, sequence
    b's nodes in rows cu_q[b]..cu_q[b+1]-1 and in the cache as its last tokens.
    A node sees the context, the nodes of its row of masks [total_q, words] int32
    (fp8kv_tree_tables) and itself; window > 0: of the context the tokens above
    pos - window and the first `sinks` (pos [total_q] int32, needed then).  The
    rest as in fp8kv_chunk_attention."""
    total_q, Hq, D = q.shape
    if D != cache.head_dim:
        raise ValueError(f"q: head dim {D}, but the cache's is {cache.head_dim}")
    if masks.dim() != 2:
        raise ValueError(f"masks: expected [total_q, words], got {tuple(masks.shape)}")
    dev, i32 = _current(cache), torch.int32
    k = _kernel(kernel)
    if out is None or workspace is None:
        with _on(stream):
            if out is None:
                out = torch.empty((total_q, Hq, D), dtype=out_dtype, device=q.device)
            if workspace is None:
                need = fp8kv_tree_workspace_bytes(cache, total_q, Hq, window, sinks, num_splits, k)
                workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    odt, words = out.dtype, masks.shape[1]
    if odt is not torch.bfloat16 and odt is not torch.float32:
        raise ValueError(f"out: expected bf16 or fp32, got {odt}")
    _check(get_lib().fp8kv_tree_attention(
        _here(q, torch.bfloat16, "q", dev), cache.struct_ref, _here(cu_q, i32, "cu_q", dev, (cache.batch + 1,)),
        _here(seq_lens, i32, "seq_lens", dev, (cache.batch,)), _here(masks, i32, "masks", dev, (total_q, words)), words,
        None if pos is None else _here(pos, i32, "pos", dev, (total_q,)), total_q, Hq,
        1.0 / math.sqrt(D) if sm_scale is None else sm_scale, window, sinks, num_splits, k,
        _here(workspace, torch.uint8, "workspace", dev), workspace.numel(), _here(out, odt, "out", dev, (total_q, Hq, D)),
        OUT_F32 if odt is torch.float32 else OUT_BF16, _raw_stream(stream, dev)), "fp8kv_tree_attention")
    return out


def fp8kv_tree_accept(caches, parents: torch.Tensor, tokens: torch.Tensor, choices: torch.Tensor, cu_new: torch.Tensor,
                      seq_lens: torch.Tensor, max_path: int, path=None, accepted=None, next_tokens=None, new_lens=None,
                      stream=None):
    """The accepted nodes of every tree, and their rows moved behind the context
    in every cache of `caches` (a list: the layers; may be empty).  parents [n],
    cu_new [B + 1], seq_lens [B] int32 as in fp8kv_tree_tables; tokens, choices [n]
    int64: drafted token of a node, the model's choice behind it.  Returns a dict
    of path [B, max_path] int32 (-1 behind the last), accepted [B] int32,
    next_tokens [B] int64 and lens [B] int32 (cached_lens of the next step)."""
    n, B, M, dev, i32, i64 = parents.numel(), seq_lens.numel(), int(max_path), torch.cuda.current_device(), torch.int32, torch.int64
    caches = list(caches)
    for c in caches:
        if c.k.get_device() != dev:
            raise ValueError(f"cache: on {c.k.device}, but the current device is {dev}")
    if path is None or accepted is None or next_tokens is None or new_lens is None:
        with _on(stream):
            def new(t, shape, dtype=torch.int32):
                return torch.empty(shape, dtype=dtype, device=parents.device) if t is None else t
            path, accepted, next_tokens, new_lens = new(path, (B, M)), new(accepted, B), new(next_tokens, B, i64), new(new_lens, B)
    refs = (ctypes.c_void_p * len(caches))(*[ctypes.addressof(c._struct) for c in caches])
    _check(get_lib().fp8kv_tree_accept(
        refs, len(caches), _here(parents, i32, "parents", dev, (n,)), _here(tokens, i64, "tokens", dev, (n,)),
        _here(choices, i64, "choices", dev, (n,)), _here(cu_new, i32, "cu_new", dev, (B + 1,)), _here(seq_lens, i32, "seq_lens", dev, (B,)),
        B, n, M, _here(path, i32, "path", dev, (B, M)), _here(accepted, i32, "accepted", dev, (B,)),
        _here(next_tokens, i64, "next_tokens", dev, (B,)), _here(new_lens, i32, "new_lens", dev, (B,)), _raw_stream(stream, dev)),
        "fp8kv_tree_accept")
    return {"path": path, "accepted": accepted, "next_tokens": next_tokens, "lens": new_lens}


def fp8kv_block_matmul(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                       bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                       stream=None):
    """Matrix product of e4m3 codes a [M, K] (activations; a_scales
    [M, ceil(K / 128)] fp32) and b [N, K] (a weight; b_scales
    [ceil(N / 128), ceil(K / 128)]): out [M, N] = the sum over blocks of 128 of
    K of both scales times the codes' products, plus bias [N] fp32.  With K a
    multiple of 128, fp8kv_quantize(x.view(M, K // 128, 128)) makes a and its
    scales (view the codes as [M, K]).  K a multiple of 16."""
    f32 = torch.float32
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError(f"a, b: expected [M, K] and [N, K], got {tuple(a.shape)} and {tuple(b.shape)}")
    M, K = a.shape
    N, KB, dev = b.shape[0], (K + 127) // 128, torch.cuda.current_device()
    if out is None:
        with _on(stream):
            out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    odt = out.dtype
    if odt is not torch.bfloat16 and odt is not f32:
        raise ValueError(f"out: expected bf16 or fp32, got {odt}")
    _check(get_lib().fp8kv_block_matmul(
        _here(a, torch.uint8, "a", dev), _here(a_scales, f32, "a_scales", dev, (M, KB)), _here(b, torch.uint8, "b", dev, (N, K)),
        _here(b_scales, f32, "b_scales", dev, ((N + 127) // 128, KB)), None if bias is None else _here(bias, f32, "bias", dev, (N,)),
        M, N, K, _here(out, odt, "out", dev, (M, N)), OUT_F32 if odt is f32 else OUT_BF16, _raw_stream(stream, dev)),
        "fp8kv_block_matmul")
    return out


def fp8kv_get_device_error(clear: bool = True) -> int:
    """Synchronise the device and return (optionally clearing) the device
    error word (bits DEVERR_*)."""
    bits = ctypes.c_uint32(0)
    st = get_lib().fp8kv_get_device_error(ctypes.byref(bits), 1 if clear else 0)
    if st not in (0, 5, 6):
        raise Fp8KVError(st, "fp8kv_get_device_error")
    return int(bits.value)


def fp8kv_status_string(status: int) -> str:
    return get_lib().fp8kv_status_string(status).decode()


__all__ = ["Fp8KVCache", "Fp8KVError", "fp8kv_quantize", "fp8kv_quantize_mx", "fp8kv_append",
           "fp8kv_decode_num_splits", "fp8kv_decode_workspace_bytes", "fp8kv_decode_split",
           "fp8kv_decode_merge", "fp8kv_decode_attention", "fp8kv_decode_step",
           "fp8kv_decode_step_workspace_bytes",
           "fp8kv_prefill_attention", "fp8kv_build_tables", "fp8kv_rope_tables", "fp8kv_rope_append",
           "fp8kv_chunk_num_splits", "fp8kv_chunk_workspace_bytes", "fp8kv_chunk_attention",
           "fp8kv_tree_tables", "fp8kv_tree_workspace_bytes", "fp8kv_tree_attention", "fp8kv_tree_accept", "fp8kv_block_matmul",
           "fp8kv_get_device_error", "fp8kv_status_string",
           "EXPORTS", "K8V8", "K16V8", "K16V16", "K8V16", "MXK8V8"]
