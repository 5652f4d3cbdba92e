"""Python binding of the B200 decoder library (liblfwd.so, C ABI in include/llama_fwd.h).

Argument marshalling only: every step of the forward pass runs in the library's
CUDA kernels. The functions below carry the C names; ``Model`` bundles a model
handle with the tensors whose device pointers it holds. There is no fallback:
if the shared library is missing, ``load()`` raises. Operations run on the stream that
they are given, ``stream=None`` being the legacy default stream and not torch's current
one: inside ``torch.cuda.stream(s)``, pass ``stream=s``.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, List, Optional

import torch

from .build import LIB as _LIB_PLAIN, LIB_CHECKED as _LIB_CHECKED

# LLM_LIB_VARIANT=checked selects the bounds-checking build (liblfwd_checked.so).
LIB_PATH = _LIB_CHECKED if os.environ.get("LLM_LIB_VARIANT") == "checked" else _LIB_PLAIN

LLM_OK = 0
LLM_ERR_BAD_CONFIG = -1
LLM_ERR_NULL_PTR = -2
LLM_ERR_SEQ_OVERFLOW = -3
LLM_ERR_BATCH = -4
LLM_ERR_CUDA = -5
LLM_ERR_DEVICE_TIMEOUT = -6
LLM_ERR_UNSUPPORTED = -7
LLM_ERR_BAD_ARG = -8
LLM_ERR_DEVICE_BOUNDS = -9
LLM_BUILD_BOUNDS_CHECK = 1
LLM_F32 = 0
LLM_BF16 = 1
LLM_FLAG_CUDA_GRAPH = 1
LLM_FLAG_DEBUG_TAPS = 2
LLM_FLAG_KERNEL_TIMING = 4
LLM_FLAG_PDL = 8
LLM_FLAG_FUSED_DECODE = 16
LLM_FLAG_KV4 = 32
KERNEL_KINDS = ("embed", "qkv", "attn", "wo", "w13", "w2", "head", "out", "step")


class llm_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("dim", "n_layers", "n_heads", "n_kv_heads", "head_dim",
                                            "ffn_hidden", "vocab", "max_seq_len", "max_batch", "max_tokens")] + \
               [("norm_eps", ctypes.c_float), ("rope_theta", ctypes.c_float)] + \
               [(n, ctypes.c_int) for n in ("dtype", "tie_embeddings", "has_embed_and_head", "flags")]


_PP = ctypes.POINTER(ctypes.c_void_p)


class llm_weights(ctypes.Structure):
    _fields_ = [("tok_emb", ctypes.c_void_p), ("out", ctypes.c_void_p), ("final_norm", ctypes.c_void_p)] + \
               [(n, _PP) for n in ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "w1", "w3", "w2")]


class LlmError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"llm error {code}: {msg}")
        self.code = code


_lib = None
_vp, _i, _sz, _i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64

_SIGS = {
    "llm_model_init": (_i, [ctypes.POINTER(llm_config), ctypes.POINTER(llm_weights), _vp, ctypes.POINTER(_vp)]),
    "llm_prefill": (_i, [_vp, _vp, _i, _i, _vp, _vp]),
    "llm_prefill_hidden": (_i, [_vp, _vp, _i, _i, _vp]),
    "llm_decode_step": (_i, [_vp, _i, _vp, _vp, _vp]),
    "llm_decode_step_hidden": (_i, [_vp, _i, _vp, _vp]),
    "llm_kv_cache_reset": (_i, [_vp]),
    "llm_kv_cache_view": (_i, [_vp, ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.POINTER(ctypes.c_int64)]),
    "llm_kv_cache_set_lens": (_i, [_vp, ctypes.POINTER(ctypes.c_int32), _i]),
    "llm_kv_cache_get_lens": (_i, [_vp, ctypes.POINTER(ctypes.c_int32), _i]),
    "llm_debug_tap": (_i, [_vp, _i, _vp, _sz]),
    "llm_kernel_times": (_i, [_vp, _i, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64), _i]),
    "llm_debug_wait_probe": (_i, [_vp, _i, ctypes.c_double]),
    "llm_synchronize": (_i, [_vp]),
    "llm_build_flags": (_i, []),
    "llm_op_synchronize": (_i, [_vp]),
    "llm_model_free": (None, [_vp]),
    "llm_last_error": (ctypes.c_char_p, []),
    "llm_op_gemm_bf16": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp]),
    "llm_op_gemv_workspace": (_sz, [_i, _i]),
    "llm_op_gemv_bf16": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _sz, _vp]),
    "llm_op_attention_prefill": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp]),
    "llm_op_attention_decode_workspace": (_sz, [_i, _i, _i, _i, _i]),
    "llm_op_attention_decode": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _sz, _vp]),
    "llm_op_attention_decode_static": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp]),
    "llm_op_attention_decode_cluster": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "llm_kv4_page_bytes": (_sz, [_i, _i, _i]),
    "llm_op_kv_pages": (_i, [_vp, _vp, _i, _i, _vp, _i, _vp, _vp, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp]),
    "llm_op_qk_norm_rope_kv4": (_i, [_vp, _vp, _vp, _i64, _i64, _i64, _i, _vp, _vp, _i, ctypes.c_float, _vp, _vp, _i,
                                     _vp, _vp, _i, _i, _i, _i, _vp, _vp, _i, _i, _vp, _vp, _vp]),
    "llm_op_attention_kv4_workspace": (_sz, [_i] * 8),
    "llm_op_attention_kv4": (_i, [_vp, _vp, _i, _i, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _sz, _vp]),
}


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load liblfwd.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"CUDA library not built: {p} is missing "
                          "(run python -m llama_decoder_forward_fwd_b200.build)")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGS.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def exported_symbols() -> List[str]:
    return list(_SIGS)


def check(rc: int):
    if rc != LLM_OK:
        raise LlmError(rc, load().llm_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        return None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ---------------------------------------------------------------- C names
def llm_model_init(cfg: llm_config, w: llm_weights, stream=None) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    check(load().llm_model_init(ctypes.byref(cfg), ctypes.byref(w), _stream_ptr(stream), ctypes.byref(h)))
    return h


def llm_prefill(m, tokens: torch.Tensor, next_tok: torch.Tensor, logits: Optional[torch.Tensor] = None):
    B, T = tokens.shape
    check(load().llm_prefill(m, _ptr(tokens), B, T, _ptr(next_tok), _ptr(logits)))


def llm_prefill_hidden(m, h_in: torch.Tensor, h_out: torch.Tensor):
    B, T, _ = h_in.shape
    check(load().llm_prefill_hidden(m, _ptr(h_in), B, T, _ptr(h_out)))


def llm_decode_step(m, in_tok: torch.Tensor, next_tok: torch.Tensor, logits: Optional[torch.Tensor] = None):
    check(load().llm_decode_step(m, in_tok.shape[0], _ptr(in_tok), _ptr(next_tok), _ptr(logits)))


def llm_decode_step_hidden(m, h_in: torch.Tensor, h_out: torch.Tensor):
    check(load().llm_decode_step_hidden(m, h_in.shape[0], _ptr(h_in), _ptr(h_out)))


def llm_kv_cache_reset(m):
    check(load().llm_kv_cache_reset(m))


def llm_kv_cache_view(m):
    k, v = ctypes.c_void_p(), ctypes.c_void_p()
    st = (ctypes.c_int64 * 4)()
    check(load().llm_kv_cache_view(m, ctypes.byref(k), ctypes.byref(v), st))
    return k.value, v.value, list(st)


def llm_kv_cache_set_lens(m, lens: List[int]):
    arr = (ctypes.c_int32 * len(lens))(*lens)
    check(load().llm_kv_cache_set_lens(m, arr, len(lens)))


def llm_kv_cache_get_lens(m, B: int) -> List[int]:
    arr = (ctypes.c_int32 * B)()
    check(load().llm_kv_cache_get_lens(m, arr, B))
    return list(arr)


def llm_debug_tap(m, layer: int, dst: torch.Tensor):
    check(load().llm_debug_tap(m, layer, _ptr(dst), dst.numel()))


def llm_kernel_times(m, reset: bool = True):
    """{kind: (total ms, launches)} since the last reset (needs LLM_FLAG_KERNEL_TIMING)."""
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    check(load().llm_kernel_times(m, n, ms, cnt, int(reset)))
    return {k: (ms[i], cnt[i]) for i, k in enumerate(KERNEL_KINDS)}


def llm_debug_wait_probe(m, which: int, limit_ms: float):
    """Queue a bounded device wait that cannot complete (0: mbarrier, 1: grid barrier)."""
    check(load().llm_debug_wait_probe(m, which, float(limit_ms)))


def llm_synchronize(m):
    check(load().llm_synchronize(m))


def llm_build_flags() -> int:
    return load().llm_build_flags()


def llm_op_synchronize(stream=None):
    check(load().llm_op_synchronize(_stream_ptr(stream)))


def llm_model_free(m):
    load().llm_model_free(m)


def llm_op_gemm_bf16(A, B, C, stream=None):
    M, K = A.shape
    N = B.shape[0]
    check(load().llm_op_gemm_bf16(_ptr(A), _ptr(B), _ptr(C), M, N, K, _stream_ptr(stream)))


def llm_op_gemv_workspace(N, K) -> int:
    return load().llm_op_gemv_workspace(N, K)


def llm_op_gemv_bf16(x, W, y, workspace, stream=None):
    M, K = x.shape
    N = W.shape[0]
    check(load().llm_op_gemv_bf16(_ptr(x), _ptr(W), _ptr(y), M, N, K, _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream_ptr(stream)))


def _dt(t: torch.Tensor) -> int:
    return LLM_BF16 if t.dtype == torch.bfloat16 else LLM_F32


def llm_op_attention_prefill(q, kc, vc, pos0, out, stream=None):
    """q [B,T,H,d]; kc, vc [B,Hk,S_max,d]; pos0 int32 [B]; out [B,T,H*d]."""
    B, T, H, d = q.shape
    Hk, S = kc.shape[1], kc.shape[2]
    check(load().llm_op_attention_prefill(_ptr(q), _ptr(kc), _ptr(vc), _ptr(pos0), _ptr(out), B, T, H, Hk, d, S,
                                          _dt(q), _stream_ptr(stream)))


def llm_op_attention_decode_workspace(B, T, H, Hk, d) -> int:
    return load().llm_op_attention_decode_workspace(B, T, H, Hk, d)


def llm_op_attention_decode(q, kc, vc, pos0, out, workspace, stream=None):
    B, T, H, d = q.shape
    Hk, S = kc.shape[1], kc.shape[2]
    check(load().llm_op_attention_decode(_ptr(q), _ptr(kc), _ptr(vc), _ptr(pos0), _ptr(out), B, T, H, Hk, d, S,
                                         _dt(q), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                         _stream_ptr(stream)))


# ---------------------------------------------------------------- convenience
def make_config(shape, max_batch: int, max_tokens: int = 0, flags: int = 0) -> llm_config:
    """llm_config from a seeded_inputs.ModelShape-like object."""
    return llm_config(dim=shape.dim, n_layers=shape.n_layers, n_heads=shape.n_heads, n_kv_heads=shape.n_kv_heads,
                      head_dim=shape.head_dim, ffn_hidden=shape.ffn_hidden, vocab=shape.vocab,
                      max_seq_len=shape.max_seq_len, max_batch=max_batch, max_tokens=max_tokens,
                      norm_eps=shape.norm_eps, rope_theta=shape.rope_theta,
                      dtype=LLM_F32 if shape.dtype == "f32" else LLM_BF16,
                      tie_embeddings=int(shape.tie_embeddings), has_embed_and_head=int(shape.has_embed_and_head),
                      flags=flags)


class Model:
    """A model handle plus the device tensors it points into.

    ``glob`` and ``layers`` are the dicts made by ``seeded_inputs.make_weights``
    (tensors are moved to the GPU if needed and kept alive here).
    """

    def __init__(self, shape, glob: Dict[str, torch.Tensor], layers: List[Dict[str, torch.Tensor]],
                 max_batch: int, max_tokens: int = 0, flags: int = 0, stream=None, device="cuda"):
        self.shape = shape
        dev = torch.device(device)
        self.glob = {k: v.to(dev).contiguous() for k, v in glob.items()}
        self.layers = [{k: v.to(dev).contiguous() for k, v in lw.items()} for lw in layers]
        self.cfg = make_config(shape, max_batch, max_tokens, flags)
        L = shape.n_layers

        def arr(key):
            a = (ctypes.c_void_p * L)(*[lw[key].data_ptr() for lw in self.layers])
            return ctypes.cast(a, _PP), a

        self._keep = []
        fields = {}
        for key in ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "w1", "w3", "w2"):
            src = {"attn_norm": "attention_norm"}.get(key, key)
            p, a = arr(src)
            fields[key] = p
            self._keep.append(a)
        g = self.glob
        self.w = llm_weights(tok_emb=g["tok_embeddings"].data_ptr() if "tok_embeddings" in g else None,
                             out=g["output"].data_ptr() if "output" in g else None,
                             final_norm=g["norm"].data_ptr() if "norm" in g else None, **fields)
        torch.cuda.synchronize(dev)
        self.h = llm_model_init(self.cfg, self.w, stream)

    def kv_cache_tensors(self):
        """torch views [n_layers, max_batch, n_kv_heads, max_seq_len, head_dim] of the library's K and V caches."""
        k, v, st = llm_kv_cache_view(self.h)
        s, c = self.shape, self.cfg
        shp = (s.n_layers, c.max_batch, s.n_kv_heads, s.max_seq_len, s.head_dim)
        typestr = "<f4" if s.dtype == "f32" else "<i2"

        class _Dev:
            def __init__(self, ptr):
                self.__cuda_array_interface__ = {"shape": shp, "typestr": typestr, "data": (ptr, False),
                                                 "version": 3, "strides": None}

        out = []
        for ptr in (k, v):
            t = torch.as_tensor(_Dev(ptr), device="cuda")
            out.append(t if s.dtype == "f32" else t.view(torch.bfloat16))
        return out[0], out[1]

    def free(self):
        if self.h:
            llm_model_free(self.h)
            self.h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def llm_op_attention_decode_cluster(q, kc, vc, pos0, out, stream=None):
    """Single-token decode attention on the tensor cores (bf16, head_dim 128, no workspace)."""
    B, T, H, d = q.shape
    Hk, S = kc.shape[1], kc.shape[2]
    check(load().llm_op_attention_decode_cluster(_ptr(q), _ptr(kc), _ptr(vc), _ptr(pos0), _ptr(out), B, H, Hk, S,
                                                 _stream_ptr(stream)))


def llm_op_attention_decode_static(q, kc, vc, pos0, out, stream=None):
    """As llm_op_attention_decode, on the library's fixed scratch (no workspace, no allocation)."""
    B, T, H, d = q.shape
    Hk, S = kc.shape[1], kc.shape[2]
    check(load().llm_op_attention_decode_static(_ptr(q), _ptr(kc), _ptr(vc), _ptr(pos0), _ptr(out), B, T, H, Hk, d,
                                                S, _dt(q), _stream_ptr(stream)))


# ---------------------------------------------------------------- the 4-bit paged cache
# These calls are a few microseconds of GPU work at their smallest, so their argument
# checks are written flat.
_I32, _I64, _BF, _F32, _U8 = torch.int32, torch.int64, torch.bfloat16, torch.float32, torch.uint8


def _device() -> int:
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -2


def _refuse(**operands):
    """Raise for the first of name=(tensor, dtype, shape) that is not what the call takes: what the C side cannot see
    in a pointer (tensors off the current device, of another type or shape, not contiguous)."""
    dev = _device()
    for name, (t, dtype, shape) in operands.items():
        if t is None or (t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
            continue
        raise LlmError(LLM_ERR_BAD_ARG, f"{name} must be {dtype}, {tuple(shape)}, contiguous and on the current CUDA "
                                        f"device; it is {t.dtype}, {tuple(t.shape)}, strides {t.stride()}, on {t.device}")


def _bad(t, dtype, shape, dev):
    return t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous()


def _rank(n, **operands):
    """Raise for the first of name=tensor that has not n dimensions."""
    for name, t in operands.items():
        if t.dim() != n:
            raise LlmError(LLM_ERR_BAD_ARG, f"{name} must have {n} dimensions; it has the shape {tuple(t.shape)}")


def _pool_pages(pool, Hk, d, page_size):
    # llm_kv4_page_bytes of the sizes that the C side takes (it refuses others), without another call into it
    shape = pool.shape
    if len(shape) != 2 or shape[1] != Hk * page_size * (d + d // 4):
        raise LlmError(LLM_ERR_BAD_ARG, "pool must be uint8 [n_pages, llm_kv4_page_bytes(Hk, d, page_size)]")
    return shape[0]


def llm_kv4_page_bytes(Hk, d, page_size) -> int:
    return load().llm_kv4_page_bytes(Hk, d, page_size)


def llm_op_kv_pages(lens, n_new, page_size, free_pages, used_in, table, q_start, positions, slots, new_lens, used_out,
                    stream=None):
    """Block tables and slot maps from request lengths. lens, n_new, new_lens int32 [B]; free_pages int32 [n_free];
    used_in (or None), used_out int32 [1]; table int32 [B, max_blocks]; q_start int32 [B+1]; positions int32 [N];
    slots int64 [N]."""
    if lens.dim() != 1 or positions.dim() != 1 or free_pages.dim() != 1 or table.dim() != 2:
        _rank(1, lens=lens, positions=positions, free_pages=free_pages)
        _rank(2, table=table)
    dev, B, N, n_free, blocks = _device(), lens.shape[0], positions.shape[0], free_pages.shape[0], table.shape[-1]
    bs, ns, one = (B,), (N,), (1,)
    if (_bad(lens, _I32, bs, dev) or _bad(n_new, _I32, bs, dev) or _bad(free_pages, _I32, (n_free,), dev)
            or _bad(table, _I32, (B, blocks), dev) or _bad(q_start, _I32, (B + 1,), dev) or _bad(positions, _I32, ns, dev)
            or _bad(slots, _I64, ns, dev) or _bad(new_lens, _I32, bs, dev) or _bad(used_out, _I32, one, dev)
            or (used_in is not None and _bad(used_in, _I32, one, dev))):
        _refuse(lens=(lens, _I32, bs), n_new=(n_new, _I32, bs), free_pages=(free_pages, _I32, (n_free,)),
                table=(table, _I32, (B, blocks)), q_start=(q_start, _I32, (B + 1,)), positions=(positions, _I32, ns),
                slots=(slots, _I64, ns), new_lens=(new_lens, _I32, bs), used_out=(used_out, _I32, one),
                used_in=(used_in, _I32, one))
    # an empty tensor has no address; the calls want one even where nothing is read
    rc = load().llm_op_kv_pages(lens.data_ptr(), n_new.data_ptr(), B, page_size, free_pages.data_ptr() or 16, n_free,
                                None if used_in is None else used_in.data_ptr(), table.data_ptr(), blocks,
                                q_start.data_ptr(), positions.data_ptr() or 16, slots.data_ptr() or 16, N,
                                new_lens.data_ptr(), used_out.data_ptr(), _stream_ptr(stream))
    if rc:
        check(rc)


def _token_rows(name, t, dtype, N, heads, d, dev):
    """The element stride between the token rows of [N, heads, d], whose rows must be contiguous."""
    ld, hs, es = t.stride()
    if t.get_device() != dev or t.dtype is not dtype or t.shape != (N, heads, d) or \
            (N and (es != 1 or (heads > 1 and hs != d))):
        raise LlmError(LLM_ERR_BAD_ARG, f"{name} must be {dtype} {(N, heads, d)} with contiguous rows, on the current CUDA device")
    return ld if N > 1 else heads * d


def llm_op_qk_norm_rope_kv4(q, k, v, positions, slots, rope_cos, rope_sin, q_out, pool, page_size, q_norm=None,
                            k_norm=None, eps=1e-5, k_out=None, v_out=None, stream=None):
    """Norms of queries and keys per head, rotation, append in 4 bits. q [N,H,d], k, v [N,Hk,d], fp32 or bf16 (any
    stride between tokens); positions int32 [N]; slots int64 [N]; rope_cos, rope_sin fp32 [n_pos, d/2]; q_out bf16
    [N,H,d]; pool uint8 [n_pages, llm_kv4_page_bytes]; q_norm, k_norm [d]; k_out, v_out bf16 [N,Hk,d] or None."""
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3 or rope_cos.dim() != 2:
        _rank(3, q=q, k=k, v=v)
        _rank(2, rope_cos=rope_cos)
    (N, H, d), Hk, t, dev, n_pos = q.shape, k.shape[1], q.dtype, _device(), rope_cos.shape[0]
    w = q_norm if q_norm is not None else k_norm
    wt = _F32 if w is None else w.dtype
    if t not in (_F32, _BF) or wt not in (_F32, _BF):
        raise LlmError(LLM_ERR_BAD_ARG, "q, k, v, q_norm and k_norm must be float32 or bfloat16")
    half, vs = (n_pos, d // 2), (N, Hk, d)
    if (_bad(positions, _I32, (N,), dev) or _bad(slots, _I64, (N,), dev) or _bad(rope_cos, _F32, half, dev)
            or _bad(rope_sin, _F32, half, dev) or _bad(q_out, _BF, (N, H, d), dev) or _bad(pool, _U8, pool.shape, dev)
            or (q_norm is not None and _bad(q_norm, wt, (d,), dev)) or (k_norm is not None and _bad(k_norm, wt, (d,), dev))
            or (k_out is not None and _bad(k_out, _BF, vs, dev)) or (v_out is not None and _bad(v_out, _BF, vs, dev))):
        _refuse(positions=(positions, _I32, (N,)), slots=(slots, _I64, (N,)), rope_cos=(rope_cos, _F32, half),
                rope_sin=(rope_sin, _F32, half), q_out=(q_out, _BF, (N, H, d)), pool=(pool, _U8, pool.shape),
                q_norm=(q_norm, wt, (d,)), k_norm=(k_norm, wt, (d,)), k_out=(k_out, _BF, vs), v_out=(v_out, _BF, vs))
    rc = load().llm_op_qk_norm_rope_kv4(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _token_rows("q", q, t, N, H, d, dev),
        _token_rows("k", k, t, N, Hk, d, dev), _token_rows("v", v, t, N, Hk, d, dev), LLM_F32 if t is _F32 else LLM_BF16,
        None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(),
        LLM_F32 if wt is _F32 else LLM_BF16, eps, rope_cos.data_ptr(), rope_sin.data_ptr(), n_pos, positions.data_ptr(),
        slots.data_ptr(), N, H, Hk, d, q_out.data_ptr(), pool.data_ptr(), _pool_pages(pool, Hk, d, page_size), page_size,
        None if k_out is None else k_out.data_ptr(), None if v_out is None else v_out.data_ptr(), _stream_ptr(stream))
    if rc:
        check(rc)


def llm_op_attention_kv4_workspace(B, N, max_new, H, Hk, d, max_blocks, page_size) -> int:
    return load().llm_op_attention_kv4_workspace(B, N, max_new, H, Hk, d, max_blocks, page_size)


def llm_op_attention_kv4(q, pool, page_size, Hk, table, lens, q_start, max_new, out, workspace, stream=None):
    """Attention over the 4-bit pages. q bf16 [N,H,d]; pool uint8 [n_pages, llm_kv4_page_bytes]; table int32
    [B, max_blocks]; lens int32 [B]; q_start int32 [B+1]; out bf16 [N, H*d]."""
    if q.dim() != 3 or table.dim() != 2:
        _rank(3, q=q)
        _rank(2, table=table)
    (N, H, d), (B, blocks), dev = q.shape, table.shape, _device()
    if (_bad(q, _BF, (N, H, d), dev) or _bad(pool, _U8, pool.shape, dev) or _bad(table, _I32, (B, blocks), dev)
            or _bad(lens, _I32, (B,), dev) or _bad(q_start, _I32, (B + 1,), dev) or _bad(out, _BF, (N, H * d), dev)
            or _bad(workspace, _U8, workspace.shape, dev)):
        _refuse(q=(q, _BF, (N, H, d)), pool=(pool, _U8, pool.shape), table=(table, _I32, (B, blocks)),
                lens=(lens, _I32, (B,)), q_start=(q_start, _I32, (B + 1,)), out=(out, _BF, (N, H * d)),
                workspace=(workspace, _U8, workspace.shape))
    rc = load().llm_op_attention_kv4(q.data_ptr(), pool.data_ptr(), _pool_pages(pool, Hk, d, page_size), page_size,
                                     table.data_ptr(), blocks, lens.data_ptr(), q_start.data_ptr(), B, N, max_new, H, Hk,
                                     d, out.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream_ptr(stream))
    if rc:
        check(rc)
