"""ctypes binding of libdflash.so: the C ABI of include/dflash.h, same names.

Argument marshalling only: torch tensors are passed as raw device pointers
and the caller's current CUDA stream is passed as the stream handle.  Every
step of the computation runs in the library's CUDA kernels.  If the shared
library is missing, loading raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libdflash.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "dflash.h")

DFLASH_F32, DFLASH_BF16, DFLASH_I32 = 0, 1, 2
DFLASH_ACCEPT_GREEDY, DFLASH_ACCEPT_ALL, DFLASH_ACCEPT_GIVEN = 0, 1, 2
DFLASH_VERIFY_LAST_ONLY = 1

STATUS = {0: "OK", 1: "INVALID_ARG", 2: "CAPACITY", 3: "OOM", 4: "CUDA", 5: "DEVICE_CHECK",
          6: "TIMEOUT", 7: "UNSUPPORTED", 8: "STATE"}


class DFlashError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"dflash status {status} ({STATUS.get(status, '?')}): {msg}")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [
        ("d_model", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("ffn_dim", ctypes.c_int32), ("vocab", ctypes.c_int32),
        ("n_target_layers", ctypes.c_int32), ("n_draft_layers", ctypes.c_int32),
        ("n_inject", ctypes.c_int32), ("inject_layers", ctypes.c_int32 * 16),
        ("rope_theta", ctypes.c_float), ("rms_eps", ctypes.c_float),
        ("block_size", ctypes.c_int32), ("max_batch", ctypes.c_int32),
        ("max_ctx", ctypes.c_int32), ("max_rows", ctypes.c_int32),
        ("max_tree_nodes", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("kv_pages", ctypes.c_int32),
    ]


PAGE_SLOTS = 128  # DFLASH_PAGE_SLOTS: cache slots per KV page


class DTree(ctypes.Structure):
    _fields_ = [
        ("tok", ctypes.c_void_p), ("parent", ctypes.c_void_p), ("depth", ctypes.c_void_p),
        ("anc", ctypes.c_void_p), ("n_nodes", ctypes.c_void_p),
        ("max_nodes", ctypes.c_int32), ("anc_words", ctypes.c_int32),
    ]


class _PagesStruct(ctypes.Structure):
    _fields_ = [
        ("page_table", ctypes.c_void_p), ("n_mapped", ctypes.c_void_p),
        ("free_pages", ctypes.c_void_p), ("n_free", ctypes.c_void_p), ("status", ctypes.c_void_p),
        ("n_pages", ctypes.c_int32), ("n_seqs", ctypes.c_int32), ("pages_per_seq", ctypes.c_int32),
    ]


class _KvqCacheStruct(ctypes.Structure):
    _fields_ = [
        ("k8", ctypes.c_void_p), ("v8", ctypes.c_void_p), ("k_exp", ctypes.c_void_p),
        ("v_exp", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("status", ctypes.c_void_p),
        ("n_pages", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("n_seqs", ctypes.c_int32),
        ("pages_per_seq", ctypes.c_int32),
    ]


_P = ctypes.c_void_p
_I = ctypes.c_int32
_L = ctypes.c_int64
_SIGS = {
    "dflash_create": ([ctypes.POINTER(Config), ctypes.POINTER(_P)], _I),
    "dflash_set_weight": ([_P, ctypes.c_char_p, _P, _I, ctypes.POINTER(ctypes.c_int64), _I], _I),
    "dflash_reset_seq": ([_P, _I, _P], _I),
    "dflash_kv_reserve": ([_P, _I, _I, _P], _I),
    "dflash_injection_rows": ([_P, ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(_P),
                               ctypes.POINTER(_I)], _I),
    "dflash_advance_lengths": ([_P, _I, _P, _P, _P], _I),
    "dflash_kv_release": ([_P, _I, _P], _I),
    "dflash_kv_free_pages": ([_P], _I),
    "dflash_kv_pool_create": ([_I, _I, _I], _P),
    "dflash_kv_pool_destroy": ([_P], None),
    "dflash_kv_pool_reserve": ([_P, _I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I)], _I),
    "dflash_kv_pool_release": ([_P, _I], _I),
    "dflash_kv_pool_pages": ([_P, _I, _P, _I], _I),
    "dflash_kv_pool_free": ([_P], _I),
    "dflash_verify": ([_P, _I, _P, _P, _I, _P, _I, _P, _P, _P, _P], _I),
    "dflash_draft_block": ([_P, _I, _P, _P, _P, _I, _P, _P, _P, _P], _I),
    "dflash_set_block_size": ([_P, _I], _I),
    "dflash_accept_commit": ([_P, _I, _P, _P, _P, ctypes.POINTER(DTree), _I, _P, _P, _P, _P], _I),
    "dflash_inject_kv": ([_P, _I, _P, _P, _P, _P], _I),
    "dtree_build": ([_P, _I, _P, _P, _P, _I, _I, ctypes.POINTER(DTree), _P], _I),
    "dtree_verify": ([_P, _I, _P, ctypes.POINTER(DTree), _P, _P, _P, _P], _I),
    "dflash_check": ([_P], _I),
    "dflash_last_error": ([_P], ctypes.c_char_p),
    "dflash_seq_lengths": ([_P], _P),
    "dflash_launch_count": ([_P], ctypes.c_int64),
    "dflash_debug_view": ([_P, ctypes.c_char_p, _I, ctypes.POINTER(_P), ctypes.POINTER(ctypes.c_int64)], _I),
    "dflash_destroy": ([_P], None),
    "dflash_block_attention": ([_I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, ctypes.c_int64, _P], _I),
    "dflash_block_attention_workspace": ([_I, _I, _I, _I, _I], ctypes.c_int64),
    "dflash_block_attention_noalloc": ([_I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P], _I),
    "dflash_debug_wait_timeout": ([_P, _P], _I),
    "dflash_sample_workspace": ([_I, _I], ctypes.c_int64),
    "dflash_sample_rows": ([_I, _I, _P, _P, _P, _P, ctypes.c_int64, _P], _I),
    "dflash_spec_accept_workspace": ([_I, _I, _I], ctypes.c_int64),
    "dflash_spec_accept_sampled": ([_I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int64, _P],
                                   _I),
    "dflash_kvq_append": ([_P, _I, _I, _P, _P, _P, _P, _P, _L, _L, _P], _I),
    "dflash_kvq_read": ([_P, _I, _I, _P, _P, _P, _P, _P, _P], _I),
    "dflash_kvq_attention": ([_P, _I, _I, _I, _I, _P, _P, _P, _P, _I, _I, _P, _L, _P, _P, _P, _L,
                              _P], _I),
    "dflash_kvq_attention_workspace": ([_I, _I, _I, _I, _I], _L),
    "dflash_kvq_score": ([_P, _I, _I, _I, _I, _P, _P, _P, _P, _I, _I, _P, _L, _P, ctypes.c_float, _P,
                          _P, _P], _I),
    "dflash_kvq_evict": ([_P, _I, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P], _I),
    "dflash_kvq_check": ([_P, _P], _I),
    "dflash_pages_map": ([_P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P], _I),
    "dflash_pages_release": ([_P, _I, _P, _P, _P], _I),
    "dflash_status_check": ([_P, _P], _I),
    "dflash_kvq_append_packed": ([_P, _I, _I, _P, _P, _P, _P, _P, _L, _L, _P], _I),
    "dflash_prompt_attention": ([_I, _I, _I, _I, _I, _P, _P, _L, _P, _L, _P, _L, _P, _P, _P, _P], _I),
    "dflash_token_logprobs": ([_I, _I, _I, _P, _L, _P, _I, _P, _P, _P, _P, _P], _I),
    "dflash_plan_gemm": ([_I, _I, _I, _I, _I, _I, _P], _I),
    "dflash_plan_attention": ([_I, _I, _I, _I, _I, ctypes.c_int64, _I, _P], _I),
    "dflash_profile": ([_P, _I], _I),
    "dflash_debug_trace": ([_P, _P, ctypes.c_int64], _I),
    "dflash_debug_trace_draft": ([_P, _P, ctypes.c_int64], _I),
    "dflash_debug_trace_draft_attn": ([_P, _P, _P, ctypes.c_int64], _I),
    "dflash_profile_list": ([_P, _I, _P, _P, ctypes.c_int64], ctypes.c_int64),
    "dflash_profile_read": ([_P, _I, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_double),
                             ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)], _I),
}

_lib: Optional[ctypes.CDLL] = None


def header_functions():
    """Names of the functions declared in include/dflash.h."""
    with open(HEADER) as f:
        src = f.read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b((?:dflash|dtree)_[a-z_]+)\s*\(", src)))


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Loads libdflash.so (raises if it has not been built).  DFLASH_LIB_PATH
    names another build of the same library (e.g. one compiled with
    different tuning flags)."""
    global _lib
    if _lib is not None:
        return _lib
    if path is None:
        path = os.environ.get("DFLASH_LIB_PATH", LIB_PATH)
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} is missing: build it with __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    for name, (args, ret) in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ret
    _lib = lib
    return lib


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def _check(ctx, status: int) -> None:
    if status != 0:
        msg = load().dflash_last_error(ctx).decode() if ctx else ""
        raise DFlashError(status, msg)


# ---------------------------------------------------------------------------
# the C ABI, one wrapper per function (raises DFlashError on a non-OK status)
# ---------------------------------------------------------------------------

def dflash_create(cfg: Config) -> int:
    h = _P()
    st = load().dflash_create(ctypes.byref(cfg), ctypes.byref(h))
    if st != 0:
        raise DFlashError(st, "dflash_create rejected the configuration")
    return h.value


def dflash_destroy(ctx: int) -> None:
    load().dflash_destroy(ctx)


def dflash_set_weight(ctx: int, name: str, tensor, dtype: int) -> None:
    shape = (ctypes.c_int64 * tensor.dim())(*tensor.shape)
    _check(ctx, load().dflash_set_weight(ctx, name.encode(), _ptr(tensor), dtype, shape, tensor.dim()))


def dflash_reset_seq(ctx: int, seq_id: int, stream=None) -> None:
    _check(ctx, load().dflash_reset_seq(ctx, seq_id, _stream(stream)))


def dflash_injection_rows(ctx):
    """(hidden, row_seq, row_pos device pointers, rows) of the pending injection queue."""
    h, rs, rp, n = _P(), _P(), _P(), _I()
    _check(ctx, load().dflash_injection_rows(ctx, ctypes.byref(h), ctypes.byref(rs), ctypes.byref(rp),
                                             ctypes.byref(n)))
    return h.value, rs.value, rp.value, n.value


def dflash_advance_lengths(ctx, batch: int, seq_ids, counts, stream=None) -> None:
    _check(ctx, load().dflash_advance_lengths(ctx, batch, _ptr(seq_ids), _ptr(counts),
                                              _stream(stream)))


def dflash_kv_reserve(ctx, seq_id: int, n_slots: int, stream=None) -> None:
    _check(ctx, load().dflash_kv_reserve(ctx, seq_id, n_slots, _stream(stream)))


def dflash_kv_release(ctx, seq_id: int, stream=None) -> None:
    _check(ctx, load().dflash_kv_release(ctx, seq_id, _stream(stream)))


def dflash_kv_free_pages(ctx) -> int:
    return load().dflash_kv_free_pages(ctx)


class KvPool:
    """The host page allocator (dflash_kv_pool_*), no GPU needed."""

    def __init__(self, n_pages: int, max_seqs: int, max_pages: int):
        self.h = load().dflash_kv_pool_create(n_pages, max_seqs, max_pages)
        if not self.h:
            raise DFlashError(1, "dflash_kv_pool_create")

    def reserve(self, seq: int, n_slots: int):
        """(first new table index, pages added); raises DFlashError when refused."""
        f, n = _I(), _I()
        st = load().dflash_kv_pool_reserve(self.h, seq, n_slots, ctypes.byref(f), ctypes.byref(n))
        if st != 0:
            raise DFlashError(st, "dflash_kv_pool_reserve")
        return f.value, n.value

    def release(self, seq: int) -> int:
        return load().dflash_kv_pool_release(self.h, seq)

    def pages(self, seq: int) -> list:
        n = load().dflash_kv_pool_pages(self.h, seq, None, 0)
        if n < 0:
            raise DFlashError(1, "dflash_kv_pool_pages")
        buf = (_I * max(n, 1))()
        load().dflash_kv_pool_pages(self.h, seq, ctypes.addressof(buf), n)
        return list(buf)[:n]

    def free(self) -> int:
        return load().dflash_kv_pool_free(self.h)

    def close(self) -> None:
        if self.h:
            load().dflash_kv_pool_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def dflash_verify(ctx, batch, seq_ids, tokens, q, q_lens, flags, argmax, margin=None, logits=None,
                  stream=None) -> None:
    _check(ctx, load().dflash_verify(ctx, batch, _ptr(seq_ids), _ptr(tokens), q, _ptr(q_lens), flags,
                                     _ptr(argmax), _ptr(margin), _ptr(logits), _stream(stream)))


def dflash_set_block_size(ctx, block: int) -> None:
    _check(ctx, load().dflash_set_block_size(ctx, block))


def dflash_draft_block(ctx, batch, seq_ids, anchor, block, topk=0, topk_ids=None, topk_logp=None,
                       logits=None, stream=None) -> None:
    _check(ctx, load().dflash_draft_block(ctx, batch, _ptr(seq_ids), _ptr(anchor), _ptr(block), topk,
                                          _ptr(topk_ids), _ptr(topk_logp), _ptr(logits),
                                          _stream(stream)))


def dflash_accept_commit(ctx, batch, seq_ids, block, argmax, tree, mode, accept_len, next_anchor,
                         emitted, stream=None) -> None:
    tp = ctypes.byref(tree) if tree is not None else None
    _check(ctx, load().dflash_accept_commit(ctx, batch, _ptr(seq_ids), _ptr(block), _ptr(argmax), tp,
                                            mode, _ptr(accept_len), _ptr(next_anchor), _ptr(emitted),
                                            _stream(stream)))


def dflash_inject_kv(ctx, n_rows=0, row_seq=None, row_pos=None, hidden=None, stream=None) -> None:
    _check(ctx, load().dflash_inject_kv(ctx, n_rows, _ptr(row_seq), _ptr(row_pos), _ptr(hidden),
                                        _stream(stream)))


def dtree_build(ctx, batch, anchor, topk_ids, topk_logp, topk, budget, tree: DTree,
                stream=None) -> None:
    _check(ctx, load().dtree_build(ctx, batch, _ptr(anchor), _ptr(topk_ids), _ptr(topk_logp), topk,
                                   budget, ctypes.byref(tree), _stream(stream)))


def dtree_verify(ctx, batch, seq_ids, tree: DTree, node_argmax, margin=None, logits=None,
                 stream=None) -> None:
    _check(ctx, load().dtree_verify(ctx, batch, _ptr(seq_ids), ctypes.byref(tree), _ptr(node_argmax),
                                    _ptr(margin), _ptr(logits), _stream(stream)))


def dflash_check(ctx) -> None:
    _check(ctx, load().dflash_check(ctx))


def dflash_last_error(ctx) -> str:
    return load().dflash_last_error(ctx).decode()


def dflash_seq_lengths(ctx) -> int:
    return load().dflash_seq_lengths(ctx)


def dflash_launch_count(ctx) -> int:
    return int(load().dflash_launch_count(ctx))


def dflash_debug_view(ctx, name: str, layer: int = 0):
    p = _P()
    n = ctypes.c_int64()
    _check(ctx, load().dflash_debug_view(ctx, name.encode(), layer, ctypes.byref(p), ctypes.byref(n)))
    return p.value, n.value


def dflash_block_attention(batch, n_heads, n_kv_heads, ctx_len, block, causal, q, k, v, out,
                           workspace=None, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().dflash_block_attention(batch, n_heads, n_kv_heads, ctx_len, block, causal, _ptr(q),
                                       _ptr(k), _ptr(v), _ptr(out), _ptr(workspace), nbytes,
                                       _stream(stream))
    if st != 0:
        raise DFlashError(st, "dflash_block_attention")


def dflash_block_attention_workspace(batch, n_heads, n_kv_heads, ctx_len, block) -> int:
    return int(load().dflash_block_attention_workspace(batch, n_heads, n_kv_heads, ctx_len, block))


def dflash_plan_gemm(sm_count, M, N, K, kind, max_splits=8) -> dict:
    """Launch plan of the tensor-core GEMM (host arithmetic; no GPU needed)."""
    out = (ctypes.c_int32 * 8)()
    st = load().dflash_plan_gemm(sm_count, M, N, K, kind, max_splits, ctypes.addressof(out))
    if st != 0:
        raise DFlashError(st, "dflash_plan_gemm")
    keys = ("BN", "m_tiles", "n_tiles", "stages", "splits", "threads", "smem_bytes", "persistent")
    return dict(zip(keys, list(out)))


def dflash_plan_attention(sm_count, batch, n_heads, n_kv_heads, q_per_seq, max_keys,
                          min_splits=1) -> dict:
    """Split-KV plan of the bf16 attention (host arithmetic; no GPU needed)."""
    out = (ctypes.c_int32 * 3)()
    st = load().dflash_plan_attention(sm_count, batch, n_heads, n_kv_heads, q_per_seq, max_keys,
                                      min_splits, ctypes.addressof(out))
    if st != 0:
        raise DFlashError(st, "dflash_plan_attention")
    return dict(zip(("splits", "keys_per_split", "ctas"), list(out)))


def dflash_profile(ctx, enable: bool) -> None:
    _check(ctx, load().dflash_profile(ctx, 1 if enable else 0))


PROF_GEMM, PROF_ATTN, PROF_ROW, PROF_VOCAB, PROF_SPEC, PROF_ALL = 0, 1, 2, 3, 4, -1


def dflash_profile_list(ctx, kind: int):
    """Per-launch (ms, flops) of the recorded launches of one class."""
    n = load().dflash_profile_list(ctx, kind, None, None, 0)
    if n < 0:
        raise DFlashError(4, "dflash_profile_list")
    ms = (ctypes.c_double * max(n, 1))()
    fl = (ctypes.c_double * max(n, 1))()
    load().dflash_profile_list(ctx, kind, ctypes.addressof(ms), ctypes.addressof(fl), n)
    return list(zip(list(ms)[:n], list(fl)[:n]))


def dflash_profile_read(ctx, kind: int):
    """(launches, ms, algorithmic bytes, flops) of one kernel class."""
    n = ctypes.c_int64()
    ms, b, f = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
    _check(ctx, load().dflash_profile_read(ctx, kind, ctypes.byref(n), ctypes.byref(ms),
                                           ctypes.byref(b), ctypes.byref(f)))
    return n.value, ms.value, b.value, f.value


def dflash_block_attention_noalloc(batch, n_heads, n_kv_heads, ctx_len, block, causal, q, k, v, out,
                                   stream=None) -> None:
    """Block attention with the library's fixed scratch array (no allocation)."""
    st = load().dflash_block_attention_noalloc(batch, n_heads, n_kv_heads, ctx_len, block, causal,
                                               _ptr(q), _ptr(k), _ptr(v), _ptr(out), _stream(stream))
    if st != 0:
        raise DFlashError(st, "dflash_block_attention_noalloc")


def dflash_debug_wait_timeout(ctx, stream=None) -> None:
    """Runs a bounded wait that expires (about 2 s) and records a timeout."""
    st = load().dflash_debug_wait_timeout(ctx, _stream(stream))
    if st != 0:
        raise DFlashError(st, "dflash_debug_wait_timeout")


def dflash_sample_workspace(rows, vocab) -> int:
    return int(load().dflash_sample_workspace(rows, vocab))


def dflash_sample_rows(rows, vocab, logits, u, tokens, workspace, stream=None) -> None:
    """One temperature-1 draw per row of fp32 logits [rows][vocab] (uniforms u [rows])."""
    nbytes = workspace.numel() * workspace.element_size()
    st = load().dflash_sample_rows(rows, vocab, _ptr(logits), _ptr(u), _ptr(tokens), _ptr(workspace),
                                   nbytes, _stream(stream))
    if st != 0:
        raise DFlashError(st, "dflash_sample_rows")


def dflash_spec_accept_workspace(batch, block, vocab) -> int:
    return int(load().dflash_spec_accept_workspace(batch, block, vocab))


def dflash_spec_accept_sampled(batch, block, vocab, draft_logits, target_logits, tokens, u_accept,
                               u_resample, accept_len, emitted, workspace, stream=None) -> None:
    """Temperature-1 acceptance of one block per sequence (speculative rejection rule)."""
    nbytes = workspace.numel() * workspace.element_size()
    st = load().dflash_spec_accept_sampled(batch, block, vocab, _ptr(draft_logits), _ptr(target_logits),
                                           _ptr(tokens), _ptr(u_accept), _ptr(u_resample),
                                           _ptr(accept_len), _ptr(emitted), _ptr(workspace), nbytes,
                                           _stream(stream))
    if st != 0:
        raise DFlashError(st, "dflash_spec_accept_sampled")


# ---------------------------------------------------------------------------
# the 8-bit KV cache (dflash_kvq_*)
# ---------------------------------------------------------------------------
MASK_NONE, MASK_CAUSAL, MASK_TREE = 0, 1, 2


def _kvq_refuse(what: str) -> None:
    raise DFlashError(1, what)


_KVQ_DTYPES: dict = {}


def _kvq_dtypes() -> dict:
    """torch dtypes by the short names used below (torch is imported on first use)."""
    if not _KVQ_DTYPES:
        import torch
        _KVQ_DTYPES.update(
            i32=(torch.int32,), i8=(torch.int8,), f32=(torch.float32,), bf16=(torch.bfloat16,),
            codes=(torch.uint8, torch.float8_e4m3fn), bits=(torch.int64, torch.uint64),
            stream=torch._C._cuda_getCurrentRawStream, device=torch.cuda.current_device)
    return _KVQ_DTYPES


def _kvq_dense(t, name: str, dtype: str, shape: tuple) -> Optional[int]:
    """Address of a contiguous tensor of this kind and shape (None passes)."""
    if t is None:
        return None
    if (t.dtype not in (_KVQ_DTYPES or _kvq_dtypes())[dtype] or t.shape != shape
            or not t.is_contiguous()):
        _kvq_refuse(f"{name}: need a contiguous {dtype} tensor of shape {shape}")
    return t.data_ptr()


def _kvq_rows(t, name: str, batch: int, rows: int, heads: int) -> int:
    """Elements between the rows of a bf16 [batch][rows][heads][128] tensor
    whose rows may be slices of wider ones."""
    if (t.dtype not in (_KVQ_DTYPES or _kvq_dtypes())["bf16"]
            or t.shape != (batch, rows, heads, 128)):
        _kvq_refuse(f"{name}: need bfloat16 of shape {(batch, rows, heads, 128)}")
    sb, sr, sh, sd = t.stride()
    if rows == 1:
        sr = sb if batch > 1 else heads * 128
    if sd != 1 or (sh != 128 and heads > 1) or (sb != rows * sr and batch > 1):
        _kvq_refuse(f"{name}: rows of {heads} * 128 elements, equally spaced, are needed")
    return sr


def _kvq_stream(stream) -> int:
    if stream is not None:
        return _stream(stream)
    d = _KVQ_DTYPES or _kvq_dtypes()
    return d["stream"](d["device"]())


class KvqCache:
    """An 8-bit KV cache over tensors the caller owns (and this keeps alive):
    k8, v8 [n_pages][n_kv_heads][128][128] uint8 or float8_e4m3fn, k_exp, v_exp
    [n_pages][n_kv_heads][8] int8, page_table [n_seqs][pages_per_seq] int32,
    status [1] int32 (zero at the start)."""

    def __init__(self, k8, v8, k_exp, v_exp, page_table, status):
        if k8.dim() != 4 or page_table.dim() != 2:
            _kvq_refuse("k8: need [n_pages][n_kv_heads][128][128], page_table: [n_seqs][pages]")
        n_pages, heads = k8.shape[0], k8.shape[1]
        for t, name in ((k8, "k8"), (v8, "v8")):
            _kvq_dense(t, name, "codes", (n_pages, heads, PAGE_SLOTS, 128))
        for t, name in ((k_exp, "k_exp"), (v_exp, "v_exp")):
            _kvq_dense(t, name, "i8", (n_pages, heads, PAGE_SLOTS // 16))
        _kvq_dense(page_table, "page_table", "i32", tuple(page_table.shape))
        _kvq_dense(status, "status", "i32", (1,))
        self.tensors = (k8, v8, k_exp, v_exp, page_table, status)
        self.n_kv_heads = heads
        self.n_seqs, self.pages_per_seq = page_table.shape
        self.slots = self.pages_per_seq * PAGE_SLOTS
        self._struct = _KvqCacheStruct(*[_ptr(t) for t in self.tensors], n_pages, heads,
                                       self.n_seqs, self.pages_per_seq)
        self.ref = ctypes.addressof(self._struct)


def _kvq_check(status: int, name: str) -> None:
    if status != 0:
        raise DFlashError(status, name)


def dflash_kvq_append(cache: KvqCache, batch, rows, seq_ids, start, counts, k, v,
                      stream=None) -> None:
    """Writes bf16 rows k, v [batch][rows][n_kv_heads][128] (rows may be slices
    of wider ones) to slots start[b] .. start[b] + counts[b] - 1."""
    one, heads = (batch,), cache.n_kv_heads
    _kvq_check(load().dflash_kvq_append(
        cache.ref, batch, rows, _kvq_dense(seq_ids, "seq_ids", "i32", one),
        _kvq_dense(start, "start", "i32", one), _kvq_dense(counts, "counts", "i32", one),
        k.data_ptr(), v.data_ptr(), _kvq_rows(k, "k", batch, rows, heads),
        _kvq_rows(v, "v", batch, rows, heads), _kvq_stream(stream)), "dflash_kvq_append")


def dflash_kvq_read(cache: KvqCache, batch, rows, seq_ids, start, counts, k_out, v_out,
                    stream=None) -> None:
    """Values of slots start[b] + j, j < counts[b], as bf16 [batch][rows][n_kv_heads][128]."""
    one, out = (batch,), (batch, rows, cache.n_kv_heads, 128)
    _kvq_check(load().dflash_kvq_read(
        cache.ref, batch, rows, _kvq_dense(seq_ids, "seq_ids", "i32", one),
        _kvq_dense(start, "start", "i32", one), _kvq_dense(counts, "counts", "i32", one),
        _kvq_dense(k_out, "k_out", "bf16", out), _kvq_dense(v_out, "v_out", "bf16", out),
        _kvq_stream(stream)), "dflash_kvq_read")


def _kvq_anc(anc, mask, batch, block):
    """(address, words) of the ancestor bits of a tree pass."""
    if mask != MASK_TREE:
        return None, 0
    if anc is None or anc.dim() != 3:
        _kvq_refuse("anc: need [batch][block][words]")
    words = anc.shape[2]
    return _kvq_dense(anc, "anc", "bits", (batch, block, words)), words


def dflash_kvq_attention_workspace(batch, n_heads, n_kv_heads, block, max_keys) -> int:
    return int(load().dflash_kvq_attention_workspace(batch, n_heads, n_kv_heads, block, max_keys))


def dflash_kvq_attention(cache: KvqCache, batch, n_heads, block, mask, seq_ids, kv_lens, q_lens,
                         anc, max_keys, q, out, lse=None, workspace=None, stream=None) -> None:
    """Attention of q [batch][block][n_heads][128] (rows may be slices of wider
    ones) over the cache: out of that shape, lse [batch][block][n_heads]."""
    one = (batch,)
    bits, words = _kvq_anc(anc, mask, batch, block)
    ws, nbytes = None, 0
    if workspace is not None:
        if not workspace.is_contiguous():  # its elements would not be all of its address range
            _kvq_refuse("workspace: need a contiguous tensor")
        ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _kvq_check(load().dflash_kvq_attention(
        cache.ref, batch, n_heads, block, mask, _kvq_dense(seq_ids, "seq_ids", "i32", one),
        _kvq_dense(kv_lens, "kv_lens", "i32", one), _kvq_dense(q_lens, "q_lens", "i32", one), bits,
        words, max_keys, q.data_ptr(), _kvq_rows(q, "q", batch, block, n_heads),
        _kvq_dense(out, "out", "bf16", (batch, block, n_heads, 128)),
        _kvq_dense(lse, "lse", "f32", (batch, block, n_heads)), ws, nbytes, _kvq_stream(stream)),
        "dflash_kvq_attention")


def dflash_kvq_score(cache: KvqCache, batch, n_heads, block, mask, seq_ids, kv_lens, q_lens, anc,
                     max_keys, q, lse, decay, score_in, score_out, stream=None) -> None:
    """score_out = decay * score_in + the weights each slot received; scores
    [n_seqs][n_kv_heads][pages_per_seq * 128] (score_in None: zero)."""
    one, row = (batch,), (cache.n_seqs, cache.n_kv_heads, cache.slots)
    bits, words = _kvq_anc(anc, mask, batch, block)
    _kvq_check(load().dflash_kvq_score(
        cache.ref, batch, n_heads, block, mask, _kvq_dense(seq_ids, "seq_ids", "i32", one),
        _kvq_dense(kv_lens, "kv_lens", "i32", one), _kvq_dense(q_lens, "q_lens", "i32", one), bits,
        words, max_keys, q.data_ptr(), _kvq_rows(q, "q", batch, block, n_heads),
        _kvq_dense(lse, "lse", "f32", (batch, block, n_heads)), decay,
        _kvq_dense(score_in, "score_in", "f32", row), _kvq_dense(score_out, "score_out", "f32", row),
        _kvq_stream(stream)), "dflash_kvq_score")


def dflash_kvq_evict(cache: KvqCache, batch, src_ids, dst_ids, kv_lens, max_keys, budget, window,
                     score, kept, new_lens, stream=None) -> None:
    """Keeps the last `window` slots and the best-scored others of sequences
    src_ids, `budget` in all, in the pages of sequences dst_ids."""
    one, heads = (batch,), cache.n_kv_heads
    _kvq_check(load().dflash_kvq_evict(
        cache.ref, batch, _kvq_dense(src_ids, "src_ids", "i32", one),
        _kvq_dense(dst_ids, "dst_ids", "i32", one), _kvq_dense(kv_lens, "kv_lens", "i32", one),
        max_keys, budget, window, _kvq_dense(score, "score", "f32", (cache.n_seqs, heads, cache.slots)),
        _kvq_dense(kept, "kept", "i32", (batch, heads, budget)),
        _kvq_dense(new_lens, "new_lens", "i32", one), _kvq_stream(stream)), "dflash_kvq_evict")


def dflash_kvq_check(cache: KvqCache, stream=None) -> None:
    """Waits for the stream, clears the cache's status word and raises if it was set."""
    _kvq_check(load().dflash_kvq_check(cache.ref, _kvq_stream(stream)), "dflash_kvq_check")


# ---------------------------------------------------------------------------
# packed batches of prompts
# ---------------------------------------------------------------------------
class Pages:
    """Pages of a cache mapped on the GPU, over tensors the caller owns (and this
    keeps alive): page_table [n_seqs][pages_per_seq], n_mapped [n_seqs], free_pages
    [n_pages], n_free [1], status [1], all int32."""

    def __init__(self, page_table, n_mapped, free_pages, n_free, status):
        if page_table.dim() != 2 or free_pages.dim() != 1:
            _kvq_refuse("page_table: need [n_seqs][pages], free_pages: [n_pages]")
        _kvq_dense(page_table, "page_table", "i32", tuple(page_table.shape))
        _kvq_dense(n_mapped, "n_mapped", "i32", (page_table.shape[0],))
        _kvq_dense(free_pages, "free_pages", "i32", tuple(free_pages.shape))
        _kvq_dense(n_free, "n_free", "i32", (1,))
        _kvq_dense(status, "status", "i32", (1,))
        self.tensors = (page_table, n_mapped, free_pages, n_free, status)
        self.n_seqs, self.pages_per_seq = page_table.shape
        self._struct = _PagesStruct(*[_ptr(t) for t in self.tensors], free_pages.shape[0],
                                    self.n_seqs, self.pages_per_seq)
        self.ref = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, n_pages, n_seqs, pages_per_seq, device="cuda", status=None):
        """A pool of n_pages free pages, the lowest ids first, nothing mapped."""
        import torch
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.full((n_seqs, pages_per_seq), -1, **i32), torch.zeros(n_seqs, **i32),
                   torch.arange(n_pages - 1, -1, -1, **i32), torch.full((1,), n_pages, **i32),
                   torch.zeros(1, **i32) if status is None else status)


def dflash_pages_map(pages: Pages, batch, n_rows, seq_ids, start, counts, offsets, kv_lens,
                     row_seq=None, row_pos=None, row_slot=None, stream=None) -> None:
    """Maps pages for counts[b] rows behind start[b] slots of each sequence and
    lays out the packed batch: offsets, lengths, and the rows' maps."""
    one, row = (batch,), (n_rows,)
    _kvq_check(load().dflash_pages_map(
        pages.ref, batch, n_rows, _kvq_dense(seq_ids, "seq_ids", "i32", one),
        _kvq_dense(start, "start", "i32", one), _kvq_dense(counts, "counts", "i32", one),
        _kvq_dense(offsets, "offsets", "i32", (batch + 1,)),
        _kvq_dense(kv_lens, "kv_lens", "i32", one), _kvq_dense(row_seq, "row_seq", "i32", row),
        _kvq_dense(row_pos, "row_pos", "i32", row), _kvq_dense(row_slot, "row_slot", "i32", row),
        _kvq_stream(stream)), "dflash_pages_map")


def dflash_pages_release(pages: Pages, batch, seq_ids=None, keep=None, stream=None) -> None:
    """Gives back the pages behind the first keep[b] slots (None: all pages)."""
    one = (batch,)
    _kvq_check(load().dflash_pages_release(
        pages.ref, batch, _kvq_dense(seq_ids, "seq_ids", "i32", one),
        _kvq_dense(keep, "keep", "i32", one), _kvq_stream(stream)), "dflash_pages_release")


def dflash_status_check(status, stream=None) -> None:
    """Waits for the stream, clears the status word and raises if it was set."""
    _kvq_check(load().dflash_status_check(_kvq_dense(status, "status", "i32", (1,)),
                                          _kvq_stream(stream)), "dflash_status_check")


def _packed_rows(t, name: str, n_rows: int, heads: int) -> int:
    """Elements between the rows of a bf16 [n_rows][heads][128] tensor whose rows
    may be slices of wider ones."""
    if (t.dtype not in (_KVQ_DTYPES or _kvq_dtypes())["bf16"]
            or t.shape != (n_rows, heads, 128)):
        _kvq_refuse(f"{name}: need bfloat16 of shape {(n_rows, heads, 128)}")
    sr, sh, sd = t.stride()
    if sd != 1 or (sh != 128 and heads > 1):
        _kvq_refuse(f"{name}: rows of {heads} * 128 elements are needed")
    return sr if n_rows > 1 else heads * 128


def dflash_kvq_append_packed(cache: KvqCache, batch, seq_ids, start, offsets, k, v,
                             stream=None) -> None:
    """Writes the packed bf16 rows k, v [n_rows][n_kv_heads][128] of each sequence to
    slots start[b] on."""
    one, heads, n_rows = (batch,), cache.n_kv_heads, k.shape[0]
    _kvq_check(load().dflash_kvq_append_packed(
        cache.ref, batch, n_rows, _kvq_dense(seq_ids, "seq_ids", "i32", one),
        _kvq_dense(start, "start", "i32", one), _kvq_dense(offsets, "offsets", "i32", (batch + 1,)),
        k.data_ptr(), v.data_ptr(), _packed_rows(k, "k", n_rows, heads),
        _packed_rows(v, "v", n_rows, heads), _kvq_stream(stream)), "dflash_kvq_append_packed")


def dflash_prompt_attention(batch, causal, offsets, q, k, v, out, lse=None, status=None,
                            stream=None) -> None:
    """Attention of a packed batch of prompts over themselves: q [n_rows][n_heads][128],
    k, v [n_rows][n_kv_heads][128] (rows may be slices of wider ones), out of
    q's shape, lse [n_rows][n_heads] or None, status [1] int32 (zero at the start; always
    needed, its default only lets lse be left out)."""
    if status is None:
        _kvq_refuse("status: need int32 [1], where bad offsets are reported")
    if q.dim() != 3 or k.dim() != 3:
        _kvq_refuse("q, k: need [n_rows][heads][128]")
    n_rows, heads, _ = rows = q.shape
    kv_heads = k.shape[1]
    _kvq_check(load().dflash_prompt_attention(
        batch, n_rows, heads, kv_heads, causal, _kvq_dense(offsets, "offsets", "i32", (batch + 1,)),
        q.data_ptr(), _packed_rows(q, "q", n_rows, heads), k.data_ptr(),
        _packed_rows(k, "k", n_rows, kv_heads), v.data_ptr(),
        _packed_rows(v, "v", n_rows, kv_heads), _kvq_dense(out, "out", "bf16", rows),
        _kvq_dense(lse, "lse", "f32", (n_rows, heads)), _kvq_dense(status, "status", "i32", (1,)),
        _kvq_stream(stream)), "dflash_prompt_attention")


def dflash_token_logprobs(logits, tokens, top=0, logp=None, entropy=None, top_ids=None,
                          top_logp=None, stream=None) -> None:
    """Log probabilities of tokens [rows] under logits [rows][vocab] (fp32 or bf16, rows
    may be slices of wider ones), entropies [rows], and the `top` best ids with theirs."""
    d = _KVQ_DTYPES or _kvq_dtypes()
    if logits.dim() != 2 or logits.dtype not in d["f32"] + d["bf16"] or (
            logits.shape[1] > 1 and logits.stride(1) != 1):
        _kvq_refuse("logits: need float32 or bfloat16 [rows][vocab], each row contiguous")
    rows, vocab = logits.shape
    dtype = DFLASH_F32 if logits.dtype in d["f32"] else DFLASH_BF16
    _kvq_check(load().dflash_token_logprobs(
        rows, vocab, dtype, logits.data_ptr(), logits.stride(0) if rows > 1 else vocab,
        _kvq_dense(tokens, "tokens", "i32", (rows,)), top, _kvq_dense(logp, "logp", "f32", (rows,)),
        _kvq_dense(entropy, "entropy", "f32", (rows,)),
        _kvq_dense(top_ids, "top_ids", "i32", (rows, top)),
        _kvq_dense(top_logp, "top_logp", "f32", (rows, top)), _kvq_stream(stream)),
        "dflash_token_logprobs")


def dflash_debug_trace(ctx, dst=None) -> None:
    """Registers (or clears with None) a [L][max_rows][d] fp32 residual trace."""
    nbytes = dst.numel() * dst.element_size() if dst is not None else 0
    _check(ctx, load().dflash_debug_trace(ctx, _ptr(dst), nbytes))


def dflash_debug_trace_draft(ctx, dst=None) -> None:
    """Registers (or clears with None) a [L_d][max_rows][d] fp32 residual trace
    of the draft passes."""
    nbytes = dst.numel() * dst.element_size() if dst is not None else 0
    _check(ctx, load().dflash_debug_trace_draft(ctx, _ptr(dst), nbytes))


def dflash_debug_trace_draft_attn(ctx, q=None, attn=None) -> None:
    """Registers (or clears with None) per-draft-layer copies of the roped
    queries and of the attention output, [L_d][max_rows][H*hd] each."""
    t = q if q is not None else attn
    nbytes = t.numel() * t.element_size() if t is not None else 0
    _check(ctx, load().dflash_debug_trace_draft_attn(ctx, _ptr(q), _ptr(attn), nbytes))
