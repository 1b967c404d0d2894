"""Python binding of libuocr.so, the B200 (sm_100a) SR-SWA / DASH block-sparse attention step.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/uocr.h``.  PyTorch provides the
device memory and the stream; there is no CPU fallback: the first call (or
any access to ``lib``) raises ``ImportError`` when ``libuocr.so`` has not been
built (``python -m block_sparse_long_uocr_b200.build``).  The library is loaded
on first use so that the build module can be imported before it exists.

Entry points (same names as the C ABI, without the ``uocr_`` prefix):

* :func:`index_score`  -- block scores of the 1-head x 128 Lightning Indexer;
* :func:`block_topk`   -- 4 local + top-12 remote block selection;
* :func:`sparse_attn`  -- exact 10-head attention over the selected 512 tokens;
* :func:`sparse_decode` -- the three fused into one decode call;
* :func:`prefill_index_score` -- the block scores of a prefill chunk on the tcgen05 tensor cores;
* :func:`sparse_prefill` -- tensor-core scoring, selection and attention for a prefill chunk;
* :func:`sparse_attn_seq` -- the block-centric attention of many queries of one sequence over a
  caller's selection (the attention stage of :func:`sparse_prefill`);
* :func:`summary_score`, :func:`block_summary_mean`, :func:`sparse_decode_summary` -- block-summary
  scoring (one vector per block) and the decode step built on it;
* :func:`block_topk_masked` -- selection under a page-aware candidate bitmap;
* :func:`rope_append` -- page2d rotary embedding of new tokens and their append to the caches;
* :func:`dense_decode` -- comparator: full causal attention, or an R-SWA-style reference
  prefix plus the 128-token window (the baselines the sparse step is measured against);
* :func:`sparse_decode_static` -- the same decode call for callers that cannot
  allocate device memory (scratch held inside the library);
* :func:`rope_append_kv8`, :func:`sparse_attn_kv8`, :func:`sparse_decode_kv8`, :func:`dense_decode_kv8`,
  :func:`sparse_attn_seq_kv8`, :func:`sparse_prefill_kv8` -- the same steps over a key / value cache
  held in e4m3 with a scale for each (page, head), optionally adding each block's attention weight to
  its running total;
* :func:`evict_blocks` -- removes the blocks with the lowest totals from tables, totals and lengths;
* :func:`workspace_bytes` and its likes.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libuocr.so")

BLOCK = 32
N_LOCAL = 4
N_REMOTE = 12
N_SEL = 16
HEAD_DIM = 128
IDX_DIM = 128

STATUS = {0: "UOCR_OK", 1: "UOCR_ERR_INVALID_ARG", 2: "UOCR_ERR_UNSUPPORTED",
          3: "UOCR_ERR_WORKSPACE", 4: "UOCR_ERR_CUDA"}
DEVERR_PAGE, DEVERR_POS, DEVERR_SEL, DEVERR_TIMEOUT = 1, 2, 4, 8


class UocrError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: {msg}")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m block_sparse_long_uocr_b200.build` "
                          "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.uocr_status_string.argtypes = [I]
    lib.uocr_status_string.restype = ctypes.c_char_p
    lib.uocr_abi_version.argtypes = []
    lib.uocr_abi_version.restype = I
    lib.uocr_last_cuda_error.argtypes = []
    lib.uocr_last_cuda_error.restype = ctypes.c_char_p
    lib.uocr_workspace_bytes.argtypes = [I, I, I]
    lib.uocr_workspace_bytes.restype = Z
    lib.uocr_index_score.argtypes = [P, P, P, P, P, P, I, I, I, I, P, P, P]
    lib.uocr_index_score.restype = I
    lib.uocr_block_topk.argtypes = [P, P, P, P, I, I, I, P, P, P]
    lib.uocr_block_topk.restype = I
    lib.uocr_sparse_attn.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, F, P, P, P]
    lib.uocr_sparse_attn.restype = I
    lib.uocr_sparse_decode.argtypes = [P, P, P, P, P, P, P, I, I, I, I, P, P, P, Z, P, P]
    lib.uocr_sparse_decode.restype = I
    lib.uocr_summary_score.argtypes = [P, P, P, P, P, P, I, I, I, I, P, P, P]
    lib.uocr_summary_score.restype = I
    lib.uocr_block_summary_mean.argtypes = [P, P, I, I, P, P, P]
    lib.uocr_block_summary_mean.restype = I
    lib.uocr_sparse_decode_summary.argtypes = [P, P, P, P, P, P, P, I, I, I, I, P, P, P, Z, P, P]
    lib.uocr_sparse_decode_summary.restype = I
    lib.uocr_block_topk_masked.argtypes = [P, P, P, P, P, I, I, I, I, P, P, P]
    lib.uocr_block_topk_masked.restype = I
    lib.uocr_rope_append.argtypes = [P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, P, P, P, P, P]
    lib.uocr_rope_append.restype = I
    lib.uocr_dense_workspace_bytes.argtypes = [I, I, I]
    lib.uocr_dense_workspace_bytes.restype = Z
    lib.uocr_dense_decode.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P, Z, P, P]
    lib.uocr_dense_decode.restype = I
    lib.uocr_prefill_workspace_bytes.argtypes = [I, I, I]
    lib.uocr_prefill_workspace_bytes.restype = Z
    lib.uocr_prefill_index_score.argtypes = [P, P, P, P, I, P, I, I, I, I, P, P, P]
    lib.uocr_prefill_index_score.restype = I
    lib.uocr_sparse_prefill.argtypes = [P, P, P, P, P, P, P, I, P, I, I, I, I, I, P, P, P, Z, P, P]
    lib.uocr_sparse_prefill.restype = I
    lib.uocr_sparse_attn_seq_workspace_bytes.argtypes = [I, I, I]
    lib.uocr_sparse_attn_seq_workspace_bytes.restype = Z
    lib.uocr_sparse_attn_seq.argtypes = [P, P, P, P, P, I, P, P, I, I, I, I, I, F, P, P, Z, P, P]
    lib.uocr_sparse_attn_seq.restype = I
    lib.uocr_sparse_decode_static.argtypes = [P, P, P, P, P, P, P, I, I, I, I, P, P, P, P]
    lib.uocr_sparse_decode_static.restype = I
    lib.uocr_rope_append_kv8.argtypes = [P] * 10 + [I] * 5 + [P] * 9
    lib.uocr_sparse_attn_kv8.argtypes = [P] * 10 + [I] * 5 + [F, P, P, P, P]
    lib.uocr_sparse_decode_kv8.argtypes = [P] * 9 + [I] * 4 + [P, P, P, P, Z, P, P]
    lib.uocr_dense_decode_kv8.argtypes = [P] * 7 + [I] * 5 + [P, P, P, Z, P, P]
    lib.uocr_sparse_attn_seq_kv8.argtypes = [P] * 7 + [I, P, P] + [I] * 5 + [F, P, P, P, Z, P, P]
    lib.uocr_sparse_prefill_kv8.argtypes = [P] * 9 + [I, P] + [I] * 5 + [P, P, P, P, Z, P, P]
    lib.uocr_evict_blocks.argtypes = [P] * 3 + [I] * 5 + [P] * 6 + [Z, P, P]
    for name in ("rope_append_kv8", "sparse_attn_kv8", "sparse_decode_kv8", "dense_decode_kv8", "sparse_attn_seq_kv8",
                 "sparse_prefill_kv8", "evict_blocks"):
        getattr(lib, "uocr_" + name).restype = I
    for name in ("dense_kv8", "sparse_attn_seq_kv8", "prefill_kv8", "evict"):
        fn = getattr(lib, f"uocr_{name}_workspace_bytes")
        fn.argtypes = [I, I, I]
        fn.restype = Z
    return lib


_LIB = None


def _lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        _LIB = _load()
    return _LIB


def __getattr__(name):
    if name == "lib":
        return _lib()
    raise AttributeError(name)


# --------------------------------------------------------------------------- helpers
def _check(fn: str, st: int):
    if st != 0:
        msg = _lib().uocr_status_string(st).decode()
        if st == 4:   # UOCR_ERR_CUDA: name the CUDA error behind it
            msg += f" ({_lib().uocr_last_cuda_error().decode()})"
        raise UocrError(fn, st, msg)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int | None = None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _opt_i32(t, name, n=None):
    if t is None:
        return None
    _dev(t, name, torch.int32, 1)
    if n is not None:
        _shape(t, name, (n,))
    return t


def _shape(t: torch.Tensor, name: str, shape) -> torch.Tensor:
    """Refuse, before any launch, a tensor whose shape differs from what the kernels will index
    (None in `shape` accepts any extent): a smaller buffer would be written or read past its end
    on the device."""
    got = tuple(t.shape)
    if len(got) != len(shape) or any(e is not None and g != e for g, e in zip(got, shape)):
        want = "[" + ", ".join("*" if e is None else str(e) for e in shape) + "]"
        raise ValueError(f"{name} must have shape {want}, got {list(got)}")
    return t


def _check_caches(k_cache, v_cache, H):
    """K / V caches [P, H, 32, 128] of the same shape."""
    _shape(k_cache, "k_cache", (None, H, BLOCK, HEAD_DIM))
    _shape(v_cache, "v_cache", tuple(k_cache.shape))


def _check_decode_args(q, k_cache, v_cache, idx_q, idx_k_cache, block_table, seq_lens, out, sel):
    """One decode query per sequence: every per-sequence tensor has B rows, the caches agree on
    the head count and the pool size, and the outputs match the queries."""
    B, H = q.shape[0], q.shape[1]
    _shape(q, "q", (B, H, HEAD_DIM))
    _check_caches(k_cache, v_cache, H)
    _shape(idx_q, "idx_q", (B, IDX_DIM))
    if idx_k_cache is not None:
        _shape(idx_k_cache, "idx_k_cache", (k_cache.shape[0], BLOCK, IDX_DIM))
    _shape(block_table, "block_table", (B, None))
    _shape(seq_lens, "seq_lens", (B,))
    if out is not None:
        _shape(out, "out", (B, H, HEAD_DIM))
    if sel is not None:
        _shape(sel, "sel", (B, N_SEL))


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def workspace_bytes(n_q: int, heads: int, max_blocks: int) -> int:
    return int(_lib().uocr_workspace_bytes(int(n_q), int(heads), int(max_blocks)))


def prefill_workspace_bytes(n_q: int, heads: int, max_blocks: int) -> int:
    return int(_lib().uocr_prefill_workspace_bytes(int(n_q), int(heads), int(max_blocks)))


def alloc_prefill_workspace(n_q: int, heads: int, max_blocks: int, device) -> torch.Tensor:
    """uint8 workspace for sparse_prefill; its first n_q*max_blocks*4 bytes hold the block scores."""
    return torch.empty(max(prefill_workspace_bytes(n_q, heads, max_blocks), 1), dtype=torch.uint8, device=device)


def sparse_attn_seq_workspace_bytes(n_q: int, heads: int, max_blocks: int) -> int:
    return int(_lib().uocr_sparse_attn_seq_workspace_bytes(int(n_q), int(heads), int(max_blocks)))


def alloc_workspace(n_q: int, heads: int, max_blocks: int, device) -> torch.Tensor:
    """A uint8 tensor of workspace_bytes(...) bytes (torch allocations are 256-byte aligned)."""
    return torch.empty(max(workspace_bytes(n_q, heads, max_blocks), 1), dtype=torch.uint8, device=device)


def _on_its_stream(fn):
    """What `fn` allocates and fills is allocated for, and filled on, the stream that it is given: memory or fills of the
    current stream would not be ordered before the kernels.  What it returns may be used on the current stream and
    dropped there."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        current = torch.cuda.current_stream(stream.device)
        with torch.cuda.stream(stream):
            got = fn(*args, stream=stream, **kw)
        for t in got if isinstance(got, tuple) else (got,):
            t.record_stream(current)
        return got

    return call


# --------------------------------------------------------------------------- entry points
@_on_its_stream
def index_score(idx_q, idx_k_cache, block_table, seq_lens, q_seq=None, q_pos=None, *,
                scores=None, dev_err=None, stream=None) -> torch.Tensor:
    """fp32 [n_q, max_blocks] block scores (entries past a query's causal blocks untouched)."""
    _dev(idx_q, "idx_q", torch.bfloat16, 2)
    _dev(idx_k_cache, "idx_k_cache", torch.bfloat16, 3)
    _dev(block_table, "block_table", torch.int32, 2)
    _dev(seq_lens, "seq_lens", torch.int32, 1)
    n_q, B, mb = idx_q.shape[0], block_table.shape[0], block_table.shape[1]
    _shape(idx_q, "idx_q", (n_q, IDX_DIM))
    _shape(idx_k_cache, "idx_k_cache", (None, BLOCK, IDX_DIM))
    _shape(seq_lens, "seq_lens", (B,))
    if scores is None:
        scores = torch.full((n_q, mb), float("-inf"), dtype=torch.float32, device=idx_q.device)
    _dev(scores, "scores", torch.float32, 2)
    _shape(scores, "scores", (n_q, mb))
    _check("uocr_index_score", _lib().uocr_index_score(
        _ptr(idx_q), _ptr(idx_k_cache), _ptr(block_table), _ptr(seq_lens), _ptr(_opt_i32(q_seq, "q_seq", n_q)),
        _ptr(_opt_i32(q_pos, "q_pos", n_q)), n_q, B, mb, idx_k_cache.shape[0], _ptr(scores),
        _ptr(dev_err), _stream(stream)))
    return scores


@_on_its_stream
def block_topk(scores, seq_lens, q_seq=None, q_pos=None, *, sel=None, dev_err=None, stream=None) -> torch.Tensor:
    """int32 [n_q, 16] selected logical blocks (ascending, -1 padded)."""
    _dev(scores, "scores", torch.float32, 2)
    _dev(seq_lens, "seq_lens", torch.int32, 1)
    n_q, mb = scores.shape
    if sel is None:
        sel = torch.empty((n_q, N_SEL), dtype=torch.int32, device=scores.device)
    _dev(sel, "sel", torch.int32, 2)
    _shape(sel, "sel", (n_q, N_SEL))
    _check("uocr_block_topk", _lib().uocr_block_topk(
        _ptr(scores), _ptr(seq_lens), _ptr(_opt_i32(q_seq, "q_seq", n_q)), _ptr(_opt_i32(q_pos, "q_pos", n_q)),
        n_q, seq_lens.shape[0], mb, _ptr(sel), _ptr(dev_err), _stream(stream)))
    return sel


@_on_its_stream
def sparse_attn(q, k_cache, v_cache, block_table, seq_lens, sel, q_seq=None, q_pos=None, *,
                scale: float | None = None, out=None, dev_err=None, stream=None) -> torch.Tensor:
    """bf16 [n_q, H, 128] attention output over the selected blocks."""
    _dev(q, "q", torch.bfloat16, 3)
    _dev(k_cache, "k_cache", torch.bfloat16, 4)
    _dev(v_cache, "v_cache", torch.bfloat16, 4)
    _dev(block_table, "block_table", torch.int32, 2)
    _dev(seq_lens, "seq_lens", torch.int32, 1)
    _dev(sel, "sel", torch.int32, 2)
    n_q, H = q.shape[0], q.shape[1]
    B, mb = block_table.shape
    _shape(q, "q", (n_q, H, HEAD_DIM))
    _check_caches(k_cache, v_cache, H)
    _shape(seq_lens, "seq_lens", (B,))
    _shape(sel, "sel", (n_q, N_SEL))
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out", torch.bfloat16, 3)
    _shape(out, "out", (n_q, H, HEAD_DIM))
    sc = float(scale) if scale is not None else HEAD_DIM ** -0.5
    _check("uocr_sparse_attn", _lib().uocr_sparse_attn(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
        _ptr(_opt_i32(q_seq, "q_seq", n_q)), _ptr(_opt_i32(q_pos, "q_pos", n_q)), _ptr(sel), n_q, B, H, mb,
        k_cache.shape[0], ctypes.c_float(sc), _ptr(out), _ptr(dev_err), _stream(stream)))
    return out


@_on_its_stream
def sparse_decode(q, k_cache, v_cache, idx_q, idx_k_cache, block_table, seq_lens, *,
                  out=None, sel=None, workspace=None, dev_err=None, stream=None):
    """One decode query per sequence at p = seq_len - 1.  Returns (out [B,H,128] bf16, sel [B,16] int32)."""
    _dev(q, "q", torch.bfloat16, 3)
    _dev(k_cache, "k_cache", torch.bfloat16, 4)
    _dev(v_cache, "v_cache", torch.bfloat16, 4)
    _dev(idx_q, "idx_q", torch.bfloat16, 2)
    _dev(idx_k_cache, "idx_k_cache", torch.bfloat16, 3)
    _dev(block_table, "block_table", torch.int32, 2)
    _dev(seq_lens, "seq_lens", torch.int32, 1)
    B, H = q.shape[0], q.shape[1]
    mb = block_table.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if sel is None:
        sel = torch.empty((B, N_SEL), dtype=torch.int32, device=q.device)
    _dev(out, "out", torch.bfloat16, 3)
    _dev(sel, "sel", torch.int32, 2)
    _check_decode_args(q, k_cache, v_cache, idx_q, idx_k_cache, block_table, seq_lens, out, sel)
    if workspace is None:
        workspace = alloc_workspace(B, H, mb, q.device)
    _check("uocr_sparse_decode", _lib().uocr_sparse_decode(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(idx_q), _ptr(idx_k_cache), _ptr(block_table),
        _ptr(seq_lens), B, H, mb, k_cache.shape[0], _ptr(out), _ptr(sel), _ptr(workspace),
        workspace.numel(), _ptr(dev_err), _stream(stream)))
    return out, sel


@_on_its_stream
def prefill_index_score(idx_q, idx_k_cache, block_table, seq_lens, seq: int, q_pos, *,
                        scores=None, dev_err=None, stream=None) -> torch.Tensor:
    """fp32 [n_q, max_blocks] block scores of n_q queries of sequence `seq` (tcgen05 GEMM)."""
    _dev(idx_q, "idx_q", torch.bfloat16, 2)
    _dev(idx_k_cache, "idx_k_cache", torch.bfloat16, 3)
    _dev(block_table, "block_table", torch.int32, 2)
    _dev(seq_lens, "seq_lens", torch.int32, 1)
    _dev(q_pos, "q_pos", torch.int32, 1)
    n_q, B, mb = idx_q.shape[0], block_table.shape[0], block_table.shape[1]
    _shape(idx_q, "idx_q", (n_q, IDX_DIM))
    _shape(idx_k_cache, "idx_k_cache", (None, BLOCK, IDX_DIM))
    _shape(seq_lens, "seq_lens", (B,))
    _shape(q_pos, "q_pos", (n_q,))
    if scores is None:
        scores = torch.full((n_q, mb), float("-inf"), dtype=torch.float32, device=idx_q.device)
    _dev(scores, "scores", torch.float32, 2)
    _shape(scores, "scores", (n_q, mb))
    _check("uocr_prefill_index_score", _lib().uocr_prefill_index_score(
        _ptr(idx_q), _ptr(idx_k_cache), _ptr(block_table), _ptr(seq_lens), int(seq), _ptr(q_pos), n_q, B, mb,
        idx_k_cache.shape[0], _ptr(scores), _ptr(dev_err), _stream(stream)))
    return scores


@_on_its_stream
def sparse_prefill(q, k_cache, v_cache, idx_q, idx_k_cache, block_table, seq_lens, seq: int, q_pos, *,
                   out=None, sel=None, workspace=None, dev_err=None, stream=None):
    """Prefill chunk of sequence `seq`.  Returns (out [n_q,H,128] bf16, sel [n_q,16] int32)."""
    for t, n, dt, nd in ((q, "q", torch.bfloat16, 3), (k_cache, "k_cache", torch.bfloat16, 4),
                         (v_cache, "v_cache", torch.bfloat16, 4), (idx_q, "idx_q", torch.bfloat16, 2),
                         (idx_k_cache, "idx_k_cache", torch.bfloat16, 3), (block_table, "block_table", torch.int32, 2),
                         (seq_lens, "seq_lens", torch.int32, 1), (q_pos, "q_pos", torch.int32, 1)):
        _dev(t, n, dt, nd)
    n_q, H = q.shape[0], q.shape[1]
    B, mb = block_table.shape
    if out is None:
        out = torch.empty_like(q)
    if sel is None:
        sel = torch.empty((n_q, N_SEL), dtype=torch.int32, device=q.device)
    _dev(out, "out", torch.bfloat16, 3)
    _dev(sel, "sel", torch.int32, 2)
    _shape(q, "q", (n_q, H, HEAD_DIM))
    _check_caches(k_cache, v_cache, H)
    _shape(idx_q, "idx_q", (n_q, IDX_DIM))
    _shape(idx_k_cache, "idx_k_cache", (k_cache.shape[0], BLOCK, IDX_DIM))
    _shape(seq_lens, "seq_lens", (B,))
    _shape(q_pos, "q_pos", (n_q,))
    _shape(out, "out", (n_q, H, HEAD_DIM))
    _shape(sel, "sel", (n_q, N_SEL))
    if workspace is None:
        workspace = alloc_prefill_workspace(n_q, H, mb, q.device)
    _check("uocr_sparse_prefill", _lib().uocr_sparse_prefill(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(idx_q), _ptr(idx_k_cache), _ptr(block_table), _ptr(seq_lens),
        int(seq), _ptr(q_pos), n_q, B, H, mb, k_cache.shape[0], _ptr(out), _ptr(sel), _ptr(workspace),
        workspace.numel(), _ptr(dev_err), _stream(stream)))
    return out, sel


@_on_its_stream
def sparse_attn_seq(q, k_cache, v_cache, block_table, seq_lens, seq: int, q_pos, sel, *, scale=None,
                    out=None, workspace=None, dev_err=None, stream=None) -> torch.Tensor:
    """Attention of many queries of sequence `seq` over the given selection (block-centric).
    Returns out [n_q,H,128] bf16."""
    for t, n, dt, nd in ((q, "q", torch.bfloat16, 3), (k_cache, "k_cache", torch.bfloat16, 4),
                         (v_cache, "v_cache", torch.bfloat16, 4), (block_table, "block_table", torch.int32, 2),
                         (seq_lens, "seq_lens", torch.int32, 1), (q_pos, "q_pos", torch.int32, 1),
                         (sel, "sel", torch.int32, 2)):
        _dev(t, n, dt, nd)
    n_q, H = q.shape[0], q.shape[1]
    B, mb = block_table.shape
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out", torch.bfloat16, 3)
    _shape(q, "q", (n_q, H, HEAD_DIM))
    _check_caches(k_cache, v_cache, H)
    _shape(seq_lens, "seq_lens", (B,))
    _shape(q_pos, "q_pos", (n_q,))
    _shape(sel, "sel", (n_q, N_SEL))
    _shape(out, "out", (n_q, H, HEAD_DIM))
    if workspace is None:
        workspace = torch.empty(max(sparse_attn_seq_workspace_bytes(n_q, H, mb), 1), dtype=torch.uint8,
                                device=q.device)
    sc = float(scale) if scale is not None else HEAD_DIM ** -0.5
    _check("uocr_sparse_attn_seq", _lib().uocr_sparse_attn_seq(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens), int(seq), _ptr(q_pos), _ptr(sel),
        n_q, B, H, mb, k_cache.shape[0], sc, _ptr(out), _ptr(workspace), workspace.numel(), _ptr(dev_err),
        _stream(stream)))
    return out


@_on_its_stream
def summary_score(idx_q, summary_cache, block_table, seq_lens, q_seq=None, q_pos=None, *,
                  scores=None, dev_err=None, stream=None) -> torch.Tensor:
    """fp32 [n_q, max_blocks]: idx_q . summary of each causal block's page."""
    _dev(idx_q, "idx_q", torch.bfloat16, 2)
    _dev(summary_cache, "summary_cache", torch.bfloat16, 2)
    _dev(block_table, "block_table", torch.int32, 2)
    _dev(seq_lens, "seq_lens", torch.int32, 1)
    n_q, B, mb = idx_q.shape[0], block_table.shape[0], block_table.shape[1]
    _shape(idx_q, "idx_q", (n_q, IDX_DIM))
    _shape(summary_cache, "summary_cache", (None, IDX_DIM))
    _shape(seq_lens, "seq_lens", (B,))
    if scores is None:
        scores = torch.full((n_q, mb), float("-inf"), dtype=torch.float32, device=idx_q.device)
    _dev(scores, "scores", torch.float32, 2)
    _shape(scores, "scores", (n_q, mb))
    _check("uocr_summary_score", _lib().uocr_summary_score(
        _ptr(idx_q), _ptr(summary_cache), _ptr(block_table), _ptr(seq_lens), _ptr(_opt_i32(q_seq, "q_seq", n_q)),
        _ptr(_opt_i32(q_pos, "q_pos", n_q)), n_q, B, mb, summary_cache.shape[0], _ptr(scores), _ptr(dev_err),
        _stream(stream)))
    return scores


@_on_its_stream
def block_summary_mean(idx_k_cache, summary_cache=None, pages=None, *, dev_err=None, stream=None) -> torch.Tensor:
    """bf16 [P, 128]: the mean of each (listed) page's indexer keys."""
    _dev(idx_k_cache, "idx_k_cache", torch.bfloat16, 3)
    P = idx_k_cache.shape[0]
    _shape(idx_k_cache, "idx_k_cache", (P, BLOCK, IDX_DIM))
    if summary_cache is None:
        summary_cache = torch.zeros((P, IDX_DIM), dtype=torch.bfloat16, device=idx_k_cache.device)
    _dev(summary_cache, "summary_cache", torch.bfloat16, 2)
    _shape(summary_cache, "summary_cache", (P, IDX_DIM))
    n = P if pages is None else _dev(pages, "pages", torch.int32, 1).shape[0]
    _check("uocr_block_summary_mean", _lib().uocr_block_summary_mean(
        _ptr(idx_k_cache), _ptr(pages), n, P, _ptr(summary_cache), _ptr(dev_err), _stream(stream)))
    return summary_cache


@_on_its_stream
def sparse_decode_summary(q, k_cache, v_cache, idx_q, summary_cache, block_table, seq_lens, *,
                          out=None, sel=None, workspace=None, dev_err=None, stream=None):
    """sparse_decode with block-summary scoring.  Returns (out, sel)."""
    for t, n, dt, nd in ((q, "q", torch.bfloat16, 3), (k_cache, "k_cache", torch.bfloat16, 4),
                         (v_cache, "v_cache", torch.bfloat16, 4), (idx_q, "idx_q", torch.bfloat16, 2),
                         (summary_cache, "summary_cache", torch.bfloat16, 2), (block_table, "block_table", torch.int32, 2),
                         (seq_lens, "seq_lens", torch.int32, 1)):
        _dev(t, n, dt, nd)
    B, H = q.shape[0], q.shape[1]
    mb = block_table.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if sel is None:
        sel = torch.empty((B, N_SEL), dtype=torch.int32, device=q.device)
    _dev(out, "out", torch.bfloat16, 3)
    _dev(sel, "sel", torch.int32, 2)
    _shape(summary_cache, "summary_cache", (k_cache.shape[0], IDX_DIM))
    _check_decode_args(q, k_cache, v_cache, idx_q, None, block_table, seq_lens, out, sel)
    if workspace is None:
        workspace = alloc_workspace(B, H, mb, q.device)
    _check("uocr_sparse_decode_summary", _lib().uocr_sparse_decode_summary(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(idx_q), _ptr(summary_cache), _ptr(block_table), _ptr(seq_lens),
        B, H, mb, k_cache.shape[0], _ptr(out), _ptr(sel), _ptr(workspace), workspace.numel(), _ptr(dev_err),
        _stream(stream)))
    return out, sel


@_on_its_stream
def block_topk_masked(scores, seq_lens, cand_mask, q_seq=None, q_pos=None, *, sel=None, dev_err=None,
                      stream=None) -> torch.Tensor:
    """Selection where remote candidate j of sequence b needs bit j of cand_mask[b] (int32 words)."""
    _dev(scores, "scores", torch.float32, 2)
    _dev(seq_lens, "seq_lens", torch.int32, 1)
    _dev(cand_mask, "cand_mask", torch.int32, 2)
    n_q, mb = scores.shape
    _shape(cand_mask, "cand_mask", (seq_lens.shape[0], None))
    if sel is None:
        sel = torch.empty((n_q, N_SEL), dtype=torch.int32, device=scores.device)
    _dev(sel, "sel", torch.int32, 2)
    _shape(sel, "sel", (n_q, N_SEL))
    _check("uocr_block_topk_masked", _lib().uocr_block_topk_masked(
        _ptr(scores), _ptr(seq_lens), _ptr(_opt_i32(q_seq, "q_seq", n_q)), _ptr(_opt_i32(q_pos, "q_pos", n_q)),
        _ptr(cand_mask), cand_mask.shape[1], n_q, seq_lens.shape[0], mb, _ptr(sel), _ptr(dev_err), _stream(stream)))
    return sel


def rope_append(q, idx_q, k_new, v_new, idx_k_new, tok_pos, page_pos, block_table, seq_lens,
                k_cache, v_cache, idx_k_cache, q_seq=None, q_pos=None, *, dev_err=None, stream=None):
    """Rotate q / idx_q in place (page2d) and write the new tokens' rotated k / idx_k and raw v into the
    caches at each token's position (default: its sequence's last cached position)."""
    for t, n, dt, nd in ((q, "q", torch.bfloat16, 3), (idx_q, "idx_q", torch.bfloat16, 2),
                         (k_new, "k_new", torch.bfloat16, 3), (v_new, "v_new", torch.bfloat16, 3),
                         (idx_k_new, "idx_k_new", torch.bfloat16, 2), (tok_pos, "tok_pos", torch.int32, 1),
                         (page_pos, "page_pos", torch.int32, 1), (block_table, "block_table", torch.int32, 2),
                         (seq_lens, "seq_lens", torch.int32, 1), (k_cache, "k_cache", torch.bfloat16, 4),
                         (v_cache, "v_cache", torch.bfloat16, 4), (idx_k_cache, "idx_k_cache", torch.bfloat16, 3)):
        _dev(t, n, dt, nd)
    n, H = q.shape[0], q.shape[1]
    B, mb = block_table.shape
    _shape(q, "q", (n, H, HEAD_DIM))
    _shape(idx_q, "idx_q", (n, IDX_DIM))
    _shape(k_new, "k_new", (n, H, HEAD_DIM))
    _shape(v_new, "v_new", (n, H, HEAD_DIM))
    _shape(idx_k_new, "idx_k_new", (n, IDX_DIM))
    _shape(tok_pos, "tok_pos", (n,))
    _shape(page_pos, "page_pos", (n,))
    _shape(seq_lens, "seq_lens", (B,))
    _check_caches(k_cache, v_cache, H)
    _shape(idx_k_cache, "idx_k_cache", (k_cache.shape[0], BLOCK, IDX_DIM))
    _check("uocr_rope_append", _lib().uocr_rope_append(
        _ptr(q), _ptr(idx_q), _ptr(k_new), _ptr(v_new), _ptr(idx_k_new), _ptr(tok_pos), _ptr(page_pos),
        _ptr(_opt_i32(q_seq, "q_seq", n)), _ptr(_opt_i32(q_pos, "q_pos", n)), _ptr(block_table), _ptr(seq_lens),
        n, B, H, mb, k_cache.shape[0], _ptr(k_cache), _ptr(v_cache), _ptr(idx_k_cache), _ptr(dev_err),
        _stream(stream)))
    return q, idx_q


def dense_workspace_bytes(n_q: int, heads: int, max_blocks: int) -> int:
    return int(_lib().uocr_dense_workspace_bytes(int(n_q), int(heads), int(max_blocks)))


@_on_its_stream
def dense_decode(q, k_cache, v_cache, block_table, seq_lens, *, ref_blocks: int | None = None,
                 out=None, workspace=None, dev_err=None, stream=None) -> torch.Tensor:
    """Decode attention over blocks [0, ref_blocks) plus the 4-block local window (all blocks when
    ref_blocks is None: full causal attention).  Returns out [B,H,128] bf16."""
    for t, n, dt, nd in ((q, "q", torch.bfloat16, 3), (k_cache, "k_cache", torch.bfloat16, 4),
                         (v_cache, "v_cache", torch.bfloat16, 4), (block_table, "block_table", torch.int32, 2),
                         (seq_lens, "seq_lens", torch.int32, 1)):
        _dev(t, n, dt, nd)
    B, H = q.shape[0], q.shape[1]
    mb = block_table.shape[1]
    rb = mb if ref_blocks is None else int(ref_blocks)
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out", torch.bfloat16, 3)
    _shape(q, "q", (B, H, HEAD_DIM))
    _check_caches(k_cache, v_cache, H)
    _shape(block_table, "block_table", (B, None))
    _shape(seq_lens, "seq_lens", (B,))
    _shape(out, "out", (B, H, HEAD_DIM))
    if workspace is None:
        workspace = torch.empty(max(dense_workspace_bytes(B, H, mb), 1), dtype=torch.uint8, device=q.device)
    _check("uocr_dense_decode", _lib().uocr_dense_decode(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens), rb, B, H, mb, k_cache.shape[0],
        _ptr(out), _ptr(workspace), workspace.numel(), _ptr(dev_err), _stream(stream)))
    return out


STATIC_SCRATCH_BYTES = 8 << 20   # UOCR_STATIC_SCRATCH_BYTES


def sparse_decode_static(q, k_cache, v_cache, idx_q, idx_k_cache, block_table, seq_lens, *,
                         out, sel, dev_err=None, stream=None):
    """Decode without a workspace, for callers that cannot allocate device memory.

    The caller passes the outputs (`out` [B,H,128] bf16, `sel` [B,16] int32); the scratch
    lives in one fixed-size device array inside libuocr.so, shared by every call on the
    device (calls that overlap on the GPU race on it), so nothing is allocated here or in
    the library.  Raises UocrError (UOCR_ERR_WORKSPACE) when the shapes need more scratch
    than STATIC_SCRATCH_BYTES.  The first call on a device looks the array up; make it
    before any stream capture.
    """
    for t, n, dt, nd in ((q, "q", torch.bfloat16, 3), (k_cache, "k_cache", torch.bfloat16, 4),
                         (v_cache, "v_cache", torch.bfloat16, 4), (idx_q, "idx_q", torch.bfloat16, 2),
                         (idx_k_cache, "idx_k_cache", torch.bfloat16, 3), (block_table, "block_table", torch.int32, 2),
                         (seq_lens, "seq_lens", torch.int32, 1), (out, "out", torch.bfloat16, 3),
                         (sel, "sel", torch.int32, 2)):
        _dev(t, n, dt, nd)
    _check_decode_args(q, k_cache, v_cache, idx_q, idx_k_cache, block_table, seq_lens, out, sel)
    B, H = q.shape[0], q.shape[1]
    _check("uocr_sparse_decode_static", _lib().uocr_sparse_decode_static(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(idx_q), _ptr(idx_k_cache), _ptr(block_table),
        _ptr(seq_lens), B, H, block_table.shape[1], k_cache.shape[0], _ptr(out), _ptr(sel),
        _ptr(dev_err), _stream(stream)))
    return out, sel


# --------------------------------------------------------------------------- the cache held in 8 bits
def dense_kv8_workspace_bytes(n_q: int, heads: int, max_blocks: int) -> int:
    return int(_lib().uocr_dense_kv8_workspace_bytes(int(n_q), int(heads), int(max_blocks)))


def sparse_attn_seq_kv8_workspace_bytes(n_q: int, heads: int, max_blocks: int) -> int:
    return int(_lib().uocr_sparse_attn_seq_kv8_workspace_bytes(int(n_q), int(heads), int(max_blocks)))


def prefill_kv8_workspace_bytes(n_q: int, heads: int, max_blocks: int) -> int:
    return int(_lib().uocr_prefill_kv8_workspace_bytes(int(n_q), int(heads), int(max_blocks)))


def evict_workspace_bytes(n_seq: int, heads: int, max_blocks: int) -> int:
    return int(_lib().uocr_evict_workspace_bytes(int(n_seq), int(heads), int(max_blocks)))


# The entry points below check their tensors on every call of a decode loop, so each asks in one
# expression, without calls, what matters of each tensor: type, shape, device and density.  Only when
# something is wrong does `_refuse` look for it and say which.  (Checks by function calls took 28 us per
# call of sparse_attn_kv8, its launch included; a function per tensor 11.3, this 9.8.)
_BF16, _F32, _I32, _E4M3, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn, torch.uint8
_WRONG = (AttributeError, TypeError, ValueError, IndexError)   # what looking at something else raises
_SCALE = HEAD_DIM ** -0.5


def _refuse(dev: int, *specs):
    """Raise for the first of (tensor, name, dtype, shape) that does not fit device `dev`; None tensors are skipped."""
    for t, name, dtype, shape in specs:
        if t is None:
            continue
        _dev(t, name, dtype, len(shape))
        _shape(t, name, shape)
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on cuda:{dev} like the other tensors, got {t.device}")


def _unfit():
    """After `_refuse` found nothing to name: what an entry point asks for and the list of it do not agree."""
    return ValueError("the tensors do not fit together (type, shape, device or density)")


def _need(t, name: str):
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    return t


def _at(t):
    return None if t is None else t.data_ptr()


def _int(x, name: str, most: int | None = None) -> int:
    """x as the library's 32-bit integer; past `most`, where that means the same, `most`.  (ctypes would cut the upper
    bits off without a word.)"""
    x = int(x)
    if most is not None and x > most:
        return most
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{name} must fit in 32 bits, got {x}")
    return x


def _launch(fn, name: str, dev: int, stream, *args):
    """fn(*args, stream) with device `dev` current, on its current stream unless one is given."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    else:
        raw = stream.cuda_stream
        if stream.device.index != dev:
            raise ValueError(f"stream must be on cuda:{dev} like the tensors, got {stream.device}")
    if torch.cuda.current_device() == dev:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, raw)
    if st != 0:
        _check("uocr_" + name, st)


def _kv8_specs(k_cache, v_cache, k_scale, v_scale, P, H):
    return ((k_cache, "k_cache", _E4M3, (P, H, BLOCK, HEAD_DIM)), (v_cache, "v_cache", _E4M3, (P, H, BLOCK, HEAD_DIM)),
            (k_scale, "k_scale", _F32, (P, H)), (v_scale, "v_scale", _F32, (P, H)))


def _empty(shape, dtype, dev: int, stream):
    """Memory on device `dev` that a call on `stream` (None: the current one) writes.  It is allocated for that stream:
    the allocator gives out memory whose last work is still queued on the stream that asks, which is safe in that
    stream's order only."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev))


def _output(given, shape, dtype, dev: int, stream):
    """The caller's output, or a new one, which the caller may use on the current stream and drop."""
    if given is not None:
        return given
    t = _empty(shape, dtype, dev, stream)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(dev))
    return t


def _space(workspace, nbytes, dev: int, stream):
    """The caller's workspace, or a new one of nbytes() bytes on device `dev`."""
    if workspace is None:
        return _empty(max(nbytes(), 1), _U8, dev, stream)
    if not (workspace.dtype is _U8 and workspace.dim() == 1 and workspace.get_device() == dev
            and workspace.is_contiguous()):
        _refuse(dev, (workspace, "workspace", _U8, (None,)))
    return workspace


def _lend(stream, *tensors):
    """For a call on a stream other than the current one: the memory of tensors that were allocated for the current one
    is not given out again before that stream is done with it."""
    if stream is not None:
        for t in tensors:
            t.record_stream(stream)


def _check_dev_err(dev_err, dev: int):
    _dev(dev_err, "dev_err", _I32)
    if dev_err.numel() < 1 or dev_err.get_device() != dev:
        raise ValueError(f"dev_err must hold one int32 on cuda:{dev}")


def rope_append_kv8(q, idx_q, k_new, v_new, idx_k_new, tok_pos, page_pos, block_table, seq_lens, k_cache, v_cache,
                    k_scale, v_scale, idx_k_cache, new_start=None, *, q_out=None, idx_q_out=None, dev_err=None,
                    stream=None):
    """Rotate q / idx_q (page2d; in place unless q_out / idx_q_out are given) and append the new tokens: rotated k
    and raw v quantised to e4m3 under one power-of-two scale per (page, head), rotated idx_k as bf16.  Sequence b's
    new tokens are rows new_start[b] .. new_start[b + 1] - 1 (None: token i belongs to sequence i) and take the
    sequence's last positions.  Returns (q_out, idx_q_out)."""
    if q_out is None:
        q_out = q
    if idx_q_out is None:
        idx_q_out = idx_q
    try:
        dev = q.get_device()
        n, H, _ = q.shape
        P = k_cache.shape[0]
        B, mb = block_table.shape
        rows, idx, toks, tile, page = (n, H, HEAD_DIM), (n, IDX_DIM), (n,), (P, H, BLOCK, HEAD_DIM), (P, H)
        good = (dev >= 0 and q.dtype is _BF16 and q.shape == rows and q.is_contiguous()
                and idx_q.dtype is _BF16 and idx_q.shape == idx and idx_q.get_device() == dev and idx_q.is_contiguous()
                and k_new.dtype is _BF16 and k_new.shape == rows and k_new.get_device() == dev and k_new.is_contiguous()
                and v_new.dtype is _BF16 and v_new.shape == rows and v_new.get_device() == dev and v_new.is_contiguous()
                and idx_k_new.dtype is _BF16 and idx_k_new.shape == idx and idx_k_new.get_device() == dev
                and idx_k_new.is_contiguous()
                and tok_pos.dtype is _I32 and tok_pos.shape == toks and tok_pos.get_device() == dev
                and tok_pos.is_contiguous()
                and page_pos.dtype is _I32 and page_pos.shape == toks and page_pos.get_device() == dev
                and page_pos.is_contiguous()
                and block_table.dtype is _I32 and block_table.get_device() == dev and block_table.is_contiguous()
                and seq_lens.dtype is _I32 and seq_lens.shape == (B,) and seq_lens.get_device() == dev
                and seq_lens.is_contiguous()
                and k_cache.dtype is _E4M3 and k_cache.shape == tile and k_cache.get_device() == dev
                and k_cache.is_contiguous()
                and v_cache.dtype is _E4M3 and v_cache.shape == tile and v_cache.get_device() == dev
                and v_cache.is_contiguous()
                and k_scale.dtype is _F32 and k_scale.shape == page and k_scale.get_device() == dev
                and k_scale.is_contiguous()
                and v_scale.dtype is _F32 and v_scale.shape == page and v_scale.get_device() == dev
                and v_scale.is_contiguous()
                and idx_k_cache.dtype is _BF16 and idx_k_cache.shape == (P, BLOCK, IDX_DIM)
                and idx_k_cache.get_device() == dev and idx_k_cache.is_contiguous()
                and (new_start is None or (new_start.dtype is _I32 and new_start.shape == (B + 1,)
                                           and new_start.get_device() == dev and new_start.is_contiguous()))
                and (q_out is q or (q_out.dtype is _BF16 and q_out.shape == rows and q_out.get_device() == dev
                                    and q_out.is_contiguous()))
                and (idx_q_out is idx_q or (idx_q_out.dtype is _BF16 and idx_q_out.shape == idx
                                            and idx_q_out.get_device() == dev and idx_q_out.is_contiguous())))
    except _WRONG:
        good = False
    if not good:
        _dev(q, "q", _BF16, 3)
        _dev(k_cache, "k_cache", _E4M3, 4)
        _dev(block_table, "block_table", _I32, 2)
        dev, (n, H, _), P, (B, mb) = q.get_device(), q.shape, k_cache.shape[0], block_table.shape
        rows, idx = (n, H, HEAD_DIM), (n, IDX_DIM)
        _refuse(dev, (q, "q", _BF16, rows), (_need(idx_q, "idx_q"), "idx_q", _BF16, idx),
                (_need(k_new, "k_new"), "k_new", _BF16, rows), (_need(v_new, "v_new"), "v_new", _BF16, rows),
                (_need(idx_k_new, "idx_k_new"), "idx_k_new", _BF16, idx),
                (_need(tok_pos, "tok_pos"), "tok_pos", _I32, (n,)), (_need(page_pos, "page_pos"), "page_pos", _I32, (n,)),
                (block_table, "block_table", _I32, (B, mb)), (_need(seq_lens, "seq_lens"), "seq_lens", _I32, (B,)),
                *_kv8_specs(k_cache, _need(v_cache, "v_cache"), _need(k_scale, "k_scale"), _need(v_scale, "v_scale"), P, H),
                (_need(idx_k_cache, "idx_k_cache"), "idx_k_cache", _BF16, (P, BLOCK, IDX_DIM)),
                (new_start, "new_start", _I32, (B + 1,)), (q_out, "q_out", _BF16, rows),
                (idx_q_out, "idx_q_out", _BF16, idx))
        raise _unfit()
    if dev_err is not None:
        _check_dev_err(dev_err, dev)
    _launch(_lib().uocr_rope_append_kv8, "rope_append_kv8", dev, stream, q.data_ptr(), idx_q.data_ptr(),
            k_new.data_ptr(), v_new.data_ptr(), idx_k_new.data_ptr(), tok_pos.data_ptr(), page_pos.data_ptr(),
            _at(new_start), block_table.data_ptr(), seq_lens.data_ptr(), n, B, H, mb, P, q_out.data_ptr(),
            idx_q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            idx_k_cache.data_ptr(), _at(dev_err))
    return q_out, idx_q_out


def _attn_args(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, per_seq, out, mass, dev_err, stream):
    """The checks that the attention entry points share; per_seq: q has a row per sequence.  Returns (device, n, H, P,
    B, max_blocks, out)."""
    if out is None and isinstance(q, torch.Tensor) and q.is_cuda:
        out = _output(None, q.shape, _BF16, q.get_device(), stream)
    try:
        dev = q.get_device()
        n, H, _ = q.shape
        P = k_cache.shape[0]
        B, mb = block_table.shape
        rows, tile, page = (n, H, HEAD_DIM), (P, H, BLOCK, HEAD_DIM), (P, H)
        good = (dev >= 0 and q.dtype is _BF16 and q.shape == rows and q.is_contiguous()
                and k_cache.dtype is _E4M3 and k_cache.shape == tile and k_cache.get_device() == dev
                and k_cache.is_contiguous()
                and v_cache.dtype is _E4M3 and v_cache.shape == tile and v_cache.get_device() == dev
                and v_cache.is_contiguous()
                and k_scale.dtype is _F32 and k_scale.shape == page and k_scale.get_device() == dev
                and k_scale.is_contiguous()
                and v_scale.dtype is _F32 and v_scale.shape == page and v_scale.get_device() == dev
                and v_scale.is_contiguous()
                and block_table.dtype is _I32 and block_table.get_device() == dev and block_table.is_contiguous()
                and seq_lens.dtype is _I32 and seq_lens.shape == (B,) and seq_lens.get_device() == dev
                and seq_lens.is_contiguous()
                and out.dtype is _BF16 and out.shape == rows and out.get_device() == dev and out.is_contiguous()
                and (not per_seq or n == B)
                and (mass is None or (mass.dtype is _F32 and mass.shape == (B, H, mb) and mass.get_device() == dev
                                      and mass.is_contiguous())))
    except _WRONG:
        good = False
    if not good:
        _dev(q, "q", _BF16, 3)
        _dev(k_cache, "k_cache", _E4M3, 4)
        _dev(block_table, "block_table", _I32, 2)
        dev, (n, H, _), P, (B, mb) = q.get_device(), q.shape, k_cache.shape[0], block_table.shape
        _refuse(dev, (q, "q", _BF16, (n, H, HEAD_DIM)), (block_table, "block_table", _I32, (n if per_seq else B, mb)),
                (_need(seq_lens, "seq_lens"), "seq_lens", _I32, (B,)),
                *_kv8_specs(k_cache, _need(v_cache, "v_cache"), _need(k_scale, "k_scale"), _need(v_scale, "v_scale"), P, H),
                (out, "out", _BF16, (n, H, HEAD_DIM)), (mass, "mass", _F32, (B, H, mb)))
        raise _unfit()
    if dev_err is not None:
        _check_dev_err(dev_err, dev)
    return dev, n, H, P, B, mb, out


def _index_args(dev, idx_q, idx_k_cache, sel, n, P, stream):
    """The indexer's tensors of a whole step, and the selection's output."""
    sel = _output(sel, (n, N_SEL), _I32, dev, stream)
    _refuse(dev, (_need(idx_q, "idx_q"), "idx_q", _BF16, (n, IDX_DIM)),
            (_need(idx_k_cache, "idx_k_cache"), "idx_k_cache", _BF16, (P, BLOCK, IDX_DIM)), (sel, "sel", _I32, (n, N_SEL)))
    return sel


def sparse_attn_kv8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, sel, q_seq=None, q_pos=None, *,
                    scale: float | None = None, out=None, mass=None, dev_err=None, stream=None) -> torch.Tensor:
    """sparse_attn over the 8-bit cache: bf16 [n_q, H, 128].  mass [B, H, max_blocks] fp32 (one query per
    sequence, q_seq None): each selected block's attention weight is added to its total."""
    dev, n_q, H, P, B, mb, out = _attn_args(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, False, out,
                                            mass, dev_err, stream)
    _need(sel, "sel")
    if not (sel.dtype is _I32 and sel.shape == (n_q, N_SEL) and sel.get_device() == dev and sel.is_contiguous()
            and q_seq is None and q_pos is None):
        _refuse(dev, (sel, "sel", _I32, (n_q, N_SEL)), (q_seq, "q_seq", _I32, (n_q,)), (q_pos, "q_pos", _I32, (n_q,)))
    if mass is not None and q_seq is not None:
        raise ValueError("mass needs one query per sequence: q_seq must be None")
    _launch(_lib().uocr_sparse_attn_kv8, "sparse_attn_kv8", dev, stream, q.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
            _at(q_seq), _at(q_pos), sel.data_ptr(), n_q, B, H, mb, P, _SCALE if scale is None else float(scale),
            out.data_ptr(), _at(mass), _at(dev_err))
    _lend(stream, out)
    return out


def sparse_decode_kv8(q, k_cache, v_cache, k_scale, v_scale, idx_q, idx_k_cache, block_table, seq_lens, *, out=None,
                      sel=None, mass=None, workspace=None, dev_err=None, stream=None):
    """sparse_decode over the 8-bit cache.  Returns (out [B,H,128] bf16, sel [B,16] int32)."""
    dev, B, H, P, _, mb, out = _attn_args(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, True, out,
                                          mass, dev_err, stream)
    sel = _index_args(dev, idx_q, idx_k_cache, sel, B, P, stream)
    workspace = _space(workspace, lambda: workspace_bytes(B, H, mb), dev, stream)
    _launch(_lib().uocr_sparse_decode_kv8, "sparse_decode_kv8", dev, stream, q.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), idx_q.data_ptr(), idx_k_cache.data_ptr(),
            block_table.data_ptr(), seq_lens.data_ptr(), B, H, mb, P, out.data_ptr(), sel.data_ptr(), _at(mass),
            workspace.data_ptr(), workspace.numel(), _at(dev_err))
    _lend(stream, out, sel, workspace)
    return out, sel


def dense_decode_kv8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, *, ref_blocks: int | None = None,
                     out=None, mass=None, workspace=None, dev_err=None, stream=None) -> torch.Tensor:
    """dense_decode over the 8-bit cache: blocks [0, ref_blocks) plus the 4-block local window, or all of them
    when ref_blocks is None.  Returns out [B,H,128] bf16; mass [B, H, max_blocks] receives every attended block's
    weight."""
    dev, B, H, P, _, mb, out = _attn_args(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, True, out,
                                          mass, dev_err, stream)
    workspace = _space(workspace, lambda: dense_kv8_workspace_bytes(B, H, mb), dev, stream)
    _launch(_lib().uocr_dense_decode_kv8, "dense_decode_kv8", dev, stream, q.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
            mb if ref_blocks is None else _int(ref_blocks, "ref_blocks", mb), B, H, mb, P, out.data_ptr(), _at(mass),
            workspace.data_ptr(), workspace.numel(), _at(dev_err))
    _lend(stream, out, workspace)
    return out


def sparse_attn_seq_kv8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, seq: int, q_pos, sel, *,
                        scale: float | None = None, out=None, mass=None, workspace=None, dev_err=None,
                        stream=None) -> torch.Tensor:
    """sparse_attn_seq over the 8-bit cache: many queries of sequence `seq` over the given selection.  Returns out
    [n_q,H,128] bf16; row `seq` of mass [B, H, max_blocks] receives the queries' weights."""
    dev, n_q, H, P, B, mb, out = _attn_args(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, False, out,
                                            mass, dev_err, stream)
    _refuse(dev, (_need(q_pos, "q_pos"), "q_pos", _I32, (n_q,)), (_need(sel, "sel"), "sel", _I32, (n_q, N_SEL)))
    workspace = _space(workspace, lambda: sparse_attn_seq_kv8_workspace_bytes(n_q, H, mb), dev, stream)
    _launch(_lib().uocr_sparse_attn_seq_kv8, "sparse_attn_seq_kv8", dev, stream, q.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
            _int(seq, "seq"), q_pos.data_ptr(), sel.data_ptr(), n_q, B, H, mb, P, _SCALE if scale is None else float(scale),
            out.data_ptr(), _at(mass), workspace.data_ptr(), workspace.numel(), _at(dev_err))
    _lend(stream, out, workspace)
    return out


def sparse_prefill_kv8(q, k_cache, v_cache, k_scale, v_scale, idx_q, idx_k_cache, block_table, seq_lens, seq: int,
                       q_pos, *, out=None, sel=None, mass=None, workspace=None, dev_err=None, stream=None):
    """sparse_prefill over the 8-bit cache.  Returns (out [n_q,H,128] bf16, sel [n_q,16] int32)."""
    dev, n_q, H, P, B, mb, out = _attn_args(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, False, out,
                                            mass, dev_err, stream)
    sel = _index_args(dev, idx_q, idx_k_cache, sel, n_q, P, stream)
    _refuse(dev, (_need(q_pos, "q_pos"), "q_pos", _I32, (n_q,)))
    workspace = _space(workspace, lambda: prefill_kv8_workspace_bytes(n_q, H, mb), dev, stream)
    _launch(_lib().uocr_sparse_prefill_kv8, "sparse_prefill_kv8", dev, stream, q.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), idx_q.data_ptr(), idx_k_cache.data_ptr(),
            block_table.data_ptr(), seq_lens.data_ptr(), _int(seq, "seq"), q_pos.data_ptr(), n_q, B, H, mb, P,
            out.data_ptr(), sel.data_ptr(), _at(mass), workspace.data_ptr(), workspace.numel(), _at(dev_err))
    _lend(stream, out, sel, workspace)
    return out, sel


def evict_blocks(mass, block_table, seq_lens, keep_blocks: int, *, n_sink: int = 0, new_mass=None, new_table=None,
                 new_lens=None, freed=None, n_freed=None, workspace=None, dev_err=None, stream=None):
    """Cut every sequence of more than keep_blocks blocks to keep_blocks: its first n_sink blocks, its 4 local ones
    and those of the others with the highest totals over the heads (lower id on ties) stay.  Returns (new_mass
    [B,H,max_blocks] fp32, new_table [B,max_blocks] int32, new_lens [B] int32, freed [B,max_blocks] int32 pages,
    n_freed [B] int32); the first three may be the inputs themselves."""
    try:
        dev = mass.get_device()
        B, H, mb = totals = mass.shape
        table, lens = (B, mb), (B,)
        if dev >= 0:
            new_mass = _output(new_mass, totals, _F32, dev, stream)
            new_table = _output(new_table, table, _I32, dev, stream)
            new_lens = _output(new_lens, lens, _I32, dev, stream)
            freed = _output(freed, table, _I32, dev, stream)
            n_freed = _output(n_freed, lens, _I32, dev, stream)
        good = (dev >= 0 and mass.dtype is _F32 and mass.is_contiguous()
                and block_table.dtype is _I32 and block_table.shape == table and block_table.get_device() == dev
                and block_table.is_contiguous()
                and seq_lens.dtype is _I32 and seq_lens.shape == lens and seq_lens.get_device() == dev
                and seq_lens.is_contiguous()
                and new_mass.dtype is _F32 and new_mass.shape == totals and new_mass.get_device() == dev
                and new_mass.is_contiguous()
                and new_table.dtype is _I32 and new_table.shape == table and new_table.get_device() == dev
                and new_table.is_contiguous()
                and new_lens.dtype is _I32 and new_lens.shape == lens and new_lens.get_device() == dev
                and new_lens.is_contiguous()
                and freed.dtype is _I32 and freed.shape == table and freed.get_device() == dev and freed.is_contiguous()
                and n_freed.dtype is _I32 and n_freed.shape == lens and n_freed.get_device() == dev
                and n_freed.is_contiguous())
    except _WRONG:
        good = False
    if not good:
        _dev(mass, "mass", _F32, 3)
        dev, (B, H, mb) = mass.get_device(), mass.shape
        _refuse(dev, (_need(block_table, "block_table"), "block_table", _I32, (B, mb)),
                (_need(seq_lens, "seq_lens"), "seq_lens", _I32, (B,)), (new_mass, "new_mass", _F32, (B, H, mb)),
                (new_table, "new_table", _I32, (B, mb)), (new_lens, "new_lens", _I32, (B,)),
                (freed, "freed", _I32, (B, mb)), (n_freed, "n_freed", _I32, (B,)))
        raise _unfit()
    if dev_err is not None:
        _check_dev_err(dev_err, dev)
    workspace = _space(workspace, lambda: evict_workspace_bytes(B, H, mb), dev, stream)
    _launch(_lib().uocr_evict_blocks, "evict_blocks", dev, stream, mass.data_ptr(), block_table.data_ptr(),
            seq_lens.data_ptr(), B, H, mb, _int(keep_blocks, "keep_blocks", (1 << 31) - 1), _int(n_sink, "n_sink"),
            new_mass.data_ptr(), new_table.data_ptr(), new_lens.data_ptr(), freed.data_ptr(), n_freed.data_ptr(),
            workspace.data_ptr(), workspace.numel(), _at(dev_err))
    _lend(stream, new_mass, new_table, new_lens, freed, n_freed, workspace)
    return new_mass, new_table, new_lens, freed, n_freed
