"""GB300 (sm_103a) low-rank KV-block predictor: Python binding of libhss.so.

The predictor ("high-speed swap" block predictor; page "metrale_storage/predictor.rs")
projects query rows and key tokens through a fixed P [head_dim, r], keeps the projected
keys of every paged KV block in A_g [num_layers, max_blocks, num_kv_heads, block_size, r]
(bf16), scores each block as the max over query heads, query rows and tokens of Qp . A_g,
and ranks eviction victims by ascending score.

Every step runs in the CUDA kernels of libhss.so (include/hss.h).  This module only
marshals arguments: torch tensors become device pointers, the current torch stream becomes
the cudaStream_t, and a non-zero status becomes an HssError.  There is no CPU fallback: if
the library is missing, importing a compute function raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libhss.so")

HSS_OK = 0
HSS_ERR_INVALID_DIMS = 1
HSS_ERR_OUT_OF_RANGE = 2
HSS_ERR_NULL_POINTER = 3
HSS_ERR_MISALIGNED = 4
HSS_ERR_WORKSPACE_TOO_SMALL = 5
HSS_ERR_UNSUPPORTED_SHAPE = 6
HSS_ERR_CUDA = 7
HSS_ERR_DEVICE_TIMEOUT = 8
HSS_ERR_INVALID_ARGUMENT = 9

HSS_PATH_AUTO = 0
HSS_PATH_DECODE = 1
HSS_PATH_TCGEN05 = 2
HSS_MAX_VICTIMS = 8192

HSS_ROPE_HALF = 0
HSS_ROPE_INTERLEAVED = 1
HSS_ROPE_SCALE_NONE = 0
HSS_ROPE_SCALE_LINEAR = 1
HSS_ROPE_SCALE_BASE = 2
HSS_ROPE_SCALE_RAMP = 3

EXPORTED = (
    "hss_status_string", "hss_version", "hss_validate_dims", "hss_a_g_bytes", "hss_project_q",
    "hss_project_kv_blocks", "hss_score_blocks", "hss_rank_victims", "hss_read_device_error",
    "hss_layer_step", "hss_layer_step_workspace_bytes", "hss_layer_step_static",
    "hss_score_blocks_masked",
    "hss_layer_step_static_max_seqs", "hss_write_kv_tokens", "hss_score_rows",
    "hss_select_rows", "hss_self_test_wait_timeout", "hss_self_test_spread_wait",
    "hss_layer_step_bound", "hss_rope_table", "hss_rope_tokens", "hss_attend_tree",
    "hss_attend_tree_workspace_bytes", "hss_evict_blocks",
    "hss_norm_rope_tokens", "hss_packed_page_bytes", "hss_pack_kv_tokens",
    "hss_unpack_kv_tokens", "hss_attend_packed_workspace_bytes", "hss_attend_packed",
    "hss_fork_pages_workspace_bytes", "hss_compact_pages_workspace_bytes", "hss_fork_pages",
    "hss_compact_pages", "hss_copy_pages",
)


class hss_dims(ctypes.Structure):
    """The seven predictor dimensions (PredictorDims on the predictor page)."""

    _fields_ = [
        ("num_layers", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("r", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("max_blocks", ctypes.c_int64),
    ]

    @classmethod
    def of(cls, d) -> "hss_dims":
        """From any object with the seven attributes (or an hss_dims)."""
        if isinstance(d, cls):
            return d
        return cls(int(d.num_layers), int(d.num_q_heads), int(d.num_kv_heads), int(d.head_dim),
                   int(d.r), int(d.block_size), int(d.max_blocks))


class HssError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib: Optional[ctypes.CDLL] = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libhss.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build the CUDA library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    dp = ctypes.POINTER(hss_dims)
    lib.hss_status_string.restype = ctypes.c_char_p
    lib.hss_status_string.argtypes = [i32]
    lib.hss_version.restype = i32
    lib.hss_version.argtypes = []
    lib.hss_validate_dims.restype = i32
    lib.hss_validate_dims.argtypes = [dp]
    lib.hss_a_g_bytes.restype = sz
    lib.hss_a_g_bytes.argtypes = [dp]
    lib.hss_project_q.restype = i32
    lib.hss_project_q.argtypes = [dp, vp, vp, i64, vp, vp]
    lib.hss_project_kv_blocks.restype = i32
    lib.hss_project_kv_blocks.argtypes = [dp, vp, vp, i32, vp, i64, vp, vp, vp]
    lib.hss_write_kv_tokens.restype = i32
    lib.hss_write_kv_tokens.argtypes = [dp, vp, vp, vp, i64, vp, vp, i32, vp, vp]
    lib.hss_score_rows.restype = i32
    lib.hss_score_rows.argtypes = [dp, vp, i32, vp, i32, vp, i64, vp, vp, vp]
    lib.hss_select_rows.restype = i32
    lib.hss_select_rows.argtypes = [vp, i32, i64, i64, i32, i32, vp, vp]
    lib.hss_score_blocks.restype = i32
    lib.hss_score_blocks.argtypes = [dp, vp, i32, vp, i32, vp, vp, i32, i64, vp, i32, vp, vp]
    lib.hss_score_blocks_masked.restype = i32
    lib.hss_score_blocks_masked.argtypes = [dp, vp, i32, vp, i32, vp, vp, i32, i64, vp, vp, vp,
                                            i32, vp, vp]
    lib.hss_self_test_wait_timeout.restype = i32
    lib.hss_self_test_wait_timeout.argtypes = [vp, i64, vp]
    lib.hss_self_test_spread_wait.restype = i32
    lib.hss_self_test_spread_wait.argtypes = [dp, vp, vp, vp, i32, vp, vp, i64, vp, i32, vp, vp,
                                              sz, i64, vp, vp]
    lib.hss_rank_victims.restype = i32
    lib.hss_rank_victims.argtypes = [vp, vp, i32, i64, i32, vp, vp]
    lib.hss_read_device_error.restype = i32
    lib.hss_read_device_error.argtypes = [ctypes.POINTER(i32), vp]
    lib.hss_layer_step_workspace_bytes.restype = sz
    lib.hss_layer_step_workspace_bytes.argtypes = [i32]
    lib.hss_layer_step_static_max_seqs.restype = i32
    lib.hss_layer_step_static_max_seqs.argtypes = []
    lib.hss_layer_step_static.restype = i32
    lib.hss_layer_step_static.argtypes = [dp, vp, vp, vp, i64, vp, i32, vp, vp, i32, vp, vp, i32,
                                          i64, vp, i32, vp, vp, vp]
    lib.hss_layer_step.restype = i32
    lib.hss_layer_step.argtypes = [dp, vp, vp, vp, i64, vp, i32, vp, vp, i32, vp, vp, i32, i64,
                                   vp, i32, vp, vp, sz, vp, vp]
    lib.hss_layer_step_bound.restype = i32
    lib.hss_layer_step_bound.argtypes = [ctypes.POINTER(hss_layer_step_args), i32, vp, vp, vp,
                                         vp, vp]
    lib.hss_rope_table.restype = i32
    lib.hss_rope_table.argtypes = [ctypes.POINTER(hss_rope), vp]
    lib.hss_rope_tokens.restype = i32
    lib.hss_rope_tokens.argtypes = [ctypes.POINTER(hss_rope_args)] + [vp] * 8
    lib.hss_attend_tree_workspace_bytes.restype = sz
    lib.hss_attend_tree_workspace_bytes.argtypes = [dp, i32, i32, i64, i32]
    lib.hss_attend_tree.restype = i32
    lib.hss_attend_tree.argtypes = [ctypes.POINTER(hss_attend_args)] + [vp] * 8
    lib.hss_evict_blocks.restype = i32
    lib.hss_evict_blocks.argtypes = [vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, vp, vp, vp, vp,
                                     vp, vp, vp]
    lib.hss_norm_rope_tokens.restype = i32
    lib.hss_norm_rope_tokens.argtypes = [ctypes.POINTER(hss_norm_rope_args)] + [vp] * 10
    lib.hss_packed_page_bytes.restype = sz
    lib.hss_packed_page_bytes.argtypes = [dp]
    lib.hss_pack_kv_tokens.restype = i32
    lib.hss_pack_kv_tokens.argtypes = [ctypes.POINTER(hss_pack_args)] + [vp] * 4
    lib.hss_unpack_kv_tokens.restype = i32
    lib.hss_unpack_kv_tokens.argtypes = [ctypes.POINTER(hss_pack_args)] + [vp] * 4
    lib.hss_attend_packed_workspace_bytes.restype = sz
    lib.hss_attend_packed_workspace_bytes.argtypes = [dp, i32, i32, i64, i32, i32]
    lib.hss_attend_packed.restype = i32
    lib.hss_attend_packed.argtypes = [ctypes.POINTER(hss_packed_args)] + [vp] * 5
    lib.hss_fork_pages_workspace_bytes.restype = sz
    lib.hss_fork_pages_workspace_bytes.argtypes = [i32, i64]
    lib.hss_compact_pages_workspace_bytes.restype = sz
    lib.hss_compact_pages_workspace_bytes.argtypes = [i64]
    lib.hss_fork_pages.restype = i32
    lib.hss_fork_pages.argtypes = [vp, vp, i32, i64, vp, i64, vp, i64, vp, vp, vp, i32, i32, i64,
                                   vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.hss_compact_pages.restype = i32
    lib.hss_compact_pages.argtypes = [vp, i64, vp, i64, i64, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.hss_copy_pages.restype = i32
    lib.hss_copy_pages.argtypes = [vp, vp, vp, i64, vp, vp, i64, i64, i32, vp, vp]
    _lib = lib
    return lib


# ----------------------------------------------------------------------------- marshalling

def _ptr(x) -> Optional[int]:
    """Device pointer of a tensor (or an int address, or None for NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch

        # The raw handle of the current stream: the same value as
        # torch.cuda.current_stream().cuda_stream without building a Stream object.
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, what: str) -> None:
    if status != HSS_OK:
        raise HssError(status, what)


def status_string(status: int) -> str:
    return load().hss_status_string(status).decode()


def hss_version() -> int:
    return load().hss_version()


def hss_validate_dims(dims) -> int:
    """Status of the dims (HSS_OK when valid and supported); never raises."""
    return load().hss_validate_dims(ctypes.byref(hss_dims.of(dims)))


def hss_a_g_bytes(dims) -> int:
    return load().hss_a_g_bytes(ctypes.byref(hss_dims.of(dims)))


def hss_project_q(dims, P, Q, num_rows: int, Qp, stream=None) -> None:
    """Qp [num_rows, num_q_heads, r] = bf16(Q [num_rows, num_q_heads, head_dim] . P)."""
    st = load().hss_project_q(ctypes.byref(hss_dims.of(dims)), _ptr(P), _ptr(Q), int(num_rows),
                              _ptr(Qp), _stream(stream))
    _check(st, "hss_project_q")


def hss_project_kv_blocks(dims, P, K, layer: int, block_ids, num_blocks: int, A_g,
                          dev_status=None, stream=None) -> None:
    """A_g[layer][block_ids[i]] = bf16(K[i] . P), head-major slots."""
    st = load().hss_project_kv_blocks(ctypes.byref(hss_dims.of(dims)), _ptr(P), _ptr(K),
                                      int(layer), _ptr(block_ids), int(num_blocks), _ptr(A_g),
                                      _ptr(dev_status), _stream(stream))
    _check(st, "hss_project_kv_blocks")


def hss_write_kv_tokens(dims, P, K_tok, slots, num_tokens: int, K_cache, A_g, layer: int,
                        dev_status=None, stream=None) -> None:
    """K_cache[slot] = K_tok[i] and A_g[layer][slot's block][h][slot's position] =
    bf16(K_tok[i][h] . P) for every new token i (K_cache may be None)."""
    st = load().hss_write_kv_tokens(ctypes.byref(hss_dims.of(dims)), _ptr(P), _ptr(K_tok),
                                    _ptr(slots), int(num_tokens), _ptr(K_cache), _ptr(A_g),
                                    int(layer), _ptr(dev_status), _stream(stream))
    _check(st, "hss_write_kv_tokens")


def hss_score_rows(dims, Qp, rows: int, A_g, layer: int, block_table, num_blocks: int, scores,
                   dev_status=None, stream=None) -> None:
    """scores[row, j] = max over heads and tokens of block_table[j] of Qp[row] . A_g."""
    st = load().hss_score_rows(ctypes.byref(hss_dims.of(dims)), _ptr(Qp), int(rows), _ptr(A_g),
                               int(layer), _ptr(block_table), int(num_blocks), _ptr(scores),
                               _ptr(dev_status), _stream(stream))
    _check(st, "hss_score_rows")


def hss_select_rows(scores, rows: int, num_blocks: int, first_pos: int, block_size: int,
                    topk: int, lists, stream=None) -> None:
    """lists[r] = the topk blocks row r has seen whole, largest score first."""
    st = load().hss_select_rows(_ptr(scores), int(rows), int(num_blocks), int(first_pos),
                                int(block_size), int(topk), _ptr(lists), _stream(stream))
    _check(st, "hss_select_rows")


def hss_score_blocks(dims, Qp, rows_per_seq: int, A_g, layer: int, block_table, seq_offsets,
                     num_seqs: int, total_blocks: int, scores, path: int = HSS_PATH_AUTO,
                     dev_status=None, stream=None) -> None:
    """scores[i] = max over rows, heads and tokens of Qp . A_g[layer][block_table[i]]."""
    st = load().hss_score_blocks(ctypes.byref(hss_dims.of(dims)), _ptr(Qp), int(rows_per_seq),
                                 _ptr(A_g), int(layer), _ptr(block_table), _ptr(seq_offsets),
                                 int(num_seqs), int(total_blocks), _ptr(scores), int(path),
                                 _ptr(dev_status), _stream(stream))
    _check(st, "hss_score_blocks")


def hss_score_blocks_masked(dims, Qp, rows_per_seq: int, A_g, layer: int, block_table,
                            seq_offsets, num_seqs: int, total_blocks: int, ctx_len, row_pos0,
                            scores, path: int = HSS_PATH_AUTO, dev_status=None,
                            stream=None) -> None:
    """hss_score_blocks over visible tokens only (length mask ctx_len, causal row_pos0)."""
    st = load().hss_score_blocks_masked(ctypes.byref(hss_dims.of(dims)), _ptr(Qp),
                                        int(rows_per_seq), _ptr(A_g), int(layer),
                                        _ptr(block_table), _ptr(seq_offsets), int(num_seqs),
                                        int(total_blocks), _ptr(ctx_len), _ptr(row_pos0),
                                        _ptr(scores), int(path), _ptr(dev_status),
                                        _stream(stream))
    _check(st, "hss_score_blocks_masked")


def hss_rank_victims(scores, seq_offsets, num_seqs: int, total_blocks: int, k: int, victims,
                     stream=None) -> None:
    """victims[s, :] = the min(k, n_s) smallest (score, index) entries of sequence s; -1 pad."""
    st = load().hss_rank_victims(_ptr(scores), _ptr(seq_offsets), int(num_seqs),
                                 int(total_blocks), int(k), _ptr(victims), _stream(stream))
    _check(st, "hss_rank_victims")


def hss_layer_step_workspace_bytes(num_seqs: int) -> int:
    return load().hss_layer_step_workspace_bytes(int(num_seqs))


def hss_layer_step(dims, P, K_new, new_ids, num_new: int, Q, rows_per_seq: int, Qp, A_g,
                   layer: int, block_table, seq_offsets, num_seqs: int, total_blocks: int,
                   scores, k: int, victims, workspace, workspace_bytes: int, dev_status=None,
                   stream=None) -> None:
    """One layer call: project new blocks and queries, score, rank (fused where possible)."""
    st = load().hss_layer_step(ctypes.byref(hss_dims.of(dims)), _ptr(P), _ptr(K_new),
                               _ptr(new_ids), int(num_new), _ptr(Q), int(rows_per_seq), _ptr(Qp),
                               _ptr(A_g), int(layer), _ptr(block_table), _ptr(seq_offsets),
                               int(num_seqs), int(total_blocks), _ptr(scores), int(k),
                               _ptr(victims), _ptr(workspace), int(workspace_bytes),
                               _ptr(dev_status), _stream(stream))
    _check(st, "hss_layer_step")


class hss_layer_step_args(ctypes.Structure):
    """The bound arguments of hss_layer_step_bound (hss_layer_step_args in hss.h)."""

    _fields_ = [
        ("dims", hss_dims),
        ("P", ctypes.c_void_p),
        ("new_ids", ctypes.c_void_p),
        ("num_new", ctypes.c_int64),
        ("rows_per_seq", ctypes.c_int32),
        ("Qp", ctypes.c_void_p),
        ("A_g", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("seq_offsets", ctypes.c_void_p),
        ("num_seqs", ctypes.c_int32),
        ("total_blocks", ctypes.c_int64),
        ("k", ctypes.c_int32),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("dev_status", ctypes.c_void_p),
    ]


class LayerStep:
    """hss_layer_step with the arguments that stay the same from call to call bound once.

    A serving loop makes one layer call per layer and step with the same dims, P, A_g,
    block table, offsets, workspace and sizes; they are bound once in an
    hss_layer_step_args struct and each call passes only the per-call ones (layer, the new
    key blocks, the queries, the score and victim buffers, the stream) to
    hss_layer_step_bound, which is exactly hss_layer_step.  Tensors or integer device
    addresses are accepted for those.
    """

    def __init__(self, dims, P, new_ids, num_new: int, rows_per_seq: int, Qp, A_g,
                 block_table, seq_offsets, num_seqs: int, total_blocks: int, k: int,
                 workspace, workspace_bytes: int, dev_status=None):
        self._fn = load().hss_layer_step_bound
        self._args = hss_layer_step_args(
            hss_dims.of(dims), _ptr(P), _ptr(new_ids), int(num_new), int(rows_per_seq),
            _ptr(Qp), _ptr(A_g), _ptr(block_table), _ptr(seq_offsets), int(num_seqs),
            int(total_blocks), int(k), _ptr(workspace), int(workspace_bytes), _ptr(dev_status))
        self._ref = ctypes.byref(self._args)  # kept alive with the struct

    def __call__(self, layer: int, K_new, Q, scores, victims, stream=None) -> None:
        st = self._fn(self._ref, int(layer), _ptr(K_new), _ptr(Q), _ptr(scores), _ptr(victims),
                      _stream(stream))
        _check(st, "hss_layer_step_bound")


class hss_rope(ctypes.Structure):
    """Rotary frequencies and their scaling for longer contexts (hss_rope in hss.h)."""

    _fields_ = [
        ("rot_dim", ctypes.c_int32),
        ("scaling", ctypes.c_int32),
        ("base", ctypes.c_double),
        ("factor", ctypes.c_double),
        ("original_ctx", ctypes.c_double),
        ("low", ctypes.c_double),
        ("high", ctypes.c_double),
    ]


def hss_rope_table(rope: hss_rope, turns) -> None:
    """turns[i] (host array of rot_dim / 2 64-bit words) = pair i's turns per position in 2^-64."""
    _check(load().hss_rope_table(ctypes.byref(rope), _ptr(turns)), "hss_rope_table")


class hss_rope_args(ctypes.Structure):
    """What the layers of one step share in hss_rope_tokens (hss_rope_args in hss.h)."""

    _fields_ = [
        ("dims", hss_dims),
        ("rot_dim", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("turns", ctypes.c_void_p),
        ("magnitude", ctypes.c_float),
        ("positions", ctypes.c_void_p),
        ("slots", ctypes.c_void_p),
        ("num_tokens", ctypes.c_int64),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("dev_status", ctypes.c_void_p),
    ]


class RopeTokens:
    """hss_rope_tokens with what the layers of one step share bound once.

    Each call rotates one layer's queries and keys and writes its keys and values into the
    paged caches; what a call does not want is None.  The tensors bound here are kept alive.
    """

    def __init__(self, dims, rot_dim: int, layout: int, turns, magnitude: float, positions, slots,
                 num_tokens: int, q_stride: int, k_stride: int, v_stride: int, dev_status=None):
        self._fn = load().hss_rope_tokens
        self._keep = (turns, positions, slots, dev_status)
        self._args = hss_rope_args(
            hss_dims.of(dims), int(rot_dim), int(layout), _ptr(turns), float(magnitude),
            _ptr(positions), _ptr(slots), int(num_tokens), int(q_stride), int(k_stride),
            int(v_stride), _ptr(dev_status))
        self._ref = ctypes.byref(self._args)

    def __call__(self, Q, K, V, Q_out, K_out, K_cache, V_cache, stream=None) -> None:
        st = self._fn(self._ref, _ptr(Q), _ptr(K), _ptr(V), _ptr(Q_out), _ptr(K_out),
                      _ptr(K_cache), _ptr(V_cache), _stream(stream))
        _check(st, "hss_rope_tokens")


class hss_attend_args(ctypes.Structure):
    """What the layers of one step share in hss_attend_tree (hss_attend_args in hss.h)."""

    _fields_ = [
        ("dims", hss_dims),
        ("q_offsets", ctypes.c_void_p),
        ("total_q", ctypes.c_int64),
        ("max_q", ctypes.c_int32),
        ("mask_words", ctypes.c_int32),
        ("tree_mask", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("seq_offsets", ctypes.c_void_p),
        ("ctx_len", ctypes.c_void_p),
        ("total_blocks", ctypes.c_int64),
        ("num_seqs", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("decay", ctypes.c_float),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("dev_status", ctypes.c_void_p),
    ]


def hss_attend_tree_workspace_bytes(dims, num_seqs: int, max_q: int, total_blocks: int,
                                    with_weights: bool) -> int:
    return load().hss_attend_tree_workspace_bytes(ctypes.byref(hss_dims.of(dims)), int(num_seqs),
                                                  int(max_q), int(total_blocks),
                                                  int(bool(with_weights)))


class AttendTree:
    """hss_attend_tree with what the layers of one step share bound once.

    Each call attends one layer's rows over its caches: out, and where asked for the rows'
    lse and the blocks' accumulated weights.  The tensors bound here are kept alive.
    """

    def __init__(self, dims, q_offsets, total_q: int, max_q: int, tree_mask, mask_words: int,
                 block_table, seq_offsets, ctx_len, num_seqs: int, total_blocks: int,
                 scale: float, decay: float, workspace, workspace_bytes: int, dev_status=None):
        self._fn = load().hss_attend_tree
        self._keep = (q_offsets, tree_mask, block_table, seq_offsets, ctx_len, workspace,
                      dev_status)
        self._args = hss_attend_args(
            hss_dims.of(dims), _ptr(q_offsets), int(total_q), int(max_q), int(mask_words),
            _ptr(tree_mask), _ptr(block_table), _ptr(seq_offsets), _ptr(ctx_len),
            int(total_blocks), int(num_seqs), float(scale), float(decay), _ptr(workspace),
            int(workspace_bytes), _ptr(dev_status))
        self._ref = ctypes.byref(self._args)

    def __call__(self, Q, K_cache, V_cache, out, lse=None, weights_in=None, weights_out=None,
                 stream=None) -> None:
        st = self._fn(self._ref, _ptr(Q), _ptr(K_cache), _ptr(V_cache), _ptr(out), _ptr(lse),
                      _ptr(weights_in), _ptr(weights_out), _stream(stream))
        _check(st, "hss_attend_tree")


def hss_evict_blocks(weights, block_table, seq_offsets, ctx_len, budgets, num_seqs: int,
                     total_blocks: int, block_size: int, keep_first: int, keep_last: int,
                     new_table, new_offsets, new_weights, new_ctx_len, freed, freed_offsets,
                     stream=None) -> None:
    """Cut every sequence's table to its budget, the blocks with the least weight going first."""
    st = load().hss_evict_blocks(_ptr(weights), _ptr(block_table), _ptr(seq_offsets),
                                 _ptr(ctx_len), _ptr(budgets), int(num_seqs), int(total_blocks),
                                 int(block_size), int(keep_first), int(keep_last),
                                 _ptr(new_table), _ptr(new_offsets), _ptr(new_weights),
                                 _ptr(new_ctx_len), _ptr(freed), _ptr(freed_offsets),
                                 _stream(stream))
    _check(st, "hss_evict_blocks")


class hss_norm_rope_args(ctypes.Structure):
    """What the layers of one step share in hss_norm_rope_tokens (hss_norm_rope_args in hss.h)."""

    _fields_ = [
        ("rope", hss_rope_args),
        ("q_weight_stride", ctypes.c_int64),
        ("k_weight_stride", ctypes.c_int64),
        ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float),
    ]


class NormRopeTokens:
    """hss_norm_rope_tokens with what the layers of one step share bound once.

    Each call norms and rotates one layer's queries and keys, with that layer's weights, and
    writes its keys and values into the paged caches; what a call does not want is None.  The
    tensors bound here are kept alive.
    """

    def __init__(self, dims, rot_dim: int, layout: int, turns, magnitude: float, positions, slots,
                 num_tokens: int, q_stride: int, k_stride: int, v_stride: int,
                 q_weight_stride: int, k_weight_stride: int, eps: float,
                 weight_offset: float = 0.0, dev_status=None):
        self._fn = load().hss_norm_rope_tokens
        self._keep = (turns, positions, slots, dev_status)
        self._args = hss_norm_rope_args(
            hss_rope_args(hss_dims.of(dims), int(rot_dim), int(layout), _ptr(turns),
                          float(magnitude), _ptr(positions), _ptr(slots), int(num_tokens),
                          int(q_stride), int(k_stride), int(v_stride), _ptr(dev_status)),
            int(q_weight_stride), int(k_weight_stride), float(eps), float(weight_offset))
        self._ref = ctypes.byref(self._args)

    def __call__(self, Q, K, V, q_weight, k_weight, Q_out, K_out, K_cache, V_cache,
                 stream=None) -> None:
        st = self._fn(self._ref, _ptr(Q), _ptr(K), _ptr(V), _ptr(q_weight), _ptr(k_weight),
                      _ptr(Q_out), _ptr(K_out), _ptr(K_cache), _ptr(V_cache), _stream(stream))
        _check(st, "hss_norm_rope_tokens")


def hss_packed_page_bytes(dims) -> int:
    """Bytes of one page of the packed cache (0 if the dims are invalid)."""
    return load().hss_packed_page_bytes(ctypes.byref(hss_dims.of(dims)))


class hss_pack_args(ctypes.Structure):
    """What the layers of one step share in packing and unpacking (hss_pack_args in hss.h)."""

    _fields_ = [
        ("dims", hss_dims),
        ("slots", ctypes.c_void_p),
        ("num_tokens", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("dev_status", ctypes.c_void_p),
    ]


class PackTokens:
    """hss_pack_kv_tokens and hss_unpack_kv_tokens with the step's slots and strides bound once.

    pack writes one layer's keys and values of the tokens into its packed cache, unpack reads
    them back; K or V may be None.  The tensors bound here are kept alive.
    """

    def __init__(self, dims, slots, num_tokens: int, k_stride: int, v_stride: int,
                 dev_status=None):
        lib = load()
        self._pack, self._unpack = lib.hss_pack_kv_tokens, lib.hss_unpack_kv_tokens
        self._keep = (slots, dev_status)
        self._args = hss_pack_args(hss_dims.of(dims), _ptr(slots), int(num_tokens), int(k_stride),
                                   int(v_stride), _ptr(dev_status))
        self._ref = ctypes.byref(self._args)

    def pack(self, K, V, cache, stream=None) -> None:
        st = self._pack(self._ref, _ptr(K), _ptr(V), _ptr(cache), _stream(stream))
        _check(st, "hss_pack_kv_tokens")

    def unpack(self, cache, K, V, stream=None) -> None:
        st = self._unpack(self._ref, _ptr(cache), _ptr(K), _ptr(V), _stream(stream))
        _check(st, "hss_unpack_kv_tokens")


class hss_packed_args(ctypes.Structure):
    """What the layers of one step share in hss_attend_packed (hss_packed_args in hss.h)."""

    _fields_ = [
        ("dims", hss_dims),
        ("q_offsets", ctypes.c_void_p),
        ("total_q", ctypes.c_int64),
        ("max_q", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("sinks", ctypes.c_int32),
        ("block_table", ctypes.c_void_p),
        ("seq_offsets", ctypes.c_void_p),
        ("ctx_len", ctypes.c_void_p),
        ("total_blocks", ctypes.c_int64),
        ("num_seqs", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("dev_status", ctypes.c_void_p),
    ]


def hss_attend_packed_workspace_bytes(dims, num_seqs: int, max_q: int, total_blocks: int,
                                      window: int = 0, sinks: int = 0) -> int:
    return load().hss_attend_packed_workspace_bytes(
        ctypes.byref(hss_dims.of(dims)), int(num_seqs), int(max_q), int(total_blocks),
        int(window), int(sinks))


class AttendPacked:
    """hss_attend_packed with what the layers of one step share bound once.

    Each call attends one layer's rows over its packed cache: out, and where asked for the rows'
    lse.  The tensors bound here are kept alive.
    """

    def __init__(self, dims, q_offsets, total_q: int, max_q: int, block_table, seq_offsets,
                 ctx_len, num_seqs: int, total_blocks: int, window: int, sinks: int,
                 scale: float, workspace, workspace_bytes: int, dev_status=None):
        self._fn = load().hss_attend_packed
        self._keep = (q_offsets, block_table, seq_offsets, ctx_len, workspace, dev_status)
        self._args = hss_packed_args(
            hss_dims.of(dims), _ptr(q_offsets), int(total_q), int(max_q), int(window), int(sinks),
            _ptr(block_table), _ptr(seq_offsets), _ptr(ctx_len), int(total_blocks),
            int(num_seqs), float(scale), _ptr(workspace), int(workspace_bytes), _ptr(dev_status))
        self._ref = ctypes.byref(self._args)

    def __call__(self, Q, cache, out, lse=None, stream=None) -> None:
        st = self._fn(self._ref, _ptr(Q), _ptr(cache), _ptr(out), _ptr(lse), _stream(stream))
        _check(st, "hss_attend_packed")


def hss_fork_pages_workspace_bytes(num_new: int, max_blocks: int) -> int:
    return load().hss_fork_pages_workspace_bytes(int(num_new), int(max_blocks))


def hss_compact_pages_workspace_bytes(max_blocks: int) -> int:
    return load().hss_compact_pages_workspace_bytes(int(max_blocks))


def hss_fork_pages(block_table, seq_offsets, num_seqs: int, total_blocks: int, refs,
                   max_blocks: int, released, num_released: int, parents, lengths, room,
                   num_new: int, block_size: int, table_room: int, new_table, new_offsets,
                   new_refs, copy_src, copy_dst, counts, workspace, workspace_bytes: int,
                   dev_status=None, stream=None) -> None:
    """The next step's tables and page counts: sequences go on, fork, are cut, dropped or grow."""
    st = load().hss_fork_pages(
        _ptr(block_table), _ptr(seq_offsets), int(num_seqs), int(total_blocks), _ptr(refs),
        int(max_blocks), _ptr(released), int(num_released), _ptr(parents), _ptr(lengths),
        _ptr(room), int(num_new), int(block_size), int(table_room), _ptr(new_table),
        _ptr(new_offsets), _ptr(new_refs), _ptr(copy_src), _ptr(copy_dst), _ptr(counts),
        _ptr(workspace), int(workspace_bytes), _ptr(dev_status), _stream(stream))
    _check(st, "hss_fork_pages")


def hss_compact_pages(block_table, total_blocks: int, refs, max_blocks: int, move_room: int,
                      new_table, new_refs, copy_src, copy_dst, counts, workspace,
                      workspace_bytes: int, dev_status=None, stream=None) -> None:
    """Plan the moves of used pages into the free ones at the front of the pool."""
    st = load().hss_compact_pages(
        _ptr(block_table), int(total_blocks), _ptr(refs), int(max_blocks), int(move_room),
        _ptr(new_table), _ptr(new_refs), _ptr(copy_src), _ptr(copy_dst), _ptr(counts),
        _ptr(workspace), int(workspace_bytes), _ptr(dev_status), _stream(stream))
    _check(st, "hss_compact_pages")


def hss_copy_pages(copy_src, copy_dst, num_copies, max_copies: int, pool0, pool1,
                   page_bytes: int, max_blocks: int, num_layers: int, dev_status=None,
                   stream=None) -> None:
    """pool[layer][copy_dst[i]] = pool[layer][copy_src[i]] for every planned copy and layer."""
    st = load().hss_copy_pages(
        _ptr(copy_src), _ptr(copy_dst), _ptr(num_copies), int(max_copies), _ptr(pool0),
        _ptr(pool1), int(page_bytes), int(max_blocks), int(num_layers), _ptr(dev_status),
        _stream(stream))
    _check(st, "hss_copy_pages")


def hss_layer_step_static_max_seqs() -> int:
    return load().hss_layer_step_static_max_seqs()


def hss_layer_step_static(dims, P, K_new, new_ids, num_new: int, Q, rows_per_seq: int, Qp, A_g,
                          layer: int, block_table, seq_offsets, num_seqs: int, total_blocks: int,
                          scores, k: int, victims, dev_status=None, stream=None) -> None:
    """hss_layer_step without a workspace, for callers that cannot allocate device memory.

    The completion counters live in a fixed array inside the library (at most
    hss_layer_step_static_max_seqs() sequences per call).  Calls share that array, so they
    must not overlap on the GPU.  The first call on a device must come before any stream
    capture on it.
    """
    st = load().hss_layer_step_static(ctypes.byref(hss_dims.of(dims)), _ptr(P), _ptr(K_new),
                                      _ptr(new_ids), int(num_new), _ptr(Q), int(rows_per_seq),
                                      _ptr(Qp), _ptr(A_g), int(layer), _ptr(block_table),
                                      _ptr(seq_offsets), int(num_seqs), int(total_blocks),
                                      _ptr(scores), int(k), _ptr(victims), _ptr(dev_status),
                                      _stream(stream))
    _check(st, "hss_layer_step_static")


def hss_self_test_wait_timeout(dev_status, limit_ns: int, stream=None) -> None:
    """Launch a kernel whose bounded pipeline wait runs out (it sets dev_status)."""
    st = load().hss_self_test_wait_timeout(_ptr(dev_status), int(limit_ns), _stream(stream))
    _check(st, "hss_self_test_wait_timeout")


def hss_self_test_spread_wait(dims, P, Q, A_g, layer: int, block_table, seq_offsets,
                              total_blocks: int, scores, k: int, victims, workspace,
                              workspace_bytes: int, limit_ns: int, dev_status=None,
                              stream=None) -> None:
    """Run the layer call's one-sequence ranking with one CTA withholding its keys, so that
    the other CTAs' bounded waits run out after limit_ns (they set dev_status)."""
    st = load().hss_self_test_spread_wait(ctypes.byref(hss_dims.of(dims)), _ptr(P), _ptr(Q),
                                          _ptr(A_g), int(layer), _ptr(block_table),
                                          _ptr(seq_offsets), int(total_blocks), _ptr(scores),
                                          int(k), _ptr(victims), _ptr(workspace),
                                          int(workspace_bytes), int(limit_ns), _ptr(dev_status),
                                          _stream(stream))
    _check(st, "hss_self_test_spread_wait")


def hss_read_device_error(stream=None) -> int:
    """Synchronise the stream; return and clear the library's device error word."""
    out = ctypes.c_int32(0)
    st = load().hss_read_device_error(ctypes.byref(out), _stream(stream))
    _check(st, "hss_read_device_error")
    return out.value


# ----------------------------------------------------------------------------- host helpers

def check_a_g_budget(dims, free_bytes: int, margin: float = 0.05) -> int:
    """Refuse an A_g that would not fit in (1 - margin) of the free HBM.

    Mirrors the budget check of Predictor::new (predictor page): the error names the
    settings that shrink A_g.  Returns the A_g size in bytes when it fits.
    """
    d = hss_dims.of(dims)
    need = (d.num_layers * d.max_blocks * d.num_kv_heads * d.block_size * d.r * 2)
    budget = int(free_bytes * (1.0 - margin))
    if need > budget:
        raise MemoryError(
            f"A_g would need {need / 2**30:.2f} GiB but only {budget / 2**30:.2f} GiB of HBM "
            f"may be used ({margin:.0%} of the free memory is left for other buffers). "
            f"Shrink one of: r (now {d.r}; r/2 halves A_g), max_blocks (now {d.max_blocks}; "
            f"set by the longest context), num_layers kept ({d.num_layers}). "
            f"A_g = num_layers x max_blocks x num_kv_heads x block_size x r x 2 bytes.")
    return need
