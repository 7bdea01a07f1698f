"""ctypes binding of libtsl.so, libtsl_block.so and libtsl_attn.so -- the entry
points of include/tsl.h, include/tsl_block.h and include/tsl_attn.h under the
same names, argument marshalling only.  Every step of the compute runs in the libraries' HIP
kernels; nothing here computes.

Pointer arguments take either an integer device address or any object with
a ``data_ptr()`` method (a torch tensor).  ``stream=None`` means the current
torch stream when torch has a GPU, else the null stream.  A non-OK status
raises TslError carrying the status code.

Importing this module loads the libraries; when one has not been built the
import fails with ImportError -- there is no fallback path.

PyTorch wheels for ROCm carry their own HIP runtime, which torch's libraries
load by a different file name than the system one.  Loading libtsl.so first
would bring in the system runtime next to torch's -- two runtimes in one
process, and launches fail.  torch is therefore imported (when installed)
before libtsl.so, whose dependency then resolves to the runtime already
loaded, so the library, torch's allocations and torch's streams share one
runtime.
"""
import ctypes
import os
import struct

try:  # see the module docstring: torch's HIP runtime must be loaded first
    import torch as _torch  # noqa: F401
except ImportError:
    _torch = None

_PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_PKG, "libtsl.so")

if not os.path.exists(LIBRARY):
    raise ImportError("libtsl.so is not built: run __graft_entry__.build() or "
                      "python tensor_sharded_linear_plan_amd/build.py")
_lib = ctypes.CDLL(LIBRARY)
BLOCK_LIBRARY = os.path.join(_PKG, "libtsl_block.so")
if not os.path.exists(BLOCK_LIBRARY):
    raise ImportError("libtsl_block.so is not built: run __graft_entry__.build() or "
                      "python tensor_sharded_linear_plan_amd/build.py")
_block = ctypes.CDLL(BLOCK_LIBRARY)
ATTN_LIBRARY = os.path.join(_PKG, "libtsl_attn.so")
if not os.path.exists(ATTN_LIBRARY):
    raise ImportError("libtsl_attn.so is not built: run __graft_entry__.build() or "
                      "python tensor_sharded_linear_plan_amd/build.py")
_attn = ctypes.CDLL(ATTN_LIBRARY)

# ---- enums (include/tsl.h) ----
OK = 0
ERR_INVALID_ARG, ERR_NOT_DIVISIBLE, ERR_TP_NOT_POW2, ERR_GROUP_ALIGN = -1, -2, -3, -4
ERR_BUFFER_TOO_SMALL, ERR_UNSUPPORTED, ERR_MISALIGNED, ERR_HIP = -5, -6, -7, -8

# bytes of the fixed device scratch behind shard_linear_group_noalloc
NOALLOC_SCRATCH_BYTES = 64 << 20
COLUMN, ROW, REPLICATED, EXPERT = 0, 1, 2, 3
MOE_EXPERT_PARALLEL, MOE_WITHIN_EXPERT = 0, 1
COMBINE_NONE, COMBINE_CONCAT, COMBINE_SUM = 0, 1, 2
Q, K, V, O, GATE, UP, DOWN = range(7)
NPROJ = 7
LINEAR = 7
EMBED, LM_HEAD = 8, 9
F32, BF16, Q4G64, E4M3 = 0, 1, 2, 3
ALL_REDUCE, REDUCE_SCATTER, ALL_GATHER = 0, 1, 2
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = range(5)
ROTARY_HALVES, ROTARY_PAIRS = 0, 1
MAX_PARTS = 64


class TslError(RuntimeError):
    def __init__(self, status, where=""):
        self.status = status
        msg = _lib.tsl_status_string(status).decode()
        if status == ERR_HIP:
            last = _block.tsl_block_last_hip_error_string if where in BLOCK_EXPORTS else \
                _attn.tsl_attn_last_hip_error_string if where in ATTN_EXPORTS else \
                _lib.tsl_last_hip_error_string
            msg += " [%s]" % last().decode()
        super().__init__("%s: %s (%d)" % (where, msg, status))


class Dims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("ffn", ctypes.c_int32), ("tp_size", ctypes.c_int32),
                ("group_size", ctypes.c_int32)]


class Shard(ctypes.Structure):
    _fields_ = [("proj", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("strategy", ctypes.c_int32), ("combine", ctypes.c_int32),
                ("K", ctypes.c_int64), ("N", ctypes.c_int64),
                ("k_off", ctypes.c_int64), ("k_len", ctypes.c_int64),
                ("n_off", ctypes.c_int64), ("n_len", ctypes.c_int64),
                ("head_off", ctypes.c_int32), ("head_cnt", ctypes.c_int32)]

    FIELDS = ("proj", "rank", "strategy", "combine", "K", "N", "k_off", "k_len",
              "n_off", "n_len", "head_off", "head_cnt")

    def as_tuple(self):
        return tuple(int(getattr(self, f)) for f in self.FIELDS)

    def __repr__(self):
        return "Shard(%s)" % ", ".join("%s=%d" % (f, getattr(self, f)) for f in self.FIELDS)


class ExpertShard(ctypes.Structure):
    """The gate/up/down shards of one expert on one rank (tsl_expert_shard)."""
    _fields_ = [("expert", ctypes.c_int32), ("rank", ctypes.c_int32), ("gate", Shard),
                ("up", Shard), ("down", Shard)]


class LinearItem(ctypes.Structure):
    """One product of shard_linear_group (tsl_linear_item)."""
    _fields_ = [("shard", ctypes.POINTER(Shard)), ("packed", ctypes.c_void_p),
                ("packed_bytes", ctypes.c_size_t), ("X", ctypes.c_void_p),
                ("ldx", ctypes.c_int64), ("Y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
                ("ydtype", ctypes.c_int32), ("accumulate", ctypes.c_int32),
                ("sum_next", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("row_index", ctypes.c_void_p), ("x_rows", ctypes.c_int64)]


class Epilogue(ctypes.Structure):
    """What a product goes through before it is stored (tsl_epilogue)."""
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("pre", ctypes.c_void_p), ("ld_res", ctypes.c_int64), ("ld_pre", ctypes.c_int64),
                ("act", ctypes.c_int32), ("bias_dtype", ctypes.c_int32),
                ("res_dtype", ctypes.c_int32), ("pre_dtype", ctypes.c_int32)]


class GatedItem(ctypes.Structure):
    """One gated feed-forward block of shard_gated_group (tsl_gated_item)."""
    _fields_ = [("gate", ctypes.POINTER(Shard)), ("up", ctypes.POINTER(Shard)),
                ("packed_gate", ctypes.c_void_p), ("packed_up", ctypes.c_void_p),
                ("packed_bytes", ctypes.c_size_t), ("X", ctypes.c_void_p),
                ("ldx", ctypes.c_int64), ("H", ctypes.c_void_p), ("ldh", ctypes.c_int64),
                ("G", ctypes.c_void_p), ("U", ctypes.c_void_p), ("ld_gu", ctypes.c_int64),
                ("row_index", ctypes.c_void_p), ("x_rows", ctypes.c_int64),
                ("hdtype", ctypes.c_int32), ("rows", ctypes.c_int32)]


class Rotary(ctypes.Structure):
    """Positions and frequencies of rotate_heads (tsl_rotary)."""
    _fields_ = [("positions", ctypes.c_void_p), ("ld_pos", ctypes.c_int64),
                ("freq", ctypes.c_void_p), ("pair_axis", ctypes.c_void_p),
                ("axes", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("style", ctypes.c_int32)]


class RotateItem(ctypes.Structure):
    """One operand of rotate_heads (tsl_rotate_item)."""
    _fields_ = [("X", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("x_head", ctypes.c_int64),
                ("Y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("y_head", ctypes.c_int64),
                ("n_heads", ctypes.c_int32), ("xdtype", ctypes.c_int32),
                ("ydtype", ctypes.c_int32)]


class Cache(ctypes.Structure):
    """A paged 4-bit cache of keys and values (tsl_cache)."""
    _fields_ = [("pages", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_tokens", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class Seqs(ctypes.Structure):
    """The sequences of a cache call (tsl_seqs)."""
    _fields_ = [("row_start", ctypes.c_void_p), ("context", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("ld_table", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("n_seqs", ctypes.c_int32),
                ("max_rows", ctypes.c_int32), ("max_context", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]


_i32, _i64, _vp, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
_P_SHARD = ctypes.POINTER(Shard)
_P_ITEM = ctypes.POINTER(LinearItem)
_lib.plan_shards.argtypes = [ctypes.POINTER(Dims), _P_SHARD, _i64]
_lib.plan_linear.argtypes = [_i64, _i64, _i32, _i32, _i32, _P_SHARD, _i64]
_lib.pack_shard_size.argtypes = [_P_SHARD, ctypes.c_int, ctypes.POINTER(_sz)]
_lib.pack_shard.argtypes = [_P_SHARD, ctypes.c_int, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp,
                            _sz, _vp]
_lib.shard_linear_workspace_size.argtypes = [_P_SHARD, ctypes.c_int, _i64, ctypes.POINTER(_sz)]
_lib.shard_linear.argtypes = [_P_SHARD, ctypes.c_int, _vp, _sz, ctypes.c_int, _vp, _i64, _i64,
                              ctypes.c_int, _vp, _i64, ctypes.c_int, _vp, _sz, _vp]
_lib.shard_linear_group_workspace_size.argtypes = [_i32, _P_ITEM, ctypes.c_int, _i64,
                                                   ctypes.POINTER(_sz)]
_lib.shard_linear_group.argtypes = [_i32, _P_ITEM, ctypes.c_int, ctypes.c_int, _i64, _vp, _sz,
                                    _vp]
_lib.shard_linear_group_noalloc.argtypes = [_i32, _P_ITEM, ctypes.c_int, ctypes.c_int, _i64, _vp]
_lib.combine_partials.argtypes = [ctypes.c_int, _i32, ctypes.POINTER(_vp), ctypes.c_int, _i64,
                                  _i64, _i64, ctypes.c_int, _vp, _i64, _vp]
_lib.combine_to_ranks.argtypes = [ctypes.c_int, _i32, ctypes.POINTER(_vp), ctypes.c_int, _i64,
                                  _i64, _i64, ctypes.c_int, ctypes.POINTER(_vp), _i64, _vp]
_lib.plan_experts.argtypes = [_i32, _i64, _i64, _i32, _i32, _i32, ctypes.POINTER(ExpertShard),
                              _i64, ctypes.POINTER(_i64)]
_lib.moe_dispatch.argtypes = [_vp, _i64, _i32, _i32, _vp, _i32, _vp, _vp, _vp]
_lib.moe_gather.argtypes = [_vp, _i64, _i64, ctypes.c_int, _vp, _i64, _i64, _vp, _i64, _vp]
_lib.moe_combine.argtypes = [_vp, _i64, _i64, _vp, _vp, _i64, _i32, _i64, ctypes.c_int, _vp, _i64,
                             _vp]
_lib.plan_vocab.argtypes = [_i64, _i64, _i32, _i32, _P_SHARD, _i64]
_lib.embed_lookup.argtypes = [_P_SHARD, ctypes.c_int, _vp, _i64, _vp, _i64, ctypes.c_int, _vp,
                              _i64, _vp]
_lib.tsl_status_string.argtypes = [ctypes.c_int]
_lib.tsl_status_string.restype = ctypes.c_char_p
_lib.tsl_last_hip_error_string.argtypes = []
_lib.tsl_last_hip_error_string.restype = ctypes.c_char_p
for _f in ("plan_shards", "plan_linear", "pack_shard_size", "pack_shard",
           "shard_linear_workspace_size", "shard_linear", "shard_linear_group_workspace_size",
           "shard_linear_group", "shard_linear_group_noalloc", "combine_partials",
           "combine_to_ranks", "plan_vocab",
           "embed_lookup", "plan_experts", "moe_dispatch", "moe_gather", "moe_combine"):
    getattr(_lib, _f).restype = ctypes.c_int

EXPORTS = ("plan_shards", "plan_linear", "pack_shard_size", "pack_shard",
           "shard_linear_workspace_size", "shard_linear", "shard_linear_group_workspace_size",
           "shard_linear_group", "shard_linear_group_noalloc", "combine_partials",
           "combine_to_ranks", "plan_vocab",
           "embed_lookup", "plan_experts", "moe_dispatch", "moe_gather", "moe_combine",
           "tsl_status_string", "tsl_last_hip_error_string")


_block.add_rms_norm.argtypes = [_i32, ctypes.POINTER(_vp), ctypes.c_int, _i64, _i64, _i64, _vp,
                              ctypes.c_int, _i64, _vp, _i64, _vp, ctypes.c_int, ctypes.c_float,
                              ctypes.c_int, _vp, _i64, _vp, _i32, _vp, _vp]
_block.add_rms_norm_grad_workspace_size.argtypes = [_i64, _i64, ctypes.POINTER(_sz)]
_block.add_rms_norm_grad.argtypes = [_i64, _i64, _vp, ctypes.c_int, _i64, _vp, ctypes.c_int, _i64,
                                   _vp, ctypes.c_int, ctypes.c_float, _vp, _vp, _i64, _vp,
                                   ctypes.c_int, _i64, _vp, ctypes.c_int, _vp, _sz, _vp]
_P_EPS = ctypes.POINTER(ctypes.POINTER(Epilogue))
_P_GATED = ctypes.POINTER(GatedItem)
_block.shard_linear_group_epilogue_workspace_size.argtypes = [_i32, _P_ITEM, _P_EPS, ctypes.c_int,
                                                              _i64, ctypes.POINTER(_sz)]
_block.shard_linear_group_epilogue.argtypes = [_i32, _P_ITEM, _P_EPS, ctypes.c_int, ctypes.c_int,
                                               _i64, _vp, _sz, _vp]
_block.shard_gated_group_workspace_size.argtypes = [_i32, _P_GATED, ctypes.c_int, _i64,
                                                    ctypes.POINTER(_sz)]
_block.shard_gated_group.argtypes = [_i32, _P_GATED, ctypes.c_int, ctypes.c_int, ctypes.c_int, _i64,
                                     _vp, _sz, _vp]
_block.transpose_shard.argtypes = [_P_SHARD, _P_SHARD]
_block.shard_linear_grad_workspace_size.argtypes = [_P_SHARD, ctypes.c_int, _i64,
                                                    ctypes.POINTER(_sz)]
_block.shard_linear_grad.argtypes = [_P_SHARD, ctypes.c_int, _vp, _sz, _i64, _vp, _i64, ctypes.c_int,
                                     _vp, _i64, _vp, _i64, ctypes.c_int, _vp, _i64, ctypes.c_int,
                                     _vp, _i64, _i64, ctypes.c_int, _vp, _vp, _sz, _vp]
_block.shard_gated_grad_workspace_size.argtypes = [_P_SHARD, _P_SHARD, ctypes.c_int, _i64,
                                                   ctypes.POINTER(_sz)]
_block.shard_gated_grad.argtypes = [_P_SHARD, _P_SHARD, ctypes.c_int, _vp, _vp, _sz, _i64, _vp, _i64,
                                    ctypes.c_int, _vp, _vp, _i64, _vp, _i64, ctypes.c_int, _vp, _i64,
                                    ctypes.c_int, _vp, _vp, _i64, _i64, ctypes.c_int, _vp, _sz, _vp]
_block.tsl_block_last_hip_error_string.argtypes = []
_block.tsl_block_last_hip_error_string.restype = ctypes.c_char_p

# the entry points of include/tsl_block.h
BLOCK_EXPORTS = ("add_rms_norm", "add_rms_norm_grad_workspace_size", "add_rms_norm_grad",
                 "shard_linear_group_epilogue_workspace_size", "shard_linear_group_epilogue",
                 "shard_gated_group_workspace_size", "shard_gated_group",
                 "transpose_shard", "shard_linear_grad_workspace_size", "shard_linear_grad",
                 "shard_gated_grad_workspace_size", "shard_gated_grad",
                 "tsl_block_last_hip_error_string")
for _f in BLOCK_EXPORTS[:-1]:
    getattr(_block, _f).restype = ctypes.c_int

# (their structures go as the bytes that a call packs: a generated token's calls
# are short enough for the marshalling to count)
_attn.rotate_heads.argtypes = [_i32, _vp, _i64, _vp, ctypes.c_int, _vp]
_attn.cache_size.argtypes = [_vp, ctypes.POINTER(_sz)]
for _f in ("cache_append", "cache_read"):
    getattr(_attn, _f).argtypes = [_vp, _vp, ctypes.c_int, _vp, _i64, _i64, _vp, _i64, _i64, _vp]
_attn.cache_attention_workspace_size.argtypes = [_vp, _vp, _i32, _i32, _i32, ctypes.POINTER(_sz)]
_attn.cache_attention.argtypes = [_vp, _vp, _i32, _vp, _i64, _i64, ctypes.c_float, _i32, _i32,
                                  ctypes.c_int, _vp, _i64, _i64, _vp, _sz, _vp]
_attn.tsl_attn_last_hip_error_string.argtypes = []
_attn.tsl_attn_last_hip_error_string.restype = ctypes.c_char_p

# the entry points of include/tsl_attn.h
ATTN_EXPORTS = ("rotate_heads", "cache_size", "cache_append", "cache_read",
                "cache_attention_workspace_size", "cache_attention",
                "tsl_attn_last_hip_error_string")
for _f in ATTN_EXPORTS[:-1]:
    getattr(_attn, _f).restype = ctypes.c_int


def _check(status, where):
    if status != OK:
        raise TslError(status, where)


def _ptr(x):
    if x is None:
        return None
    try:
        return x.data_ptr()
    except AttributeError:
        return int(x)


_raw_stream = getattr(getattr(_torch, "_C", None), "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is not None:
        return getattr(stream, "cuda_stream", stream)
    if _torch is None:
        return None
    # the current stream's handle, without building a Stream object per call
    if _raw_stream is not None and _torch.cuda.is_initialized():
        return _raw_stream(_torch.cuda.current_device())
    if _torch.cuda.is_available():
        return _torch.cuda.current_stream().cuda_stream
    return None


def tsl_status_string(status):
    return _lib.tsl_status_string(status).decode()


def tsl_last_hip_error_string():
    return _lib.tsl_last_hip_error_string().decode()


def plan_shards(hidden, n_q_heads, n_kv_heads, head_dim, ffn, tp_size, group_size=0):
    """Shards for every (rank, projection): a list indexed [rank * NPROJ + proj]."""
    d = Dims(hidden, n_q_heads, n_kv_heads, head_dim, ffn, tp_size, group_size)
    n = max(int(tp_size), 1) * NPROJ
    out = (Shard * n)()
    _check(_lib.plan_shards(ctypes.byref(d), out, n), "plan_shards")
    return list(out)


def plan_linear(K, N, tp_size, strategy, group_size=0):
    n = max(int(tp_size), 1)
    out = (Shard * n)()
    _check(_lib.plan_linear(K, N, tp_size, strategy, group_size, out, n), "plan_linear")
    return list(out)


def plan_vocab(vocab, hidden, tp_size, group_size=0):
    """[embedding shard, LM-head shard] of every rank: a list of 2*tp shards."""
    n = 2 * max(int(tp_size), 1)
    out = (Shard * n)()
    _check(_lib.plan_vocab(vocab, hidden, tp_size, group_size, out, n), "plan_vocab")
    return list(out)


def plan_experts(n_experts, hidden, expert_ffn, tp_size, mode, group_size=0):
    """Every rank's expert shards, rank-major: a list of ExpertShard."""
    n = n_experts * (max(int(tp_size), 1) if mode == MOE_WITHIN_EXPERT else 1)
    out = (ExpertShard * max(n, 1))()
    got = _i64(0)
    _check(_lib.plan_experts(n_experts, hidden, expert_ffn, tp_size, mode, group_size, out, n,
                             ctypes.byref(got)), "plan_experts")
    return list(out)[:got.value]


def moe_dispatch(topk, n_experts, experts):
    """Host routing -> (offsets int64 [n_local + 1], row_slot int32 [rows],
    slot_row int32 [T*k]); topk is an int32 array [T][k] (host)."""
    import numpy as np
    topk = np.ascontiguousarray(topk, dtype=np.int32)
    T, k = topk.shape
    ex = np.ascontiguousarray(experts, dtype=np.int32)
    offsets = np.zeros(len(ex) + 1, dtype=np.int64)
    row_slot = np.zeros(max(T * k, 1), dtype=np.int32)
    slot_row = np.zeros(max(T * k, 1), dtype=np.int32)
    _check(_lib.moe_dispatch(topk.ctypes.data, T, k, n_experts, ex.ctypes.data if len(ex) else None,
                             len(ex), offsets.ctypes.data, row_slot.ctypes.data,
                             slot_row.ctypes.data), "moe_dispatch")
    return offsets, row_slot[:offsets[-1]].copy(), slot_row[:T * k].copy()


def moe_gather(src, ld_src, n_src, dtype, idx, n, width, out, ldo, stream=None):
    _check(_lib.moe_gather(_ptr(src), ld_src, n_src, dtype, _ptr(idx), n, width, _ptr(out), ldo,
                           _stream(stream)), "moe_gather")


def moe_combine(P, ldp, n_rows, slot_row, weights, T, k, n, ydtype, Y, ldy, stream=None):
    _check(_lib.moe_combine(_ptr(P), ldp, n_rows, _ptr(slot_row), _ptr(weights), T, k, n, ydtype,
                            _ptr(Y), ldy, _stream(stream)), "moe_combine")


def embed_lookup(shard, tdtype, table, ld_table, tokens, M, ydtype, Y, ldy, stream=None):
    _check(_lib.embed_lookup(ctypes.byref(shard), tdtype, _ptr(table), ld_table, _ptr(tokens), M,
                             ydtype, _ptr(Y), ldy, _stream(stream)), "embed_lookup")


def pack_shard_size(shard, wdtype):
    b = _sz(0)
    _check(_lib.pack_shard_size(ctypes.byref(shard), wdtype, ctypes.byref(b)), "pack_shard_size")
    return b.value


def pack_shard(shard, wdtype, W, stride_k, stride_n, scales, biases, sb_stride_g, sb_stride_n,
               packed, packed_bytes, stream=None):
    _check(_lib.pack_shard(ctypes.byref(shard), wdtype, _ptr(W), stride_k, stride_n,
                           _ptr(scales), _ptr(biases), sb_stride_g, sb_stride_n, _ptr(packed),
                           packed_bytes, _stream(stream)), "pack_shard")


def shard_linear_workspace_size(shard, wdtype, M):
    b = _sz(0)
    _check(_lib.shard_linear_workspace_size(ctypes.byref(shard), wdtype, M, ctypes.byref(b)),
           "shard_linear_workspace_size")
    return b.value


def shard_linear(shard, wdtype, packed, packed_bytes, xdtype, X, ldx, M, ydtype, Y, ldy,
                 accumulate=0, workspace=None, ws_bytes=0, stream=None):
    _check(_lib.shard_linear(ctypes.byref(shard), wdtype, _ptr(packed), packed_bytes, xdtype,
                             _ptr(X), ldx, M, ydtype, _ptr(Y), ldy, accumulate, _ptr(workspace),
                             ws_bytes, _stream(stream)), "shard_linear")


def _shard(sh):
    """A Shard, or a copy of any object with its as_tuple."""
    return sh if isinstance(sh, Shard) else Shard(*sh.as_tuple())


def _items(items):
    """items: sequence of dicts (or LinearItem) with the tsl_linear_item
    fields (ydtype defaults to F32, accumulate, sum_next and rows to 0,
    row_index to None); shard as _shard; a set member's Y may be None.
    Returns the ctypes array (which keeps the shards alive) and its length."""
    n = len(items)
    arr = (LinearItem * (n or 1))()
    keep = []
    for i, it in enumerate(items):
        if isinstance(it, LinearItem):
            arr[i] = it
            continue
        get = it.get
        sh = _shard(it["shard"])
        keep.append(sh)
        arr[i] = LinearItem(ctypes.pointer(sh), _ptr(it["packed"]), it["packed_bytes"],
                            _ptr(it["X"]), it["ldx"], _ptr(get("Y")), get("ldy", 0),
                            get("ydtype", F32), get("accumulate", 0), get("sum_next", 0),
                            get("rows", 0), _ptr(get("row_index")), get("x_rows", 0))
    arr._keep = keep
    return arr, n


def shard_linear_group_workspace_size(items, wdtype, M):
    arr, n = _items(items)
    b = _sz(0)
    _check(_lib.shard_linear_group_workspace_size(n, arr, wdtype, M, ctypes.byref(b)),
           "shard_linear_group_workspace_size")
    return b.value


def shard_linear_group(items, wdtype, xdtype, M, workspace=None, ws_bytes=0, stream=None):
    arr, n = _items(items)
    _check(_lib.shard_linear_group(n, arr, wdtype, xdtype, M, _ptr(workspace), ws_bytes,
                                   _stream(stream)), "shard_linear_group")


def shard_linear_group_noalloc(items, wdtype, xdtype, M, stream=None):
    arr, n = _items(items)
    _check(_lib.shard_linear_group_noalloc(n, arr, wdtype, xdtype, M, _stream(stream)),
           "shard_linear_group_noalloc")


def combine_partials(mode, parts, pdtype, M, n_each, ld_part, ydtype, Y, ldy, stream=None):
    arr = (_vp * max(len(parts), 1))(*[_ptr(p) for p in parts])
    _check(_lib.combine_partials(mode, len(parts), arr, pdtype, M, n_each, ld_part, ydtype,
                                 _ptr(Y), ldy, _stream(stream)), "combine_partials")


def combine_to_ranks(op, parts, pdtype, M, n_each, ld_part, odtype, outs, ldo, stream=None):
    n = len(parts)
    parr = (_vp * max(n, 1))(*[_ptr(p) for p in parts])
    oarr = (_vp * max(len(outs), 1))(*[_ptr(o) for o in outs])
    if len(outs) != n:
        raise ValueError("combine_to_ranks: one output per part")
    _check(_lib.combine_to_ranks(op, n, parr, pdtype, M, n_each, ld_part, odtype, oarr, ldo,
                                 _stream(stream)), "combine_to_ranks")


def add_rms_norm(parts, pdtype, ld_part, M, n, residual, rdtype, ldr, sum_out, ld_sum, weight,
                 wdtype, eps, ydtype, Y, ldy, scales=None, group=0, rstd=None, stream=None):
    arr = (_vp * max(len(parts), 1))(*[_ptr(p) for p in parts])
    _check(_block.add_rms_norm(len(parts), arr, pdtype, ld_part, M, n, _ptr(residual), rdtype, ldr,
                             _ptr(sum_out), ld_sum, _ptr(weight), wdtype, eps, ydtype, _ptr(Y), ldy,
                             _ptr(scales), group, _ptr(rstd), _stream(stream)), "add_rms_norm")


def add_rms_norm_grad_workspace_size(M, n):
    b = _sz(0)
    _check(_block.add_rms_norm_grad_workspace_size(M, n, ctypes.byref(b)),
           "add_rms_norm_grad_workspace_size")
    return b.value


def add_rms_norm_grad(M, n, dY, dydtype, lddy, X, xdtype, ldx, weight, wdtype, eps, rstd, dres,
                      ld_dres, dX, dxdtype, lddx, dW, accumulate_dw=0, workspace=None, ws_bytes=0,
                      stream=None):
    _check(_block.add_rms_norm_grad(M, n, _ptr(dY), dydtype, lddy, _ptr(X), xdtype, ldx, _ptr(weight),
                                  wdtype, eps, _ptr(rstd), _ptr(dres), ld_dres, _ptr(dX), dxdtype,
                                  lddx, _ptr(dW), accumulate_dw, _ptr(workspace), ws_bytes,
                                  _stream(stream)), "add_rms_norm_grad")


def _epilogues(eps, n):
    """eps: one dict (or Epilogue) per item with the tsl_epilogue fields
    (types default to F32, act to ACT_NONE), or None for a plain product."""
    if len(eps) != n:
        raise ValueError("one epilogue (or None) per item")
    arr = (ctypes.POINTER(Epilogue) * max(n, 1))()
    for i, e in enumerate(eps):
        if e is None:
            continue
        if not isinstance(e, Epilogue):
            get = e.get
            e = Epilogue(_ptr(get("bias")), _ptr(get("residual")), _ptr(get("pre")),
                         get("ld_res", 0), get("ld_pre", 0), get("act", ACT_NONE),
                         get("bias_dtype", F32), get("res_dtype", F32), get("pre_dtype", F32))
        arr[i] = ctypes.pointer(e)
    return arr


def shard_linear_group_epilogue_workspace_size(items, epilogues, wdtype, M):
    arr, n = _items(items)
    b = _sz(0)
    _check(_block.shard_linear_group_epilogue_workspace_size(n, arr, _epilogues(epilogues, n), wdtype,
                                                             M, ctypes.byref(b)),
           "shard_linear_group_epilogue_workspace_size")
    return b.value


def shard_linear_group_epilogue(items, epilogues, wdtype, xdtype, M, workspace=None, ws_bytes=0,
                                stream=None):
    arr, n = _items(items)
    _check(_block.shard_linear_group_epilogue(n, arr, _epilogues(epilogues, n), wdtype, xdtype, M,
                                              _ptr(workspace), ws_bytes, _stream(stream)),
           "shard_linear_group_epilogue")


def _gated(items):
    """items: sequence of dicts (or GatedItem) with the tsl_gated_item fields
    (gate and up as _shard; hdtype defaults to F32, rows to 0, G, U and
    row_index to None)."""
    n = len(items)
    arr = (GatedItem * (n or 1))()
    keep = []
    for i, it in enumerate(items):
        if isinstance(it, GatedItem):
            arr[i] = it
            continue
        get, g, u = it.get, _shard(it["gate"]), _shard(it["up"])
        keep += [g, u]
        arr[i] = GatedItem(ctypes.pointer(g), ctypes.pointer(u), _ptr(it["packed_gate"]),
                           _ptr(it["packed_up"]), it["packed_bytes"], _ptr(it["X"]), it["ldx"],
                           _ptr(it["H"]), it["ldh"], _ptr(get("G")), _ptr(get("U")),
                           get("ld_gu", 0), _ptr(get("row_index")), get("x_rows", 0),
                           get("hdtype", F32), get("rows", 0))
    arr._keep = keep
    return arr, n


def shard_gated_group_workspace_size(items, wdtype, M):
    arr, n = _gated(items)
    b = _sz(0)
    _check(_block.shard_gated_group_workspace_size(n, arr, wdtype, M, ctypes.byref(b)),
           "shard_gated_group_workspace_size")
    return b.value


def shard_gated_group(items, act, wdtype, xdtype, M, workspace=None, ws_bytes=0, stream=None):
    arr, n = _gated(items)
    _check(_block.shard_gated_group(n, arr, act, wdtype, xdtype, M, _ptr(workspace), ws_bytes,
                                    _stream(stream)), "shard_gated_group")


def transpose_shard(shard):
    sh, out = _shard(shard), Shard()
    _check(_block.transpose_shard(ctypes.byref(sh), ctypes.byref(out)), "transpose_shard")
    return out


def shard_linear_grad_workspace_size(shard, wdtype, M):
    sh, b = _shard(shard), _sz(0)
    _check(_block.shard_linear_grad_workspace_size(ctypes.byref(sh), wdtype, M, ctypes.byref(b)),
           "shard_linear_grad_workspace_size")
    return b.value


def shard_linear_grad(shard, wdtype, packed_t, packed_t_bytes, M, X, ldx, act, Z, ldz, dY, lddy,
                      dxdtype, dX, lddx, dwdtype, dW, dw_stride_k, dw_stride_n, accumulate_dw=0,
                      db=None, workspace=None, ws_bytes=0, stream=None):
    sh = _shard(shard)
    _check(_block.shard_linear_grad(ctypes.byref(sh), wdtype, _ptr(packed_t), packed_t_bytes, M,
                                    _ptr(X), ldx, act, _ptr(Z), ldz, _ptr(dY), lddy, dxdtype,
                                    _ptr(dX), lddx, dwdtype, _ptr(dW), dw_stride_k, dw_stride_n,
                                    accumulate_dw, _ptr(db), _ptr(workspace), ws_bytes,
                                    _stream(stream)), "shard_linear_grad")


def shard_gated_grad_workspace_size(gate, up, wdtype, M):
    g, u, b = _shard(gate), _shard(up), _sz(0)
    _check(_block.shard_gated_grad_workspace_size(ctypes.byref(g), ctypes.byref(u), wdtype, M,
                                                  ctypes.byref(b)),
           "shard_gated_grad_workspace_size")
    return b.value


def shard_gated_grad(gate, up, wdtype, packed_gate_t, packed_up_t, packed_t_bytes, M, X, ldx, act, G,
                     U, ld_gu, dH, lddh, dxdtype, dX, lddx, dwdtype, dW_gate, dW_up, dw_stride_k,
                     dw_stride_n, accumulate_dw=0, workspace=None, ws_bytes=0, stream=None):
    g, u = _shard(gate), _shard(up)
    _check(_block.shard_gated_grad(ctypes.byref(g), ctypes.byref(u), wdtype, _ptr(packed_gate_t),
                                   _ptr(packed_up_t), packed_t_bytes, M, _ptr(X), ldx, act, _ptr(G),
                                   _ptr(U), ld_gu, _ptr(dH), lddh, dxdtype, _ptr(dX), lddx, dwdtype,
                                   _ptr(dW_gate), _ptr(dW_up), dw_stride_k, dw_stride_n,
                                   accumulate_dw, _ptr(workspace), ws_bytes, _stream(stream)),
           "shard_gated_grad")


# layouts of Rotary, RotateItem, Cache and Seqs
_ROTARY, _ROTATE_ITEM = struct.Struct("=QqQQiiii"), struct.Struct("=QqqQqqiii4x")
_CACHE, _SEQS = struct.Struct("=Qqiii4x"), struct.Struct("=QQQqqiiii")


def _rotary(r):
    """r: a dict (or Rotary) with the tsl_rotary fields; pair_axis a sequence of
    axes or None (style defaults to ROTARY_HALVES, axes to 1, ld_pos to 0).
    Returns its bytes and what they point to."""
    if isinstance(r, Rotary):
        return bytes(r), None
    get, axis, keep = r.get, r.get("pair_axis"), None
    if axis is not None:
        if len(axis) != r["rot_dim"] // 2:
            raise ValueError("one axis per pair")
        keep = ctypes.create_string_buffer(bytes(axis), max(len(axis), 1))
    return _ROTARY.pack(_ptr(r["positions"]) or 0, get("ld_pos", 0), _ptr(r["freq"]) or 0,
                        ctypes.addressof(keep) if keep is not None else 0, get("axes", 1),
                        r["rot_dim"], r["head_dim"], get("style", ROTARY_HALVES)), keep


def rotate_heads(items, M, rotary, inverse=0, stream=None):
    """items: sequence of dicts (or RotateItem) with the tsl_rotate_item fields."""
    arr = b"".join([bytes(i) if isinstance(i, RotateItem) else
                    _ROTATE_ITEM.pack(_ptr(i["X"]) or 0, i["ldx"], i["x_head"], _ptr(i["Y"]) or 0,
                                      i["ldy"], i["y_head"], i["n_heads"], i["xdtype"], i["ydtype"])
                    for i in items])
    r, keep = _rotary(rotary)
    _check(_attn.rotate_heads(len(items), arr, M, r, inverse, _stream(stream)), "rotate_heads")


def _cache(c):
    """c: a dict (or Cache) with the tsl_cache fields."""
    if isinstance(c, Cache):
        return bytes(c)
    return _CACHE.pack(_ptr(c.get("pages")) or 0, c["n_pages"], c["page_tokens"], c["n_kv_heads"],
                       c["head_dim"])


def _seqs(q):
    """q: a dict (or Seqs) with the tsl_seqs fields (the arrays default to
    None, for size queries)."""
    if isinstance(q, Seqs):
        return bytes(q)
    get = q.get
    return _SEQS.pack(_ptr(get("row_start")) or 0, _ptr(get("context")) or 0,
                      _ptr(get("page_table")) or 0, get("ld_table", 0), q["rows"], q["n_seqs"],
                      q["max_rows"], q["max_context"], q["max_pages"])


def cache_size(cache):
    b = _sz(0)
    _check(_attn.cache_size(_cache(cache), ctypes.byref(b)), "cache_size")
    return b.value


def cache_append(cache, seqs, dtype, K, ldk, k_head, V, ldv, v_head, stream=None):
    _check(_attn.cache_append(_cache(cache), _seqs(seqs), dtype, _ptr(K), ldk, k_head, _ptr(V), ldv,
                              v_head, _stream(stream)), "cache_append")


def cache_read(cache, seqs, dtype, K, ldk, k_head, V, ldv, v_head, stream=None):
    _check(_attn.cache_read(_cache(cache), _seqs(seqs), dtype, _ptr(K), ldk, k_head, _ptr(V), ldv,
                            v_head, _stream(stream)), "cache_read")


def cache_attention_workspace_size(cache, seqs, n_q_heads, window=0, sinks=0):
    b = _sz(0)
    _check(_attn.cache_attention_workspace_size(_cache(cache), _seqs(seqs), n_q_heads, window, sinks,
                                                ctypes.byref(b)), "cache_attention_workspace_size")
    return b.value


def cache_attention(cache, seqs, n_q_heads, Q, ldq, q_head, scale, window, sinks, odtype, O, ldo,
                    o_head, workspace=None, ws_bytes=0, stream=None):
    _check(_attn.cache_attention(_cache(cache), _seqs(seqs), n_q_heads, _ptr(Q), ldq, q_head, scale,
                                 window, sinks, odtype, _ptr(O), ldo, o_head, _ptr(workspace),
                                 ws_bytes, _stream(stream)), "cache_attention")
