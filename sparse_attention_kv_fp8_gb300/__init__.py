"""GB300 (sm_103a) ECHO decode step: thin ctypes binding over libecho_gb300.

Every function here marshals arguments (torch tensors -> raw pointers, the
current CUDA stream) and calls the C ABI of include/echo.h with the same name;
all work runs in the library's CUDA kernels.  There is no CPU or PyTorch
fallback: importing the binding without the built library raises.

Buffers are plain torch tensors: device tensors for the GPU side, a pinned
(page-locked, mapped) CPU tensor for the host KV pool.  `Pool`, `Workspace`,
`Stage` and `Stats` are small holders that allocate those tensors and build the
C structs.
"""
from __future__ import annotations

import ctypes
import os
import platform

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, f"libecho_gb300_{platform.machine()}.so")

ECHO_OK, ECHO_EINVAL, ECHO_ECUDA, ECHO_ENOTSUP = 0, 1, 2, 3
DEV_POOL_EXHAUSTED, DEV_BAD_INDEX, DEV_WAIT_TIMEOUT, DEV_PREFETCH_CAP_HIT, DEV_INVARIANT = 1, 2, 4, 8, 16
VAL_FIELDS = ("slot_state", "slot_map", "row_map", "counter", "reserve", "free", "occupied", "reserved",
              "resident", "reserve_balance")
INF = 0x7FFFFFFF
H_INDEX, D_INDEX, KV_ELEMS, KV_BYTES = 64, 128, 576, 1152
STAGE_APPEND, STAGE_INDEXER, STAGE_TOPK, STAGE_RECALL, STAGE_EMA, NUM_STAGES = range(6)
BLOCK_BF16, BLOCK_FP4 = 0, 1
STAT_FIELDS = ("steps", "selected", "unique_rows", "hits", "misses", "recalled", "unrecalled",
               "evicted", "staged", "staged_used", "appended")

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64


class EchoError(RuntimeError):
    pass


class c_pool(ctypes.Structure):
    _fields_ = [("n_g", _I32), ("n_h", _I32), ("gpu_token_free", _P), ("gpu_token_priority", _P),
                ("gpu_indices_buffer", _P), ("gpu_token_to_host", _P), ("host_token_to_gpu", _P),
                ("gpu_kv", _P), ("host_kv", _P), ("counters", _P), ("row_elems", _I32)]


class c_workspace(ctypes.Structure):
    _fields_ = [("base", _P), ("bytes", ctypes.c_size_t), ("n_g", _I32), ("max_rows", _I32)]


class c_stage(ctypes.Structure):
    _fields_ = [("rows", _P), ("host_row", _P), ("count", _P), ("stride", _I32), ("cap_div", _I32),
                ("reserve", _P), ("reserve_ctl", _P), ("reserve_cap", _I32), ("flags", _I32)]


class c_indexer_args(ctypes.Structure):
    _fields_ = [("q", _P), ("w", _P), ("k_index", _P), ("ctx_len", _P), ("B", _I32), ("n_q", _I32),
                ("L_max", _I32), ("scores", _P), ("s_hat", _P), ("req_to_host", _P),
                ("pool", ctypes.POINTER(c_pool)), ("stage", ctypes.POINTER(c_stage)), ("dev_status", _P)]


class c_prefill_args(ctypes.Structure):
    _fields_ = [("q", _P), ("w", _P), ("k_index", _P), ("ctx_len", _P), ("B", _I32), ("C", _I32),
                ("L_max", _I32), ("scores", _P), ("s_shift", _P), ("k", _I32), ("thr_bin", _P), ("subset_n", _P),
                ("req_to_host", _P), ("pool", ctypes.POINTER(c_pool)), ("stage", ctypes.POINTER(c_stage)),
                ("dev_status", _P)]


class c_mla_args(ctypes.Structure):
    _fields_ = [("q", _P), ("gpu_kv", _P), ("n_g", _I32), ("out_slot", _P), ("B", _I32), ("n_q", _I32),
                ("k", _I32), ("scale", ctypes.c_float), ("out", _P), ("lse", _P), ("workspace", _P),
                ("workspace_bytes", ctypes.c_size_t), ("dev_status", _P)]


class c_step_args(ctypes.Structure):
    _fields_ = [("pool", ctypes.POINTER(c_pool)), ("ws", ctypes.POINTER(c_workspace)),
                ("stage", ctypes.POINTER(c_stage)), ("q", _P), ("w", _P), ("k_index", _P), ("ctx_len", _P),
                ("req_to_host", _P), ("B", _I32), ("n_q", _I32), ("L_max", _I32), ("k", _I32),
                ("scores", _P), ("sel", _P), ("kth", _P), ("out_slot", _P), ("s_hat", _P),
                ("alpha", ctypes.c_float), ("new_kv", _P), ("new_k_index", _P), ("clock", _I32),
                ("clock_dev", _P), ("advance_clock", _I32), ("stats", _P), ("dev_status", _P),
                ("stage_events", ctypes.POINTER(_P))]


class c_block_tables_args(ctypes.Structure):
    _fields_ = [("old_len", _P), ("new_len", _P), ("B", _I32), ("block_tokens", _I32), ("table", _P),
                ("free_blocks", _P), ("max_blocks", _I32), ("n_blocks", _I32), ("free_count", _P),
                ("free_count_out", _P), ("slot_map", _P), ("positions", _P), ("cu_new", _P), ("len_out", _P),
                ("max_new", _I32), ("dev_status", _P)]


class c_qk_norm_rope_args(ctypes.Structure):
    _fields_ = [("q", _P), ("k", _P), ("v", _P), ("q_stride", _I64), ("k_stride", _I64), ("v_stride", _I64),
                ("T", _I32), ("n_heads", _I32), ("n_kv_heads", _I32), ("head_dim", _I32), ("q_weight", _P),
                ("k_weight", _P), ("eps", ctypes.c_float), ("interleaved", _I32), ("cos_sin", _P), ("max_pos", _I32),
                ("rope_dim", _I32), ("positions", _P), ("q_out", _P), ("k_out", _P), ("v_out", _P), ("slot_map", _P),
                ("rows", _P), ("n_rows", _I32), ("format", _I32), ("block_tokens", _I32), ("dev_status", _P),
                ("k_shift", _I32), ("v_shift", _I32)]


class c_block_attention_args(ctypes.Structure):
    _fields_ = [("q", _P), ("rows", _P), ("n_rows", _I32), ("format", _I32), ("block_tokens", _I32),
                ("head_dim", _I32), ("table", _P), ("sel", _P), ("table_heads", _I32), ("max_blocks", _I32),
                ("ctx_len", _P), ("B", _I32), ("n_q", _I32), ("n_heads", _I32), ("n_kv_heads", _I32),
                ("sinks", _I32), ("window", _I32), ("scale", ctypes.c_float), ("out", _P), ("lse", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t), ("dev_status", _P),
                ("k_shift", _I32), ("v_shift", _I32)]


class c_block_summary_args(ctypes.Structure):
    _fields_ = [("rows", _P), ("n_rows", _I32), ("format", _I32), ("block_tokens", _I32), ("head_dim", _I32),
                ("table", _P), ("table_heads", _I32), ("max_blocks", _I32), ("old_len", _P), ("new_len", _P),
                ("B", _I32), ("n_kv_heads", _I32), ("summary", _P), ("k_shift", _I32), ("dev_status", _P)]


class c_block_scores_args(ctypes.Structure):
    _fields_ = [("q", _P), ("summary", _P), ("n_rows", _I32), ("block_tokens", _I32), ("head_dim", _I32),
                ("table", _P), ("table_heads", _I32), ("max_blocks", _I32), ("ctx_len", _P), ("B", _I32),
                ("n_q", _I32), ("n_heads", _I32), ("n_kv_heads", _I32), ("scale", ctypes.c_float), ("scores", _P),
                ("dev_status", _P)]


class c_block_select_args(ctypes.Structure):
    _fields_ = [("scores", _P), ("ctx_len", _P), ("B", _I32), ("n_q", _I32), ("n_kv_heads", _I32),
                ("block_tokens", _I32), ("k", _I32), ("first", _I32), ("last", _I32), ("table", _P),
                ("table_heads", _I32), ("max_blocks", _I32), ("sel", _P), ("sel_rows", _P), ("len_out", _P),
                ("dev_status", _P), ("n_rows", _I32)]


class c_block_weights_args(ctypes.Structure):
    _fields_ = [("q", _P), ("rows", _P), ("n_rows", _I32), ("format", _I32), ("block_tokens", _I32),
                ("head_dim", _I32), ("table", _P), ("table_heads", _I32), ("max_blocks", _I32), ("ctx_len", _P),
                ("old_len", _P), ("B", _I32), ("n_q", _I32), ("n_heads", _I32), ("n_kv_heads", _I32),
                ("scale", ctypes.c_float), ("lse", _P), ("acc", _P), ("acc_out", _P), ("decay", ctypes.c_float),
                ("k_shift", _I32), ("dev_status", _P)]


class c_block_evict_args(ctypes.Structure):
    _fields_ = [("rows", _P), ("n_rows", _I32), ("format", _I32), ("block_tokens", _I32), ("head_dim", _I32),
                ("table", _P), ("table_heads", _I32), ("max_blocks", _I32), ("len", _P), ("len_out", _P), ("B", _I32),
                ("n_kv_heads", _I32), ("keep", _I32), ("sinks", _I32), ("recent", _I32), ("acc", _P), ("acc_out", _P),
                ("pos", _P), ("pos_out", _P), ("pos_len", _P), ("next_pos", _P), ("workspace", _P),
                ("workspace_bytes", ctypes.c_size_t), ("dev_status", _P)]


class c_prefix_attention_args(ctypes.Structure):
    _fields_ = [("q", _P), ("rows", _P), ("n_rows", _I32), ("format", _I32), ("block_tokens", _I32),
                ("head_dim", _I32), ("prefix_table", _P), ("prefix_len", _P), ("group_start", _P), ("n_groups", _I32),
                ("prefix_heads", _I32), ("max_prefix_blocks", _I32), ("table", _P), ("table_heads", _I32),
                ("max_blocks", _I32), ("ctx_len", _P), ("B", _I32), ("n_q", _I32), ("n_heads", _I32),
                ("n_kv_heads", _I32), ("scale", ctypes.c_float), ("out", _P), ("lse", _P), ("workspace", _P),
                ("workspace_bytes", ctypes.c_size_t), ("dev_status", _P), ("k_shift", _I32), ("v_shift", _I32)]


_lib = None


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load the built library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise EchoError(f"libecho_gb300 is not built ({path}); run __graft_entry__.build()")
    L = ctypes.CDLL(path)
    S = ctypes.c_int
    sig = {
        "echo_indexer_score": ([ctypes.POINTER(c_indexer_args), _P], S),
        "echo_select_topk": ([_P, _P, _I32, _I32, _I32, _I32, _P, _P, _P], S),
        "echo_workspace_bytes": ([_I32, _I32, ctypes.POINTER(ctypes.c_size_t)], S),
        "echo_selftest_wait_timeout": ([_I32, _P, _P], S),
        "echo_workspace_init": ([ctypes.POINTER(c_workspace), _P], S),
        "echo_pool_init": ([ctypes.POINTER(c_pool), _P], S),
        "echo_pool_alloc": ([ctypes.POINTER(c_pool), ctypes.POINTER(c_workspace), _P, _P, _I32, _I32, _P, _P, _P, _P], S),
        "echo_pool_evict": ([ctypes.POINTER(c_pool), ctypes.POINTER(c_workspace), _P, _I32, _P, _P, _P], S),
        "echo_prefetch_recall": ([ctypes.POINTER(c_pool), ctypes.POINTER(c_workspace), _P, _P, _P, _I32, _I32, _I32,
                                  _I32, ctypes.POINTER(c_stage), _I32, _P, _P, _P, _P, _P], S),
        "echo_append": ([ctypes.POINTER(c_pool), ctypes.POINTER(c_workspace), _P, _P, _P, _I32, _I32, _P, _P, _I32,
                         _P, _P, _P, _P], S),
        "echo_prefetch_recall_noalloc": ([ctypes.POINTER(c_pool), _P, _P, _P, _I32, _I32, _I32, _I32,
                                          ctypes.POINTER(c_stage), _I32, _P, _P, _P, _P, _P], S),
        "echo_ema_update": ([_P, _P, _I32, ctypes.c_float, _P], S),
        "echo_ema_update_strided": ([_P, _P, _I32, _I32, ctypes.c_float, _P], S),
        "echo_prefill_indexer_score": ([ctypes.POINTER(c_prefill_args), _P], S),
        "echo_mla_workspace_bytes": ([_I32, _I32, _I32, ctypes.POINTER(ctypes.c_size_t)], S),
        "echo_sparse_mla_decode": ([ctypes.POINTER(c_mla_args), _P], S),
        "echo_block_row_elems": ([_I32, _I32, _I32, ctypes.POINTER(_I32)], S),
        "echo_block_tables": ([ctypes.POINTER(c_block_tables_args), _P], S),
        "echo_qk_norm_rope": ([ctypes.POINTER(c_qk_norm_rope_args), _P], S),
        "echo_block_attention_workspace_bytes": ([_I32, _I32, ctypes.POINTER(ctypes.c_size_t)], S),
        "echo_block_attention": ([ctypes.POINTER(c_block_attention_args), _P], S),
        "echo_block_summary": ([ctypes.POINTER(c_block_summary_args), _P], S),
        "echo_block_scores": ([ctypes.POINTER(c_block_scores_args), _P], S),
        "echo_block_select": ([ctypes.POINTER(c_block_select_args), _P], S),
        "echo_block_weights": ([ctypes.POINTER(c_block_weights_args), _P], S),
        "echo_block_evict_workspace_bytes": ([_I32, _I32, _I32, ctypes.POINTER(ctypes.c_size_t)], S),
        "echo_block_evict": ([ctypes.POINTER(c_block_evict_args), _P], S),
        "echo_prefix_attention_workspace_bytes": ([_I32, _I32, _I32, _I32, _I32, ctypes.POINTER(ctypes.c_size_t)], S),
        "echo_prefix_attention": ([ctypes.POINTER(c_prefix_attention_args), _P], S),
        "echo_decode_step": ([ctypes.POINTER(c_step_args), _P], S),
        "echo_decode_step_host": ([ctypes.POINTER(c_step_args), _P, _P, _P, _I32], S),
        "echo_step_graph_create": ([ctypes.POINTER(c_step_args), ctypes.POINTER(_P)], S),
        "echo_step_graph_launch": ([_P, _P, _P, _P, _I32], S),
        "echo_step_graph_destroy": ([_P], S),
        "echo_pool_validate": ([ctypes.POINTER(c_pool), ctypes.POINTER(c_stage), _P, _P, _P], S),
        "echo_pool_validate_host": ([ctypes.POINTER(c_pool), _P, _I32, _P], S),
        "echo_last_error_string": ([], ctypes.c_char_p),
        "echo_version": ([], _I32),
        "echo_metadata_bytes": ([ctypes.c_int64, ctypes.c_int64], ctypes.c_int64),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def _check(rc: int, what: str):
    if rc != ECHO_OK:
        msg = load_library().echo_last_error_string().decode()
        raise EchoError(f"{what} failed (code {rc}): {msg}")


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_contiguous():
        raise EchoError("tensors passed to libecho_gb300 must be contiguous")
    return t.data_ptr()


def _dev(t: torch.Tensor | None, name: str):
    if t is not None and not t.is_cuda:
        raise EchoError(f"{name} must be a CUDA tensor")
    return _ptr(t)


def _current_stream_handle():
    return torch.cuda.current_stream().cuda_stream


try:  # the raw handle of the current stream without building a Stream object
    _raw_stream, _cur_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice

    def _current_stream_handle():  # noqa: F811
        return _raw_stream(_cur_device())
except AttributeError:
    pass


def _stream(stream):
    if stream is None:
        return _current_stream_handle()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ---------------------------------------------------------------------------
# holders
# ---------------------------------------------------------------------------

class Pool:
    """One layer's GPU pool plus a view of the (per-model) pinned host pool.  A row is
    host_kv's last dimension: 576 (MLA's latent row of one token) or, for the
    block-level / GQA variant, any multiple of 8 up to 65536 bf16 (a block of tokens
    of one KV head)."""

    def __init__(self, n_g: int, host_kv: torch.Tensor, device="cuda"):
        if host_kv.device.type != "cpu" or not host_kv.is_pinned():
            raise EchoError("host_kv must be a pinned CPU tensor")
        R = int(host_kv.shape[-1]) if host_kv.dim() == 2 else -1
        if host_kv.dtype not in (torch.int16, torch.uint16, torch.bfloat16) or R <= 0 or R % 8 or R > 65536:
            raise EchoError("host_kv must be [n_h][R] 16-bit with R a multiple of 8 up to 65536")
        self.n_g = int(n_g)
        self.n_h = int(host_kv.shape[0])
        self.row_elems = R
        self.host_kv = host_kv
        self.free = torch.empty(n_g, dtype=torch.uint8, device=device)
        self.prio = torch.empty(n_g, dtype=torch.int32, device=device)
        self.idxbuf = torch.empty(n_g, dtype=torch.int32, device=device)
        self.to_host = torch.empty(n_g, dtype=torch.int32, device=device)
        self.host_to_gpu = torch.empty(self.n_h, dtype=torch.int32, device=device)
        self.gpu_kv = torch.zeros((n_g, R), dtype=torch.int16, device=device)
        self.counters = torch.zeros(4, dtype=torch.int32, device=device)
        self.c = c_pool(self.n_g, self.n_h, _ptr(self.free), _ptr(self.prio), _ptr(self.idxbuf),
                        _ptr(self.to_host), _ptr(self.host_to_gpu), _ptr(self.gpu_kv), _ptr(host_kv),
                        _ptr(self.counters), R)

    def load_state(self, st, gpu_kv=None):
        """Install a workload.PoolState (metadata arrays + counters); gpu_kv defaults
        to the host rows of the occupied slots."""
        import numpy as np
        self.free.copy_(torch.from_numpy(st.gpu_token_free))
        self.prio.copy_(torch.from_numpy(st.gpu_token_priority))
        self.idxbuf.copy_(torch.from_numpy(st.gpu_indices_buffer))
        self.to_host.copy_(torch.from_numpy(st.gpu_token_to_host))
        self.host_to_gpu.copy_(torch.from_numpy(st.host_token_to_gpu))
        self.counters.copy_(torch.tensor([st.n_free, st.idx_count, 0, 0], dtype=torch.int32))
        if gpu_kv is None:
            occ = np.nonzero(st.gpu_token_free == 0)[0]
            kv = torch.zeros((self.n_g, self.row_elems), dtype=torch.int16)
            if occ.size:
                hk = self.host_kv.view(torch.int16)
                kv[torch.from_numpy(occ)] = hk[torch.from_numpy(st.gpu_token_to_host[occ].astype(np.int64))]
            self.gpu_kv.copy_(kv)
        else:
            self.gpu_kv.copy_(gpu_kv)

    def metadata(self):
        return dict(free=self.free.cpu().numpy(), prio=self.prio.cpu().numpy(), idxbuf=self.idxbuf.cpu().numpy(),
                    to_host=self.to_host.cpu().numpy(), host_to_gpu=self.host_to_gpu.cpu().numpy(),
                    n_free=int(self.counters[0]), idx_count=int(self.counters[1]))


class Workspace:
    def __init__(self, n_g: int, max_rows: int, device="cuda", stream=None):
        n = ctypes.c_size_t()
        _check(load_library().echo_workspace_bytes(n_g, max_rows, ctypes.byref(n)), "echo_workspace_bytes")
        self.buf = torch.empty(n.value + 256, dtype=torch.uint8, device=device)
        base = (self.buf.data_ptr() + 255) & ~255
        self.c = c_workspace(base, n.value, n_g, max_rows)
        _check(load_library().echo_workspace_init(ctypes.byref(self.c), _stream(stream)), "echo_workspace_init")


class Stage:
    """Where the prefetch puts rows: a staging area of `stride` rows per request, or,
    with reserve=R, straight into R GPU-pool slots each recall sets aside (direct to
    slot; the staging buffers are not allocated then).  while_scoring: the decode
    indexer drops candidates still queued when a CTA's scoring ends."""

    def __init__(self, B: int, stride: int = 1, cap_div: int = 16, device="cuda", reserve: int | None = None,
                 while_scoring: bool = False):
        self.direct = reserve is not None
        self.stride, self.cap_div = int(stride), int(cap_div)
        self.count = torch.zeros(B, dtype=torch.int32, device=device)
        if self.direct:
            self.rows = self.host_row = None
            self.reserve_cap = int(reserve)
            self.reserve = torch.full((max(self.reserve_cap, 1),), -1, dtype=torch.int32, device=device)
            self.reserve_ctl = torch.zeros(2, dtype=torch.int32, device=device)
            self.c = c_stage(None, None, _ptr(self.count), self.stride, self.cap_div, _ptr(self.reserve),
                             _ptr(self.reserve_ctl), self.reserve_cap, int(bool(while_scoring)))
        else:
            self.rows = torch.zeros((B, stride, KV_ELEMS), dtype=torch.int16, device=device)
            self.host_row = torch.full((B, stride), -1, dtype=torch.int32, device=device)
            self.reserve = self.reserve_ctl = None
            self.reserve_cap = 0
            self.c = c_stage(_ptr(self.rows), _ptr(self.host_row), _ptr(self.count), self.stride, self.cap_div,
                             None, None, 0, int(bool(while_scoring)))

    def set_reserve_cap(self, R: int):
        """Slots each recall sets aside from now on (at most the capacity allocated)."""
        if not self.direct or not 0 <= R <= self.reserve.numel():
            raise EchoError(f"reserve_cap {R} outside [0, {self.reserve.numel()}] or stage not direct")
        self.reserve_cap = int(R)
        self.c.reserve_cap = int(R)

    def reserved_slots(self):
        """The current reserve (direct to slot), as a numpy array."""
        n = int(self.reserve_ctl[1])
        return self.reserve[:n].cpu().numpy()


class Stats:
    def __init__(self, device="cuda"):
        self.t = torch.zeros(len(STAT_FIELDS), dtype=torch.int64, device=device)

    def as_dict(self):
        v = self.t.cpu().tolist()
        return dict(zip(STAT_FIELDS, v))


# ---------------------------------------------------------------------------
# C-ABI calls
# ---------------------------------------------------------------------------

def echo_indexer_score(q, w, k_index, ctx_len, scores, s_hat=None, req_to_host=None, pool: Pool | None = None,
                       stage: Stage | None = None, dev_status=None, stream=None):
    B, n_q = q.shape[0], q.shape[1]
    a = c_indexer_args(_dev(q, "q"), _dev(w, "w"), _dev(k_index, "k_index"), _dev(ctx_len, "ctx_len"), B, n_q,
                       k_index.shape[1], _dev(scores, "scores"), _dev(s_hat, "s_hat"),
                       _dev(req_to_host, "req_to_host"),
                       ctypes.pointer(pool.c) if pool is not None else None,
                       ctypes.pointer(stage.c) if stage is not None else None, _dev(dev_status, "dev_status"))
    _check(load_library().echo_indexer_score(ctypes.byref(a), _stream(stream)), "echo_indexer_score")


def echo_prefill_indexer_score(q, w, k_index, ctx_len, scores, s_shift=None, k: int = 0, thr_bin=None,
                               subset_n=None, req_to_host=None, pool: Pool | None = None,
                               stage: Stage | None = None, dev_status=None, stream=None):
    """q [B][C][64][128] e4m3: the chunk's C queries per request (see include/echo.h)."""
    B, C = q.shape[0], q.shape[1]
    a = c_prefill_args(_dev(q, "q"), _dev(w, "w"), _dev(k_index, "k_index"), _dev(ctx_len, "ctx_len"), B, C,
                       k_index.shape[1], _dev(scores, "scores"), _dev(s_shift, "s_shift"), int(k),
                       _dev(thr_bin, "thr_bin"), _dev(subset_n, "subset_n"), _dev(req_to_host, "req_to_host"),
                       ctypes.pointer(pool.c) if pool is not None else None,
                       ctypes.pointer(stage.c) if stage is not None else None, _dev(dev_status, "dev_status"))
    _check(load_library().echo_prefill_indexer_score(ctypes.byref(a), _stream(stream)),
           "echo_prefill_indexer_score")


def echo_select_topk(scores, ctx_len, k: int, sel, kth, stream=None):
    B, n_q, L_max = scores.shape
    _check(load_library().echo_select_topk(_dev(scores, "scores"), _dev(ctx_len, "ctx_len"), B, n_q, L_max, k,
                                           _dev(sel, "sel"), _dev(kth, "kth"), _stream(stream)), "echo_select_topk")


def echo_pool_init(pool: Pool, stream=None):
    _check(load_library().echo_pool_init(ctypes.byref(pool.c), _stream(stream)), "echo_pool_init")


def echo_pool_alloc(pool: Pool, ws: Workspace, host_idx, n_dev, clock: int, out_slots, dev_status=None,
                    clock_dev=None, stream=None):
    _check(load_library().echo_pool_alloc(ctypes.byref(pool.c), ctypes.byref(ws.c), _dev(host_idx, "host_idx"),
                                          _dev(n_dev, "n_dev"), int(host_idx.numel()), int(clock),
                                          _dev(clock_dev, "clock_dev"), _dev(out_slots, "out_slots"),
                                          _dev(dev_status, "dev_status"), _stream(stream)), "echo_pool_alloc")


def echo_pool_evict(pool: Pool, ws: Workspace, n_needed_dev, clock: int, dev_status=None, clock_dev=None,
                    stream=None):
    _check(load_library().echo_pool_evict(ctypes.byref(pool.c), ctypes.byref(ws.c), _dev(n_needed_dev, "n_needed"),
                                          int(clock), _dev(clock_dev, "clock_dev"), _dev(dev_status, "dev_status"),
                                          _stream(stream)), "echo_pool_evict")


def echo_prefetch_recall(pool: Pool, ws: Workspace, sel, req_to_host, ctx_len, clock: int, out_slot,
                         stage: Stage | None = None, stats: Stats | None = None, dev_status=None, clock_dev=None,
                         stream=None):
    B, n_q, k = sel.shape
    _check(load_library().echo_prefetch_recall(
        ctypes.byref(pool.c), ctypes.byref(ws.c), _dev(sel, "sel"), _dev(req_to_host, "req_to_host"),
        _dev(ctx_len, "ctx_len"), B, n_q, k, req_to_host.shape[1],
        ctypes.pointer(stage.c) if stage is not None else None, int(clock), _dev(clock_dev, "clock_dev"),
        _dev(out_slot, "out_slot"), _dev(stats.t, "stats") if stats is not None else None,
        _dev(dev_status, "dev_status"), _stream(stream)), "echo_prefetch_recall")


def echo_prefetch_recall_noalloc(pool: Pool, sel, req_to_host, ctx_len, clock: int, out_slot,
                                 stage: Stage | None = None, stats: Stats | None = None, dev_status=None,
                                 clock_dev=None, stream=None):
    """Guaranteed recall without a caller workspace (the library's own fixed scratch)."""
    B, n_q, k = sel.shape
    _check(load_library().echo_prefetch_recall_noalloc(
        ctypes.byref(pool.c), _dev(sel, "sel"), _dev(req_to_host, "req_to_host"), _dev(ctx_len, "ctx_len"), B, n_q,
        k, req_to_host.shape[1], ctypes.pointer(stage.c) if stage is not None else None, int(clock),
        _dev(clock_dev, "clock_dev"), _dev(out_slot, "out_slot"), _dev(stats.t, "stats") if stats is not None else None,
        _dev(dev_status, "dev_status"), _stream(stream)), "echo_prefetch_recall_noalloc")


def echo_selftest_wait_timeout(which: int, dev_status, stream=None):
    """A wait nothing satisfies gives up after a second and flags WAIT_TIMEOUT."""
    _check(load_library().echo_selftest_wait_timeout(int(which), _dev(dev_status, "dev_status"), _stream(stream)),
           "echo_selftest_wait_timeout")


def echo_append(pool: Pool, ws: Workspace, k_index, ctx_len, req_to_host, new_kv, new_k_index, clock: int,
                stats: Stats | None = None, dev_status=None, clock_dev=None, stream=None):
    B, L_max = k_index.shape[0], k_index.shape[1]
    _check(load_library().echo_append(
        ctypes.byref(pool.c), ctypes.byref(ws.c), _dev(k_index, "k_index"), _dev(ctx_len, "ctx_len"),
        _dev(req_to_host, "req_to_host"), B, L_max, _dev(new_kv, "new_kv"), _dev(new_k_index, "new_k_index"),
        int(clock), _dev(clock_dev, "clock_dev"), _dev(stats.t, "stats") if stats is not None else None,
        _dev(dev_status, "dev_status"), _stream(stream)), "echo_append")


def echo_ema_update(s_hat, kth, alpha: float = 0.5, stream=None):
    _check(load_library().echo_ema_update(_dev(s_hat, "s_hat"), _dev(kth, "kth"), int(s_hat.numel()),
                                          float(alpha), _stream(stream)), "echo_ema_update")


class MlaWorkspace:
    """Scratch of echo_sparse_mla_decode for B requests, n_q queries, k selected rows."""

    def __init__(self, B: int, n_q: int, k: int, device="cuda"):
        n = ctypes.c_size_t()
        _check(load_library().echo_mla_workspace_bytes(B, n_q, k, ctypes.byref(n)), "echo_mla_workspace_bytes")
        self.buf = torch.empty(n.value + 256, dtype=torch.uint8, device=device)
        self.base = (self.buf.data_ptr() + 255) & ~255
        self.bytes = n.value


def echo_sparse_mla_decode(q, gpu_kv, out_slot, scale: float, out, lse, ws: MlaWorkspace, dev_status=None,
                           stream=None):
    """q [B][n_q][128][576] bf16 (int16 bits), gpu_kv [n_g][576] (the pool's rows),
    out_slot [B][n_q][k]; out [B][n_q][128][512] fp32, lse [B][n_q][128] fp32."""
    B, n_q, k = out_slot.shape
    a = c_mla_args(_dev(q, "q"), _dev(gpu_kv, "gpu_kv"), int(gpu_kv.shape[0]), _dev(out_slot, "out_slot"), B, n_q,
                   k, float(scale), _dev(out, "out"), _dev(lse, "lse"), ws.base, ws.bytes,
                   _dev(dev_status, "dev_status"))
    _check(load_library().echo_sparse_mla_decode(ctypes.byref(a), _stream(stream)), "echo_sparse_mla_decode")


def echo_ema_update_strided(s_hat, kth, kth_stride: int, alpha: float = 0.5, stream=None):
    """s_hat[i] from kth[i * kth_stride] (kth a flat device tensor view)."""
    _check(load_library().echo_ema_update_strided(_dev(s_hat, "s_hat"), _dev(kth, "kth"), int(s_hat.numel()),
                                                  int(kth_stride), float(alpha), _stream(stream)),
           "echo_ema_update_strided")


# ---------------------------------------------------------------------------
# block rows (block-level / GQA): tables, norm + rotation into the cache, attention
# ---------------------------------------------------------------------------

def block_row_elems(fmt: int, block_tokens: int, head_dim: int) -> int:
    """16-bit elements of one block row (BLOCK_BF16 or BLOCK_FP4): the row length of a
    Pool whose rows the block calls read."""
    n = _I32()
    _check(load_library().echo_block_row_elems(fmt, block_tokens, head_dim, ctypes.byref(n)), "echo_block_row_elems")
    return n.value


def rope_table(max_pos: int, rope_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """cos_sin [max_pos][rope_dim] fp32 of echo_qk_norm_rope: rope_dim / 2 cosines, then the
    sines, of position * base^(-2i / rope_dim), angles in 64 bits."""
    inv = float(base) ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64) / rope_dim)
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float().to(device)


def _typed(t, name: str, dtypes, shape=None, contiguous: bool = True):
    """The pointer of an optional CUDA tensor on the current device, its type and shape
    checked (None in `shape`: any size)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise EchoError(f"{name} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        raise EchoError(f"{name} is on cuda:{t.device.index}, the current device is cuda:{torch.cuda.current_device()}")
    if t.dtype not in dtypes:
        raise EchoError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if shape is not None and (t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape))):
        raise EchoError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise EchoError(f"{name} must be contiguous")
    return t.data_ptr()


_BF16 = (torch.bfloat16, torch.int16)
_INT = (torch.int32,)
_F32 = (torch.float32,)


def make_block_tables_args(old_len, new_len, block_tokens: int, table, free_blocks, free_count, free_count_out,
                           slot_map, positions=None, cu_new=None, len_out=None,
                           dev_status=None) -> c_block_tables_args:
    """Arguments of echo_block_tables (see include/echo.h): built once, used step after step;
    keeps its tensors alive.  All int32: old_len, new_len, len_out [B], table
    [B][max_blocks], free_blocks [n_blocks], free_count, free_count_out [1], slot_map,
    positions [max_new], cu_new [B + 1]."""
    B = int(old_len.shape[0])
    a = c_block_tables_args()
    a.old_len, a.new_len = _typed(old_len, "old_len", _INT, (B,)), _typed(new_len, "new_len", _INT, (B,))
    a.B, a.block_tokens = B, int(block_tokens)
    a.table = _typed(table, "table", _INT, (B, None))
    a.free_blocks = _typed(free_blocks, "free_blocks", _INT, (None,))
    a.max_blocks, a.n_blocks = int(table.shape[1]), int(free_blocks.shape[0])
    a.free_count = _typed(free_count, "free_count", _INT, (1,))
    a.free_count_out = _typed(free_count_out, "free_count_out", _INT, (1,))
    a.slot_map, a.max_new = _typed(slot_map, "slot_map", _INT, (None,)), int(slot_map.shape[0])
    a.positions = _typed(positions, "positions", _INT, (a.max_new,))
    a.cu_new = _typed(cu_new, "cu_new", _INT, (B + 1,))
    a.len_out = _typed(len_out, "len_out", _INT, (B,))
    a.dev_status = _typed(dev_status, "dev_status", _INT)
    a._keep = (old_len, new_len, table, free_blocks, free_count, free_count_out, slot_map, positions, cu_new,
               len_out, dev_status)
    return a


def echo_block_tables(args: c_block_tables_args, stream=None):
    """Block tables, slot map and positions of a step from request lengths."""
    _check((_lib or load_library()).echo_block_tables(ctypes.byref(args), _stream(stream)), "echo_block_tables")


def _heads(t, name: str, T: int, H, D: int):
    """A [T][H][D] bf16 view whose heads are contiguous: its pointer and token stride."""
    if t is None:
        return None, 0
    p = _typed(t, name, _BF16, (T, H, D), contiguous=False)
    if T and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != D)):
        raise EchoError(f"{name} must have contiguous heads (strides (any, {D}, 1), got {t.stride()})")
    return p, (t.stride(0) if T > 1 else t.shape[1] * D)


def make_qk_norm_rope_args(q, k, v, positions, cos_sin, q_out, q_weight=None, k_weight=None, eps: float = 1e-6,
                           interleaved: bool = False, slot_map=None, rows=None, fmt: int = BLOCK_BF16,
                           block_tokens: int = 16, k_out=None, v_out=None, dev_status=None, k_shift: int = 0,
                           v_shift: int = 0) -> c_qk_norm_rope_args:
    """Arguments of echo_qk_norm_rope (see include/echo.h).  q [T][n_heads][D], k, v
    [T][n_kv_heads][D] bf16 (views of a fused projection: heads contiguous, any token
    stride); positions, slot_map [T] int32; cos_sin [max_pos][rope_dim] fp32; weights [D]
    fp32; rows [n_rows][R] 16-bit, device or pinned host; outputs contiguous.  4-bit rows hold
    keys * 2^k_shift and values * 2^v_shift: raise them where entries lie below about 0.1."""
    T, H, D = (int(n) for n in q.shape)
    Hk = int(k.shape[1])
    a = c_qk_norm_rope_args()
    (a.q, a.q_stride), (a.k, a.k_stride) = _heads(q, "q", T, H, D), _heads(k, "k", T, Hk, D)
    a.v, a.v_stride = _heads(v, "v", T, Hk, D)
    a.T, a.n_heads, a.n_kv_heads, a.head_dim = T, H, Hk, D
    a.q_weight, a.k_weight = _typed(q_weight, "q_weight", _F32, (D,)), _typed(k_weight, "k_weight", _F32, (D,))
    a.eps, a.interleaved = float(eps), int(bool(interleaved))
    a.cos_sin = _typed(cos_sin, "cos_sin", _F32, (None, None))
    a.max_pos, a.rope_dim = int(cos_sin.shape[0]), int(cos_sin.shape[1])
    a.positions = _typed(positions, "positions", _INT, (T,))
    a.q_out = _typed(q_out, "q_out", _BF16, (T, H, D))
    a.k_out, a.v_out = _typed(k_out, "k_out", _BF16, (T, Hk, D)), _typed(v_out, "v_out", _BF16, (T, Hk, D))
    a.format, a.block_tokens = int(fmt), int(block_tokens)
    if slot_map is not None:
        if rows is None or rows.dim() != 2 or rows.element_size() != 2 or not rows.is_contiguous():
            raise EchoError("a slot_map needs contiguous 16-bit rows [n_rows][R]")
        R = block_row_elems(a.format, a.block_tokens, D)
        if int(rows.shape[1]) != R:
            raise EchoError(f"rows have {rows.shape[1]} elements, blocks of {block_tokens} tokens need {R}")
        if not rows.is_cuda and not rows.is_pinned():
            raise EchoError("rows must be a CUDA tensor or pinned host memory")
        a.slot_map = _typed(slot_map, "slot_map", _INT, (T,))
        a.rows, a.n_rows = _typed(rows, "rows", (rows.dtype,)) if rows.is_cuda else rows.data_ptr(), int(rows.shape[0])
    a.dev_status, a.k_shift, a.v_shift = _typed(dev_status, "dev_status", _INT), int(k_shift), int(v_shift)
    a._keep = (q, k, v, positions, cos_sin, q_out, q_weight, k_weight, slot_map, rows, k_out, v_out, dev_status)
    return a


def echo_qk_norm_rope(args: c_qk_norm_rope_args, stream=None):
    """Per-head norm and rotation of q and k, k and v written to their cache rows."""
    _check((_lib or load_library()).echo_qk_norm_rope(ctypes.byref(args), _stream(stream)), "echo_qk_norm_rope")


class BlockAttentionWorkspace:
    """Scratch of echo_block_attention for n_q * n_heads / n_kv_heads query rows per KV head
    (any batch size and context length).  Serves calls that run one after another: two
    streams, or two graphs that may be replayed at once, need one each."""

    def __init__(self, rows_per_kv_head: int, head_dim: int, device="cuda"):
        n = ctypes.c_size_t()
        _check(load_library().echo_block_attention_workspace_bytes(rows_per_kv_head, head_dim, ctypes.byref(n)),
               "echo_block_attention_workspace_bytes")
        self.buf = torch.empty(n.value + 256, dtype=torch.uint8, device=device)
        self.base = (self.buf.data_ptr() + 255) & ~255
        self.bytes = n.value


def make_block_attention_args(q, rows, table, ctx_len, n_kv_heads: int, scale: float, out, lse,
                              ws: BlockAttentionWorkspace, fmt: int = BLOCK_BF16, block_tokens: int = 64, sel=None,
                              sinks: int = 0, window: int = 0, dev_status=None, k_shift: int = 0,
                              v_shift: int = 0) -> c_block_attention_args:
    """Arguments of echo_block_attention (see include/echo.h).  q, out [B][n_q][n_heads][D]
    bf16; rows [n_rows][R] 16-bit; table (and sel) int32 [B][max_blocks] of block ids shared
    by the KV heads, or [B][n_kv_heads][max_blocks] of rows; ctx_len [B] int32; lse
    [B][n_q][n_heads] fp32 or None; k_shift, v_shift as the (4-bit) rows were written."""
    B, n_q, H, D = (int(n) for n in q.shape)
    if rows.dim() != 2 or rows.element_size() != 2:
        raise EchoError("rows must be 16-bit [n_rows][R]")
    R = block_row_elems(fmt, block_tokens, D)
    if int(rows.shape[1]) != R:
        raise EchoError(f"rows have {rows.shape[1]} elements, blocks of {block_tokens} tokens need {R}")
    shape = (B, None) if table.dim() == 2 else (B, int(n_kv_heads), None)
    a = c_block_attention_args()
    a.q, a.rows = _typed(q, "q", _BF16, (B, n_q, H, D)), _typed(rows, "rows", (rows.dtype,))
    a.n_rows, a.format, a.block_tokens, a.head_dim = int(rows.shape[0]), int(fmt), int(block_tokens), D
    a.table = _typed(table, "table", _INT, shape)
    a.sel = _typed(sel, "sel", _INT, tuple(table.shape))
    a.table_heads, a.max_blocks = 1 if table.dim() == 2 else int(n_kv_heads), int(table.shape[-1])
    a.ctx_len = _typed(ctx_len, "ctx_len", _INT, (B,))
    a.B, a.n_q, a.n_heads, a.n_kv_heads = B, n_q, H, int(n_kv_heads)
    a.sinks, a.window, a.scale = int(sinks), int(window), float(scale)
    a.out = _typed(out, "out", _BF16, (B, n_q, H, D))
    a.lse = _typed(lse, "lse", _F32, (B, n_q, H))
    _typed(ws.buf, "workspace", (torch.uint8,))
    a.workspace, a.workspace_bytes = ws.base, ws.bytes
    a.dev_status, a.k_shift, a.v_shift = _typed(dev_status, "dev_status", _INT), int(k_shift), int(v_shift)
    a._keep = (q, rows, table, ctx_len, out, lse, ws, sel, dev_status)
    return a


def echo_block_attention(args: c_block_attention_args, stream=None):
    """Decode attention over block rows."""
    _check((_lib or load_library()).echo_block_attention(ctypes.byref(args), _stream(stream)), "echo_block_attention")


def _table_arg(a, table, B: int, n_kv_heads: int, name: str = "table"):
    """Sets table, table_heads and max_blocks: [B][max_blocks] ids or [B][n_kv_heads][max_blocks] rows."""
    a.table = _typed(table, name, _INT, (B, None) if table.dim() == 2 else (B, int(n_kv_heads), None))
    a.table_heads, a.max_blocks = 1 if table.dim() == 2 else int(n_kv_heads), int(table.shape[-1])


def _rows_arg(a, rows, fmt: int, block_tokens: int, head_dim: int):
    """Sets rows, n_rows, format, block_tokens and head_dim."""
    if rows.dim() != 2 or rows.element_size() != 2:
        raise EchoError("rows must be 16-bit [n_rows][R]")
    R = block_row_elems(fmt, block_tokens, head_dim)
    if int(rows.shape[1]) != R:
        raise EchoError(f"rows have {rows.shape[1]} elements, blocks of {block_tokens} tokens need {R}")
    a.rows, a.n_rows = _typed(rows, "rows", (rows.dtype,)), int(rows.shape[0])
    a.format, a.block_tokens, a.head_dim = int(fmt), int(block_tokens), int(head_dim)


def make_block_summary_args(rows, table, new_len, n_kv_heads: int, summary, old_len=None, fmt: int = BLOCK_BF16,
                            block_tokens: int = 64, k_shift: int = 0, dev_status=None) -> c_block_summary_args:
    """Arguments of echo_block_summary (see include/echo.h).  rows [n_rows][R] 16-bit; table int32
    [B][max_blocks] of block ids or [B][n_kv_heads][max_blocks] of rows; old_len, new_len [B]
    int32; summary [n_rows][2][D] bf16."""
    B = int(new_len.shape[0])
    a = c_block_summary_args()
    if summary.dim() != 3:
        raise EchoError("summary must be [n_rows][2][head_dim]")
    _rows_arg(a, rows, fmt, block_tokens, int(summary.shape[2]))
    _table_arg(a, table, B, n_kv_heads)
    a.old_len, a.new_len = _typed(old_len, "old_len", _INT, (B,)), _typed(new_len, "new_len", _INT, (B,))
    a.B, a.n_kv_heads = B, int(n_kv_heads)
    a.summary = _typed(summary, "summary", _BF16, (a.n_rows, 2, a.head_dim))
    a.k_shift, a.dev_status = int(k_shift), _typed(dev_status, "dev_status", _INT)
    a._keep = (rows, table, new_len, summary, old_len, dev_status)
    return a


def echo_block_summary(args: c_block_summary_args, stream=None):
    """Smallest and largest keys of the blocks that changed."""
    _check((_lib or load_library()).echo_block_summary(ctypes.byref(args), _stream(stream)), "echo_block_summary")


def make_block_scores_args(q, summary, table, ctx_len, n_kv_heads: int, scale: float, scores, block_tokens: int = 64,
                           dev_status=None) -> c_block_scores_args:
    """Arguments of echo_block_scores (see include/echo.h).  q [B][n_q][n_heads][D] bf16; summary
    [n_rows][2][D] bf16; table as above; ctx_len [B] int32; scores
    [B][n_q][n_kv_heads][max_blocks] fp32."""
    B, n_q, H, D = (int(n) for n in q.shape)
    a = c_block_scores_args()
    a.q, a.summary = _typed(q, "q", _BF16, (B, n_q, H, D)), _typed(summary, "summary", _BF16, (None, 2, D))
    a.n_rows, a.block_tokens, a.head_dim = int(summary.shape[0]), int(block_tokens), D
    _table_arg(a, table, B, n_kv_heads)
    a.ctx_len = _typed(ctx_len, "ctx_len", _INT, (B,))
    a.B, a.n_q, a.n_heads, a.n_kv_heads, a.scale = B, n_q, H, int(n_kv_heads), float(scale)
    a.scores = _typed(scores, "scores", _F32, (B, n_q, int(n_kv_heads), a.max_blocks))
    a.dev_status = _typed(dev_status, "dev_status", _INT)
    a._keep = (q, summary, table, ctx_len, scores, dev_status)
    return a


def echo_block_scores(args: c_block_scores_args, stream=None):
    """A bound on the scores that each query can have in each block."""
    _check((_lib or load_library()).echo_block_scores(ctypes.byref(args), _stream(stream)), "echo_block_scores")


def make_block_select_args(scores, ctx_len, sel, block_tokens: int = 64, first: int = 0, last: int = 0, table=None,
                           sel_rows=None, len_out=None, dev_status=None, n_rows: int = 0) -> c_block_select_args:
    """Arguments of echo_block_select (see include/echo.h).  scores [B][n_q][n_kv_heads][max_blocks]
    fp32; ctx_len [B], sel and sel_rows [B][n_q][n_kv_heads][k], len_out [B][n_q] int32; table as
    above or None; n_rows the cache's rows (0: not given), outside which no block is chosen."""
    B, n_q, Hk, n = (int(x) for x in scores.shape)
    a = c_block_select_args()
    a.scores, a.ctx_len = _typed(scores, "scores", _F32, (B, n_q, Hk, n)), _typed(ctx_len, "ctx_len", _INT, (B,))
    a.B, a.n_q, a.n_kv_heads, a.block_tokens = B, n_q, Hk, int(block_tokens)
    a.table, a.table_heads, a.max_blocks = None, 1, n
    if table is not None:
        _table_arg(a, table, B, Hk)
        if a.max_blocks != n:
            raise EchoError(f"table has {a.max_blocks} blocks, scores have {n}")
    a.sel = _typed(sel, "sel", _INT, (B, n_q, Hk, None))
    a.k, a.first, a.last = int(sel.shape[3]), int(first), int(last)
    a.sel_rows = _typed(sel_rows, "sel_rows", _INT, tuple(sel.shape))
    a.len_out = _typed(len_out, "len_out", _INT, (B, n_q))
    a.dev_status, a.n_rows = _typed(dev_status, "dev_status", _INT), int(n_rows)
    a._keep = (scores, ctx_len, sel, table, sel_rows, len_out, dev_status)
    return a


def echo_block_select(args: c_block_select_args, stream=None):
    """The k best blocks of each query token and KV head."""
    _check((_lib or load_library()).echo_block_select(ctypes.byref(args), _stream(stream)), "echo_block_select")


def make_block_weights_args(q, rows, table, ctx_len, n_kv_heads: int, scale: float, lse, acc, acc_out, old_len=None,
                            decay: float = 1.0, fmt: int = BLOCK_BF16, block_tokens: int = 64, k_shift: int = 0,
                            dev_status=None) -> c_block_weights_args:
    """Arguments of echo_block_weights (see include/echo.h).  q, rows, table, ctx_len as to
    make_block_attention_args, lse [B][n_q][n_heads] fp32 as it returned it; acc (or None) and
    acc_out [B][n_kv_heads][max_blocks * block_tokens] fp32; old_len [B] int32 or None."""
    B, n_q, H, D = (int(n) for n in q.shape)
    a = c_block_weights_args()
    a.q = _typed(q, "q", _BF16, (B, n_q, H, D))
    _rows_arg(a, rows, fmt, block_tokens, D)
    _table_arg(a, table, B, n_kv_heads)
    a.ctx_len, a.old_len = _typed(ctx_len, "ctx_len", _INT, (B,)), _typed(old_len, "old_len", _INT, (B,))
    a.B, a.n_q, a.n_heads, a.n_kv_heads, a.scale = B, n_q, H, int(n_kv_heads), float(scale)
    shape = (B, int(n_kv_heads), a.max_blocks * a.block_tokens)
    a.lse, a.acc = _typed(lse, "lse", _F32, (B, n_q, H)), _typed(acc, "acc", _F32, shape)
    a.acc_out, a.decay = _typed(acc_out, "acc_out", _F32, shape), float(decay)
    a.k_shift, a.dev_status = int(k_shift), _typed(dev_status, "dev_status", _INT)
    a._keep = (q, rows, table, ctx_len, lse, acc, acc_out, old_len, dev_status)
    return a


def echo_block_weights(args: c_block_weights_args, stream=None):
    """The softmax weight that cached tokens gather."""
    _check((_lib or load_library()).echo_block_weights(ctypes.byref(args), _stream(stream)), "echo_block_weights")


class BlockEvictWorkspace:
    """Scratch of echo_block_evict for B requests.  Serves calls that run one after another: two
    streams, or two graphs that may be replayed at once, need one each."""

    def __init__(self, B: int, n_kv_heads: int, keep: int, device="cuda"):
        n = ctypes.c_size_t()
        _check(load_library().echo_block_evict_workspace_bytes(B, n_kv_heads, keep, ctypes.byref(n)),
               "echo_block_evict_workspace_bytes")
        self.buf = torch.empty(n.value + 256, dtype=torch.uint8, device=device)
        self.base = (self.buf.data_ptr() + 255) & ~255
        self.bytes = n.value


def make_block_evict_args(rows, table, length, len_out, n_kv_heads: int, keep: int, acc, acc_out,
                          ws: BlockEvictWorkspace, sinks: int = 0, recent: int = 0, pos=None, pos_out=None, pos_len=None,
                          next_pos=None, fmt: int = BLOCK_BF16, block_tokens: int = 64,
                          dev_status=None) -> c_block_evict_args:
    """Arguments of echo_block_evict (see include/echo.h).  length, len_out, pos_len, next_pos [B]
    int32; acc, acc_out fp32 and pos, pos_out int32 [B][n_kv_heads][max_blocks * block_tokens]."""
    B = int(length.shape[0])
    a = c_block_evict_args()
    R, bs = int(rows.shape[-1]), int(block_tokens)
    D = R * 16 // (9 * bs) if fmt == BLOCK_FP4 and bs > 0 else R // (2 * bs) if bs > 0 else 0
    _rows_arg(a, rows, fmt, block_tokens, D)
    _table_arg(a, table, B, n_kv_heads)
    a.len, a.len_out = _typed(length, "length", _INT, (B,)), _typed(len_out, "len_out", _INT, (B,))
    a.B, a.n_kv_heads, a.keep, a.sinks, a.recent = B, int(n_kv_heads), int(keep), int(sinks), int(recent)
    shape = (B, int(n_kv_heads), a.max_blocks * a.block_tokens)
    a.acc, a.acc_out = _typed(acc, "acc", _F32, shape), _typed(acc_out, "acc_out", _F32, shape)
    a.pos, a.pos_out = _typed(pos, "pos", _INT, shape), _typed(pos_out, "pos_out", _INT, shape)
    a.pos_len, a.next_pos = _typed(pos_len, "pos_len", _INT, (B,)), _typed(next_pos, "next_pos", _INT, (B,))
    _typed(ws.buf, "workspace", (torch.uint8,))
    a.workspace, a.workspace_bytes, a.dev_status = ws.base, ws.bytes, _typed(dev_status, "dev_status", _INT)
    a._keep = (rows, table, length, len_out, acc, acc_out, ws, pos, pos_out, pos_len, next_pos, dev_status)
    return a


def echo_block_evict(args: c_block_evict_args, stream=None):
    """Requests cut to the tokens that gathered the most weight."""
    _check((_lib or load_library()).echo_block_evict(ctypes.byref(args), _stream(stream)), "echo_block_evict")


class PrefixAttentionWorkspace:
    """Scratch of echo_prefix_attention for B requests (any prefixes and contexts).  Serves calls
    that run one after another: two streams, or two graphs that may be replayed at once, need one
    each."""

    def __init__(self, B: int, n_q: int, n_heads: int, n_kv_heads: int, head_dim: int, device="cuda"):
        n = ctypes.c_size_t()
        _check(load_library().echo_prefix_attention_workspace_bytes(B, n_q, n_heads, n_kv_heads, head_dim,
                                                                    ctypes.byref(n)),
               "echo_prefix_attention_workspace_bytes")
        self.buf = torch.empty(n.value + 256, dtype=torch.uint8, device=device)
        self.base = (self.buf.data_ptr() + 255) & ~255
        self.bytes = n.value


def make_prefix_attention_args(q, rows, prefix_table, prefix_len, group_start, table, ctx_len, n_kv_heads: int,
                               scale: float, out, lse, ws: PrefixAttentionWorkspace, fmt: int = BLOCK_BF16,
                               block_tokens: int = 64, dev_status=None, k_shift: int = 0,
                               v_shift: int = 0) -> c_prefix_attention_args:
    """Arguments of echo_prefix_attention (see include/echo.h).  q, rows, table, ctx_len, out and lse
    as to make_block_attention_args (table and ctx_len None: no own tokens); prefix_table int32
    [n_groups][max_prefix_blocks] of block ids or [n_groups][n_kv_heads][max_prefix_blocks] of
    rows; prefix_len [n_groups], group_start [n_groups + 1] int32."""
    B, n_q, H, D = (int(n) for n in q.shape)
    a = c_prefix_attention_args()
    a.q = _typed(q, "q", _BF16, (B, n_q, H, D))
    _rows_arg(a, rows, fmt, block_tokens, D)
    G = int(prefix_len.shape[0])
    shape = (G, None) if prefix_table.dim() == 2 else (G, int(n_kv_heads), None)
    a.prefix_table = _typed(prefix_table, "prefix_table", _INT, shape)
    a.prefix_len = _typed(prefix_len, "prefix_len", _INT, (G,))
    a.group_start = _typed(group_start, "group_start", _INT, (G + 1,))
    a.n_groups, a.max_prefix_blocks = G, int(prefix_table.shape[-1])
    a.prefix_heads = 1 if prefix_table.dim() == 2 else int(n_kv_heads)
    a.table, a.table_heads, a.max_blocks = None, 1, 1
    if table is not None:
        _table_arg(a, table, B, n_kv_heads)
    a.ctx_len = _typed(ctx_len, "ctx_len", _INT, (B,))
    a.B, a.n_q, a.n_heads, a.n_kv_heads, a.scale = B, n_q, H, int(n_kv_heads), float(scale)
    a.out, a.lse = _typed(out, "out", _BF16, (B, n_q, H, D)), _typed(lse, "lse", _F32, (B, n_q, H))
    _typed(ws.buf, "workspace", (torch.uint8,))
    a.workspace, a.workspace_bytes = ws.base, ws.bytes
    a.dev_status, a.k_shift, a.v_shift = _typed(dev_status, "dev_status", _INT), int(k_shift), int(v_shift)
    a._keep = (q, rows, prefix_table, prefix_len, group_start, table, ctx_len, out, lse, ws, dev_status)
    return a


def echo_prefix_attention(args: c_prefix_attention_args, stream=None):
    """Decode attention of requests that share a prefix."""
    _check((_lib or load_library()).echo_prefix_attention(ctypes.byref(args), _stream(stream)), "echo_prefix_attention")


class StepBuffers:
    """Device outputs of one decode step for B requests, n_q queries, k."""

    def __init__(self, B: int, n_q: int, L_max: int, k: int, device="cuda"):
        # entries past each row's context are never written: NaN marks them
        self.scores = torch.full((B, n_q, L_max), float("nan"), dtype=torch.float32, device=device)
        self.sel = torch.empty((B, n_q, k), dtype=torch.int32, device=device)
        self.kth = torch.empty((B, n_q), dtype=torch.float32, device=device)
        self.out_slot = torch.empty((B, n_q, k), dtype=torch.int32, device=device)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=device)


def make_step_args(pool: Pool, ws: Workspace, q, w, k_index, ctx_len, req_to_host, k: int, out: StepBuffers,
                   stage: Stage | None = None, s_hat=None, alpha: float = 0.5, new_kv=None, new_k_index=None,
                   clock: int = 0, clock_dev=None, advance_clock: bool = False, stats: Stats | None = None,
                   events=None) -> c_step_args:
    """Build the C struct once (e.g. before graph capture); keep the returned object
    alive while it is in use."""
    B, n_q = q.shape[0], q.shape[1]
    a = c_step_args()
    a.pool = ctypes.pointer(pool.c)
    a.ws = ctypes.pointer(ws.c)
    a.stage = ctypes.pointer(stage.c) if stage is not None else None
    a.q, a.w, a.k_index = _dev(q, "q"), _dev(w, "w"), _dev(k_index, "k_index")
    a.ctx_len, a.req_to_host = _dev(ctx_len, "ctx_len"), _dev(req_to_host, "req_to_host")
    a.B, a.n_q, a.L_max, a.k = B, n_q, k_index.shape[1], int(k)
    a.scores, a.sel, a.kth, a.out_slot = _ptr(out.scores), _ptr(out.sel), _ptr(out.kth), _ptr(out.out_slot)
    a.s_hat = _dev(s_hat, "s_hat")
    a.alpha = float(alpha)
    a.new_kv, a.new_k_index = _dev(new_kv, "new_kv"), _dev(new_k_index, "new_k_index")
    a.clock = int(clock)
    a.clock_dev = _dev(clock_dev, "clock_dev")
    a.advance_clock = 1 if advance_clock else 0
    a.stats = _dev(stats.t, "stats") if stats is not None else None
    a.dev_status = _ptr(out.dev_status)
    if events is not None:
        arr = (_P * (NUM_STAGES + 1))(*[e.cuda_event for e in events])
        a._events_keepalive = arr
        a.stage_events = arr
    # keep the referenced holders alive with the struct
    a._keep = (pool, ws, stage, q, w, k_index, ctx_len, req_to_host, out, s_hat, new_kv, new_k_index, clock_dev,
               stats)
    return a


def echo_pool_validate(pool: Pool, report, dev_status, stage: Stage | None = None, stream=None):
    """Metadata invariants on the device: report [len(VAL_FIELDS)] int32 (device) gets the
    counts, DEV_INVARIANT is OR-ed into dev_status when one is broken."""
    _check(load_library().echo_pool_validate(ctypes.byref(pool.c), ctypes.pointer(stage.c) if stage is not None
                                             else None, _dev(report, "report"), _dev(dev_status, "dev_status"),
                                             _stream(stream)), "echo_pool_validate")


def echo_pool_validate_host(free, prio, to_host, host_to_gpu, n_free: int, reserve=None):
    """The same invariants over host copies (numpy arrays: free uint8 [n_g], prio /
    to_host int32 [n_g], host_to_gpu int32 [n_h]).  Returns (violation found, counts)."""
    import numpy as np
    arrs = [np.ascontiguousarray(free, np.uint8), np.ascontiguousarray(prio, np.int32),
            np.ascontiguousarray(to_host, np.int32), np.ascontiguousarray(host_to_gpu, np.int32)]
    counters = np.array([n_free, 0, 0, 0], np.int32)
    idx = np.full(arrs[0].size, -1, np.int32)
    res = None if reserve is None else np.ascontiguousarray(reserve, np.int32)
    report = np.zeros(len(VAL_FIELDS), np.int32)
    ptr = lambda a: a.ctypes.data if a is not None and a.size else None
    c = c_pool(arrs[0].size, arrs[3].size, ptr(arrs[0]), ptr(arrs[1]), ptr(idx), ptr(arrs[2]), ptr(arrs[3]),
               None, None, ptr(counters), 0)
    rc = load_library().echo_pool_validate_host(ctypes.byref(c), ptr(res), 0 if res is None else res.size,
                                                ptr(report))
    if rc < 0:
        _check(-rc, "echo_pool_validate_host")
    return rc == DEV_INVARIANT, dict(zip(VAL_FIELDS, report.tolist()))


def echo_decode_step(args: c_step_args, stream=None):
    _check((_lib or load_library()).echo_decode_step(ctypes.byref(args), _stream(stream)), "echo_decode_step")


def _host_inputs(q_host, w_host):
    for t, name in ((q_host, "q_host"), (w_host, "w_host")):
        if t.is_cuda or not t.is_contiguous():
            raise EchoError(f"{name} must be a contiguous host tensor")
    return q_host.data_ptr(), w_host.data_ptr()


def echo_decode_step_host(args: c_step_args, q_host, w_host, stream=None, wait: bool = True):
    """One decode step whose q and w come from host tensors (pinned for an asynchronous
    copy) laid out as the step's device q and w; wait: return after the step is done."""
    qp, wp = _host_inputs(q_host, w_host)
    _check((_lib or load_library()).echo_decode_step_host(ctypes.byref(args), qp, wp, _stream(stream),
                                                          1 if wait else 0), "echo_decode_step_host")


class StepGraph:
    """A decode step captured into a CUDA graph by the library (echo_step_graph_*).
    The step's arguments (and every buffer they name) are kept alive with it."""

    def __init__(self, args: c_step_args):
        h = _P()
        _check(load_library().echo_step_graph_create(ctypes.byref(args), ctypes.byref(h)), "echo_step_graph_create")
        self._h, self._args = h, args

    def launch(self, q_host=None, w_host=None, stream=None, wait: bool = True):
        qp, wp = _host_inputs(q_host, w_host) if q_host is not None else (None, None)
        _check(_lib.echo_step_graph_launch(self._h, qp, wp, _stream(stream), 1 if wait else 0),
               "echo_step_graph_launch")

    def close(self):
        if self._h:
            _check(_lib.echo_step_graph_destroy(self._h), "echo_step_graph_destroy")
            self._h = _P()

    def __del__(self):
        try:
            if self._h and _lib is not None:
                _lib.echo_step_graph_destroy(self._h)
        except Exception:
            pass


def version() -> int:
    return int(load_library().echo_version())
