"""ctypes binding of libs3r (include/s3r.h): argument marshalling only.

Each function has the name of the C entry point it calls and takes torch
tensors (device memory) or raw device addresses; every step of the computation
runs in the library's CUDA kernels. A non-OK status raises S3RError. The
library must have been built (``python -m self_sparse_speculative_b200.build``);
if it is missing, importing this module raises ImportError - there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libs3r.so")

S3R_OK, S3R_ERR_INVALID_ARG, S3R_ERR_UNSUPPORTED, S3R_ERR_WORKSPACE, S3R_ERR_CUDA, S3R_ERR_DEVICE_CHECK = range(6)
S3R_F32, S3R_BF16 = 0, 1
S3R_DEV_BAD_CONTEXT_LEN, S3R_DEV_BAD_PAGE_ID, S3R_DEV_BAD_TOKEN_ID, S3R_DEV_WAIT_TIMEOUT = 0x1, 0x2, 0x4, 0x8
S3R_DEV_BAD_TREE = 0x10

EXPORTED = [
    "s3r_page_summaries", "s3r_page_summaries_checked", "s3r_sparse_draft_attn", "s3r_verify_attn",
    "s3r_spec_sample", "s3r_spec_sample_noalloc", "s3r_sample_tokens", "s3r_attn_workspace_bytes", "s3r_sample_workspace_bytes",
    "s3r_device_status", "s3r_status_str", "s3r_version", "s3r_sparse_draft_kernels",
    "s3r_sample_tokens_ex", "s3r_spec_sample_ex", "s3r_kv_append", "s3r_kv_rollback", "s3r_kv_workspace_bytes",
    "s3r_debug_exp64", "s3r_gamma_policy_init", "s3r_gamma_policy_update", "s3r_gamma_policy_choose",
    "s3r_attend_cost_us", "s3r_round_cost_us", "s3r_verify_attn_tree", "s3r_tree_spec_sample",
    "s3r_tree_sample_workspace_bytes", "s3r_tree_node_budget",
    "s3r_kvq_page_bytes", "s3r_kvq_append", "s3r_kvq_pack", "s3r_kvq_read", "s3r_kvq_rollback",
    "s3r_kvq_attn_workspace_bytes", "s3r_kvq_attn",
]


class S3RError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_str(status)}")


class GammaPolicy(ctypes.Structure):
    _fields_ = [("gamma_max", ctypes.c_int32), ("decay", ctypes.c_double), ("accepted", ctypes.c_double),
                ("tested", ctypes.c_double), ("cost_us", ctypes.c_double * 17)]


class PagedKV(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32), ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
        ("num_pages_total", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("context_lens", ctypes.c_void_p),
    ]


class PagedKVQ(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32), ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
        ("num_pages_total", ctypes.c_int32), ("bits", ctypes.c_int32),
        ("pages", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("context_lens", ctypes.c_void_p),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libs3r.so is not built ({LIB_PATH}); run python -m self_sparse_speculative_b200.build")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, f32, sz, f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t, ctypes.c_double
    kvp, kqp = ctypes.POINTER(PagedKV), ctypes.POINTER(PagedKVQ)
    sig = {
        "s3r_page_summaries": ([kvp, i32, vp, vp, vp], i32),
        "s3r_page_summaries_checked": ([kvp, i32, vp, vp, vp, vp], i32),
        "s3r_sparse_draft_attn": ([kvp, vp, vp, vp, i32, f32, vp, vp, vp, vp, sz, vp], i32),
        "s3r_verify_attn": ([kvp, vp, i32, f32, vp, vp, vp, sz, vp], i32),
        "s3r_spec_sample": ([vp, vp, i32, vp, vp, vp, i32, i32, i32, f32, vp, vp, vp, sz, vp], i32),
        "s3r_spec_sample_noalloc": ([vp, vp, i32, vp, vp, vp, i32, i32, i32, f32, vp, vp, vp], i32),
        "s3r_sample_tokens": ([vp, i32, i32, i32, f32, vp, vp, vp, sz, vp], i32),
        "s3r_sample_tokens_ex": ([vp, i32, i32, i32, f32, vp, vp, vp, vp, sz, vp], i32),
        "s3r_spec_sample_ex": ([vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, f32, vp, vp, vp, sz, vp], i32),
        "s3r_kv_append": ([kvp, vp, vp, vp, i32, i32, vp, vp, vp, sz, vp], i32),
        "s3r_kv_rollback": ([kvp, vp, vp, i32, vp, vp, vp, sz, vp], i32),
        "s3r_kv_workspace_bytes": ([i32], sz),
        "s3r_debug_exp64": ([vp, vp, vp, i32, vp], i32),
        "s3r_gamma_policy_init": ([ctypes.POINTER(GammaPolicy), i32, f64, f64, f64, ctypes.POINTER(f64)], i32),
        "s3r_gamma_policy_update": ([ctypes.POINTER(GammaPolicy), ctypes.POINTER(i32), i32, i32], i32),
        "s3r_gamma_policy_choose": ([ctypes.POINTER(GammaPolicy), ctypes.POINTER(i32), ctypes.POINTER(f64),
                                     ctypes.POINTER(f64)], i32),
        "s3r_attend_cost_us": ([i32, i32, i32, i32, i32, f64, i32, f64, f64], f64),
        "s3r_round_cost_us": ([i32, i32, i32, i32, i32, i32, f64, i32, i32, i32, i32, f64, f64], f64),
        "s3r_attn_workspace_bytes": ([kvp, i32, i32], sz),
        "s3r_sample_workspace_bytes": ([i32, i32, i32], sz),
        "s3r_device_status": ([vp, ctypes.POINTER(ctypes.c_uint32), vp], i32),
        "s3r_status_str": ([i32], ctypes.c_char_p),
        "s3r_sparse_draft_kernels": ([kvp, i32], i32),
        "s3r_version": ([], i32),
        "s3r_verify_attn_tree": ([kvp, vp, i32, vp, f32, vp, vp, vp, sz, vp], i32),
        "s3r_tree_sample_workspace_bytes": ([i32, i32, i32], sz),
        "s3r_tree_spec_sample": ([vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, f32, vp, vp, vp, vp, sz, vp], i32),
        "s3r_tree_node_budget": ([ctypes.c_int64, i32, i32, i32], i32),
        "s3r_kvq_page_bytes": ([i32, i32, i32], sz),
        "s3r_kvq_append": ([kqp, vp, vp, vp, i32, i32, i32, vp, sz, vp], i32),
        "s3r_kvq_pack": ([kvp, kqp, i32, vp, sz, vp], i32),
        "s3r_kvq_read": ([kqp, vp, i32, i32, vp, vp, vp, sz, vp], i32),
        "s3r_kvq_rollback": ([kqp, vp, vp, i32, vp, sz, vp], i32),
        "s3r_kvq_attn_workspace_bytes": ([kqp, i32, i32, i32], sz),
        "s3r_kvq_attn": ([kqp, vp, i32, i32, vp, i32, f32, vp, vp, vp, sz, vp], i32),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


_lib = _load()


def lib():
    return _lib


def status_str(status: int) -> str:
    return _lib.s3r_status_str(int(status)).decode()


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, st):
    if st != S3R_OK:
        raise S3RError(fn, st)


def dtype_code(dt) -> int:
    import torch
    if dt in (torch.bfloat16, "bf16", S3R_BF16):
        return S3R_BF16
    if dt in (torch.float32, "f32", S3R_F32):
        return S3R_F32
    raise ValueError(f"unsupported dtype {dt}")


def paged_kv(k_cache, v_cache, block_table, context_lens, num_q_heads: int) -> PagedKV:
    """Describe a cache [num_pages_total, Hkv, P, D] with its block table."""
    n, h, p, d = k_cache.shape
    kv = PagedKV(int(block_table.shape[0]), int(num_q_heads), int(h), int(d), int(p),
                 int(block_table.shape[1]), int(n), dtype_code(k_cache.dtype),
                 _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(context_lens))
    kv.devices = {x.get_device() for x in (k_cache, v_cache, block_table, context_lens) if hasattr(x, "get_device")}
    return kv


def s3r_attn_workspace_bytes(kv: PagedKV, rows: int, budget_pages: int) -> int:
    return int(_lib.s3r_attn_workspace_bytes(ctypes.byref(kv), rows, budget_pages))


def s3r_sample_workspace_bytes(num_seqs: int, gamma: int, vocab: int) -> int:
    return int(_lib.s3r_sample_workspace_bytes(num_seqs, gamma, vocab))


def s3r_page_summaries(kv: PagedKV, tail_only: int, kmin, kmax, stream=None, status_word=None):
    if status_word is None:
        st = _lib.s3r_page_summaries(ctypes.byref(kv), int(tail_only), _ptr(kmin), _ptr(kmax), _stream(stream))
    else:
        st = _lib.s3r_page_summaries_checked(ctypes.byref(kv), int(tail_only), _ptr(kmin), _ptr(kmax),
                                             _ptr(status_word), _stream(stream))
    _check("s3r_page_summaries", st)


def s3r_sparse_draft_attn(kv: PagedKV, kmin, kmax, q, budget_pages: int, scale: float, selected, out,
                          lse, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = _lib.s3r_sparse_draft_attn(ctypes.byref(kv), _ptr(kmin), _ptr(kmax), _ptr(q), int(budget_pages),
                                    float(scale), _ptr(selected), _ptr(out), _ptr(lse), _ptr(workspace), wb,
                                    _stream(stream))
    _check("s3r_sparse_draft_attn", st)


def s3r_verify_attn(kv: PagedKV, q, rows: int, scale: float, out, lse, workspace, workspace_bytes=None,
                    stream=None):
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = _lib.s3r_verify_attn(ctypes.byref(kv), _ptr(q), int(rows), float(scale), _ptr(out), _ptr(lse),
                              _ptr(workspace), wb, _stream(stream))
    _check("s3r_verify_attn", st)


def s3r_verify_attn_tree(kv: PagedKV, q, nodes: int, parents, scale: float, out, lse, workspace,
                         workspace_bytes=None, stream=None):
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = _lib.s3r_verify_attn_tree(ctypes.byref(kv), _ptr(q), int(nodes), _ptr(parents), float(scale), _ptr(out),
                                   _ptr(lse), _ptr(workspace), wb, _stream(stream))
    _check("s3r_verify_attn_tree", st)


def s3r_tree_sample_workspace_bytes(num_seqs: int, nodes: int, vocab: int) -> int:
    return int(_lib.s3r_tree_sample_workspace_bytes(num_seqs, nodes, vocab))


def s3r_tree_spec_sample(target_logits, draft_logits, logit_dtype, tokens, parents, u_accept, u_sample,
                         num_seqs: int, nodes: int, vocab: int, temperature: float, out_tokens, num_accepted,
                         path, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = _lib.s3r_tree_spec_sample(_ptr(target_logits), _ptr(draft_logits), dtype_code(logit_dtype), _ptr(tokens),
                                   _ptr(parents), _ptr(u_accept), _ptr(u_sample), int(num_seqs), int(nodes),
                                   int(vocab), float(temperature), _ptr(out_tokens), _ptr(num_accepted), _ptr(path),
                                   _ptr(workspace), wb, _stream(stream))
    _check("s3r_tree_spec_sample", st)


def s3r_tree_node_budget(capacity: int, active: int, n_min: int, n_max: int) -> int:
    """N_t = clip(floor(capacity / active), n_min, n_max); -1 for bad arguments."""
    return int(_lib.s3r_tree_node_budget(int(capacity), int(active), int(n_min), int(n_max)))


def s3r_spec_sample(target_logits, draft_logits, logit_dtype, draft_tokens, u_accept, u_sample,
                    num_seqs: int, gamma: int, vocab: int, temperature: float, out_tokens, num_accepted,
                    workspace, workspace_bytes=None, stream=None, draft_stats=None):
    """draft_stats (float64 [S, gamma, 2] from s3r_sample_tokens(..., row_stats=...)) selects
    s3r_spec_sample_ex."""
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    if draft_stats is None:
        st = _lib.s3r_spec_sample(_ptr(target_logits), _ptr(draft_logits), dtype_code(logit_dtype),
                                  _ptr(draft_tokens), _ptr(u_accept), _ptr(u_sample), int(num_seqs), int(gamma),
                                  int(vocab), float(temperature), _ptr(out_tokens), _ptr(num_accepted),
                                  _ptr(workspace), wb, _stream(stream))
        _check("s3r_spec_sample", st)
        return
    st = _lib.s3r_spec_sample_ex(_ptr(target_logits), _ptr(draft_logits), dtype_code(logit_dtype),
                                 _ptr(draft_tokens), _ptr(u_accept), _ptr(u_sample), _ptr(draft_stats),
                                 int(num_seqs), int(gamma), int(vocab), float(temperature), _ptr(out_tokens),
                                 _ptr(num_accepted), _ptr(workspace), wb, _stream(stream))
    _check("s3r_spec_sample_ex", st)


def s3r_spec_sample_noalloc(target_logits, draft_logits, logit_dtype, draft_tokens, u_accept, u_sample,
                            num_seqs: int, gamma: int, vocab: int, temperature: float, out_tokens,
                            num_accepted, stream=None):
    """s3r_spec_sample with the library's own static device scratch instead of a workspace
    (for callers that cannot allocate device memory; calls must not overlap on the GPU)."""
    st = _lib.s3r_spec_sample_noalloc(_ptr(target_logits), _ptr(draft_logits), dtype_code(logit_dtype),
                                      _ptr(draft_tokens), _ptr(u_accept), _ptr(u_sample), int(num_seqs),
                                      int(gamma), int(vocab), float(temperature), _ptr(out_tokens),
                                      _ptr(num_accepted), _stream(stream))
    _check("s3r_spec_sample_noalloc", st)


def s3r_sample_tokens(logits, logit_dtype, num_rows: int, vocab: int, temperature: float, u, tokens,
                      workspace, workspace_bytes=None, stream=None, row_stats=None):
    """row_stats (float64 [num_rows, 2]) selects s3r_sample_tokens_ex, which also writes each
    row's {max, exact Z}."""
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    if row_stats is None:
        st = _lib.s3r_sample_tokens(_ptr(logits), dtype_code(logit_dtype), int(num_rows), int(vocab),
                                    float(temperature), _ptr(u), _ptr(tokens), _ptr(workspace), wb,
                                    _stream(stream))
        _check("s3r_sample_tokens", st)
        return
    st = _lib.s3r_sample_tokens_ex(_ptr(logits), dtype_code(logit_dtype), int(num_rows), int(vocab),
                                   float(temperature), _ptr(u), _ptr(tokens), _ptr(row_stats), _ptr(workspace),
                                   wb, _stream(stream))
    _check("s3r_sample_tokens_ex", st)


def s3r_device_status(workspace, stream=None):
    """(status, bits) of the most recent call that used `workspace` (synchronises)."""
    bits = ctypes.c_uint32(0)
    st = _lib.s3r_device_status(_ptr(workspace), ctypes.byref(bits), _stream(stream))
    return int(st), int(bits.value)


def s3r_sparse_draft_kernels(kv: PagedKV, budget_pages: int) -> int:
    """Kernels one s3r_sparse_draft_attn call launches (1 fused, 2 select + attention)."""
    return int(_lib.s3r_sparse_draft_kernels(ctypes.byref(kv), int(budget_pages)))


def s3r_kv_workspace_bytes(num_seqs: int) -> int:
    return int(_lib.s3r_kv_workspace_bytes(int(num_seqs)))


def s3r_kv_append(kv: PagedKV, context_lens, k_new, v_new, n: int, overwrite: int, kmin, kmax, workspace,
                  workspace_bytes=None, stream=None):
    """Write n rows per sequence at L - overwrite.. (updating L and the touched pages' summaries)."""
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = _lib.s3r_kv_append(ctypes.byref(kv), _ptr(context_lens), _ptr(k_new), _ptr(v_new), int(n),
                            int(overwrite), _ptr(kmin), _ptr(kmax), _ptr(workspace), wb, _stream(stream))
    _check("s3r_kv_append", st)


def s3r_kv_rollback(kv: PagedKV, context_lens, num_accepted, rows: int, kmin, kmax, workspace,
                    workspace_bytes=None, stream=None):
    """L <- L - rows + n_acc + 1, and the new tail page's summary."""
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = _lib.s3r_kv_rollback(ctypes.byref(kv), _ptr(context_lens), _ptr(num_accepted), int(rows), _ptr(kmin),
                              _ptr(kmax), _ptr(workspace), wb, _stream(stream))
    _check("s3r_kv_rollback", st)


def s3r_kvq_page_bytes(head_dim: int, page_size: int, bits: int) -> int:
    """Bytes of one (page, KV head) of a quantised cache; 0 for unsupported sizes."""
    return int(_lib.s3r_kvq_page_bytes(int(head_dim), int(page_size), int(bits)))


_torch = None
_kvq_types = {}                  # name of a type -> (torch type, code)


def _expect(device, *args):
    """Checks (name, tensor, dtype, shape) arguments: the library would read or write past a tensor of another type,
    shape or layout. device: index of the current device. None and raw addresses pass."""
    for name, x, dtype, shape in args:
        if x is None or isinstance(x, int):
            continue
        if x.shape != shape or x.dtype != dtype or not x.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                             f"got {x.dtype} {tuple(x.shape)}")
        at = x.get_device()                                  # -1 on the host
        if at < 0:
            raise ValueError(f"{name} must live on the GPU")
        if at != device:
            raise ValueError(f"{name} lives on {x.device}, the current device is cuda:{device}")


def _kvq_env(dtype):
    """(current device index, torch dtype, its code); -1 before CUDA is in use (there are no GPU tensors then)."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    known = _kvq_types.get(dtype)
    if known is None:
        code = dtype_code(dtype) if dtype is not None else S3R_BF16
        known = _kvq_types[dtype] = (_torch.bfloat16 if code == S3R_BF16 else _torch.float32, code)
    device = _torch.cuda.current_device() if _torch.cuda.is_initialized() else -1
    return device, known[0], known[1]


def _same_device(device, kvq, workspace):
    """Refuses a cache or a workspace of another device: the launch goes to the current one."""
    if getattr(kvq, "device", device) != device:
        raise ValueError(f"the quantised cache lives on cuda:{kvq.device}, the current device is cuda:{device}")
    if hasattr(workspace, "get_device") and workspace.get_device() != device:
        raise ValueError(f"workspace lives on {workspace.device}, the current device is cuda:{device}")


def _stream_on(stream, device):
    """_stream(stream), without building a stream object for the current one (3 us of a small call)."""
    if stream is None and device >= 0:
        raw = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(device)
    return _stream(stream)


def paged_kvq(pages, block_table, context_lens, num_q_heads: int, head_dim: int, page_size: int, bits: int) -> PagedKVQ:
    """Describe a quantised cache: pages uint8 [num_pages_total, Hkv, s3r_kvq_page_bytes(D, P, bits)]."""
    device, _, _ = _kvq_env(None)
    n, h, nb = pages.shape
    if nb != s3r_kvq_page_bytes(head_dim, page_size, bits):
        raise ValueError(f"pages have {nb} bytes per head, head_dim {head_dim}, page_size {page_size} and {bits} bits "
                         f"need {s3r_kvq_page_bytes(head_dim, page_size, bits)}")
    _expect(device, ("pages", pages, _torch.uint8, (n, h, nb)),
            ("block_table", block_table, _torch.int32, block_table.shape),
            ("context_lens", context_lens, _torch.int32, (block_table.shape[0],)))
    kvq = PagedKVQ(int(block_table.shape[0]), int(num_q_heads), int(h), int(head_dim), int(page_size),
                   int(block_table.shape[1]), int(n), int(bits), _ptr(pages), _ptr(block_table), _ptr(context_lens))
    kvq.tensors = (pages, block_table, context_lens)     # alive as long as the description
    kvq.device = device
    return kvq


def s3r_kvq_append(kvq: PagedKVQ, context_lens, k_new, v_new, dtype, n: int, overwrite: int, workspace,
                   workspace_bytes=None, stream=None):
    """Quantise n rows per sequence into positions L - overwrite.. (updating L; context_lens None: L stays)."""
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    device, dt, code = _kvq_env(dtype)
    shape = (kvq.num_seqs, n, kvq.num_kv_heads, kvq.head_dim)
    _expect(device, ("k_new", k_new, dt, shape), ("v_new", v_new, dt, shape))
    _same_device(device, kvq, workspace)
    st = _lib.s3r_kvq_append(ctypes.byref(kvq), _ptr(context_lens), _ptr(k_new), _ptr(v_new), code, int(n),
                             int(overwrite), _ptr(workspace), wb, _stream_on(stream, device))
    _check("s3r_kvq_append", st)


def s3r_kvq_pack(kv: PagedKV, kvq: PagedKVQ, last_n: int, workspace, workspace_bytes=None, stream=None):
    """Quantise the last last_n positions (0: all) of each sequence of kv into kvq."""
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    device, _, _ = _kvq_env(None)
    for at in getattr(kv, "devices", ()):
        if at != device or at < 0:
            raise ValueError(f"the source cache lives on {'the host' if at < 0 else f'cuda:{at}'}, "
                             f"the current device is cuda:{device}")
    _same_device(device, kvq, workspace)
    st = _lib.s3r_kvq_pack(ctypes.byref(kv), ctypes.byref(kvq), int(last_n), _ptr(workspace), wb, _stream_on(stream, device))
    _check("s3r_kvq_pack", st)


def s3r_kvq_read(kvq: PagedKVQ, start, n: int, dtype, k_out, v_out, workspace, workspace_bytes=None, stream=None):
    """Positions start[b] + t (start None: 0) of each sequence to rows k_out[b, t], v_out[b, t]."""
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    device, dt, code = _kvq_env(dtype)
    shape = (kvq.num_seqs, n, kvq.num_kv_heads, kvq.head_dim)
    _expect(device, ("start", start, _torch.int32, (kvq.num_seqs,)), ("k_out", k_out, dt, shape), ("v_out", v_out, dt, shape))
    _same_device(device, kvq, workspace)
    st = _lib.s3r_kvq_read(ctypes.byref(kvq), _ptr(start), int(n), code, _ptr(k_out), _ptr(v_out),
                           _ptr(workspace), wb, _stream_on(stream, device))
    _check("s3r_kvq_read", st)


def s3r_kvq_rollback(kvq: PagedKVQ, context_lens, num_accepted, rows: int, workspace, workspace_bytes=None, stream=None):
    """L <- L - rows + n_acc + 1."""
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    device, _, _ = _kvq_env(None)
    _expect(device, ("num_accepted", num_accepted, _torch.int32, (kvq.num_seqs,)))
    _same_device(device, kvq, workspace)
    st = _lib.s3r_kvq_rollback(ctypes.byref(kvq), _ptr(context_lens), _ptr(num_accepted), int(rows), _ptr(workspace), wb,
                               _stream_on(stream, device))
    _check("s3r_kvq_rollback", st)


def s3r_kvq_attn_workspace_bytes(kvq: PagedKVQ, dtype, rows: int, budget_pages: int = 0) -> int:
    return int(_lib.s3r_kvq_attn_workspace_bytes(ctypes.byref(kvq), dtype_code(dtype), int(rows), int(budget_pages)))


def s3r_kvq_attn(kvq: PagedKVQ, q, dtype, rows: int, scale: float, out, lse, workspace, pages=None, budget_pages: int = 0,
                 workspace_bytes=None, stream=None):
    """Causal attention of `rows` rows per sequence over the quantised cache (pages: the list of kept pages, or all)."""
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    device, dt, code = _kvq_env(dtype)
    shape = (kvq.num_seqs, rows, kvq.num_q_heads, kvq.head_dim)
    _expect(device, ("q", q, dt, shape), ("out", out, dt, shape), ("lse", lse, _torch.float32, shape[:3]),
            ("pages", pages, _torch.int32, (kvq.num_seqs, kvq.num_kv_heads, budget_pages)))
    _same_device(device, kvq, workspace)
    st = _lib.s3r_kvq_attn(ctypes.byref(kvq), _ptr(q), code, int(rows), _ptr(pages), int(budget_pages),
                           float(scale), _ptr(out), _ptr(lse), _ptr(workspace), wb, _stream_on(stream, device))
    _check("s3r_kvq_attn", st)


def s3r_debug_exp64(x, y_tbl, y_ref, stream=None):
    """The sampler's float64 exponential of x (y_tbl) and CUDA's exp (y_ref), float64 device tensors."""
    st = _lib.s3r_debug_exp64(_ptr(x), _ptr(y_tbl), _ptr(y_ref), int(x.numel()), _stream(stream))
    _check("s3r_debug_exp64", st)


class GammaPolicyHandle:
    """The library's draft-length policy (host code): init, update with a round's
    acceptance counts, choose the next gamma (0: drafting off)."""

    def __init__(self, gamma_max: int, decay: float, prior_accept: float, prior_weight: float, cost_us):
        self.p = GammaPolicy()
        c = (ctypes.c_double * 17)(*[float(x) for x in cost_us])
        _check("s3r_gamma_policy_init", _lib.s3r_gamma_policy_init(ctypes.byref(self.p), int(gamma_max),
                                                                   float(decay), float(prior_accept),
                                                                   float(prior_weight), c))

    def update(self, num_accepted, gamma_used: int):
        n = [int(x) for x in num_accepted]
        arr = (ctypes.c_int32 * len(n))(*n)
        _check("s3r_gamma_policy_update", _lib.s3r_gamma_policy_update(ctypes.byref(self.p), arr, len(n),
                                                                       int(gamma_used)))

    def choose(self):
        """(gamma, alpha, rate)."""
        g, a, r = ctypes.c_int32(0), ctypes.c_double(0), ctypes.c_double(0)
        _check("s3r_gamma_policy_choose", _lib.s3r_gamma_policy_choose(ctypes.byref(self.p), ctypes.byref(g),
                                                                       ctypes.byref(a), ctypes.byref(r)))
        return int(g.value), float(a.value), float(r.value)


def s3r_attend_cost_us(*args) -> float:
    return float(_lib.s3r_attend_cost_us(*args))


def s3r_round_cost_us(*args) -> float:
    return float(_lib.s3r_round_cost_us(*args))


def s3r_version() -> int:
    return int(_lib.s3r_version())
