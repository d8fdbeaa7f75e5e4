"""Python binding of libtreespec (the C ABI declared in include/treespec.h).

Argument marshalling only: every function here checks shapes/dtypes of torch
tensors, passes raw device pointers and the current CUDA stream to the
function of the same name in libtreespec.so, and raises TreespecError when it
returns an error. All computation happens in the library's CUDA kernels; there
is no CPU fallback -- without the built library every call raises.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtreespec.so")

TS_OK, TS_ERR_INVALID_ARG, TS_ERR_CUDA, TS_ERR_UNSUPPORTED = 0, 1, 2, 3
TS_F32, TS_BF16 = 0, 1
TS_OP_ATTENTION, TS_OP_VERIFY_GREEDY, TS_OP_VERIFY_MSS = 0, 1, 2
STATUS_BAD_TREE, STATUS_NONFINITE, STATUS_ZERO_RESID, STATUS_INDEX, STATUS_TIMEOUT = 1, 2, 4, 8, 16
STATUS_NO_PAGES = 32
MAX_NODES = 256
PAGE_KEYS = 64   # TS_PAGE_KEYS
DROPPED_LOGIT = -1e30   # TS_DROPPED_LOGIT

#: every entry point of the C ABI (include/treespec.h)
EXPORTS = ("tree_build", "tree_build_chains", "kv_append", "tree_attention", "verify_greedy", "verify_mss",
           "kv_commit", "treespec_workspace_size", "treespec_workspace_init", "treespec_last_error",
           "treespec_version", "tree_attention_noalloc", "treespec_attention_kernel", "verify_naive",
           "tree_expand_topk", "kv_append_paged", "tree_attention_paged", "kv_commit_paged", "tree_build_append",
           "tree_attention_append", "tree_qk_norm_rope", "kv8_append", "kv8_read", "tree_attention_kv8", "kv8_commit",
           "treespec_kv8_workspace_size", "kv_pages_build", "kv_append_slots", "decode_attention_paged",
           "treespec_decode_workspace_size", "sample_tokens")
#: bytes of the scratch array compiled into the library (TS_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 8 << 20


class TreespecError(RuntimeError):
    pass


class ts_tree(C.Structure):
    _fields_ = [("B", C.c_int32), ("n_max", C.c_int32)] + [
        (name, C.c_void_p) for name in ("n_nodes", "perm", "dfs_of", "parent", "token", "depth", "pos", "sub_end",
                                        "anc")]


class ts_paged_kv(C.Structure):
    _fields_ = [("k_pages", C.c_void_p), ("v_pages", C.c_void_p), ("block_table", C.c_void_p),
                ("num_pages", C.c_int32), ("max_pages", C.c_int32)]


class ts_qk_rope(C.Structure):
    _fields_ = [("inv_freq", C.c_void_p), ("q_weight", C.c_void_p), ("k_weight", C.c_void_p), ("eps", C.c_float),
                ("norm", C.c_int32), ("rot_dim", C.c_int32), ("interleaved", C.c_int32)]


class ts_kv8(C.Structure):
    _fields_ = [(name, C.c_void_p) for name in ("k", "v", "k_scale", "v_scale", "block_table")] + [
        (name, C.c_int32) for name in ("B", "H", "d", "L_max", "num_pages", "max_pages")]


class ts_page_pool(C.Structure):
    _fields_ = [(name, C.c_void_p) for name in ("block_table", "held", "ring", "ring_state")] + [
        (name, C.c_int32) for name in ("B", "max_pages", "num_pages")]


_lib = None


def load_library(path: str | None = None):
    """Load libtreespec.so (built by tree_speculative_verification_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise TreespecError(f"{path} is missing: build the CUDA library first "
                            "(python -m tree_speculative_verification_gb300.build)")
    lib = C.CDLL(path)
    P, I, F, Z = C.c_void_p, C.c_int, C.c_float, C.c_size_t
    T, KV, R, S = C.POINTER(ts_tree), C.POINTER(ts_kv8), C.POINTER(ts_qk_rope), C.c_longlong
    sig = {
        "tree_build": [T, P, P, P, P, I, P, P, P],
        "tree_build_chains": [T, P, P, I, I, P, P, P, P, P, P],
        "kv_append": [P, P, P, P, P, T, I, I, I, I, P, P],
        "tree_build_append": [T, P, P, I, P, P, P, P, P, I, I, I, I, P, P],
        "tree_attention": [P, P, P, P, P, T, I, I, I, I, F, P, Z, P, P],
        "tree_attention_append": [P, P, P, P, P, P, P, T, I, I, I, I, F, P, Z, P, P],
        "verify_greedy": [P, P, P, P, P, T, I, P, Z, P, P],
        "verify_mss": [P, P, P, P, P, P, I, P, P, I, P, F, T, I, P, P],
        "verify_naive": [P, P, P, P, P, P, I, P, F, T, I, P, P],
        "tree_expand_topk": [P, P, P, I, I, I, P, I, I, P, P],
        "kv_append_paged": [C.POINTER(ts_paged_kv), P, P, P, T, I, I, P, P],
        "tree_attention_paged": [P, P, C.POINTER(ts_paged_kv), P, T, I, I, F, P, Z, P, P],
        "kv_commit_paged": [C.POINTER(ts_paged_kv), P, P, P, P, T, I, I, P, P],
        "kv_commit": [P, P, P, P, P, P, T, I, I, I, I, P, P],
        "treespec_workspace_init": [P, Z, P],
        "tree_attention_noalloc": [P, P, P, P, P, T, I, I, I, I, F, P, P],
        "tree_qk_norm_rope": [P, P, P, P, I, I, I, S, S, R, T, I, P, P],
        "kv8_append": [KV, P, P, S, S, R, P, P, I, S, P, T, I, P, P],
        "kv8_read": [P, P, KV, P, P, I, I, P, P],
        "tree_attention_kv8": [P, P, KV, I, P, T, F, P, Z, P, P],
        "kv8_commit": [KV, P, P, P, P, T, P, P],
        "kv_pages_build": [C.POINTER(ts_page_pool), P, P, P, I, P, P, P, P, P],
        "kv_append_slots": [C.POINTER(ts_paged_kv), P, P, S, S, P, I, I, I, P, P],
        "decode_attention_paged": [P, P, S, C.POINTER(ts_paged_kv), P, I, I, I, I, F, P, Z, P, P],
        "sample_tokens": [P, P, P, P, S, I, P, P, P, P, P, I, I, P, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = C.c_int
    lib.treespec_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.treespec_workspace_size.restype = C.c_size_t
    lib.treespec_kv8_workspace_size.argtypes = [I, I, I, I, I, I]
    lib.treespec_kv8_workspace_size.restype = C.c_size_t
    lib.treespec_decode_workspace_size.argtypes = [I, I, I, I]
    lib.treespec_decode_workspace_size.restype = C.c_size_t
    lib.treespec_attention_kernel.argtypes = [I, I, I, I, I, I]
    lib.treespec_attention_kernel.restype = C.c_char_p
    lib.treespec_last_error.restype = C.c_char_p
    lib.treespec_version.restype = C.c_char_p
    _lib = lib
    return lib


def _check(rc: int, what: str):
    if rc != TS_OK:
        msg = load_library().treespec_last_error().decode()
        raise TreespecError(f"{what} failed ({rc}): {msg}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise TreespecError("tensors passed to the library must live on a CUDA device")
    if not t.is_contiguous():
        raise TreespecError("tensors passed to the library must be contiguous")
    return C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _i32(t, name):
    if t is not None and t.dtype != torch.int32:
        raise TreespecError(f"{name} must be int32")
    return t


def _dtype(t):
    if t.dtype == torch.bfloat16:
        return TS_BF16
    if t.dtype == torch.float32:
        return TS_F32
    raise TreespecError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")


class Tree:
    """Device arrays of a linearised tree batch (the ts_tree of the C ABI)."""

    def __init__(self, B: int, n_max: int, device="cuda"):
        if not 1 <= n_max <= MAX_NODES:
            raise TreespecError(f"n_max={n_max} outside [1, {MAX_NODES}]")
        self.B, self.n_max = B, n_max
        W = (n_max + 31) // 32
        z = lambda *s: torch.full(s, -1, dtype=torch.int32, device=device)
        self.n_nodes = torch.zeros(B, dtype=torch.int32, device=device)
        self.perm, self.dfs_of, self.parent, self.token = z(B, n_max), z(B, n_max), z(B, n_max), z(B, n_max)
        self.depth, self.pos, self.sub_end = z(B, n_max), z(B, n_max), z(B, n_max)
        self.anc = torch.zeros(B, n_max, W, dtype=torch.int32, device=device)   # uint32 bit patterns
        self._c = ts_tree(B, n_max, *[t.data_ptr() for t in (self.n_nodes, self.perm, self.dfs_of, self.parent,
                                                              self.token, self.depth, self.pos, self.sub_end,
                                                              self.anc)])

    @property
    def c(self):
        return C.byref(self._c)


def tree_build(tree: Tree, tokens, parent=None, n_nodes=None, widths=None, prefix_len=None, status=None,
               stream=None):
    lib = load_library()
    w_arr, m = None, 0
    if widths is not None:
        m = len(widths)
        w_arr = (C.c_int32 * max(1, m))(*[int(k) for k in widths])
    _check(lib.tree_build(tree.c, _ptr(_i32(tokens, "tokens")), _ptr(_i32(parent, "parent")),
                          _ptr(_i32(n_nodes, "n_nodes")), w_arr, m, _ptr(_i32(prefix_len, "prefix_len")),
                          _ptr(status), _stream(stream)), "tree_build")


def tree_build_append(tree: Tree, tokens, widths, prefix_len, k_cache, v_cache, k_new, v_new, status=None,
                      stream=None):
    """tree_build (widths mode) and kv_append in one launch (dense cache)."""
    lib = load_library()
    m = len(widths)
    w_arr = (C.c_int32 * max(1, m))(*[int(k) for k in widths])
    B, H, L_max, d = k_cache.shape
    _check(lib.tree_build_append(tree.c, _ptr(_i32(tokens, "tokens")), w_arr, m, _ptr(_i32(prefix_len, "prefix_len")),
                                 _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new), H, d, L_max,
                                 _dtype(k_cache), _ptr(status), _stream(stream)), "tree_build_append")


def tree_build_chains(tree: Tree, root_token, chains, tokens_out=None, p_row=None, q_row=None, prefix_len=None,
                      status=None, stream=None):
    lib = load_library()
    Cn, ln = chains.shape[1], chains.shape[2]
    _check(lib.tree_build_chains(tree.c, _ptr(_i32(root_token, "root_token")), _ptr(_i32(chains, "chains")), Cn, ln,
                                 _ptr(_i32(tokens_out, "tokens_out")), _ptr(_i32(p_row, "p_row")),
                                 _ptr(_i32(q_row, "q_row")), _ptr(_i32(prefix_len, "prefix_len")), _ptr(status),
                                 _stream(stream)), "tree_build_chains")


def tree_expand_topk(tokens, root_token, ssm_probs, widths, status=None, stream=None):
    """Draft the expansion tree <widths> from drafter rows into tokens [B][n_max]."""
    lib = load_library()
    B, n_max = tokens.shape
    NQ, V = ssm_probs.shape[1], ssm_probs.shape[2]
    m = len(widths)
    w_arr = (C.c_int32 * max(1, m))(*[int(k) for k in widths])
    _check(lib.tree_expand_topk(_ptr(_i32(tokens, "tokens")), _ptr(_i32(root_token, "root_token")), _ptr(ssm_probs),
                                NQ, B, n_max, w_arr, m, V, _ptr(status), _stream(stream)), "tree_expand_topk")


def kv_append(k_cache, v_cache, k_new, v_new, prefix_len, tree: Tree, status=None, stream=None):
    lib = load_library()
    B, H, L_max, d = k_cache.shape
    _check(lib.kv_append(_ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new), _ptr(_i32(prefix_len, "prefix_len")),
                         tree.c, H, d, L_max, _dtype(k_cache), _ptr(status), _stream(stream)), "kv_append")


def workspace_size(op: int, B: int, H: int, n_max: int, d: int, L_max: int, V: int) -> int:
    return int(load_library().treespec_workspace_size(op, B, H, n_max, d, L_max, V))


def attention_kernel(B: int, H: int, n_max: int, d: int, L_max: int, dtype: int) -> str:
    """Name of the kernel tree_attention launches for these sizes ("" if rejected)."""
    return load_library().treespec_attention_kernel(B, H, n_max, d, L_max, dtype).decode()


def workspace(op: int, B: int, H: int = 1, n_max: int = 1, d: int = 128, L_max: int = 1, V: int = 1,
              device="cuda"):
    """A zero-filled workspace of the size the op needs (at least 256 bytes)."""
    return torch.zeros(max(256, workspace_size(op, B, H, n_max, d, L_max, V)), dtype=torch.uint8, device=device)


def tree_attention(out, q, k_cache, v_cache, prefix_len, tree: Tree, scale: float = 0.0, ws=None, status=None,
                   stream=None):
    lib = load_library()
    B, H, L_max, d = k_cache.shape
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.tree_attention(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(_i32(prefix_len, "prefix_len")),
                              tree.c, H, d, L_max, _dtype(k_cache), float(scale), _ptr(ws), nbytes, _ptr(status),
                              _stream(stream)), "tree_attention")


def tree_attention_append(out, q, k_cache, v_cache, k_new, v_new, prefix_len, tree: Tree, scale: float = 0.0,
                          ws=None, status=None, stream=None):
    """kv_append and tree_attention in one call (one launch with the persistent
    tcgen05 kernel, else the two launches)."""
    lib = load_library()
    B, H, L_max, d = k_cache.shape
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.tree_attention_append(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new),
                                     _ptr(_i32(prefix_len, "prefix_len")), tree.c, H, d, L_max, _dtype(k_cache),
                                     float(scale), _ptr(ws), nbytes, _ptr(status), _stream(stream)),
           "tree_attention_append")


def tree_attention_noalloc(out, q, k_cache, v_cache, prefix_len, tree: Tree, scale: float = 0.0, status=None,
                           stream=None):
    """tree_attention without a workspace argument, for callers that cannot
    allocate device memory: the library's built-in scratch array (shared by all
    calls on a device; calls must not overlap on the GPU) holds the partials."""
    lib = load_library()
    B, H, L_max, d = k_cache.shape
    _check(lib.tree_attention_noalloc(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                      _ptr(_i32(prefix_len, "prefix_len")), tree.c, H, d, L_max, _dtype(k_cache),
                                      float(scale), _ptr(status), _stream(stream)), "tree_attention_noalloc")


def verify_greedy(out_tokens, out_path, out_count, logits, tree: Tree, argmax_out=None, ws=None, status=None,
                  stream=None):
    lib = load_library()
    V = logits.shape[-1]
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.verify_greedy(_ptr(out_tokens), _ptr(out_path), _ptr(out_count), _ptr(argmax_out), _ptr(logits),
                             tree.c, V, _ptr(ws), nbytes, _ptr(status), _stream(stream)), "verify_greedy")


def verify_mss(out_tokens, out_path, out_count, target_logits, ssm_probs, q_row, uniforms, temperature, tree: Tree,
               p_row=None, status=None, stream=None, lowmargin=None):
    """lowmargin: optional int32 [B], the number of decisions per request taken
    with a margin below 1e-6."""
    lib = load_library()
    NP, V = target_logits.shape[1], target_logits.shape[2]
    NQ = ssm_probs.shape[1]
    _check(lib.verify_mss(_ptr(out_tokens), _ptr(out_path), _ptr(out_count), _ptr(_i32(lowmargin, "lowmargin")),
                          _ptr(target_logits),
                          _ptr(_i32(p_row, "p_row")), NP, _ptr(ssm_probs), _ptr(_i32(q_row, "q_row")), NQ,
                          _ptr(uniforms), float(temperature), tree.c, V, _ptr(status), _stream(stream)), "verify_mss")


def verify_naive(out_tokens, out_path, out_count, target_logits, uniforms, temperature, tree: Tree, p_row=None,
                 status=None, stream=None, lowmargin=None):
    lib = load_library()
    NP, V = target_logits.shape[1], target_logits.shape[2]
    _check(lib.verify_naive(_ptr(out_tokens), _ptr(out_path), _ptr(out_count), _ptr(_i32(lowmargin, "lowmargin")),
                            _ptr(target_logits),
                            _ptr(_i32(p_row, "p_row")), NP, _ptr(uniforms), float(temperature), tree.c, V,
                            _ptr(status), _stream(stream)), "verify_naive")


def kv_commit(k_cache, v_cache, prefix_len, new_prefix_len, out_path, out_count, tree: Tree, status=None,
              stream=None):
    lib = load_library()
    B, H, L_max, d = k_cache.shape
    _check(lib.kv_commit(_ptr(k_cache), _ptr(v_cache), _ptr(_i32(prefix_len, "prefix_len")),
                         _ptr(_i32(new_prefix_len, "new_prefix_len")), _ptr(out_path), _ptr(out_count), tree.c, H, d,
                         L_max, _dtype(k_cache), _ptr(status), _stream(stream)), "kv_commit")


class PagedKV:
    """A paged KV cache (the ts_paged_kv of the C ABI): k_pages / v_pages
    [num_pages][H][PAGE_KEYS][d] bf16 and block_table [B][max_pages] int32."""

    def __init__(self, k_pages, v_pages, block_table):
        if k_pages.dtype != torch.bfloat16 or v_pages.shape != k_pages.shape:
            raise TreespecError("pages must be two bf16 tensors of one shape [num_pages][H][64][d]")
        if k_pages.shape[2] != PAGE_KEYS:
            raise TreespecError(f"a page holds {PAGE_KEYS} keys")
        self.k_pages, self.v_pages, self.block_table = k_pages, v_pages, _i32(block_table, "block_table")
        self.H, self.d, self.device = k_pages.shape[1], k_pages.shape[3], k_pages.get_device()
        self._whole = k_pages.is_cuda and all(x.is_contiguous() and x.device == k_pages.device
                                              for x in (k_pages, v_pages, block_table)) and block_table.dim() == 2
        self.B = block_table.shape[0]
        self._c = ts_paged_kv(k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(), k_pages.shape[0],
                              block_table.shape[1])
        self._ref = C.byref(self._c)

    @property
    def c(self):
        return self._ref

    @property
    def L_max(self) -> int:
        return self.block_table.shape[1] * PAGE_KEYS


def kv_append_paged(kv: PagedKV, k_new, v_new, prefix_len, tree: Tree, status=None, stream=None):
    _check(load_library().kv_append_paged(kv.c, _ptr(k_new), _ptr(v_new), _ptr(_i32(prefix_len, "prefix_len")), tree.c,
                                          kv.H, kv.d, _ptr(status), _stream(stream)), "kv_append_paged")


def tree_attention_paged(out, q, kv: PagedKV, prefix_len, tree: Tree, scale=0.0, ws=None, status=None, stream=None):
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load_library().tree_attention_paged(_ptr(out), _ptr(q), kv.c, _ptr(_i32(prefix_len, "prefix_len")), tree.c,
                                               kv.H, kv.d, float(scale), _ptr(ws), nbytes, _ptr(status),
                                               _stream(stream)), "tree_attention_paged")


def kv_commit_paged(kv: PagedKV, prefix_len, new_prefix_len, out_path, out_count, tree: Tree, status=None,
                    stream=None):
    _check(load_library().kv_commit_paged(kv.c, _ptr(_i32(prefix_len, "prefix_len")),
                                          _ptr(_i32(new_prefix_len, "new_prefix_len")), _ptr(out_path),
                                          _ptr(out_count), tree.c, kv.H, kv.d, _ptr(status), _stream(stream)),
           "kv_commit_paged")


# -- head norms with rotation, and the 8-bit KV cache -----------------------------
# A short call's time is the host's, so checks are tests around a raise (a call that passes builds no message), devices
# are compared by their index, and contiguous rows take no look at strides.
def _int_array(t, n, name, device):
    """Pointer of an int32 tensor of at least n entries on CUDA device number `device`."""
    if t.dtype is not torch.int32 or t.numel() < n or t.get_device() != device or not t.is_contiguous():
        raise TreespecError(f"{name} must be a contiguous int32 tensor of {n} entries on CUDA device {device}")
    return t.data_ptr()


def _status_ptr(status, device):
    return None if status is None else _int_array(status, 1, "status", device)


def _node_rows(t, shape, name, dtype, device):
    """(pointer, elements from one node to the next) of node rows `shape` = (B, n_max, H, d): heads contiguous, nodes
    and requests a constant stride apart (a slice of a wider projection output)."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape:
        raise TreespecError(f"{name} must be a {dtype} tensor {shape} on CUDA device {device}, not {t.dtype} "
                            f"{tuple(t.shape)} on {t.device}")
    B, n, H, d = shape
    if t.is_contiguous():
        return t.data_ptr(), H * d
    sb, sn, sh, sd = t.stride()
    if n == 1:
        sn = sb if B > 1 else H * d
    if sd != 1 or (H > 1 and sh != d) or (B > 1 and sb != n * sn):
        raise TreespecError(f"{name}: heads must be contiguous, nodes and requests a constant stride apart")
    return t.data_ptr(), sn


def _out_rows(t, shape, name, dtype, device):
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise TreespecError(f"{name} must be a contiguous {dtype} tensor {shape} on CUDA device {device}")
    return t.data_ptr()


def _same_device(tree, device):
    if tree.n_nodes.get_device() != device:
        raise TreespecError(f"the tree is on {tree.n_nodes.device}, not on CUDA device {device}")


def _run(fn, what, device, stream, *args):
    """Call an entry point on the current stream of CUDA device number `device` (or on the given one)."""
    # the stream's handle alone: torch.cuda.current_stream() makes an object of it, a quarter of a short call's time
    handle = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
    if device == torch._C._cuda_getDevice():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
    if rc != TS_OK:
        _check(rc, what)


class QKRope:
    """Norm and rotation of query and key heads (the ts_qk_rope of the C ABI). inv_freq: fp32 [rot_dim / 2] (None: no
    rotation); q_weight, k_weight: fp32 [d] norm weights (None: ones); norm=False rotates only."""

    def __init__(self, inv_freq=None, q_weight=None, k_weight=None, eps: float = 1e-6, norm: bool = True,
                 interleaved: bool = False):
        given = [x for x in (inv_freq, q_weight, k_weight) if x is not None]
        for x in given:
            if not (x.dtype == torch.float32 and x.is_contiguous() and x.dim() == 1 and x.is_cuda
                    and x.device == given[0].device):
                raise TreespecError("inv_freq and weights must be contiguous fp32 vectors on one CUDA device")
        self.inv_freq, self.q_weight, self.k_weight = inv_freq, q_weight, k_weight
        self.device = given[0].get_device() if given else None
        self.rot_dim = 0 if inv_freq is None else 2 * inv_freq.numel()
        p = lambda x: None if x is None else x.data_ptr()
        self._c = ts_qk_rope(p(inv_freq), p(q_weight), p(k_weight), float(eps), int(bool(norm)), self.rot_dim,
                             int(bool(interleaved)))
        self._ref = C.byref(self._c)

    def _for(self, d, device):
        if self.device is not None and self.device != device:
            raise TreespecError(f"the rotation's tensors are on CUDA device {self.device}, not {device}")
        for w in (self.q_weight, self.k_weight):
            if w is not None and w.numel() != d:
                raise TreespecError(f"norm weights must have head_dim {d} entries")
        return self._ref

    @staticmethod
    def frequencies(rot_dim: int, theta: float = 10000.0, device="cuda"):
        """theta^(-2j / rot_dim), j = 0 .. rot_dim / 2 - 1, in fp32."""
        return (theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)).float().to(device)


def tree_qk_norm_rope(q_out, k_out, q, k, rope: QKRope, tree: Tree, status=None, stream=None):
    """Norm every head of q and k [B][n_max][H][d] and rotate it to its node's position (tree.pos); q or k may be
    None with its output. Outputs are contiguous, and may be the inputs where those are."""
    x = q if q is not None else k
    if x is None or not x.is_cuda or x.dim() != 4:
        raise TreespecError("q or k [B][n_max][H][d] on a CUDA device is needed")
    dev, d, dt, dtype = x.get_device(), x.shape[3], _dtype(x), x.dtype
    _same_device(tree, dev)
    B, n = tree.B, tree.n_max
    qp = kp = qo = ko = None
    Hq = Hk = qs = ks = 0
    if q is not None:
        Hq = q.shape[2]
        shape = (B, n, Hq, d)
        (qp, qs), qo = _node_rows(q, shape, "q", dtype, dev), _out_rows(q_out, shape, "q_out", dtype, dev)
    if k is not None:
        Hk = k.shape[2]
        shape = (B, n, Hk, d)
        (kp, ks), ko = _node_rows(k, shape, "k", dtype, dev), _out_rows(k_out, shape, "k_out", dtype, dev)
    _run(load_library().tree_qk_norm_rope, "tree_qk_norm_rope", dev, stream, qo, ko, qp, kp, Hq, Hk, d, qs, ks,
         rope._for(d, dev), tree.c, dt, _status_ptr(status, dev))


class KV8:
    """An 8-bit KV cache (the ts_kv8 of the C ABI): e4m3 codes and one fp32 scale per row and head. Dense: k, v
    [B][H][L_max][d] torch.float8_e4m3fn, k_scale, v_scale [B][H][L_max]; with block_table [B][max_pages] int32 paged:
    k, v [num_pages][H][PAGE_KEYS][d], scales [num_pages][H][PAGE_KEYS]."""

    def __init__(self, k, v, k_scale, v_scale, block_table=None):
        if not (k.dim() == 4 and k.dtype == torch.float8_e4m3fn and v.dtype == k.dtype and v.shape == k.shape):
            raise TreespecError("k and v must be two float8_e4m3fn tensors of one shape [B or pages][H][rows][d]")
        if not (k_scale.dtype == torch.float32 and v_scale.dtype == torch.float32 and k_scale.shape == k.shape[:3]
                and v_scale.shape == k.shape[:3]):
            raise TreespecError("scales must be fp32 of the codes' shape without head_dim")
        for x in (k, v, k_scale, v_scale):
            if not (x.is_cuda and x.is_contiguous() and x.device == k.device):
                raise TreespecError("cache tensors must be contiguous on one CUDA device")
        self.k, self.v, self.k_scale, self.v_scale, self.block_table = k, v, k_scale, v_scale, block_table
        self.H, self.d, self.device = k.shape[1], k.shape[3], k.get_device()
        pages = 0
        if block_table is not None:
            if k.shape[2] != PAGE_KEYS:
                raise TreespecError(f"a page holds {PAGE_KEYS} keys")
            if block_table.dim() != 2:
                raise TreespecError("block_table must be [B][max_pages]")
            _int_array(block_table, 1, "block_table", self.device)
            self.B, pages = block_table.shape
            self.L_max = pages * PAGE_KEYS
        else:
            self.B, self.L_max = k.shape[0], k.shape[2]
        self._c = ts_kv8(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                         None if block_table is None else block_table.data_ptr(), self.B, self.H, self.d,
                         self.L_max if block_table is None else 0, 0 if block_table is None else k.shape[0], pages)
        self._ref = C.byref(self._c)

    @classmethod
    def dense(cls, B: int, H: int, L_max: int, d: int, device="cuda"):
        """A dense cache of zeros."""
        z = lambda *s, t=torch.float8_e4m3fn: torch.zeros(s, dtype=t, device=device)
        return cls(z(B, H, L_max, d), z(B, H, L_max, d), z(B, H, L_max, t=torch.float32), z(B, H, L_max, t=torch.float32))

    @classmethod
    def paged(cls, num_pages: int, H: int, d: int, block_table):
        """A paged cache of zeros on the block table's device."""
        z = lambda *s, t=torch.float8_e4m3fn: torch.zeros(s, dtype=t, device=block_table.device)
        s = (num_pages, H, PAGE_KEYS)
        return cls(z(*s, d), z(*s, d), z(*s, t=torch.float32), z(*s, t=torch.float32), block_table)

    def _with(self, tree: Tree):
        if tree.B != self.B:
            raise TreespecError(f"cache of {self.B} requests, tree of {tree.B}")
        _same_device(tree, self.device)
        return self._ref


def kv8_append(kv: KV8, k_new, v_new, prefix_len, tree: Tree, rope: QKRope | None = None, q=None, q_out=None,
               status=None, stream=None):
    """Quantise the pass's K/V [B][n_max][H][d] into the cache rows P + dfs; with rope the keys are normed and rotated
    on the way, and the queries q, if given, into q_out."""
    ref, dev, d = kv._with(tree), kv.device, kv.d
    dt, dtype, shape = _dtype(k_new), k_new.dtype, (tree.B, tree.n_max, kv.H, d)
    kp, ks = _node_rows(k_new, shape, "k_new", dtype, dev)
    vp, vs = _node_rows(v_new, shape, "v_new", dtype, dev)
    qp = qo = r = None
    Hq = qs = 0
    if q is not None:
        if rope is None or q_out is None:
            raise TreespecError("queries are only taken with rope, and need q_out")
        Hq = q.shape[2]
        shape = (tree.B, tree.n_max, Hq, d)
        qp, qs = _node_rows(q, shape, "q", dtype, dev)
        qo = _out_rows(q_out, shape, "q_out", dtype, dev)
    if rope is not None:
        r = rope._for(d, dev)
    _run(load_library().kv8_append, "kv8_append", dev, stream, ref, kp, vp, ks, vs, r, qo, qp, Hq, qs,
         _int_array(prefix_len, tree.B, "prefix_len", dev), tree.c, dt, _status_ptr(status, dev))


def kv8_read(k_out, v_out, kv: KV8, row_end, row_begin=None, status=None, stream=None):
    """Cache rows row_begin[b] .. row_end[b] - 1 as values into rows 0 .. of k_out, v_out [B][H][L_out][d] (bfloat16
    or float32)."""
    dev = kv.device
    shape = (kv.B, kv.H, k_out.shape[2] if k_out.dim() == 4 else 0, kv.d)
    for x in (k_out, v_out):
        if x.shape != shape or x.dtype is not k_out.dtype or x.get_device() != dev or not x.is_contiguous():
            raise TreespecError(f"k_out and v_out must be contiguous tensors {shape} of one dtype on CUDA device {dev}")
    begin = None if row_begin is None else _int_array(row_begin, kv.B, "row_begin", dev)
    _run(load_library().kv8_read, "kv8_read", dev, stream, k_out.data_ptr(), v_out.data_ptr(), kv._ref, begin,
         _int_array(row_end, kv.B, "row_end", dev), shape[2], _dtype(k_out), _status_ptr(status, dev))


def kv8_workspace(B: int, Hq: int, Hkv: int, n_max: int, d: int, L_max: int, device="cuda"):
    """A zero-filled workspace of the size tree_attention_kv8 needs (L_max: KV8.L_max)."""
    with torch.cuda.device(device):
        need = int(load_library().treespec_kv8_workspace_size(B, Hq, Hkv, n_max, d, L_max))
    return torch.zeros(max(256, need), dtype=torch.uint8, device=device)


def tree_attention_kv8(out, q, kv: KV8, prefix_len, tree: Tree, scale: float = 0.0, ws=None, status=None, stream=None):
    """tree_attention over an 8-bit cache; q, out [B][n_max][Hq][d] bfloat16, Hq a multiple of kv.H."""
    ref, dev = kv._with(tree), kv.device
    if q.dim() != 4:
        raise TreespecError("q must be [B][n_max][Hq][d]")
    Hq = q.shape[2]
    shape = (tree.B, tree.n_max, Hq, kv.d)
    op = _out_rows(out, shape, "out", torch.bfloat16, dev)
    qp = _out_rows(q, shape, "q", torch.bfloat16, dev)
    if ws is None or ws.get_device() != dev or not ws.is_contiguous():
        raise TreespecError(f"a workspace (kv8_workspace) on CUDA device {dev} is needed")
    _run(load_library().tree_attention_kv8, "tree_attention_kv8", dev, stream, op, qp, ref, Hq,
         _int_array(prefix_len, tree.B, "prefix_len", dev), tree.c, float(scale), ws.data_ptr(),
         ws.numel() * ws.element_size(), _status_ptr(status, dev))


def kv8_commit(kv: KV8, prefix_len, new_prefix_len, out_path, out_count, tree: Tree, status=None, stream=None):
    """kv_commit over an 8-bit cache."""
    ref, dev, B = kv._with(tree), kv.device, tree.B
    _run(load_library().kv8_commit, "kv8_commit", dev, stream, ref, _int_array(prefix_len, B, "prefix_len", dev),
         _int_array(new_prefix_len, B, "new_prefix_len", dev),
         _int_array(out_path, B * (tree.n_max + 1), "out_path", dev), _int_array(out_count, B, "out_count", dev),
         tree.c, _status_ptr(status, dev))


# -- a decode step on the paged cache ------------------------------------------------
class PagePool:
    """Cache pages and who holds them (the ts_page_pool of the C ABI): block_table [B][max_pages], of which request b
    holds the first held[b] entries, and the free pages in a ring [num_pages]; state [3] is its first free entry, the
    number of free pages, and a counter that is 0 between calls. int32 tensors on one CUDA device."""

    def __init__(self, block_table, held, ring, state):
        if block_table.dim() != 2 or not block_table.is_cuda:
            raise TreespecError("block_table must be [B][max_pages] on a CUDA device")
        self.B, self.max_pages = block_table.shape
        self.device = dev = block_table.get_device()
        self.num_pages = ring.numel()
        self.block_table, self.held, self.ring, self.state = block_table, held, ring, state
        self._c = ts_page_pool(_int_array(block_table, 1, "block_table", dev), _int_array(held, self.B, "held", dev),
                               _int_array(ring, 1, "ring", dev), _int_array(state, 3, "state", dev), self.B,
                               self.max_pages, self.num_pages)
        self._ref = C.byref(self._c)

    @classmethod
    def empty(cls, B: int, max_pages: int, num_pages: int, device="cuda"):
        """A pool whose pages are all free."""
        i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=device)
        return cls(torch.full((B, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(B, dtype=torch.int32, device=device),
                   torch.arange(num_pages, dtype=torch.int32, device=device), i32(0, num_pages, 0))


def kv_pages_build(pool: PagePool, row_end, row_begin=None, slot=None, slot_offset=None, new_held=None, new_state=None,
                   status=None, stream=None):
    """Pages for rows 0 .. row_end[b] - 1 of every request, and the slots of rows row_begin[b] .. row_end[b] - 1 into
    slot (entries behind the last row are -1) with each request's first one in slot_offset [B + 1]. Without new_held and
    new_state the pool itself is brought up to date; with them it can serve the same call again."""
    dev, B = pool.device, pool.B
    sp = so = rb = None
    n = 0
    if slot is not None:
        n = slot.numel()
        sp = _int_array(slot, 1, "slot", dev)
        if row_begin is None:
            raise TreespecError("slots need row_begin")
        rb = _int_array(row_begin, B, "row_begin", dev)
        if slot_offset is not None:
            so = _int_array(slot_offset, B + 1, "slot_offset", dev)
    elif slot_offset is not None:
        raise TreespecError("slot_offset without slot")
    _run(load_library().kv_pages_build, "kv_pages_build", dev, stream, pool._ref,
         pool._c.held if new_held is None else _int_array(new_held, B, "new_held", dev),
         pool._c.ring_state if new_state is None else _int_array(new_state, 3, "new_state", dev), sp, n, so, rb,
         _int_array(row_end, B, "row_end", dev), _status_ptr(status, dev))


def _whole_pages(kv: PagedKV):
    if not kv._whole:
        raise TreespecError("pages and block table must be contiguous on one CUDA device")
    return kv._ref


def _token_rows(t, H, d, name, dtype, device):
    """(pointer, elements from one token to the next) of rows [T][H][d] whose heads are contiguous."""
    if t.dtype is not dtype or t.get_device() != device or t.dim() != 3 or t.shape[1] != H or t.shape[2] != d:
        raise TreespecError(f"{name} must be a {dtype} tensor [T][{H}][{d}] on CUDA device {device}, not {t.dtype} "
                            f"{tuple(t.shape)} on {t.device}")
    if t.is_contiguous():
        return t.data_ptr(), H * d
    st, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (H > 1 and sh != d):
        raise TreespecError(f"{name}: heads must be contiguous")
    return t.data_ptr(), H * d if t.shape[0] == 1 else st


def kv_append_slots(kv: PagedKV, k_new, v_new, slot, status=None, stream=None):
    """Rows k_new, v_new [T][H][d] into the pages by their slots (-1: left out). H * d apart or more."""
    ref, dev = _whole_pages(kv), kv.device
    kp, ks = _token_rows(k_new, kv.H, kv.d, "k_new", torch.bfloat16, dev)
    vp, vs = _token_rows(v_new, kv.H, kv.d, "v_new", torch.bfloat16, dev)
    T = k_new.shape[0]
    if v_new.shape[0] != T:
        raise TreespecError(f"k_new of {T} tokens, v_new of {v_new.shape[0]}")
    _run(load_library().kv_append_slots, "kv_append_slots", dev, stream, ref, kp, vp, ks, vs,
         _int_array(slot, T, "slot", dev), T, kv.H, kv.d, _status_ptr(status, dev))


def decode_workspace(B: int, Hq: int, Hkv: int, d: int, device="cuda"):
    """A zero-filled workspace of the size decode_attention_paged needs."""
    with torch.cuda.device(device):
        need = int(load_library().treespec_decode_workspace_size(B, Hq, Hkv, d))
    return torch.zeros(max(256, need), dtype=torch.uint8, device=device)


def decode_attention_paged(out, q, kv: PagedKV, kv_len, scale: float = 0.0, ws=None, status=None, stream=None):
    """Attention of one new token a request to the first kv_len[b] rows of its pages; q, out [B][Hq][d] bfloat16, Hq a
    multiple of kv.H, the rows of q Hq * d apart or more."""
    ref, dev, d, B = _whole_pages(kv), kv.device, kv.d, kv.B
    if q.dim() != 3 or q.shape[0] != B:
        raise TreespecError(f"q must be [{B}][Hq][{d}]")
    Hq = q.shape[1]
    qp, qs = _token_rows(q, Hq, d, "q", torch.bfloat16, dev)
    op = _out_rows(out, (B, Hq, d), "out", torch.bfloat16, dev)
    if ws is None or ws.get_device() != dev or not ws.is_contiguous():
        raise TreespecError(f"a workspace (decode_workspace) on CUDA device {dev} is needed")
    _run(load_library().decode_attention_paged, "decode_attention_paged", dev, stream, op, qp, qs, ref,
         _int_array(kv_len, B, "kv_len", dev), B, Hq, kv.H, d, float(scale), ws.data_ptr(),
         ws.numel() * ws.element_size(), _status_ptr(status, dev))


def _f32_array(t, n, name, device):
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.numel() < n or t.get_device() != device or not t.is_contiguous():
        raise TreespecError(f"{name} must be a contiguous float32 tensor of {n} entries on CUDA device {device}")
    return t.data_ptr()


def sample_tokens(token, logits, u=None, temperature=None, top_k=None, top_p=None, min_p=None, probs=None, kept=None,
                  status=None, stream=None):
    """A token for each row of logits [R][V] (bfloat16 or float32, rows V apart or more) from u [R], under each row's
    temperature, top_k, top_p and min_p [R] (None: 1, all, 1, 0). probs [R][V] float32: the filtered distribution;
    kept [R][V] float32: the logits of what is kept, DROPPED_LOGIT elsewhere (may be the logits themselves). token may
    be None where one of these is asked for."""
    if logits.dim() != 2 or not logits.is_cuda:
        raise TreespecError("logits must be [R][V] on a CUDA device")
    R, V = logits.shape
    dev, stride = logits.get_device(), logits.stride()
    if stride[1] != 1 and V > 1:
        raise TreespecError("a row of logits must be contiguous")
    rows = [None if x is None else _out_rows(x, (R, V), name, torch.float32, dev)
            for x, name in ((probs, "probs"), (kept, "kept"))]
    _run(load_library().sample_tokens, "sample_tokens", dev, stream,
         None if token is None else _int_array(token, R, "token", dev), rows[0], rows[1], logits.data_ptr(),
         stride[0] if R > 1 else V, _dtype(logits), _f32_array(u, R, "u", dev),
         _f32_array(temperature, R, "temperature", dev), None if top_k is None else _int_array(top_k, R, "top_k", dev),
         _f32_array(top_p, R, "top_p", dev), _f32_array(min_p, R, "min_p", dev), R, V, _status_ptr(status, dev))


def version() -> str:
    return load_library().treespec_version().decode()
