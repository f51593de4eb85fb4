"""FreeSolo sparse-attention forward pass on NVIDIA B200 (sm_100a).

Thin Python binding of the C-ABI library libfreesolo.so (include/freesolo.h): it only
marshals arguments (tensor pointers, sizes, the current CUDA stream).  Every step of the
computation runs in the library's CUDA kernels; there is no Python or CPU fallback, and
loading fails loudly if the library has not been built (python -m
long_context_sparse_head_b200.build).

The entry points mirror the C names: `workspace_size`, `cell_summaries`, `select_topk`,
`forward`, `host_scratch_size`, `forward_host`, `sync_status`, `status_string`, and the
FS-L streaming cache `cache_bytes`, `cache_reset`, `cache_append`, `cache_attend`,
`cache_status`.  Serving many sequences at once: `Rotary`, `rope`, `rope_backward` (rotary
positions), `PagedParams`, `paged_append`, `paged_attend` (a cache in pages and attention of
one new token per sequence over it) and `pages_reserve`, `pages_copy`, `pages_fork`,
`pages_free`, `pages_compact` (its pages).
"""
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfreesolo.so")

FS_BF16, FS_F32, FS_F16 = 0, 1, 2
FS_ROPE_MAX_R = 256
STATUS = {0: "FS_OK", 1: "FS_ERR_INVALID_ARG", 2: "FS_ERR_UNSUPPORTED", 3: "FS_ERR_WORKSPACE",
          4: "FS_ERR_CUDA", 5: "FS_ERR_TIMEOUT", 6: "FS_ERR_KERNEL_CHECK"}
EXPORTS = ("fs_workspace_size", "fs_cell_summaries", "fs_select_topk", "fs_forward",
           "fs_host_scratch_size", "fs_forward_host", "fs_sync_status", "fs_status_string",
           "fs_launch_count", "fs_timing_enable", "fs_kernel_times", "fs_kernel_name",
           "fs_select_topk_noalloc", "fs_cache_bytes", "fs_cache_reset", "fs_cache_append",
           "fs_cache_attend", "fs_cache_status", "fs_select_topk_rerank", "fs_forward_rerank",
           "fs_backward_workspace_size", "fs_backward", "fs_forest_bytes", "fs_forest_build",
           "fs_select_topk_tree", "fs_forward_tree", "fs_forest_append", "fs_selftest_timeout",
           "fs_rotary_init", "fs_rope", "fs_rope_backward", "fs_paged_workspace_size", "fs_paged_append",
           "fs_paged_attend", "fs_pages_reserve", "fs_pages_copy", "fs_pages_fork", "fs_pages_free",
           "fs_pages_compact")


class FsError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__("%s: %s (%s)" % (where, STATUS.get(code, code), status_string(code)))


class FsParams(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("H", ctypes.c_int), ("Nq", ctypes.c_int), ("Nk", ctypes.c_int),
        ("d", ctypes.c_int), ("w", ctypes.c_int), ("s", ctypes.c_int), ("K", ctypes.c_int),
        ("W", ctypes.c_int), ("P", ctypes.c_int),
        ("rope_base", ctypes.c_float),
        ("alpha", ctypes.POINTER(ctypes.c_float)),
        ("lambda_", ctypes.POINTER(ctypes.c_float)),
        ("sigma", ctypes.POINTER(ctypes.c_float)),
        ("rms_eps", ctypes.c_float),
        ("dtype", ctypes.c_int),
    ]


class FsRotary(ctypes.Structure):
    _fields_ = [("r", ctypes.c_int), ("layout", ctypes.c_int), ("mscale", ctypes.c_float),
                ("turns", ctypes.c_uint64 * (FS_ROPE_MAX_R // 2))]


class FsRopeParams(ctypes.Structure):
    # the strides q[3], qo[3], k[3], ko[3] field by field (quicker to fill than arrays)
    _fields_ = ([(n, ctypes.c_int) for n in ("B", "N", "H", "Hk", "d")] +
                [(t + "_" + x, ctypes.c_longlong) for t in ("q", "qo", "k", "ko") for x in "bhn"] +
                [("dtype", ctypes.c_int)])


class FsPagedParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("B", "H", "Hkv", "d", "page_size", "num_pages", "max_pages")] +
                [(n, ctypes.c_longlong) for n in ("page_stride", "head_stride", "token_stride")] +
                [("dtype", ctypes.c_int)])


_lib = None


def load():
    """Load libfreesolo.so (raises if it is missing: there is no fallback path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libfreesolo.so is not built; run "
                               "`python -m long_context_sparse_head_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(FsParams)
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        L.fs_workspace_size.argtypes = [P, ctypes.POINTER(sz)]
        L.fs_cell_summaries.argtypes = [P, vp, vp, vp, vp]
        L.fs_select_topk.argtypes = [P, vp, vp, vp, vp, vp, sz, vp]
        L.fs_select_topk_noalloc.argtypes = [P, vp, vp, vp, vp, vp]
        L.fs_select_topk_rerank.argtypes = [P, vp, vp, vp, vp, ctypes.c_int, vp, vp, sz, vp]
        L.fs_forward_rerank.argtypes = [P, vp, vp, vp, vp, vp, ctypes.c_int, vp, vp, vp, sz, vp]
        L.fs_forward.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.fs_host_scratch_size.argtypes = [P, ctypes.POINTER(sz)]
        L.fs_forward_host.argtypes = [P, vp, vp, vp, vp, vp, sz, vp]
        L.fs_sync_status.argtypes = [vp, vp]
        L.fs_status_string.argtypes = [ctypes.c_int]
        L.fs_status_string.restype = ctypes.c_char_p
        L.fs_launch_count.argtypes = []
        L.fs_launch_count.restype = ctypes.c_longlong
        L.fs_timing_enable.argtypes = [ctypes.c_int]
        L.fs_kernel_times.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_longlong),
                                      ctypes.POINTER(ctypes.c_double)]
        L.fs_cache_bytes.argtypes = [P, ctypes.c_int, ctypes.POINTER(sz)]
        L.fs_cache_reset.argtypes = [P, ctypes.c_int, vp, sz, vp]
        L.fs_cache_append.argtypes = [P, ctypes.c_int, vp, sz, vp, vp, ctypes.c_int, vp]
        L.fs_cache_attend.argtypes = [P, ctypes.c_int, vp, sz, vp, ctypes.c_int, vp, vp, vp]
        L.fs_cache_status.argtypes = [vp, vp]
        L.fs_kernel_name.argtypes = [ctypes.c_int]
        L.fs_kernel_name.restype = ctypes.c_char_p
        L.fs_backward_workspace_size.argtypes = [P, ctypes.POINTER(sz)]
        L.fs_backward.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        fp = ctypes.POINTER(ctypes.c_float)
        L.fs_forest_bytes.argtypes = [P, ctypes.POINTER(sz)]
        L.fs_forest_build.argtypes = [P, vp, vp, fp, vp, sz, vp]
        L.fs_forest_append.argtypes = [P, ctypes.c_int, vp, vp, fp, vp, sz, vp]
        L.fs_select_topk_tree.argtypes = [P, vp, vp, sz, ctypes.c_int, ctypes.c_float, vp, vp, sz, vp]
        L.fs_forward_tree.argtypes = [P, vp, vp, vp, fp, ctypes.c_int, ctypes.c_float, vp, vp, vp, sz, vp,
                                      sz, vp]
        L.fs_selftest_timeout.argtypes = [vp, vp]
        i32, i64, f32, f64 = ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_double
        PP = ctypes.POINTER(FsPagedParams)
        L.fs_rotary_init.argtypes = [i32, i32, f64, i32, f64, f64, f64, f64, f64, ctypes.POINTER(FsRotary)]
        L.fs_rope.argtypes = [ctypes.POINTER(FsRopeParams), ctypes.POINTER(FsRotary), vp, vp, vp, vp, vp, i64, i64, vp]
        L.fs_rope_backward.argtypes = L.fs_rope.argtypes
        L.fs_paged_workspace_size.argtypes = [PP, ctypes.POINTER(sz)]
        L.fs_paged_append.argtypes = [PP, ctypes.POINTER(FsRotary), i32, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp,
                                      vp, vp, vp, vp, sz, vp]
        L.fs_paged_attend.argtypes = [PP, vp, i64, vp, vp, vp, vp, i32, f32, vp, i64, vp, vp, sz, vp]
        L.fs_pages_reserve.argtypes = [PP, vp, vp, vp, vp, vp, sz, vp]
        L.fs_pages_copy.argtypes = [PP, vp, vp, vp, vp, i32, vp, sz, vp]
        L.fs_pages_fork.argtypes = [PP, vp, vp, vp, vp, vp, vp, vp, i32, vp, sz, vp]
        L.fs_pages_free.argtypes = [PP, vp, vp, vp, vp, i32, vp, sz, vp]
        L.fs_pages_compact.argtypes = [PP, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        for name in EXPORTS:
            if name not in ("fs_status_string", "fs_launch_count", "fs_kernel_name"):
                getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(code):
    return load().fs_status_string(int(code)).decode()


class Params:
    """fs_params plus the host arrays it points to (kept alive with it).

    Q [B,H,Nq,d], K/V [B,H,Nk,d]; W = P = -1 turns pruning off; lam/sigma None turns the
    erf prior off.  dtype: "bf16" or "f32".
    """

    def __init__(self, *, B, H, Nq, Nk, d=64, w=512, s=32, K=16, W=16, P=48, alpha,
                 lam=None, sigma=None, rope_base=10000.0, rms_eps=1e-6, dtype="bf16"):
        self.alpha = np.ascontiguousarray(alpha, np.float32)
        self.lam = None if lam is None else np.ascontiguousarray(lam, np.float32)
        self.sigma = None if sigma is None else np.ascontiguousarray(sigma, np.float32)
        fp = ctypes.POINTER(ctypes.c_float)
        c = FsParams()
        c.B, c.H, c.Nq, c.Nk, c.d, c.w, c.s, c.K, c.W, c.P = B, H, Nq, Nk, d, w, s, K, W, P
        c.rope_base, c.rms_eps = rope_base, rms_eps
        c.alpha = self.alpha.ctypes.data_as(fp)
        c.lambda_ = self.lam.ctypes.data_as(fp) if self.lam is not None else fp()
        c.sigma = self.sigma.ctypes.data_as(fp) if self.sigma is not None else fp()
        c.dtype = {"bf16": FS_BF16, "f16": FS_F16}.get(dtype, FS_F32)     # f16: refused by these calls
        self.c = c
        self.B, self.H, self.Nq, self.Nk, self.d, self.s, self.K = B, H, Nq, Nk, d, s, K
        self.dtype = dtype

    @property
    def C(self):
        return self.Nk // self.s

    def ref(self):
        return ctypes.byref(self.c)


def _ptr(t):
    # a plain int converts to void * through the argtypes (cheaper than a c_void_p object)
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return getattr(stream, "cuda_stream", stream)


def _check(code, where):
    if code != 0:
        raise FsError(code, where)


def workspace_size(params):
    n = ctypes.c_size_t()
    _check(load().fs_workspace_size(params.ref(), ctypes.byref(n)), "fs_workspace_size")
    return n.value


def host_scratch_size(params):
    n = ctypes.c_size_t()
    _check(load().fs_host_scratch_size(params.ref(), ctypes.byref(n)), "fs_host_scratch_size")
    return n.value


def alloc_workspace(params, device="cuda"):
    """A zero-filled workspace (the device error flag must start at zero)."""
    import torch
    return torch.zeros(workspace_size(params), dtype=torch.uint8, device=device)


def cell_summaries(params, K, kbar, amax, stream=None):
    _check(load().fs_cell_summaries(params.ref(), _ptr(K), _ptr(kbar), _ptr(amax),
                                    _stream(stream)), "fs_cell_summaries")


def select_topk(params, Q, kbar, amax, idx, ws, stream=None):
    _check(load().fs_select_topk(params.ref(), _ptr(Q), _ptr(kbar), _ptr(amax), _ptr(idx),
                                 _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "fs_select_topk")


def select_topk_rerank(params, Q, K, kbar, amax, idx, ws, shortlist=0, stream=None):
    """Selection by the eq. (12) token-level rerank of a shortlist of A_i (0: all of A_i)."""
    _check(load().fs_select_topk_rerank(params.ref(), _ptr(Q), _ptr(K), _ptr(kbar), _ptr(amax),
                                        int(shortlist), _ptr(idx), _ptr(ws),
                                        ws.numel() * ws.element_size(), _stream(stream)),
           "fs_select_topk_rerank")


def forward_rerank(params, Q, K, V, O, ws, kbar=None, amax=None, idx=None, shortlist=0, stream=None):
    """The forward pass with the eq. (12) rerank as its selection (idx: optional output)."""
    _check(load().fs_forward_rerank(params.ref(), _ptr(Q), _ptr(K), _ptr(V), _ptr(kbar), _ptr(amax),
                                    int(shortlist), _ptr(idx), _ptr(O), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)), "fs_forward_rerank")


def select_topk_noalloc(params, Q, kbar, amax, idx, stream=None):
    """fs_select_topk without a workspace, for callers that cannot allocate device memory:
    its scratch is a fixed array inside the library (see include/freesolo.h)."""
    _check(load().fs_select_topk_noalloc(params.ref(), _ptr(Q), _ptr(kbar), _ptr(amax),
                                         _ptr(idx), _stream(stream)), "fs_select_topk_noalloc")


def forward(params, Q, K, V, O, ws, kbar=None, amax=None, idx=None, stream=None):
    _check(load().fs_forward(params.ref(), _ptr(Q), _ptr(K), _ptr(V), _ptr(kbar), _ptr(amax),
                             _ptr(idx), _ptr(O), _ptr(ws), ws.numel() * ws.element_size(),
                             _stream(stream)), "fs_forward")


def forward_host(params, hQ, hK, hV, hO, dscratch, stream=None):
    _check(load().fs_forward_host(params.ref(), _ptr(hQ), _ptr(hK), _ptr(hV), _ptr(hO),
                                  _ptr(dscratch), dscratch.numel() * dscratch.element_size(),
                                  _stream(stream)), "fs_forward_host")


# ---- FS-B: balanced-tree search (eqs. (10)-(11)) --------------------------------------
def forest_bytes(params):
    n = ctypes.c_size_t()
    _check(load().fs_forest_bytes(params.ref(), ctypes.byref(n)), "fs_forest_bytes")
    return n.value


def alloc_forest(params, device="cuda"):
    import torch
    return torch.empty(forest_bytes(params), dtype=torch.uint8, device=device)


def _tau(params, tau):
    if tau is None:
        return None
    arr = (ctypes.c_float * params.H)(*[float(x) for x in tau])
    return ctypes.cast(arr, ctypes.POINTER(ctypes.c_float)), arr


def forest_build(params, kbar, amax, forest, tau=None, stream=None):
    """Both FS-B forests from the cell summaries; tau: per-head thresholds (None: forest 0 only)."""
    t = _tau(params, tau)
    _check(load().fs_forest_build(params.ref(), _ptr(kbar), _ptr(amax), t[0] if t else None, _ptr(forest),
                                  forest.numel() * forest.element_size(), _stream(stream)), "fs_forest_build")


def forest_append(params, prev_cells, kbar, amax, forest, tau=None, stream=None):
    """Rebuild only the trees whose blocks end after cell prev_cells (growing archive)."""
    t = _tau(params, tau)
    _check(load().fs_forest_append(params.ref(), int(prev_cells), _ptr(kbar), _ptr(amax), t[0] if t else None,
                                   _ptr(forest), forest.numel() * forest.element_size(), _stream(stream)),
           "fs_forest_append")


def select_topk_tree(params, Q, forest, idx, ws, beam, c_explore=1.0, stream=None):
    _check(load().fs_select_topk_tree(params.ref(), _ptr(Q), _ptr(forest), forest.numel() * forest.element_size(),
                                      int(beam), ctypes.c_float(c_explore), _ptr(idx), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)), "fs_select_topk_tree")


def forward_tree(params, Q, K, V, O, ws, forest, beam, c_explore=1.0, tau=None, idx=None, stream=None):
    """The forward pass with the FS-B selection (idx: optional output of the selection)."""
    t = _tau(params, tau)
    _check(load().fs_forward_tree(params.ref(), _ptr(Q), _ptr(K), _ptr(V), t[0] if t else None, int(beam),
                                  ctypes.c_float(c_explore), _ptr(idx), _ptr(O), _ptr(ws),
                                  ws.numel() * ws.element_size(), _ptr(forest),
                                  forest.numel() * forest.element_size(), _stream(stream)), "fs_forward_tree")


def backward_workspace_size(params):
    n = ctypes.c_size_t()
    _check(load().fs_backward_workspace_size(params.ref(), ctypes.byref(n)), "fs_backward_workspace_size")
    return n.value


def alloc_backward_workspace(params, device="cuda"):
    """A zero-filled backward workspace (its device error flag must start at zero)."""
    import torch
    return torch.zeros(backward_workspace_size(params), dtype=torch.uint8, device=device)


def backward(params, Q, K, V, idx, dO, dQ, dK, dV, dalpha, bws, stream=None):
    """Gradients of eq. (2) for the upstream gradient dO with the cells idx held fixed:
    dQ, dK, dV (float32, [B,H,N,d]) and dalpha (float32 [H], or None)."""
    _check(load().fs_backward(params.ref(), _ptr(Q), _ptr(K), _ptr(V), _ptr(idx), _ptr(dO),
                              _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(dalpha), _ptr(bws),
                              bws.numel() * bws.element_size(), _stream(stream)), "fs_backward")


def selftest_timeout(ws, stream=None):
    """Enqueue a kernel whose bounded wait runs out (about 2 s): the next sync_status(ws)
    raises FsError with FS_ERR_TIMEOUT."""
    _check(load().fs_selftest_timeout(_ptr(ws), _stream(stream)), "fs_selftest_timeout")


def sync_status(ws, stream=None):
    code = load().fs_sync_status(_ptr(ws), _stream(stream))
    _check(code, "fs_sync_status")


# ---- FS-L streaming cache ----------------------------------------------------------
def cache_bytes(params, max_block):
    n = ctypes.c_size_t()
    _check(load().fs_cache_bytes(params.ref(), int(max_block), ctypes.byref(n)), "fs_cache_bytes")
    return n.value


def alloc_cache(params, max_block, device="cuda", stream=None):
    """A cache buffer of cache_bytes(params, max_block) bytes, emptied by fs_cache_reset."""
    import torch
    cache = torch.empty(cache_bytes(params, max_block), dtype=torch.uint8, device=device)
    cache_reset(params, max_block, cache, stream)
    return cache


def cache_reset(params, max_block, cache, stream=None):
    _check(load().fs_cache_reset(params.ref(), int(max_block), _ptr(cache), cache.numel(),
                                 _stream(stream)), "fs_cache_reset")


def cache_append(params, max_block, cache, K_new, V_new, stream=None):
    """Appends K_new, V_new [B,H,n_new,d] (n_new <= max_block) to the stream."""
    _check(load().fs_cache_append(params.ref(), int(max_block), _ptr(cache), cache.numel(),
                                  _ptr(K_new), _ptr(V_new), int(K_new.shape[2]), _stream(stream)),
           "fs_cache_append")


def cache_attend(params, max_block, cache, Q_new, O, idx=None, stream=None):
    """O [B,H,n_q,d] for the n_q = Q_new.shape[2] most recent positions."""
    _check(load().fs_cache_attend(params.ref(), int(max_block), _ptr(cache), cache.numel(),
                                  _ptr(Q_new), int(Q_new.shape[2]), _ptr(idx), _ptr(O),
                                  _stream(stream)), "fs_cache_attend")


def cache_status(cache, stream=None):
    _check(load().fs_cache_status(_ptr(cache), _stream(stream)), "fs_cache_status")


# ---- serving: what the calls below share ---------------------------------------------
# A decoding step makes a few of these calls, each a few microseconds on the GPU, so the checks
# compare whole tuples first and look closer only where those differ.
_INT = 0x7fffffff                              # the library counts in C ints; ctypes would cut what is larger


def _refuse(where, what):
    raise FsError(1, "%s: %s" % (where, what))


def _too_many(where):
    raise FsError(2, "%s: a size past 2^31 - 1" % where)


_torch = _raw_stream = _raw_device = None
_DTYPES = {}


def _types():
    """torch, once it is imported, and the element types of the serving calls."""
    global _torch, _raw_stream, _raw_device
    if _torch is None:
        import torch
        # handles of the current stream and device (the public call makes a stream object, 1.2 us)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        _raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _DTYPES.update({torch.bfloat16: FS_BF16, torch.float32: FS_F32, torch.float16: FS_F16})
        _torch = torch
    return _torch


def _dtype(t, where):
    if _torch is None:
        _types()
    code = _DTYPES.get(t.dtype)
    if code is None:
        _refuse(where, "tensors are bf16, f16 or f32")
    return code


def _one_device(where, *tensors):
    dev = tensors[0].get_device()
    if dev < 0:
        _refuse(where, "tensors are on a CUDA device")
    for t in tensors:
        if t.get_device() != dev:
            _refuse(where, "all tensors are on one device")
    return dev


def _call(fn, where, dev, stream, *args):
    """fn(*args, stream) with device dev current; on that device's current stream unless given."""
    if _torch is None:
        _types()
    stream = _raw_stream(dev) if stream is None else _stream(stream)
    if _raw_device() == dev:
        code = fn(*args, stream)
    else:
        with _torch.cuda.device(dev):
            code = fn(*args, stream)
    if code:
        raise FsError(code, where)


def _run(fn, where, stream, tensors, *args):
    _call(fn, where, _one_device(where, *tensors), stream, *args)


# ---- rotary positions ----------------------------------------------------------------
class Rotary:
    """A rotation of the first r elements of a row: layout "interleaved" (pairs 2m, 2m+1) or
    "half" (pairs m, m + r/2); frequencies base^(-2m/r), for contexts longer by `factor` scaled
    "linear", "ntk" or "by_parts" (orig_len, slow, fast); mscale multiplies what is rotated."""
    LAYOUTS = {"interleaved": 0, "half": 1}
    SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}

    def __init__(self, r, layout="interleaved", base=10000.0, scaling="none", factor=1.0, orig_len=0.0, slow=1.0,
                 fast=32.0, mscale=1.0):
        if layout not in self.LAYOUTS or scaling not in self.SCALINGS:
            _refuse("Rotary", "layout or scaling unknown")
        self.c = FsRotary()
        _check(load().fs_rotary_init(int(r), self.LAYOUTS[layout], base, self.SCALINGS[scaling], factor, orig_len,
                                     slow, fast, mscale, ctypes.byref(self.c)), "fs_rotary_init")
        self.r, self.layout = int(r), layout

    def ref(self):
        return ctypes.byref(self.c)


def _rope(fn, where, rotary, Q, Qo, K, Ko, positions, pos0, stream):
    shape = Q.shape
    if len(shape) != 4 or Qo.shape != shape or Qo.dtype != Q.dtype:
        _refuse(where, "Q and its output are [B,H,N,d] of one type")
    B, H, N, d = shape
    Hk, ts, ks_, kos = 0, [Q, Qo], (0, 0, 0, 1), (0, 0, 0, 1)
    if K is not None and Ko is not None:
        ks = K.shape
        if len(ks) != 4 or Ko.shape != ks or not K.dtype == Ko.dtype == Q.dtype or (ks[0], ks[2], ks[3]) != (B, N, d):
            _refuse(where, "K and its output are [B,Hk,N,d] of Q's type")
        Hk, ks_, kos = ks[1], K.stride(), Ko.stride()
        ts += [K, Ko]
    elif K is not None or Ko is not None:
        _refuse(where, "K and its output come together")
    if max(shape) > _INT or Hk > _INT:
        _too_many(where)
    qs, qos = Q.stride(), Qo.stride()
    if d > 1 and not qs[3] == qos[3] == ks_[3] == kos[3] == 1:
        _refuse(where, "a row's elements are contiguous")
    ps = 0
    if positions is not None:
        if positions.dtype is not (_torch or _types()).int32:
            _refuse(where, "positions are int32")
        st = positions.stride()
        if positions.shape not in ((B, N), (N,)) or (N > 1 and st[-1] != 1):
            _refuse(where, "positions are [N] or [B,N], a row contiguous")
        if len(st) == 2:
            ps = st[0]
        ts.append(positions)
    c = FsRopeParams(B, N, H, Hk, d, qs[0], qs[1], qs[2], qos[0], qos[1], qos[2], ks_[0], ks_[1], ks_[2], kos[0], kos[1],
                     kos[2], _dtype(Q, where))
    _run(fn, where, stream, ts, c, rotary.c, Q.data_ptr(), Qo.data_ptr(), _ptr(K), _ptr(Ko), _ptr(positions), ps, int(pos0))


def rope(rotary, Q, Qo, K=None, Ko=None, positions=None, pos0=0, stream=None):
    """Rotates Q [B,H,N,d] into Qo and K [B,Hk,N,d] into Ko (views of any strides with contiguous
    rows; an output may be its input): token (b, n) by positions[b, n] or [n] (int32), or pos0 + n."""
    _rope(load().fs_rope, "fs_rope", rotary, Q, Qo, K, Ko, positions, pos0, stream)


def rope_backward(rotary, dQo, dQ, dKo=None, dK=None, positions=None, pos0=0, stream=None):
    """Gradients of rope: dQ, dK from the gradients dQo, dKo of its outputs."""
    _rope(load().fs_rope_backward, "fs_rope_backward", rotary, dQo, dQ, dKo, dK, positions, pos0, stream)


# ---- paged key-value cache -----------------------------------------------------------
class PagedParams:
    """fs_paged_params: B sequences over a pool of num_pages pages of page_size tokens; H query
    and Hkv key-value heads of dim d.  The pools are tensors [num_pages, Hkv, page_size, d] with
    these strides (elements): layout "heads_first" (contiguous) or "tokens_first" (a view of
    [num_pages, page_size, Hkv, d]), or `strides` of one's own (page, head, token)."""

    def __init__(self, *, B, H, Hkv, page_size, num_pages, max_pages, d=64, dtype="bf16", layout="heads_first",
                 strides=None):
        if max(B, H, Hkv, d, page_size, num_pages, max_pages) > _INT:
            _too_many("PagedParams")
        if dtype not in ("bf16", "f32", "f16") or layout not in ("heads_first", "tokens_first"):
            _refuse("PagedParams", "dtype or layout unknown")
        if strides is None:
            page = Hkv * page_size * d
            strides = (page, page_size * d, d) if layout == "heads_first" else (page, d, Hkv * d)
        self.B, self.H, self.Hkv, self.d, self.dtype = B, H, Hkv, d, dtype
        self.page_size, self.num_pages, self.max_pages = page_size, num_pages, max_pages
        self.shape, self.strides = (num_pages, Hkv, page_size, d), tuple(int(x) for x in strides)
        self.scale = d ** -0.5 if d > 0 else 0.0
        self.stride4, self.table_shape, self.table_stride = self.strides + (1,), (B, max_pages), (max_pages, 1)
        self.code = {"bf16": FS_BF16, "f32": FS_F32, "f16": FS_F16}[dtype]
        torch = _types()
        self.dt = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}[dtype]
        self.int32, self.row_shape, self.lens_shape = torch.int32, (B, H, d), (B,)
        self.c = FsPagedParams(B, H, Hkv, d, page_size, num_pages, max_pages, *self.strides, self.code)
        paged_workspace_size(self)             # refuses what is not supported

    def ref(self):
        return ctypes.byref(self.c)


def paged_workspace_size(params):
    n = ctypes.c_size_t()
    _check(load().fs_paged_workspace_size(params.ref(), ctypes.byref(n)), "fs_paged_workspace_size")
    return n.value


def alloc_paged_workspace(params, device="cuda"):
    """A zero-filled workspace for the paged calls (its flag and counters must start at zero)."""
    import torch
    return torch.zeros(paged_workspace_size(params), dtype=torch.uint8, device=device)


def alloc_pages(params, device="cuda"):
    """An empty cache: pools Kp, Vp (contents undefined), refs, table and lens."""
    import torch
    size = sum((n - 1) * s for n, s in zip(params.shape, params.strides)) + params.d
    Kp, Vp = (torch.empty(size, dtype=params.dt, device=device).as_strided(params.shape, params.strides + (1,))
              for _ in range(2))
    refs = torch.zeros(params.num_pages, dtype=torch.int32, device=device)
    table = torch.full((params.B, params.max_pages), -1, dtype=torch.int32, device=device)
    return Kp, Vp, refs, table, torch.zeros(params.B, dtype=torch.int32, device=device)


def _pools(p, where, Kp, Vp):
    if not Kp.shape == Vp.shape == p.shape or Kp.dtype is not p.dt or Vp.dtype is not p.dt:
        _refuse(where, "pools have the shape and type of the parameters")
    if not Kp.stride() == Vp.stride() == p.stride4:
        for t in (Kp, Vp):                     # the stride of a dimension of one says nothing
            st = t.stride()
            if st[3] != 1 or any(n > 1 and a != b for n, a, b in zip(p.shape, st, p.strides)):
                _refuse(where, "pools have the strides of the parameters")


def _ints(where, n, *tensors):
    int32 = (_torch or _types()).int32
    if n > _INT:
        _too_many(where)
    for t in tensors:
        if t.dtype is not int32 or t.shape != (n,) or (n > 1 and t.stride(0) != 1):
            _refuse(where, "a list is contiguous int32 of the length that goes with the others")


def _table(p, where, table, lens=None):
    if table.dtype is not p.int32 or table.shape != p.table_shape or not (
            table.stride() == p.table_stride or table.is_contiguous()):
        _refuse(where, "table is contiguous int32 [B, max_pages]")
    if lens is not None and (lens.dtype is not p.int32 or lens.shape != p.lens_shape or not lens.is_contiguous()):
        _refuse(where, "lens is contiguous int32 [B]")


def _rows(p, where, t, shape):
    """A [rows, heads, d] tensor with heads d apart: its row stride."""
    st = t.stride()
    if t.shape != shape or t.dtype is not p.dt or st[2] != 1 or (st[1] != p.d and shape[1] > 1):
        _refuse(where, "rows are [rows, heads, d] of the cache's type and sizes, a row's heads contiguous")
    return st[0]


def paged_append(params, K_new, V_new, Kp, Vp, table, lens, ws, cu=None, rotary=None, Q=None, Qo=None, stream=None):
    """Writes the newest tokens into their pages: K_new, V_new [T, Hkv, d]; sequence b's are the
    rows cu[b] .. cu[b+1]-1 at its last positions (cu None: row b at lens[b] - 1).  With `rotary`
    the keys are rotated on the way and Q [T, H, d] into Qo."""
    where, p, T = "fs_paged_append", params, K_new.shape[0]
    dt, d, kv = p.dt, p.d, (T, p.Hkv, p.d)
    if T > _INT:
        _too_many(where)
    ks, vs = K_new.stride(), V_new.stride()
    if not (K_new.shape == V_new.shape == kv and Kp.shape == Vp.shape == p.shape and
            K_new.dtype is dt and V_new.dtype is dt and Kp.dtype is dt and Vp.dtype is dt and
            ks[1] == vs[1] == d and ks[2] == vs[2] == 1 and Kp.stride() == Vp.stride() == p.stride4):
        _rows(p, where, K_new, kv)             # what is wrong, or a dimension of one, whose stride says nothing
        _rows(p, where, V_new, kv)
        _pools(p, where, Kp, Vp)
    _table(p, where, table, lens)
    dev = K_new.get_device()
    if not V_new.get_device() == Kp.get_device() == Vp.get_device() == table.get_device() == lens.get_device() == \
            ws.get_device() == dev >= 0:
        _one_device(where, K_new, V_new, Kp, Vp, table, lens, ws)
    qs = qos = 0
    if Q is not None and Qo is not None:
        q = (T, p.H, d)
        qs, qos = _rows(p, where, Q, q), _rows(p, where, Qo, q)
        if not Q.get_device() == Qo.get_device() == dev:
            _refuse(where, "all tensors are on one device")
    elif Q is not None or Qo is not None:
        _refuse(where, "Q and Qo come together")
    if cu is not None:
        _ints(where, p.B + 1, cu)
        if cu.get_device() != dev:
            _refuse(where, "all tensors are on one device")
    _call(load().fs_paged_append, where, dev, stream, p.c, None if rotary is None else rotary.c, T, _ptr(Q), qs, _ptr(Qo),
          qos, K_new.data_ptr(), ks[0], V_new.data_ptr(), vs[0], _ptr(cu), Kp.data_ptr(), Vp.data_ptr(),
          table.data_ptr(), lens.data_ptr(), ws.data_ptr(), ws.nbytes)


def paged_attend(params, Q, Kp, Vp, table, lens, O, ws, lse=None, window=-1, scale=None, stream=None):
    """O [B, H, d] = attention of each sequence's newest token, query row Q[b], over its pages: all
    of them, or the last window + 1 tokens.  scale None: 1/sqrt(d).  lse: optional float32 [B, H]."""
    where, p = "fs_paged_attend", params
    qs, os_, dt, d = Q.stride(), O.stride(), p.dt, p.d
    if not (Q.shape == O.shape == p.row_shape and Kp.shape == Vp.shape == p.shape and
            Q.dtype is dt and O.dtype is dt and Kp.dtype is dt and Vp.dtype is dt and
            qs[1] == os_[1] == d and qs[2] == os_[2] == 1 and Kp.stride() == Vp.stride() == p.stride4):
        _rows(p, where, Q, p.row_shape)        # what is wrong, or a dimension of one, whose stride says nothing
        _rows(p, where, O, p.row_shape)
        _pools(p, where, Kp, Vp)
    _table(p, where, table, lens)
    dev = Q.get_device()
    if not Kp.get_device() == Vp.get_device() == table.get_device() == lens.get_device() == O.get_device() == \
            ws.get_device() == dev >= 0:
        _one_device(where, Q, Kp, Vp, table, lens, O, ws)
    if lse is not None:
        if _dtype(lse, where) != FS_F32 or lse.shape != (p.B, p.H) or not lse.is_contiguous():
            _refuse(where, "lse is contiguous float32 [B, H]")
        if lse.get_device() != dev:
            _refuse(where, "all tensors are on one device")
    if not -1 <= window <= _INT:
        window = -1 if window < 0 else _INT
    _call(load().fs_paged_attend, where, dev, stream, p.c, Q.data_ptr(), qs[0], Kp.data_ptr(), Vp.data_ptr(),
          table.data_ptr(), lens.data_ptr(), int(window), p.scale if scale is None else scale, O.data_ptr(), os_[0],
          _ptr(lse), ws.data_ptr(), ws.nbytes)


def pages_reserve(params, n_new, refs, table, lens, ws, stream=None):
    """Room for n_new[b] (int32) more tokens of every sequence; lens grows by them."""
    where, p = "fs_pages_reserve", params
    _ints(where, p.B, n_new)
    _ints(where, p.num_pages, refs)
    _table(p, where, table, lens)
    _run(load().fs_pages_reserve, where, stream, (n_new, refs, table, lens, ws), p.c, n_new.data_ptr(), refs.data_ptr(),
         table.data_ptr(), lens.data_ptr(), ws.data_ptr(), ws.nbytes)


def pages_copy(params, Kp, Vp, src, dst, ws, stream=None):
    """Page dst[i] of both pools becomes a copy of page src[i] (int32)."""
    where, p, n = "fs_pages_copy", params, src.numel()
    _pools(p, where, Kp, Vp)
    _ints(where, n, src, dst)
    _run(load().fs_pages_copy, where, stream, (Kp, Vp, src, dst, ws), p.c, Kp.data_ptr(), Vp.data_ptr(), src.data_ptr(),
         dst.data_ptr(), n, ws.data_ptr(), ws.nbytes)


def pages_fork(params, Kp, Vp, refs, table, lens, src, dst, ws, stream=None):
    """The empty sequences dst[i] become branches of src[i] (int32): whole pages shared, a
    part-filled last page copied."""
    where, p, n = "fs_pages_fork", params, src.numel()
    _pools(p, where, Kp, Vp)
    _ints(where, p.num_pages, refs)
    _table(p, where, table, lens)
    _ints(where, n, src, dst)
    _run(load().fs_pages_fork, where, stream, (Kp, Vp, refs, table, lens, src, dst, ws), p.c, Kp.data_ptr(),
         Vp.data_ptr(), refs.data_ptr(), table.data_ptr(), lens.data_ptr(), src.data_ptr(), dst.data_ptr(), n,
         ws.data_ptr(), ws.nbytes)


def pages_free(params, refs, table, lens, rows, ws, stream=None):
    """The sequences rows[i] (int32) give their pages back and are empty."""
    where, p, n = "fs_pages_free", params, rows.numel()
    _ints(where, p.num_pages, refs)
    _table(p, where, table, lens)
    _ints(where, n, rows)
    _run(load().fs_pages_free, where, stream, (refs, table, lens, rows, ws), p.c, refs.data_ptr(), table.data_ptr(),
         lens.data_ptr(), rows.data_ptr(), n, ws.data_ptr(), ws.nbytes)


def pages_compact(params, Kp, Vp, refs, table, ws, live=None, refs_out=None, table_out=None, stream=None):
    """Packs the pages in use to the pool's front.  refs and table are rewritten, or refs_out and
    table_out receive the packed cache's; live (int32 [1]) receives the number of pages in use."""
    where, p = "fs_pages_compact", params
    refs_out, table_out = refs if refs_out is None else refs_out, table if table_out is None else table_out
    _pools(p, where, Kp, Vp)
    _ints(where, p.num_pages, refs, refs_out)
    _table(p, where, table)
    _table(p, where, table_out)
    ts = [Kp, Vp, refs, table, refs_out, table_out, ws]
    if live is not None:
        _ints(where, 1, live)
        ts.append(live)
    _run(load().fs_pages_compact, where, stream, ts, p.c, Kp.data_ptr(), Vp.data_ptr(), refs.data_ptr(),
         table.data_ptr(), refs_out.data_ptr(), table_out.data_ptr(), _ptr(live), ws.data_ptr(), ws.nbytes)


# ---- diagnostics -------------------------------------------------------------------
def launch_count():
    """Kernels the library has launched since it was loaded."""
    return load().fs_launch_count()


def timing_enable(on=True):
    load().fs_timing_enable(1 if on else 0)


def kernel_times():
    """{kernel name: (launches, summed device ms)} since the previous read (then cleared)."""
    n = 64
    cnt = (ctypes.c_longlong * n)()
    ms = (ctypes.c_double * n)()
    k = load().fs_kernel_times(n, cnt, ms)
    out = {}
    for i in range(min(k, n)):
        name = load().fs_kernel_name(i).decode()
        out[name] = (cnt[i], ms[i])
    return out
