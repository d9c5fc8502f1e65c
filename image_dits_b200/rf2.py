"""Python binding of the C ABI in ``include/rf2.h`` (ctypes; marshalling only).

Every step of the path runs in ``librf2.so``'s CUDA kernels.  PyTorch only
provides device memory and the current stream.  There is no fallback: if the
library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librf2.so")
CHECKED_LIB_PATH = os.path.join(_HERE, "librf2_checked.so")     # built with RF2_CHECKED=1

RF2_OK = 0
RF2_ERR_INVALID_ARGUMENT = 1
RF2_ERR_UNSUPPORTED = 2
RF2_ERR_INSUFFICIENT_WORKSPACE = 3
RF2_ERR_CUDA = 4
RF2_ERR_TIMEOUT = 5
RF2_ERR_RANGE = 6

# Every entry point declared in include/rf2.h.
EXPORTED = (
    "rf2_status_string", "rf2_query", "rf2_permutation_index", "rf2_permute", "rf2_unpermute",
    "rf2_predict_mask", "rf2_predict_mask_static", "rf2_permute_qk_pool", "rf2_predict_mask_pooled",
    "rf2_predict_mask_cdf", "rf2_predict_mask_cdf_pooled",
    "rf2_block_sparse_attn", "rf2_device_status", "rf2_selftest_wait_timeout",
    "rf2_attention_host_query", "rf2_attention_host", "rf2_host_events_create", "rf2_host_events_destroy",
    "rf2_layer_query", "rf2_rope_table_floats", "rf2_rope_table", "rf2_norm_rope_permute",
    "rf2_norm_rope_permute_backward", "rf2_block_sparse_attn_mod", "rf2_block_sparse_attn_backward",
    "rf2_predict_mask_visible",
)


class Geometry(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "heads", "head_dim", "frames", "height", "width",
        "win_t", "win_h", "win_w", "block", "first_frame_sink", "text_tokens")]


class Sizes(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("num_blocks", ctypes.c_int32),
        ("n_keep", ctypes.c_int32),
        ("sink_first", ctypes.c_int32),
        ("row_capacity", ctypes.c_int32),
        ("num_rows", ctypes.c_int64),
        ("col_idx_capacity", ctypes.c_int64),
        ("mask_workspace_bytes", ctypes.c_size_t),
    ]


class LayerSizes(ctypes.Structure):
    _fields_ = [("norm_rope_backward_bytes", ctypes.c_size_t), ("score_mod_bytes", ctypes.c_size_t),
                ("attn_backward_bytes", ctypes.c_size_t)]


class View(ctypes.Structure):
    """rf2_view: a bf16 tensor [B, H, N, d] by element strides."""
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64)]


class NormRope(ctypes.Structure):
    _fields_ = [("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("rope", ctypes.c_void_p), ("rope_split", ctypes.c_int32 * 3),
                ("interleaved", ctypes.c_int32)]


class ScoreModStruct(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("distance_t", ctypes.c_float), ("distance_h", ctypes.c_float),
                ("distance_w", ctypes.c_float), ("slopes", ctypes.c_void_p), ("document", ctypes.c_void_p),
                ("order", ctypes.c_void_p)]


class Rf2Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


_lib = None


def lib():
    """Load librf2.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        _lib = load(LIB_PATH)
    return _lib


def use_library(path: str):
    """Route every call of this module through the library at `path` (for
    example CHECKED_LIB_PATH); returns the one it replaces (None if none was
    loaded yet)."""
    global _lib
    old = _lib
    _lib = load(path)
    return old


def load(path: str):
    """Load a build of the library and declare its entry points."""
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} (run image_dits_b200.build.build())")
    L = ctypes.CDLL(path)
    vp, i32, f64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_double, ctypes.c_size_t
    G = ctypes.POINTER(Geometry)
    L.rf2_status_string.argtypes = [i32]
    L.rf2_status_string.restype = ctypes.c_char_p
    L.rf2_query.argtypes = [G, f64, ctypes.POINTER(Sizes)]
    L.rf2_permutation_index.argtypes = [G, vp]
    L.rf2_permute.argtypes = [G, vp, vp, vp]
    L.rf2_unpermute.argtypes = [G, vp, vp, vp]
    L.rf2_predict_mask.argtypes = [G, vp, vp, f64, vp, vp, vp, vp, sz, vp]
    L.rf2_predict_mask_static.argtypes = [G, vp, vp, f64, vp, vp, vp, vp]
    L.rf2_permute_qk_pool.argtypes = [G, vp, vp, vp, vp, vp, sz, vp]
    L.rf2_predict_mask_pooled.argtypes = [G, f64, vp, vp, vp, vp, sz, vp]
    L.rf2_predict_mask_cdf.argtypes = [G, vp, vp, f64, vp, vp, vp, vp, sz, vp]
    L.rf2_predict_mask_cdf_pooled.argtypes = [G, f64, vp, vp, vp, vp, sz, vp]
    L.rf2_block_sparse_attn.argtypes = [G, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.rf2_device_status.argtypes = [vp]
    L.rf2_selftest_wait_timeout.argtypes = [ctypes.c_uint32, ctypes.POINTER(ctypes.c_int32), vp]
    L.rf2_attention_host_query.argtypes = [G, f64, f64, i32, ctypes.POINTER(HostSizes)]
    L.rf2_attention_host.argtypes = [G, f64, f64, i32, vp, vp, vp, vp, vp, sz, vp, vp, vp,
                                     ctypes.POINTER(vp), i32]
    L.rf2_host_events_create.argtypes = [i32, ctypes.POINTER(vp)]
    L.rf2_host_events_destroy.argtypes = [i32, ctypes.POINTER(vp)]
    P, V, M = ctypes.POINTER(NormRope), ctypes.POINTER(View), ctypes.POINTER(ScoreModStruct)
    L.rf2_layer_query.argtypes = [G, ctypes.POINTER(LayerSizes)]
    L.rf2_rope_table_floats.argtypes = [G, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int64)]
    L.rf2_rope_table.argtypes = [G, ctypes.POINTER(ctypes.c_int32), f64, vp]
    L.rf2_norm_rope_permute.argtypes = [G, P, V, V, V, vp, vp, vp, vp, sz, vp]
    L.rf2_norm_rope_permute_backward.argtypes = [G, P, V, V, vp, vp, vp, V, V, V, vp, vp, vp, sz, vp]
    L.rf2_block_sparse_attn_mod.argtypes = [G, vp, vp, vp, vp, vp, vp, M, vp, vp, vp, sz, vp]
    L.rf2_block_sparse_attn_backward.argtypes = [G, vp, vp, vp, vp, vp, vp, vp, vp, vp, M, vp, vp, vp, vp, sz, vp]
    L.rf2_predict_mask_visible.argtypes = [G, f64, M, vp, vp, vp, vp, sz, vp, sz, vp]
    for name in EXPORTED:
        if name != "rf2_status_string":
            getattr(L, name).restype = i32
    return L


def status_string(status: int) -> str:
    return lib().rf2_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != RF2_OK:
        raise Rf2Error(status, what)


def make_geometry(batch, heads, head_dim, frames, height, width, win_t, win_h, win_w, sink, block=64,
                  text=0) -> Geometry:
    return Geometry(batch, heads, head_dim, frames, height, width, win_t, win_h, win_w, block, int(bool(sink)),
                    int(text))


def num_tokens(geom: Geometry) -> int:
    """Sequence length N: video tokens, then text tokens."""
    return geom.frames * geom.height * geom.width + geom.text_tokens


def geometry_of(wl, batch: int | None = None) -> Geometry:
    """Geometry of a ``workload.Workload``."""
    return make_geometry(wl.batch if batch is None else batch, wl.heads, wl.head_dim, wl.frames, wl.height,
                         wl.width, wl.win_t, wl.win_h, wl.win_w, wl.sink, text=wl.text_tokens)


def query(geom: Geometry, keep: float = 1.0) -> Sizes:
    out = Sizes()
    _check(lib().rf2_query(ctypes.byref(geom), float(keep), ctypes.byref(out)), "rf2_query")
    return out


def permutation_index(geom: Geometry) -> np.ndarray:
    perm = np.empty(num_tokens(geom), dtype=np.int32)
    _check(lib().rf2_permutation_index(ctypes.byref(geom), perm.ctypes.data), "rf2_permutation_index")
    return perm


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _shape(geom: Geometry) -> tuple:
    return geom.batch, geom.heads, num_tokens(geom), geom.head_dim


def _check_qkv(geom: Geometry, *ts):
    shape = _shape(geom)
    for t in ts:
        if not (t.is_cuda and t.dtype is torch.bfloat16 and t.is_contiguous() and t.shape == shape):
            raise ValueError(f"expected a contiguous CUDA bf16 tensor of shape {shape}, got "
                             f"{tuple(t.shape)} {t.dtype} {t.device}")


def permute(geom: Geometry, x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _check_qkv(geom, x)
    out = torch.empty_like(x) if out is None else out
    _check_qkv(geom, out)
    _check(lib().rf2_permute(ctypes.byref(geom), x.data_ptr(), out.data_ptr(), _stream(stream)), "rf2_permute")
    return out


def unpermute(geom: Geometry, xp: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _check_qkv(geom, xp)
    out = torch.empty_like(xp) if out is None else out
    _check_qkv(geom, out)
    _check(lib().rf2_unpermute(ctypes.byref(geom), xp.data_ptr(), out.data_ptr(), _stream(stream)), "rf2_unpermute")
    return out


@dataclass
class BlockMask:
    """CSR block mask: row r = (b*heads + h)*T_b + i keeps
    col_idx[row_start[r] : row_start[r] + row_count[r]] (ascending)."""
    row_start: torch.Tensor
    row_count: torch.Tensor
    col_idx: torch.Tensor
    sizes: Sizes

    def dense(self) -> np.ndarray:
        """[B*H, T_b, T_b] uint8 on the host (for tests)."""
        Tb = self.sizes.num_blocks
        rs = self.row_start.cpu().numpy().astype(np.int64)
        rc = self.row_count.cpu().numpy().astype(np.int64)
        ci = self.col_idx.cpu().numpy()
        out = np.zeros((rs.size, Tb), np.uint8)
        for r in range(rs.size):
            out[r, ci[rs[r]:rs[r] + rc[r]]] = 1
        return out.reshape(-1, Tb, Tb)

    def kept_pairs(self) -> int:
        return int(self.row_count.sum().item())


def alloc_mask(geom: Geometry, keep: float, device) -> tuple:
    sz = query(geom, keep)
    row_start = torch.empty(sz.num_rows, dtype=torch.int32, device=device)
    row_count = torch.empty(sz.num_rows, dtype=torch.int32, device=device)
    col_idx = torch.empty(max(1, sz.col_idx_capacity), dtype=torch.int32, device=device)
    ws = torch.empty(max(16, sz.mask_workspace_bytes), dtype=torch.uint8, device=device)
    return BlockMask(row_start, row_count, col_idx, sz), ws


def predict_mask(geom: Geometry, qp: torch.Tensor, kp: torch.Tensor, keep: float, mask: BlockMask | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> BlockMask:
    _check_qkv(geom, qp, kp)
    if mask is None or workspace is None:
        m2, ws2 = alloc_mask(geom, keep, qp.device)
        mask = mask or m2
        workspace = ws2 if workspace is None else workspace
    _check(lib().rf2_predict_mask(ctypes.byref(geom), qp.data_ptr(), kp.data_ptr(), float(keep),
                                  mask.row_start.data_ptr(), mask.row_count.data_ptr(), mask.col_idx.data_ptr(),
                                  workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                  _stream(stream)), "rf2_predict_mask")
    return mask


def predict_mask_cdf(geom: Geometry, qp: torch.Tensor, kp: torch.Tensor, tau: float, mask: BlockMask | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> BlockMask:
    """CDF-threshold mask (rows sized at full capacity: alloc_mask(geom, 1.0, ...))."""
    _check_qkv(geom, qp, kp)
    if mask is None or workspace is None:
        m2, ws2 = alloc_mask(geom, 1.0, qp.device)
        mask = mask or m2
        workspace = ws2 if workspace is None else workspace
    _check(lib().rf2_predict_mask_cdf(ctypes.byref(geom), qp.data_ptr(), kp.data_ptr(), float(tau),
                                      mask.row_start.data_ptr(), mask.row_count.data_ptr(), mask.col_idx.data_ptr(),
                                      workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                      _stream(stream)), "rf2_predict_mask_cdf")
    return mask


def predict_mask_cdf_pooled(geom: Geometry, tau: float, mask: BlockMask, workspace: torch.Tensor,
                            stream=None) -> BlockMask:
    """CDF-threshold mask from the block means rf2_permute_qk_pool left in `workspace`."""
    _check(lib().rf2_predict_mask_cdf_pooled(ctypes.byref(geom), float(tau), mask.row_start.data_ptr(),
                                             mask.row_count.data_ptr(), mask.col_idx.data_ptr(),
                                             workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                             _stream(stream)), "rf2_predict_mask_cdf_pooled")
    return mask


def permute_qk_pool(geom: Geometry, q: torch.Tensor, k: torch.Tensor, workspace: torch.Tensor,
                    qp: torch.Tensor | None = None, kp: torch.Tensor | None = None, stream=None):
    """Permute Q and K and leave their block means in the mask workspace."""
    _check_qkv(geom, q, k)
    qp = torch.empty_like(q) if qp is None else qp
    kp = torch.empty_like(k) if kp is None else kp
    _check_qkv(geom, qp, kp)
    _check(lib().rf2_permute_qk_pool(ctypes.byref(geom), q.data_ptr(), k.data_ptr(), qp.data_ptr(), kp.data_ptr(),
                                     workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                     _stream(stream)), "rf2_permute_qk_pool")
    return qp, kp


def predict_mask_pooled(geom: Geometry, keep: float, mask: BlockMask, workspace: torch.Tensor,
                        stream=None) -> BlockMask:
    """Mask prediction from the block means rf2_permute_qk_pool left in `workspace`."""
    _check(lib().rf2_predict_mask_pooled(ctypes.byref(geom), float(keep), mask.row_start.data_ptr(),
                                         mask.row_count.data_ptr(), mask.col_idx.data_ptr(), workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(), _stream(stream)),
           "rf2_predict_mask_pooled")
    return mask


def block_sparse_attn(geom: Geometry, qp, kp, vp, mask: BlockMask, out: torch.Tensor | None = None,
                      lse: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _check_qkv(geom, qp, kp, vp)
    out = torch.empty_like(qp) if out is None else out
    _check_qkv(geom, out)
    if lse is not None:
        n = num_tokens(geom)
        if not (lse.is_cuda and lse.dtype == torch.float32 and lse.is_contiguous()
                and lse.numel() == geom.batch * geom.heads * n):
            raise ValueError("lse must be a contiguous CUDA float32 tensor of B*H*N elements")
    _check(lib().rf2_block_sparse_attn(ctypes.byref(geom), qp.data_ptr(), kp.data_ptr(), vp.data_ptr(),
                                       mask.row_start.data_ptr(), mask.row_count.data_ptr(),
                                       mask.col_idx.data_ptr(), out.data_ptr(),
                                       lse.data_ptr() if lse is not None else None, _stream(stream)),
           "rf2_block_sparse_attn")
    return out


def device_status(stream=None) -> int:
    """Synchronize and return (and clear) the device status word."""
    return int(lib().rf2_device_status(_stream(stream)))


def selftest_wait_timeout(limit_us: int = 1000, stream=None) -> int:
    """Run the library's timeout self-test (a bounded wait on a barrier that
    nothing completes, and a second wait left through the abort flag); returns
    how many of the two waits gave up.  The timeout is then in the device
    status word (``device_status()`` returns RF2_ERR_TIMEOUT once)."""
    n = ctypes.c_int32(-1)
    _check(lib().rf2_selftest_wait_timeout(ctypes.c_uint32(int(limit_us)), ctypes.byref(n), _stream(stream)),
           "rf2_selftest_wait_timeout")
    return int(n.value)


def rainfusion_attention(geom: Geometry, q, k, v, keep: float, stream=None):
    """The whole path for one attention call: permute Q/K/V (block means of Q
    and K taken on the way), predict the block mask, block-sparse attention,
    unpermute.  Returns (O, mask)."""
    mask, ws = alloc_mask(geom, keep, q.device)
    qp, kp = permute_qk_pool(geom, q, k, ws, stream=stream)
    vp = permute(geom, v, stream=stream)
    predict_mask_pooled(geom, keep, mask, ws, stream=stream)
    op = block_sparse_attn(geom, qp, kp, vp, mask, stream=stream)
    return unpermute(geom, op, stream=stream), mask


# --------------------------------------------------------------------------
# The layer around the attention: norms, rotation, score modifications, gradients.
# The calls record nothing for autograd: what they return has no graph behind it,
# whatever requires_grad its inputs have; the gradients are the *_backward calls.


def layer_query(geom: Geometry) -> LayerSizes:
    """rf2_layer_query: device scratch of the calls below."""
    out = LayerSizes()
    _check(lib().rf2_layer_query(ctypes.byref(geom), ctypes.byref(out)), "rf2_layer_query")
    return out


# torch.cuda.current_stream(index).cuda_stream without making the stream object (4 us a call).
_raw_stream = torch._C._cuda_getCurrentRawStream


class _On:
    """Device of a tensor current, and `stream` (torch stream or raw handle;
    None: the device's current one) too, so that outputs and scratch allocated
    inside belong to the stream the kernels run on.  Enters as its handle."""
    __slots__ = ("device", "stream", "contexts")

    def __init__(self, t: torch.Tensor, stream):
        if not t.is_cuda:
            raise ValueError(f"expected a CUDA tensor, got one on {t.device}")
        self.device, self.stream, self.contexts = t.device, stream, ()

    def __enter__(self) -> int:
        dev, stream = self.device, self.stream
        if stream is None and dev.index == torch.cuda.current_device():
            return _raw_stream(dev.index)
        if stream is not None and not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=dev) if int(stream) else torch.cuda.default_stream(dev)
        self.contexts = (torch.cuda.device(dev), torch.cuda.stream(stream))
        for c in self.contexts:
            c.__enter__()
        return _raw_stream(dev.index)

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)


def _same_device(first, *ts):
    dev = first.device
    for t in ts:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on different devices: {dev} and {t.device}")


def _scratch(nbytes: int, like: torch.Tensor, given: torch.Tensor | None = None) -> torch.Tensor:
    if given is None:
        return torch.empty(max(16, nbytes), dtype=torch.uint8, device=like.device)
    if not (given.is_cuda and given.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _same_device(like, given)
    return given


def _check_three(out, names: str):
    """Another number of outputs would shift the pointers behind them."""
    if out is not None and len(out) != 3:
        raise ValueError(f"out: expected three tensors {names}, got {len(out)}")


def _bytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


@dataclass
class RopeTable:
    """Rotation table on the device (see rf2_norm_rope in include/rf2.h) and
    the channels turned by frame, row and column."""
    table: torch.Tensor
    split: tuple


def rope_table(geom: Geometry, split, theta: float = 10000.0, device=None) -> RopeTable:
    """Rotation table of the angles position * theta^(-2k/size), text tokens
    unturned.  split: channels turned by (frame, row, column).  For other
    angles (scaled positions, turned text) fill a table of the same layout."""
    sp = (ctypes.c_int32 * 3)(*(int(c) for c in split))
    n = ctypes.c_int64()
    _check(lib().rf2_rope_table_floats(ctypes.byref(geom), sp, ctypes.byref(n)), "rf2_rope_table_floats")
    host = np.empty(n.value, dtype=np.float32)
    _check(lib().rf2_rope_table(ctypes.byref(geom), sp, float(theta), host.ctypes.data), "rf2_rope_table")
    return RopeTable(torch.from_numpy(host).to("cuda" if device is None else device), tuple(int(c) for c in split))


def _rope_floats(geom: Geometry, split) -> int:
    """Values of a rotation table (rf2_rope_table_floats)."""
    t, y, x = split
    return (geom.frames * (t // 2) + geom.height * (y // 2) + geom.width * (x // 2)
            + geom.text_tokens * (geom.head_dim // 2)) * 2


def _view(shape: tuple, t: torch.Tensor, name: str) -> View:
    if not (t.is_cuda and t.dtype is torch.bfloat16 and t.shape == shape and t.stride(3) == 1):
        raise ValueError(f"{name}: expected a CUDA bf16 tensor of shape {shape} with contiguous channels, got "
                         f"{tuple(t.shape)} {t.dtype} {t.device} strides {tuple(t.stride())}")
    b, h, n, _ = t.stride()
    return View(t.data_ptr(), b, h, n)


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _norm_rope(geom: Geometry, q_weight, k_weight, rope, eps, norm, interleaved) -> NormRope:
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and not (w.is_cuda and w.dtype == torch.float32 and w.is_contiguous()
                                  and tuple(w.shape) == (geom.head_dim,)):
            raise ValueError(f"{name}: expected a contiguous CUDA float32 tensor of shape ({geom.head_dim},)")
    split = (0, 0, 0)
    if rope is not None:
        split, t = rope.split, rope.table
        n = _rope_floats(geom, split)
        if not (t.is_cuda and t.dtype is torch.float32 and t.is_contiguous() and t.numel() == n):
            raise ValueError(f"rope: expected a contiguous CUDA float32 table of {n} values")
    return NormRope(int(bool(norm)), float(eps), _ptr(q_weight), _ptr(k_weight),
                    None if rope is None else rope.table.data_ptr(), tuple(split), int(bool(interleaved)))


def norm_rope_permute(geom: Geometry, q, k, v=None, *, q_weight=None, k_weight=None, rope: RopeTable | None = None,
                      eps: float = 1e-6, norm: bool = True, interleaved: bool = True,
                      workspace: torch.Tensor | None = None, out=None, stream=None):
    """Per-head RMS norm and rotation of Q and K, and the window permutation of
    Q, K (and V), in one pass.  q, k, v: CUDA bf16 [B, H, N, d] of any strides
    with contiguous channels (views of a fused projection, say).  Returns (qp,
    kp, vp), dense; with `workspace` (the mask workspace of alloc_mask) the
    block means are left there as permute_qk_pool does."""
    _check_three(out, "(qp, kp, vp; None without v)")
    _same_device(q, k, v, q_weight, k_weight, rope and rope.table, workspace)
    with _On(q, stream) as s:
        if workspace is not None:
            _scratch(0, q, workspace)
        shape = _shape(geom)
        views = [None if t is None else _view(shape, t, n) for t, n in ((q, "q"), (k, "k"), (v, "v"))]
        p = _norm_rope(geom, q_weight, k_weight, rope, eps, norm, interleaved)
        if out is None:
            out = tuple(None if t is None else torch.empty(shape, dtype=torch.bfloat16, device=q.device) for t in (q, k, v))
        else:
            _check_qkv(geom, *(t for t in out if t is not None))
            _same_device(q, *out)
        _check(lib().rf2_norm_rope_permute(ctypes.byref(geom), ctypes.byref(p), *(_ref(w) for w in views),
                                           *(_ptr(t) for t in out), _ptr(workspace),
                                           0 if workspace is None else _bytes(workspace), s),
               "rf2_norm_rope_permute")
    return tuple(out)


def norm_rope_permute_backward(geom: Geometry, q, k, dqp, dkp, dvp=None, *, q_weight=None, k_weight=None,
                               rope: RopeTable | None = None, eps: float = 1e-6, norm: bool = True,
                               interleaved: bool = True, out=None, weight_grads: bool = True,
                               workspace: torch.Tensor | None = None, stream=None):
    """Gradient of norm_rope_permute: returns (dq, dk, dv, dq_weight, dk_weight)
    from those of its outputs.  `out`: tensors (dq, dk, dv) to write, of any
    strides (views of a fused projection's gradient, say).  The weight
    gradients are fp32 [d] (None with weight_grads=False or norm=False)."""
    _check_three(out, "(dq, dk, dv; None without dvp)")
    _same_device(dqp, dkp, dvp, q_weight, k_weight, rope and rope.table, workspace, *((q, k) if norm else ()))
    with _On(dqp, stream) as s:
        _check_qkv(geom, *(t for t in (dqp, dkp, dvp) if t is not None))
        p = _norm_rope(geom, q_weight, k_weight, rope, eps, norm, interleaved)
        shape = _shape(geom)
        xs = [_view(shape, q, "q"), _view(shape, k, "k")] if norm else [None, None]
        if out is None:
            out = tuple(None if t is None else torch.empty_like(t) for t in (dqp, dkp, dvp))
        _same_device(dqp, *out)
        outs = [None if t is None else _view(shape, t, n) for t, n in zip(out, ("dq", "dk", "dv"))]
        dws = [None, None]
        if weight_grads and norm:
            dws = [torch.empty(geom.head_dim, dtype=torch.float32, device=dqp.device) for _ in range(2)]
            workspace = _scratch(layer_query(geom).norm_rope_backward_bytes, dqp, workspace)
        _check(lib().rf2_norm_rope_permute_backward(
            ctypes.byref(geom), ctypes.byref(p), *(_ref(w) for w in xs), dqp.data_ptr(), dkp.data_ptr(), _ptr(dvp),
            *(_ref(w) for w in outs), *(_ptr(t) for t in dws), _ptr(workspace),
            0 if workspace is None else _bytes(workspace), s), "rf2_norm_rope_permute_backward")
    return (*out, *dws)


@dataclass
class ScoreMod:
    """Modifications of the attention scores (rf2_score_mod in include/rf2.h):
    tanh cap, distance bias slopes[h] * (distance . |grid offset|), document
    and order of every token in model order (int32 [B, N]; negative documents
    are padding; a token sees those of its document whose order is not later)."""
    softcap: float = 0.0
    slopes: torch.Tensor | None = None
    distance: tuple = (1.0, 1.0, 1.0)
    document: torch.Tensor | None = None
    order: torch.Tensor | None = None

    def _struct(self, geom: Geometry, like: torch.Tensor) -> ScoreModStruct:
        _same_device(like, self.slopes, self.document, self.order)
        if len(self.distance) != 3:
            raise ValueError(f"distance: expected three weights (frame, row, column), got {len(self.distance)}")
        if self.slopes is not None and not (self.slopes.is_cuda and self.slopes.dtype == torch.float32
                                            and self.slopes.is_contiguous()
                                            and tuple(self.slopes.shape) == (geom.heads,)):
            raise ValueError(f"slopes: expected a contiguous CUDA float32 tensor of shape ({geom.heads},)")
        shape = (geom.batch, num_tokens(geom))
        for name, t in (("document", self.document), ("order", self.order)):
            if t is not None and not (t.is_cuda and t.dtype == torch.int32 and t.is_contiguous()
                                      and tuple(t.shape) == shape):
                raise ValueError(f"{name}: expected a contiguous CUDA int32 tensor of shape {shape}")
        return ScoreModStruct(float(self.softcap), *(float(w) for w in self.distance), _ptr(self.slopes),
                              _ptr(self.document), _ptr(self.order))


def _check_mask(geom: Geometry, mask: BlockMask, like: torch.Tensor):
    rows = geom.batch * geom.heads * ((num_tokens(geom) + 63) // 64)
    for t in (mask.row_start, mask.row_count, mask.col_idx):
        if not (t.is_cuda and t.dtype == torch.int32 and t.is_contiguous()):
            raise ValueError("mask: expected contiguous CUDA int32 tensors")
    if mask.row_start.numel() < rows or mask.row_count.numel() < rows:
        raise ValueError(f"mask: expected {rows} rows")
    _same_device(like, mask.row_start, mask.row_count, mask.col_idx)


def _check_capacity(geom: Geometry, keep: float, mask: BlockMask):
    """A prediction at `keep` writes up to that many columns; the kernels know `keep`, not the allocation."""
    need = query(geom, keep).col_idx_capacity
    if mask.col_idx.numel() < need:
        raise ValueError(f"mask: col_idx holds {mask.col_idx.numel()} columns, keep {keep} needs {need}")


def _check_lse(geom: Geometry, lse: torch.Tensor, like: torch.Tensor):
    if not (lse.is_cuda and lse.dtype == torch.float32 and lse.is_contiguous()
            and lse.numel() == geom.batch * geom.heads * num_tokens(geom)):
        raise ValueError("lse must be a contiguous CUDA float32 tensor of B*H*N elements")
    _same_device(like, lse)


def block_sparse_attn_mod(geom: Geometry, qp, kp, vp, mask: BlockMask, mod: ScoreMod,
                          out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """block_sparse_attn with modified scores."""
    with _On(qp, stream) as s:
        _check_qkv(geom, qp, kp, vp)
        if out is None:
            out = torch.empty_like(qp)
        else:
            _check_qkv(geom, out)
        _same_device(qp, kp, vp, out)
        _check_mask(geom, mask, qp)
        if lse is not None:
            _check_lse(geom, lse, qp)
        m = mod._struct(geom, qp)
        ws = _scratch(layer_query(geom).score_mod_bytes, qp, workspace)
        _check(lib().rf2_block_sparse_attn_mod(ctypes.byref(geom), qp.data_ptr(), kp.data_ptr(), vp.data_ptr(),
                                               mask.row_start.data_ptr(), mask.row_count.data_ptr(),
                                               mask.col_idx.data_ptr(), ctypes.byref(m), out.data_ptr(), _ptr(lse),
                                               ws.data_ptr(), _bytes(ws), s), "rf2_block_sparse_attn_mod")
    return out


def block_sparse_attn_backward(geom: Geometry, qp, kp, vp, op, lse, dop, mask: BlockMask, mod: ScoreMod | None = None,
                               out=None, workspace: torch.Tensor | None = None, stream=None):
    """Gradients (dqp, dkp, dvp) of block_sparse_attn (mod None) or
    block_sparse_attn_mod, from its inputs, output and log-sum-exp and the
    output's gradient."""
    _check_three(out, "(dqp, dkp, dvp)")
    with _On(qp, stream) as s:
        _check_qkv(geom, qp, kp, vp, op, dop)
        if out is None:
            out = tuple(torch.empty_like(qp) for _ in range(3))
        else:
            _check_qkv(geom, *out)
        _same_device(qp, kp, vp, op, dop, *out)
        _check_mask(geom, mask, qp)
        _check_lse(geom, lse, qp)
        m = None if mod is None else mod._struct(geom, qp)
        ws = _scratch(layer_query(geom).attn_backward_bytes, qp, workspace)
        _check(lib().rf2_block_sparse_attn_backward(
            ctypes.byref(geom), qp.data_ptr(), kp.data_ptr(), vp.data_ptr(), op.data_ptr(), lse.data_ptr(),
            dop.data_ptr(), mask.row_start.data_ptr(), mask.row_count.data_ptr(), mask.col_idx.data_ptr(), _ref(m),
            *(t.data_ptr() for t in out), ws.data_ptr(), _bytes(ws), s), "rf2_block_sparse_attn_backward")
    return out


def predict_mask_visible(geom: Geometry, keep: float, mask: BlockMask, workspace: torch.Tensor, mod: ScoreMod,
                         mod_workspace: torch.Tensor | None = None, stream=None) -> BlockMask:
    """predict_mask_pooled that ranks the key blocks `mod`'s documents and
    order let a query block see before all others.  The block means include
    padding tokens as they are: their Q and K should be finite."""
    _check_capacity(geom, keep, mask)
    with _On(workspace, stream) as s:
        _scratch(0, workspace, workspace)
        _check_mask(geom, mask, workspace)
        m = mod._struct(geom, workspace)
        ws = _scratch(layer_query(geom).score_mod_bytes, workspace, mod_workspace)
        _check(lib().rf2_predict_mask_visible(ctypes.byref(geom), float(keep), ctypes.byref(m),
                                              mask.row_start.data_ptr(), mask.row_count.data_ptr(),
                                              mask.col_idx.data_ptr(), workspace.data_ptr(), _bytes(workspace),
                                              ws.data_ptr(), _bytes(ws), s), "rf2_predict_mask_visible")
    return mask


@dataclass
class LayerState:
    """What layer_attention keeps for its gradient."""
    geom: Geometry
    q: torch.Tensor
    k: torch.Tensor
    qp: torch.Tensor
    kp: torch.Tensor
    vp: torch.Tensor
    op: torch.Tensor
    lse: torch.Tensor
    mask: BlockMask
    mod: ScoreMod | None
    params: dict


def layer_attention(geom: Geometry, q, k, v, keep: float, *, q_weight=None, k_weight=None,
                    rope: RopeTable | None = None, eps: float = 1e-6, norm: bool = True, interleaved: bool = True,
                    mod: ScoreMod | None = None, stream=None):
    """A layer's attention from its projections: norm, rotation and permutation
    of Q, K, V (block means on the way), mask prediction (over the visible
    blocks under a document or order mask), block-sparse attention with the
    score modifications, unpermute.  Returns (O, LayerState); the state is what
    layer_attention_backward needs, with the BlockMask in it.  The Q and K of
    padding tokens (document < 0) should be finite: block means include them.
    Like every call here it is not seen by autograd (wrap it and
    layer_attention_backward in a torch.autograd.Function); norm weights are fp32."""
    params = dict(q_weight=q_weight, k_weight=k_weight, rope=rope, eps=eps, norm=norm, interleaved=interleaved)
    with _On(q, stream) as s:
        mask, ws = alloc_mask(geom, keep, q.device)
        qp, kp, vp = norm_rope_permute(geom, q, k, v, workspace=ws, **params)
        if mod is not None and (mod.document is not None or mod.order is not None):
            predict_mask_visible(geom, keep, mask, ws, mod)
        else:
            predict_mask_pooled(geom, keep, mask, ws, stream=s)
        lse = torch.empty((geom.batch, geom.heads, num_tokens(geom)), dtype=torch.float32, device=q.device)
        if mod is None:
            op = block_sparse_attn(geom, qp, kp, vp, mask, lse=lse, stream=s)
        else:
            op = block_sparse_attn_mod(geom, qp, kp, vp, mask, mod, lse=lse)
        o = unpermute(geom, op, stream=s)
    return o, LayerState(geom, q, k, qp, kp, vp, op, lse, mask, mod, params)


def layer_attention_backward(state: LayerState, do: torch.Tensor, out=None, weight_grads: bool = True, stream=None):
    """Gradient of layer_attention: (dq, dk, dv, dq_weight, dk_weight) from the
    output's gradient [B, H, N, d].  `out`: tensors (dq, dk, dv) to write."""
    st = state
    with _On(do, stream) as s:
        dop = permute(st.geom, do.contiguous(), stream=s)
        dqp, dkp, dvp = block_sparse_attn_backward(st.geom, st.qp, st.kp, st.vp, st.op, st.lse, dop, st.mask, st.mod)
        return norm_rope_permute_backward(st.geom, st.q, st.k, dqp, dkp, dvp, out=out, weight_grads=weight_grads,
                                          **st.params)


def chunk_sizes(heads: int, chunks: int, tail_split: bool = True) -> list:
    """Heads per chunk of a HostPipeline: `chunks` near-equal chunks; with
    `tail_split` the last one is further split in shrinking parts down to one
    head (the host-to-device copies set the pace, and what follows the last of
    them is the last chunk's compute and copy back)."""
    n = max(1, min(int(chunks), int(heads)))
    cuts = [round(c * heads / n) for c in range(n + 1)]
    sizes = [cuts[c + 1] - cuts[c] for c in range(n)]
    if tail_split:
        r, tail = sizes.pop(), []
        while r > 1:
            h = (r + 1) // 2
            tail.append(h)
            r -= h
        sizes += tail + ([r] if r else [])
    return sizes


class HostSizes(ctypes.Structure):
    _fields_ = [("num_chunks", ctypes.c_int32), ("max_chunk_heads", ctypes.c_int32), ("work_bytes", ctypes.c_size_t)]


def host_query(geom: Geometry, keep: float | None = None, tau: float | None = None, chunks: int = 8) -> HostSizes:
    """rf2_attention_host_query: chunk count and device scratch of rf2_attention_host."""
    out = HostSizes()
    _check(lib().rf2_attention_host_query(ctypes.byref(geom), float(keep or 0.0), float(tau or 0.0), int(chunks),
                                          ctypes.byref(out)), "rf2_attention_host_query")
    return out


class HostPipeline:
    """One attention call on host (pinned) tensors, copies overlapped with
    compute: a thin wrapper over the C call rf2_attention_host, which copies
    head chunks in on one stream, computes them on a second and copies them
    back on a third (see include/rf2.h).  Output bits equal those of the calls
    on the whole device tensors.

    Build once (the device scratch and the three streams are allocated here),
    then call `run(q, k, v, o)` with pinned host bf16 tensors [B, H, N, d].
    Selection: top-n with `keep`, or the CDF threshold with `tau`.  The B*H
    heads go in `chunks` near-equal chunks, the last of them further split in
    shrinking parts down to one head (`chunk_sizes`).
    """

    def __init__(self, geom: Geometry, keep: float | None = None, tau: float | None = None, chunks: int = 8,
                 device=None, chunk_events: bool = True):
        if (keep is None) == (tau is None):
            raise ValueError("give exactly one of keep and tau")
        self.geom, self.keep, self.tau, self.chunks = geom, keep, tau, int(chunks)
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.device = dev
        sz = host_query(geom, keep, tau, self.chunks)
        self.parts = chunk_sizes(geom.batch * geom.heads, self.chunks)
        assert len(self.parts) == sz.num_chunks and max(self.parts) == sz.max_chunk_heads
        self.work = torch.empty(max(256, sz.work_bytes), dtype=torch.uint8, device=dev)
        self.shape = (geom.batch, geom.heads, num_tokens(geom), geom.head_dim)
        self.h2d, self.comp, self.d2h = (torch.cuda.Stream(device=dev) for _ in range(3))
        # chunk-by-chunk ordering of consecutive runs (chunk c waits only for chunk c of the
        # last run); without, each run waits for the whole previous one
        self.num_events = 2 * sz.num_chunks if chunk_events else 0
        self.events = (ctypes.c_void_p * self.num_events)() if chunk_events else None
        if chunk_events:
            with torch.cuda.device(dev):
                _check(lib().rf2_host_events_create(self.num_events, self.events), "rf2_host_events_create")
        self._lib = lib()

    def __del__(self):
        events = getattr(self, "events", None)
        if events is not None:
            try:
                self.d2h.synchronize()
                self._lib.rf2_host_events_destroy(self.num_events, events)
            except Exception:
                pass

    def run(self, q_host: torch.Tensor, k_host: torch.Tensor, v_host: torch.Tensor, o_host: torch.Tensor):
        for t in (q_host, k_host, v_host, o_host):
            if not (t.device.type == "cpu" and t.is_pinned() and t.dtype == torch.bfloat16 and t.is_contiguous()
                    and tuple(t.shape) == self.shape):
                raise ValueError(f"expected pinned contiguous host bf16 tensors of shape {self.shape}")
        _check(lib().rf2_attention_host(ctypes.byref(self.geom), float(self.keep or 0.0), float(self.tau or 0.0),
                                        self.chunks, q_host.data_ptr(), k_host.data_ptr(), v_host.data_ptr(),
                                        o_host.data_ptr(), self.work.data_ptr(), self.work.numel(),
                                        self.h2d.cuda_stream, self.comp.cuda_stream, self.d2h.cuda_stream,
                                        self.events, self.num_events),
               "rf2_attention_host")
        return o_host

    def synchronize(self):
        self.d2h.synchronize()
