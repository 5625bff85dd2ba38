"""Python binding of the CSA2 C ABI (``include/csa2.h``): argument marshalling only.

Every function has the ABI call's name without the ``csa2_`` prefix, takes
torch CUDA tensors, passes their device pointers and the current CUDA stream,
and raises ``Csa2Error`` on a non-zero status. All arithmetic runs in the CUDA
kernels of ``libcsa2.so``; nothing here computes on the data.

``LayerCache`` and ``IndexKeyCache`` allocate one layer's per-sequence buffers
with PyTorch (device memory is PyTorch's job) and build the device arrays of
per-sequence base pointers the ABI takes.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass

import torch

from ._lib import Csa2Error, Pages, Params, check, lib  # noqa: F401

F32, NVFP4, E4M3, BF16 = 0, 1, 2, 3
WIN_RING, WIN_LINEAR = 0, 1
ROPE_PAIRS, ROPE_HALF, ROPE_CLEAR = 0, 1, 16
D, H, HI, DI, W, BLK, KB, KP = 512, 64, 32, 128, 128, 8, 2048, 512
KEY_TILE, KEY_TILE_BYTES = 128, 9216


def default_params(**over) -> Params:
    p = Params()
    lib().csa2_default_params(ctypes.byref(p))
    for k, v in over.items():
        setattr(p, k, v)
    return p


def version() -> int:
    return lib().csa2_version()


TRACE_KERNELS = {0: "none", 1: "compress_append", 2: "index_scores", 3: "select_topk",
                 4: "sparse_attn_layers"}


def trace_attach():
    """Attach a zeroed pinned record to the library's launch trace (csa2_trace_attach)
    and return it; read it with trace_read() after an error."""
    rec = torch.zeros(4, dtype=torch.int32, pin_memory=True)
    check(lib().csa2_trace_attach(ctypes.c_void_p(rec.data_ptr())), "trace_attach")
    return rec


def trace_read(rec) -> str:
    """The trace record as text: the last launch that started and the last whose
    first CTA finished."""
    v = [int(x) for x in rec.tolist()]
    return "last launch started: %s #%d; last first-CTA finish: %s #%d" % (
        TRACE_KERNELS.get(v[0], str(v[0])), v[1], TRACE_KERNELS.get(v[2], str(v[2])), v[3])


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise Csa2Error("expected a CUDA tensor")
    return t.data_ptr()


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def ptr_array(tensors, device=None) -> torch.Tensor:
    """Device int64 array of the base addresses of `tensors` (one per sequence)."""
    addrs = [t.data_ptr() for t in tensors]
    dev = device or tensors[0].device
    return torch.tensor(addrs, dtype=torch.int64, device=dev)


# --------------------------------------------------------------------------- calls
def compress_append(params, kv_new, gate_new, pend_kv, pend_gate, comp_ptrs, comp_scale_ptrs,
                    comp_cap, win_ptrs, n_tokens, dev_status=None, stream=None):
    B = n_tokens.numel()
    n_new = kv_new.shape[1] if kv_new.dim() == 3 else 0
    check(lib().csa2_compress_append(
        ctypes.byref(params), B, n_new, _ptr(kv_new), _ptr(gate_new), _ptr(pend_kv),
        _ptr(pend_gate), _ptr(comp_ptrs), _ptr(comp_scale_ptrs), _ptr(comp_cap), _ptr(win_ptrs),
        _ptr(n_tokens), _ptr(dev_status), _stream(stream)), "compress_append")


def window_linear(params, kv_new, win_ptrs, n_tokens, out, stream=None):
    """Linear FP8 windows of a prefill chunk (before its append): out [B, W-1+n_new, D]."""
    B, n_new = n_tokens.numel(), kv_new.shape[1]
    check(lib().csa2_window_linear(ctypes.byref(params), B, n_new, _ptr(kv_new), _ptr(win_ptrs),
                                   _ptr(n_tokens), _ptr(out), _stream(stream)), "window_linear")


def nvfp4_quantize(x, vals, scales, stream=None):
    check(lib().csa2_nvfp4_quantize(_ptr(x), x.numel() // x.shape[-1], x.shape[-1], _ptr(vals),
                                    _ptr(scales), _stream(stream)), "nvfp4_quantize")


def index_keys_write(params, vals, scales, pos0, dst_ptrs, cap, dev_status=None, stream=None):
    """Plain NVFP4 index keys vals [B, n, 64] / scales [B, n, 8] -> tiled caches."""
    B, n = vals.shape[0], vals.shape[1]
    check(lib().csa2_index_keys_write(
        ctypes.byref(params), B, n, _ptr(vals), _ptr(scales), _ptr(pos0), _ptr(dst_ptrs),
        _ptr(cap), _ptr(dev_status), _stream(stream)), "index_keys_write")


def index_scores(params, max_ncomp, q_vals, q_scales, w, key_cache_ptrs, n_tokens, scores,
                 block_max, dev_status=None, stream=None, cuda_cores=False):
    B = n_tokens.numel()
    f = lib().csa2_index_scores_cuda_cores if cuda_cores else lib().csa2_index_scores
    check(f(ctypes.byref(params), B, max_ncomp, _ptr(q_vals), _ptr(q_scales), _ptr(w),
            _ptr(key_cache_ptrs), _ptr(n_tokens), _ptr(scores), _ptr(block_max), _ptr(dev_status),
            _stream(stream)), "index_scores")


def index_scores_shared(params, max_ncomp, q_vals, q_scales, w, key_cache, n_tokens, scores,
                        block_max, dev_status=None, stream=None):
    """Q queries against ONE tiled key cache (a uint8 device tensor): the prefill
    Indexer. q_vals [Q,32,64], q_scales [Q,32,8], w [Q,32], n_tokens [Q]."""
    Q = n_tokens.numel()
    check(lib().csa2_index_scores_shared(
        ctypes.byref(params), Q, max_ncomp, _ptr(q_vals), _ptr(q_scales), _ptr(w), _ptr(key_cache),
        _ptr(n_tokens), _ptr(scores), _ptr(block_max), _ptr(dev_status), _stream(stream)),
        "index_scores_shared")


def select_topk(params, max_ncomp, scores, block_max, n_tokens, idx, n_sel=None, dev_status=None,
                stream=None):
    B = n_tokens.numel()
    check(lib().csa2_select_topk(
        ctypes.byref(params), B, max_ncomp, _ptr(scores), _ptr(block_max), _ptr(n_tokens),
        _ptr(idx), _ptr(n_sel), _ptr(dev_status), _stream(stream)), "select_topk")


def sparse_attn_workspace_size(params, B) -> int:
    return lib().csa2_sparse_attn_workspace_size(ctypes.byref(params), B)


def sparse_attn(params, q, sink, win_ptrs, n_tokens, comp_ptrs, comp_scale_ptrs, idx, out,
                workspace, dev_status=None, stream=None, mma_sync=False):
    """One layer (csa2_sparse_attn: tcgen05 for the quantised formats); mma_sync=True
    runs the legacy mma.sync split-KV implementation (csa2_sparse_attn_mma)."""
    B = n_tokens.numel()
    fn = lib().csa2_sparse_attn_mma if mma_sync else lib().csa2_sparse_attn
    check(fn(
        ctypes.byref(params), B, _ptr(q), _ptr(sink), _ptr(win_ptrs), _ptr(n_tokens),
        _ptr(comp_ptrs), _ptr(comp_scale_ptrs), _ptr(idx), _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream(stream)),
        "sparse_attn_mma" if mma_sync else "sparse_attn")


def sparse_attn_layers_split_workspace(params, L, B, device="cuda"):
    """Zero-filled workspace for sparse_attn_layers(..., workspace=...) on the
    current device (one partial-result slot per CTA boundary + the counts)."""
    n = lib().csa2_sparse_attn_layers_split_workspace_size(ctypes.byref(params), L, B)
    return torch.zeros(max(int(n), 256), dtype=torch.uint8, device=device)


def sparse_attn_layers(params, q, sink, win_ptrs, n_tokens, comp_ptrs, comp_scale_ptrs, idx, out,
                       dev_status=None, stream=None, mma_sync=False, workspace=None):
    """L layers sharing one compressed cache and selection: q/out [L, B, H, D] bf16,
    sink [L, H], win_ptrs [L*B] (layer-major), n_tokens [B]. mma_sync=True runs
    the legacy warp-level tensor-core implementation of the same contract. With a
    workspace (sparse_attn_layers_split_workspace) the tcgen05 path spreads the
    (unit, tile) work evenly over the CTAs (csa2_sparse_attn_layers_split)."""
    L, B = q.shape[0], q.shape[1]
    if workspace is not None and not mma_sync:
        check(lib().csa2_sparse_attn_layers_split(
            ctypes.byref(params), L, B, _ptr(q), _ptr(sink), _ptr(win_ptrs), _ptr(n_tokens),
            _ptr(comp_ptrs), _ptr(comp_scale_ptrs), _ptr(idx), _ptr(out), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream(stream)),
            "sparse_attn_layers_split")
        return
    fn = lib().csa2_sparse_attn_layers_mma if mma_sync else lib().csa2_sparse_attn_layers
    check(fn(
        ctypes.byref(params), L, B, _ptr(q), _ptr(sink), _ptr(win_ptrs), _ptr(n_tokens),
        _ptr(comp_ptrs), _ptr(comp_scale_ptrs), _ptr(idx), _ptr(out), _ptr(dev_status),
        _stream(stream)), "sparse_attn_layers_mma" if mma_sync else "sparse_attn_layers")


def sparse_attn_layers_part(params, b0, nb, q, sink, win_ptrs, n_tokens, comp_ptrs, comp_scale_ptrs,
                            idx, out, dev_status=None, stream=None):
    """sparse_attn_layers for the sequences [b0, b0 + nb) only; every array keeps
    its full-batch shape (q/out [L, B, H, D], win_ptrs [L*B], n_tokens [B], ...)."""
    L, B = q.shape[0], q.shape[1]
    check(lib().csa2_sparse_attn_layers_part(
        ctypes.byref(params), L, B, b0, nb, _ptr(q), _ptr(sink), _ptr(win_ptrs), _ptr(n_tokens),
        _ptr(comp_ptrs), _ptr(comp_scale_ptrs), _ptr(idx), _ptr(out), _ptr(dev_status),
        _stream(stream)), "sparse_attn_layers_part")


def sparse_attn_noalloc(params, q, sink, win_ptrs, n_tokens, comp_ptrs, comp_scale_ptrs, idx, out,
                        dev_status=None, stream=None):
    """csa2_sparse_attn without a workspace: for callers that cannot allocate device
    memory (their HBM already belongs to an engine's pool, or an allocation would
    synchronise a latency-critical path). At most 32 sequences per call; calls that
    overlap on the GPU share the library's one scratch array and must be ordered."""
    B = n_tokens.numel()
    check(lib().csa2_sparse_attn_noalloc(
        ctypes.byref(params), B, _ptr(q), _ptr(sink), _ptr(win_ptrs), _ptr(n_tokens),
        _ptr(comp_ptrs), _ptr(comp_scale_ptrs), _ptr(idx), _ptr(out), _ptr(dev_status),
        _stream(stream)), "sparse_attn_noalloc")


# --------------------------------------------------------------------------- paged cache
# These calls check what the pointers stand for (types, shapes, devices, strides) before
# they hand them on; everything else is checked by the library. A decode step's kernels run
# for a few microseconds each, so the checks are kept to what costs tenths of one.
_FORMATS = {torch.bfloat16: BF16, torch.float32: F32}
# Of a device index, without a Stream object. A torch built without CUDA has neither: the module
# still imports there, for what needs no device.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _fail(what):
    raise Csa2Error(what)


def _elsewhere(name, t, index):
    _fail("%s is on %s, the call's other tensors on cuda:%d" % (name, t.device, index))


def _i32(name, t, n, index):
    """Address of a contiguous int32 tensor of n elements on device `index`."""
    if t.dtype is not torch.int32 or t.numel() != n or not t.is_contiguous():
        _fail("%s must be a contiguous int32 tensor of %d elements" % (name, n))
    if t.get_device() != index:
        _elsewhere(name, t, index)
    return t.data_ptr()


def _at(name, t, index):
    if t.get_device() != index:
        _elsewhere(name, t, index)
    return t.data_ptr()


def _status(t, index):
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.numel() < 1:
        _fail("dev_status must be an int32 tensor")
    return _at("dev_status", t, index)


def _run(name, index, stream, fn, *args):
    """fn(*args, stream) with device `index` current, on `stream` or the device's current one."""
    if index < 0:
        _fail("expected a CUDA tensor")
    if _current_device() != index:
        with torch.cuda.device(index):
            return _run(name, index, stream, fn, *args)
    rc = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        check(rc, name)


def _new_like(x, stream):
    """An uninitialised tensor as x that a call on `stream` (None: the current one) writes. It
    comes from that stream's memory: a block that the current stream has let go of may still be
    in use by what is queued there. Letting go of it waits for the current stream too, where the
    caller is likely to read it."""
    here = None if stream is None or x.get_device() < 0 else torch.cuda.current_stream(x.device)
    if here is None or here == stream:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    with torch.cuda.stream(stream):
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    out.record_stream(here)
    return out


def rope(params, x, pos, out=None, layout=ROPE_PAIRS, first=-1, inverse=False, stream=None):
    """Rotary embedding (csa2_rope): x [N, heads, channels] bf16 or fp32 with contiguous
    channels, pos [N] int32; out as x (None: a new tensor; x itself: in place).
    A row with pos < 0 is padding: zeros in a new tensor, left as it is in a given one.
    inverse=True turns back, which is also the gradient of the call. Returns out."""
    dt, shape = x.dtype, x.shape
    fmt = _FORMATS.get(dt)
    if fmt is None or len(shape) != 3:
        _fail("rope: x must be [N, heads, channels], bf16 or fp32")
    if out is None:
        out = _new_like(x, stream)
        layout |= ROPE_CLEAR
    elif out.shape != shape or out.dtype is not dt:
        _fail("rope: out must have x's shape and type")
    N, heads, ch = shape
    if N == 0 or heads == 0:
        return out
    x0, x1, x2 = x.stride()
    o0, o1, o2 = out.stride()
    if (x2 != 1 or o2 != 1) and ch > 1:
        _fail("rope: the channels of x and out must be contiguous")
    dev = x.get_device()
    _run("rope", dev, stream, lib().csa2_rope, params, layout, 1 if inverse else 0, N, heads, ch,
         first, fmt, x.data_ptr(), x0, x1, _at("out", out, dev), o0, o1, _i32("pos", pos, N, dev))
    return out


def _rows_of(params, cache):
    """The pool's rows are params.kv_format (a wider one would read past its end)."""
    if params.kv_format != cache.kv_format:
        _fail("the cache holds rows of another format than params.kv_format")


def page_reserve(params, cache, seq, n_from, n_to, dev_status=None, stream=None):
    """Give sequences seq [N] the pages of positions n_from .. n_to-1 (csa2_page_reserve)."""
    N, dev = seq.numel(), cache.index
    _run("page_reserve", dev, stream, lib().csa2_page_reserve, params, cache.c, N,
         _i32("seq", seq, N, dev), _i32("n_from", n_from, N, dev), _i32("n_to", n_to, N, dev),
         cache.ws_ptr, cache.ws_bytes, _status(dev_status, dev))


def page_release(params, cache, seq, n_tokens=None, window=0, n_first=0, dev_status=None, stream=None):
    """Let go of every page of sequences seq [N], or with n_tokens [N] of those that no later
    token sees through window and n_first (csa2_page_release)."""
    N, dev = seq.numel(), cache.index
    _run("page_release", dev, stream, lib().csa2_page_release, params, cache.c, N,
         _i32("seq", seq, N, dev), None if n_tokens is None else _i32("n_tokens", n_tokens, N, dev),
         window, n_first, _status(dev_status, dev))


def page_fork(params, cache, parent, child, n_tokens, dev_status=None, stream=None):
    """child[i] continues the first n_tokens[i] positions of parent[i] (csa2_page_fork)."""
    _rows_of(params, cache)
    N, dev = child.numel(), cache.index
    _run("page_fork", dev, stream, lib().csa2_page_fork, params, cache.c, N,
         _i32("parent", parent, N, dev), _i32("child", child, N, dev),
         _i32("n_tokens", n_tokens, N, dev), cache.ws_ptr, cache.ws_bytes, _status(dev_status, dev))


def page_compact(params, cache, n_used=None, dev_status=None, stream=None):
    """Move the used pages to the front of the pool (csa2_page_compact); n_used [1] int32
    receives their number."""
    _rows_of(params, cache)
    dev = cache.index
    _run("page_compact", dev, stream, lib().csa2_page_compact, params, cache.c,
         None if n_used is None else _i32("n_used", n_used, 1, dev), cache.ws_ptr, cache.ws_bytes,
         _status(dev_status, dev))


def page_write(params, cache, layer, x, seq, pos, dev_status=None, stream=None):
    """Write rows x [N, 512] (fp32 or bf16) as positions pos [N] of sequences seq [N]
    (csa2_page_write), turned first when params.rope_dim > 0."""
    dt = x.dtype
    if x.dim() != 2 or x.shape[1] != D or dt not in _FORMATS or x.stride(1) != 1:
        _fail("page_write: x must be [N, %d], bf16 or fp32, with contiguous rows" % D)
    _rows_of(params, cache)
    N, dev = x.shape[0], cache.index
    _run("page_write", dev, stream, lib().csa2_page_write, params, cache.c, layer, N,
         _at("x", x, dev), _FORMATS[dt], x.stride(0), _i32("seq", seq, N, dev),
         _i32("pos", pos, N, dev), _status(dev_status, dev))


def paged_attn_workspace(params, cache, B):
    """Workspace tensor of paged_attn for batches of up to B sequences."""
    if cache.index < 0:
        _fail("expected a CUDA tensor")
    with torch.cuda.device(cache.index):
        n = lib().csa2_paged_attn_workspace_size(params, cache.c, B)
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device=cache.device)


def paged_attn(params, cache, layer, q, sink, seq, n_tokens, out, workspace, window=0, n_first=0,
               dev_status=None, stream=None):
    """Attention of one new token per sequence over a layer's pages (csa2_paged_attn):
    q [B, heads, 512] bf16 with contiguous channels, sink [heads] fp32 or None, seq [B] int32
    or None (row b of the table), n_tokens [B] int32, out [B, heads, 512] bf16. A window of 0
    sees everything; n_first positions stay visible before it."""
    shape = q.shape
    if len(shape) != 3 or q.dtype is not torch.bfloat16 or shape[2] != D or q.stride(2) != 1:
        _fail("paged_attn: q must be [B, heads, %d] bf16 with contiguous channels" % D)
    B, heads, _ = shape
    if heads != params.heads:
        _fail("paged_attn: q has %d heads, the parameters say %d" % (heads, params.heads))
    if out.shape != shape or out.dtype is not torch.bfloat16 or not out.is_contiguous():
        _fail("paged_attn: out must be contiguous bf16 of q's shape")
    if sink is not None and (sink.dtype is not torch.float32 or sink.numel() != heads or not sink.is_contiguous()):
        _fail("paged_attn: sink must be %d contiguous fp32 values" % heads)
    _rows_of(params, cache)
    dev = cache.index
    _run("paged_attn", dev, stream, lib().csa2_paged_attn, params, cache.c, layer, B,
         _at("q", q, dev), q.stride(0), q.stride(1), None if sink is None else _at("sink", sink, dev),
         None if seq is None else _i32("seq", seq, B, dev), _i32("n_tokens", n_tokens, B, dev),
         window, n_first, _at("out", out, dev), _at("workspace", workspace, dev), workspace.nbytes,
         _status(dev_status, dev))


def fp4_mma_peak(ctas, iters, dev_status=None, stream=None):
    """Enqueue the FP4 tensor-core rate measurement (csa2_fp4_mma_peak): ctas x iters
    MMA pairs of 2 x 128 x 128 x 128 flop each. The caller times it."""
    check(lib().csa2_fp4_mma_peak(int(ctas), int(iters), _ptr(dev_status), _stream(stream)),
          "fp4_mma_peak")


# --------------------------------------------------------------------------- buffers
@dataclass
class LayerCache:
    """One layer's per-sequence state: compressed cache (NVFP4 or fp32, absent
    for window-only layers), ring window, pending half-pair, token counts."""
    B: int
    caps: list
    params: Params
    has_comp: bool = True
    device: str = "cuda"

    def __post_init__(self):
        dev, B, p = self.device, self.B, self.params
        nv = p.kv_format == NVFP4
        self.comp, self.comp_scales = [], []
        if self.has_comp:
            for cap in self.caps:
                cap = max(1, int(cap))
                if nv:
                    self.comp.append(torch.zeros(cap, D // 2, dtype=torch.uint8, device=dev))
                    self.comp_scales.append(torch.zeros(cap, D // 16, dtype=torch.uint8, device=dev))
                else:
                    self.comp.append(torch.zeros(cap, D, dtype=torch.float32, device=dev))
        wdt = torch.uint8 if p.win_format == E4M3 else torch.float32
        self.win = torch.zeros(B, W, D, dtype=wdt, device=dev)
        self.pend_kv = torch.zeros(B, D, dtype=torch.float32, device=dev)
        self.pend_gate = torch.zeros(B, D, dtype=torch.float32, device=dev)
        self.n_tokens = torch.zeros(B, dtype=torch.int32, device=dev)
        self.comp_cap = torch.tensor([max(1, int(c)) for c in self.caps], dtype=torch.int64,
                                     device=dev)
        self.comp_ptrs = ptr_array(self.comp) if self.has_comp else None
        self.comp_scale_ptrs = ptr_array(self.comp_scales) if (self.has_comp and nv) else None
        self.win_ptrs = ptr_array(list(self.win.unbind(0)))

    def append(self, kv_new, gate_new=None, dev_status=None, stream=None):
        compress_append(self.params, kv_new, gate_new if self.has_comp else None,
                        self.pend_kv if self.has_comp else None,
                        self.pend_gate if self.has_comp else None,
                        self.comp_ptrs, self.comp_scale_ptrs,
                        self.comp_cap if self.has_comp else None, self.win_ptrs, self.n_tokens,
                        dev_status, stream)

    def shares_compressed_cache_of(self, other: "LayerCache"):
        """Point this (window-only) layer's compressed-cache arrays at `other`'s."""
        self.comp_ptrs, self.comp_scale_ptrs = other.comp_ptrs, other.comp_scale_ptrs


@dataclass
class IndexKeyCache:
    """Per-sequence tiled FP4 index-key caches (include/csa2.h layout): ceil(cap/128)
    tiles of 9216 bytes each."""
    caps: list
    device: str = "cuda"

    def __post_init__(self):
        self.tiles = [max(1, -(-int(c) // KEY_TILE)) for c in self.caps]
        self.buf = [torch.zeros(t * KEY_TILE_BYTES, dtype=torch.uint8, device=self.device)
                    for t in self.tiles]
        self.ptrs = ptr_array(self.buf)
        self.cap = torch.tensor([t * KEY_TILE for t in self.tiles], dtype=torch.int64,
                                device=self.device)

    def write(self, params, vals, scales, pos0, dev_status=None, stream=None):
        """Write plain rows vals [B, n, 64], scales [B, n, 8] at positions pos0[b]..."""
        index_keys_write(params, vals, scales, pos0, self.ptrs, self.cap, dev_status, stream)

    def write_seq(self, params, b, vals, scales, pos0=0, dev_status=None, stream=None):
        """Write plain rows [n, 64] / [n, 8] of one sequence starting at pos0."""
        p0 = torch.tensor([pos0], dtype=torch.int64, device=self.device)
        index_keys_write(params, vals[None], scales[None], p0, self.ptrs[b:b + 1],
                         self.cap[b:b + 1], dev_status, stream)


class PagedCache:
    """A cache in pages (csa2_pages): the pool of `layers` layers, the page table and the
    counts, allocated here from sizes, or the caller's own tensors. pool [layers, n_pages,
    page_size, 512] of bf16 or float8_e4m3fn (params.kv_format), table [max_seqs, max_pages]
    and ref [n_pages] int32; a page of a layer is contiguous. Holds the scratch of the page
    calls too, so calls on one cache are ordered: one stream, or events between streams. The
    tensors' contents are the state; the tensors themselves stay (c holds their addresses)."""

    def __init__(self, params, n_pages=0, page_size=0, max_seqs=0, max_pages=0, layers=1,
                 device="cuda", pool=None, table=None, ref=None):
        types = {BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn}
        if params.kv_format not in types:
            _fail("PagedCache: pages hold BF16 or E4M3 rows")
        dt = types[params.kv_format]
        if pool is None:
            pool = torch.zeros(layers, n_pages, page_size, D, dtype=torch.int8 if dt.itemsize == 1
                               else torch.int16, device=device).view(dt)
        if table is None:
            table = torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=pool.device)
        if ref is None:
            ref = torch.zeros(pool.shape[1], dtype=torch.int32, device=pool.device)
        if pool.dim() != 4 or pool.shape[3] != D or pool.dtype != dt or (
                pool.stride()[1:] != (pool.shape[2] * D, D, 1)):
            _fail("PagedCache: pool must be [layers, n_pages, page_size, %d] of %s with contiguous layers" % (D, dt))
        if table.dim() != 2 or table.dtype != torch.int32 or not table.is_contiguous():
            _fail("PagedCache: table must be contiguous int32 [max_seqs, max_pages]")
        _i32("ref", ref, pool.shape[1], pool.get_device())
        _at("table", table, pool.get_device())
        self.device, self.index, self.kv_format = pool.device, pool.get_device(), params.kv_format
        self.pool, self.table, self.ref = pool, table, ref
        self.c = Pages(pool.data_ptr(), pool.stride(0) * pool.element_size(), table.data_ptr(),
                       ref.data_ptr(), pool.shape[0], pool.shape[1], pool.shape[2], table.shape[0],
                       table.shape[1])
        n = lib().csa2_page_workspace_size(self.c)
        self.workspace = torch.empty(max(int(n), 256), dtype=torch.uint8, device=self.device)
        self.ws_ptr, self.ws_bytes = self.workspace.data_ptr(), self.workspace.numel()


def n_blocks(n: int) -> int:
    return math.ceil(n / BLK)
