"""libjointattn: generalized-causal GQA attention with generalized 2D RoPE
(HunyuanImage-3.0) for B200 / sm_100a.

Thin ctypes binding over the C ABI in ``include/jointattn.h``: these functions
only marshal arguments (torch tensors -> pointers and strides, the current
torch CUDA stream); every step runs in the library's CUDA kernels.  There is no
CPU fallback: if ``libjointattn.so`` is missing or fails to load, every call
raises.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "HiaError", "Segments", "lib", "hia_segments_build", "hia_rope2d_tables", "hia_attn_fwd",
    "hia_attn_bwd", "hia_attn_fwd_workspace_bytes", "hia_attn_bwd_workspace_bytes",
    "hia_get_device_status", "hia_debug_wait_timeout", "hia_profile_begin", "hia_profile_end",
    "hia_rope_plan", "hia_rope_axes_tables", "hia_rope_axes_fwd", "hia_rope_axes_bwd", "hia_cache",
    "hia_cache_chunk", "hia_cache_append", "hia_attn_cache_fwd", "hia_attn_cache_workspace_bytes",
    "Step", "hia_step_create", "hia_attn_step_host", "hia_segments_build_packed", "hia_segments_build_multi",
    "LIB_PATH",
    "EXPORTED_SYMBOLS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libjointattn.so")

EXPORTED_SYMBOLS = (
    "hia_segments_build", "hia_segments_upload", "hia_segments_destroy", "hia_segments_info",
    "hia_segments_row_bound", "hia_segments_mask", "hia_segments_tile_classes", "hia_rope2d_tables",
    "hia_attn_fwd_workspace_bytes", "hia_attn_fwd", "hia_attn_bwd_workspace_bytes", "hia_attn_bwd",
    "hia_get_device_status", "hia_debug_wait_timeout", "hia_status_string", "hia_profile_begin",
    "hia_profile_end", "hia_attn_fwd_noalloc", "hia_debug_exp2", "hia_step_create", "hia_step_destroy",
    "hia_attn_step_host", "hia_attn_fwd_ex", "hia_attn_bwd_ex", "hia_segments_build_packed",
    "hia_segments_layout", "hia_segments_build_multi", "hia_attn_bwd_reuse_fwd",
    "hia_moe_workspace_bytes", "hia_moe_fwd", "hia_segments_set_bwd_split", "hia_segments_bwd_schedule",
    "hia_segments_bwd_choice", "hia_rope_plan_init", "hia_rope_axes_tables", "hia_rope_axes_fwd",
    "hia_rope_axes_bwd", "hia_cache_append", "hia_attn_cache_workspace_bytes", "hia_attn_cache_fwd",
)


class HiaError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        super().__init__(f"{what}: {_status_string(code)} (status {code})")


class _Sample(ctypes.Structure):
    _fields_ = [("prefix_len", ctypes.c_int32), ("img_h", ctypes.c_int32),
                ("img_w", ctypes.c_int32), ("suffix_len", ctypes.c_int32)]


class _Tensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_s", ctypes.c_int64),
                ("stride_hkv", ctypes.c_int64), ("stride_hq", ctypes.c_int64)]


class SegmentsInfo(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("S", ctypes.c_int32), ("visible_pairs", ctypes.c_int64),
                ("fwd_q_tiles", ctypes.c_int32), ("fwd_kv_tiles", ctypes.c_int32),
                ("fwd_tiles_full", ctypes.c_int64), ("fwd_tiles_partial", ctypes.c_int64),
                ("fwd_tiles_skipped", ctypes.c_int64), ("bwd_q_tiles", ctypes.c_int32),
                ("bwd_kv_tiles", ctypes.c_int32), ("packed", ctypes.c_int32), ("bwd_split_units", ctypes.c_int32),
                ("total_rows", ctypes.c_int64)]


class _QkNorm(ctypes.Structure):
    _fields_ = [("wq", ctypes.c_void_p), ("wk", ctypes.c_void_p), ("eps", ctypes.c_float)]


class _Image(ctypes.Structure):
    _fields_ = [("text_before", ctypes.c_int32), ("img_h", ctypes.c_int32), ("img_w", ctypes.c_int32)]


class _MoeDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
                ("topk", ctypes.c_int32)]


class RopePlan(ctypes.Structure):
    """hia_rope_plan: plain host data; axis and freq may be changed (e.g. for
    a rescaled ladder) before it is used."""
    _fields_ = [("D", ctypes.c_int32), ("n_axes", ctypes.c_int32), ("axis", ctypes.c_uint8 * 128),
                ("freq", ctypes.c_double * 128)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("stride_page", ctypes.c_int64),
                ("stride_s", ctypes.c_int64), ("stride_h", ctypes.c_int64), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class _Chunk(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("past", ctypes.c_void_p), ("pages", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("B", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class _KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int32), ("total_ms", ctypes.c_double)]


_lib = None


def lib():
    """The loaded libjointattn.so (raises if it is missing: no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                              "or python joint_text_image_b200/build.py")
        L = ctypes.CDLL(LIB_PATH)
        P, I, Z, T = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, _Tensor
        L.hia_segments_build.argtypes = [ctypes.POINTER(_Sample), I, I, ctypes.POINTER(P)]
        L.hia_segments_build_packed.argtypes = [ctypes.POINTER(_Sample), I, ctypes.POINTER(P)]
        L.hia_segments_build_multi.argtypes = [ctypes.POINTER(_Image), P, P, I, I, I, ctypes.POINTER(P)]
        L.hia_segments_upload.argtypes = [P, P]
        L.hia_segments_destroy.argtypes = [P]
        L.hia_segments_destroy.restype = None
        L.hia_segments_info.argtypes = [P, ctypes.POINTER(SegmentsInfo)]
        L.hia_segments_set_bwd_split.argtypes = [P, I]
        L.hia_segments_bwd_schedule.argtypes = [P, I, P, P, P]
        L.hia_segments_bwd_choice.argtypes = [P, I, I, I, P]
        L.hia_segments_row_bound.argtypes = [P, P]
        L.hia_segments_layout.argtypes = [P, P, P]
        L.hia_segments_mask.argtypes = [P, P]
        L.hia_segments_tile_classes.argtypes = [P, P]
        L.hia_rope2d_tables.argtypes = [P, I, ctypes.c_double, P, P, P]
        L.hia_attn_fwd_workspace_bytes.argtypes = [P, I, I, I]
        L.hia_attn_fwd_workspace_bytes.restype = Z
        L.hia_attn_bwd_workspace_bytes.argtypes = [P, I, I, I]
        L.hia_attn_bwd_workspace_bytes.restype = Z
        L.hia_attn_fwd.argtypes = [P, I, I, I, T, T, T, P, P, ctypes.c_float, T, P, P, Z, P]
        L.hia_attn_bwd.argtypes = [P, I, I, I, T, T, T, P, P, ctypes.c_float, T, P, T, T, T, T, P, Z, P]
        L.hia_attn_bwd_reuse_fwd.argtypes = [P, I, I, I, T, T, T, P, P, ctypes.c_float, P, T, P, T, T, T, T, P, P,
                                             P, Z, P, Z, P]
        L.hia_moe_workspace_bytes.argtypes = [ctypes.POINTER(_MoeDims)]
        L.hia_moe_workspace_bytes.restype = Z
        L.hia_moe_fwd.argtypes = [ctypes.POINTER(_MoeDims), P, P, P, P, P, P, P, P, Z, P]
        L.hia_get_device_status.argtypes = [P]
        L.hia_debug_wait_timeout.argtypes = [ctypes.c_uint64, P]
        QN = ctypes.POINTER(_QkNorm)
        L.hia_attn_fwd_ex.argtypes = [P, I, I, I, T, T, T, P, P, ctypes.c_float, QN, T, P, P, Z, P]
        L.hia_attn_bwd_ex.argtypes = [P, I, I, I, T, T, T, P, P, ctypes.c_float, QN, T, P, T, T, T, T, P, P, P,
                                      Z, P]
        L.hia_attn_fwd_noalloc.argtypes = [P, I, I, I, T, T, T, P, P, ctypes.c_float, T, P, P]
        L.hia_debug_exp2.argtypes = [P, P, I, P]
        L.hia_step_create.argtypes = [P, I, I, I, ctypes.c_double, ctypes.POINTER(P)]
        L.hia_step_destroy.argtypes = [P]
        L.hia_step_destroy.restype = None
        L.hia_attn_step_host.argtypes = [P, P, P, P, P, ctypes.c_float, P, P, P, P, P, P]
        L.hia_profile_begin.argtypes = []
        L.hia_profile_end.argtypes = [ctypes.POINTER(_KernelTime), I, ctypes.POINTER(I)]
        RP, KC, KK, I64 = ctypes.POINTER(RopePlan), ctypes.POINTER(_Cache), ctypes.POINTER(_Chunk), ctypes.c_int64
        L.hia_rope_plan_init.argtypes = [RP, I, I, P, ctypes.c_double, I]
        L.hia_rope_axes_tables.argtypes = [RP, I64, P, P, P, P]
        L.hia_rope_axes_fwd.argtypes = [RP, I64, P, I, I, I, T, T, T, T, P]
        L.hia_rope_axes_bwd.argtypes = [RP, I64, P, I, I, I, T, T, T, T, P]
        L.hia_cache_append.argtypes = [KC, KK, I64, I, RP, P, QN, T, T, T, T, P]
        L.hia_attn_cache_workspace_bytes.argtypes = [KC, KK, I64, I]
        L.hia_attn_cache_workspace_bytes.restype = Z
        L.hia_attn_cache_fwd.argtypes = [KC, KK, I64, I, T, P, ctypes.c_float, T, P, P, Z, P]
        L.hia_status_string.argtypes = [I]
        L.hia_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _status_string(code):
    try:
        return lib().hia_status_string(int(code)).decode()
    except Exception:  # library missing: still report the code
        return "status"


def _check(rc, what):
    if rc != 0:
        raise HiaError(rc, what)


_raw_stream = None


def _stream():
    """The current CUDA stream of the current device, as a cudaStream_t."""
    import torch
    return ctypes.c_void_p(_raw(torch.cuda.current_device()))


def _raw(dev):
    """The current stream of device dev, as a number."""
    global _raw_stream
    if _raw_stream is None:  # the handle alone, without a Stream object (3.4 us less per call)
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    return _raw_stream(dev)


class Segments:
    """Owner of a library hia_segments object (host tables + device copies)."""

    def __init__(self, samples, S, packed=False):
        """samples: (prefix, img_h, img_w, suffix) per sample, or, for several
        images, (images, suffix) with images a list of (text_before, h, w)."""
        h = ctypes.c_void_p()
        multi = any(len(x) == 2 for x in samples)
        if multi:
            norm = [x if len(x) == 2 else (([(x[0], x[1], x[2])], x[3]) if x[1] * x[2] > 0 else ([], x[0] + x[3]))
                    for x in samples]
            imgs = [im for (ims, _) in norm for im in ims]
            iarr = (_Image * max(1, len(imgs)))(*[_Image(*map(int, im)) for im in imgs])
            import numpy as np
            n_img = np.asarray([len(ims) for (ims, _) in norm] or [0], dtype=np.int32)
            suf = np.asarray([sf for (_, sf) in norm] or [0], dtype=np.int32)
            _check(lib().hia_segments_build_multi(iarr, n_img.ctypes.data_as(ctypes.c_void_p),
                                                  suf.ctypes.data_as(ctypes.c_void_p), len(samples), int(S),
                                                  int(bool(packed)), ctypes.byref(h)), "hia_segments_build_multi")
            self.samples = [([tuple(map(int, im)) for im in ims], int(sf)) for (ims, sf) in norm]
            self.lengths = [sum(t + hh * ww for (t, hh, ww) in ims) + sf for (ims, sf) in self.samples]
        else:
            arr = (_Sample * max(1, len(samples)))(*[_Sample(*map(int, x)) for x in samples])
            if packed:
                _check(lib().hia_segments_build_packed(arr, len(samples), ctypes.byref(h)),
                       "hia_segments_build_packed")
            else:
                _check(lib().hia_segments_build(arr, len(samples), int(S), ctypes.byref(h)), "hia_segments_build")
            self.samples = [tuple(map(int, x)) for x in samples]
            self.lengths = [p + hh * ww + sf for (p, hh, ww, sf) in self.samples]
        self.handle = h
        inf = self.info()
        self.B, self.S = len(samples), int(inf.S)
        self.packed = bool(inf.packed)
        self.total_rows = int(inf.total_rows)
        self.rows, self.offsets = self.layout()
        self.on_device = False

    def upload(self):
        _check(lib().hia_segments_upload(self.handle, _stream()), "hia_segments_upload")
        self.on_device = True
        return self

    def info(self) -> SegmentsInfo:
        out = SegmentsInfo()
        _check(lib().hia_segments_info(self.handle, ctypes.byref(out)), "hia_segments_info")
        return out

    def layout(self):
        """(rows, offsets) per sample, from the library: a sample's rows in a
        tensor of this layout and its first row."""
        import numpy as np
        r = np.zeros(max(self.B, 1), dtype=np.int32)
        o = np.zeros(max(self.B, 1), dtype=np.int32)
        _check(lib().hia_segments_layout(self.handle, r.ctypes.data_as(ctypes.c_void_p),
                                         o.ctypes.data_as(ctypes.c_void_p)), "hia_segments_layout")
        return [int(x) for x in r[:self.B]], [int(x) for x in o[:self.B]]

    def row_bound(self):
        import numpy as np
        e = np.zeros((self.B, self.S), dtype=np.int32)
        _check(lib().hia_segments_row_bound(self.handle, e.ctypes.data_as(ctypes.c_void_p)), "row_bound")
        return e

    def set_bwd_split(self, mode):
        """Backward schedule (hia_segments_set_bwd_split): 0 auto (default),
        1 never split, 2 the best split schedule, 3 / 4 / 5 the best one
        cutting the longest kv tiles into exactly 2 / 3 / 4 parts."""
        _check(lib().hia_segments_set_bwd_split(self.handle, int(mode)), "hia_segments_set_bwd_split")
        return self

    def bwd_schedules(self):
        """Every backward schedule of the descriptor as (parts, entries):
        entries int32 [n, 8] = (b, kv tile, first query tile, end query tile,
        slot, part, parts, 0) in launch order (hia_segments_bwd_schedule)."""
        import numpy as np
        out = []
        while True:
            parts, n = ctypes.c_int32(0), ctypes.c_int64(0)
            rc = lib().hia_segments_bwd_schedule(self.handle, len(out), ctypes.byref(parts), ctypes.byref(n), None)
            if rc != 0:
                return out
            e = np.zeros((max(n.value, 1), 8), dtype=np.int32)
            _check(lib().hia_segments_bwd_schedule(self.handle, len(out), ctypes.byref(parts), ctypes.byref(n),
                                                   e.ctypes.data_as(ctypes.c_void_p)), "hia_segments_bwd_schedule")
            out.append((parts.value, e[:n.value]))

    def bwd_choice(self, Hkv, g, n_sm):
        """Index into bwd_schedules() of the schedule a backward launch takes
        (hia_segments_bwd_choice)."""
        i = ctypes.c_int(0)
        _check(lib().hia_segments_bwd_choice(self.handle, int(Hkv), int(g), int(n_sm), ctypes.byref(i)),
               "hia_segments_bwd_choice")
        return i.value

    def mask(self):
        import numpy as np
        m = np.zeros((self.B, self.S, self.S), dtype=np.uint8)
        _check(lib().hia_segments_mask(self.handle, m.ctypes.data_as(ctypes.c_void_p)), "mask")
        return m

    def tile_classes(self):
        import numpy as np
        inf = self.info()
        c = np.zeros((self.B, inf.fwd_q_tiles, inf.fwd_kv_tiles), dtype=np.uint8)
        _check(lib().hia_segments_tile_classes(self.handle, c.ctypes.data_as(ctypes.c_void_p)), "tile_classes")
        return c

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib is not None:
            _lib.hia_segments_destroy(h)
            self.handle = None


def hia_segments_build(samples, S, upload=True) -> Segments:
    """Segment descriptor for samples [(prefix, img_h, img_w, suffix)] padded to S."""
    seg = Segments(samples, S)
    return seg.upload() if upload else seg


def hia_segments_build_packed(samples, upload=True) -> Segments:
    """Segment descriptor for the packed (varlen) layout: samples back to back,
    tensors [total_rows, heads, D], lse [Hq, total_rows]."""
    seg = Segments(samples, 0, packed=True)
    return seg.upload() if upload else seg


def hia_segments_build_multi(samples, S=0, packed=False, upload=True) -> Segments:
    """Segment descriptor for samples with any number of images: each sample
    (images, suffix), images a list of (text_before, img_h, img_w); every
    image but a sample's last is hidden from all tokens after it."""
    seg = Segments([x if len(x) == 2 else x for x in samples], S, packed=packed)
    return seg.upload() if upload else seg


def _view(seg, x):
    """A packed [T,H,D] (or grouped [T,Hkv,g,D]) tensor as one batch row."""
    return x.unsqueeze(0) if (x is not None and seg.packed) else x


def _t(x, q_heads, g):
    """hia_tensor from a [B,S,H,D] torch view (or a [B,S,Hkv,g+2,D] fused slice)."""
    if x is None:
        return _Tensor(None, 0, 0, 0, 0)
    if x.dim() == 4:
        sb, ss, sh, sd = x.stride()
        if sd != 1:
            raise ValueError("last dimension must be contiguous")
        return _Tensor(x.data_ptr(), sb, ss, sh * g if q_heads else sh, sh if q_heads else 0)
    if x.dim() == 5:  # [B, S, Hkv, g, D] grouped view
        sb, ss, shkv, shq, sd = x.stride()
        if sd != 1:
            raise ValueError("last dimension must be contiguous")
        return _Tensor(x.data_ptr(), sb, ss, shkv, shq)
    raise ValueError("expected a 4-D [B,S,H,D] or 5-D [B,S,Hkv,g,D] tensor")


def _heads(x):
    return x.shape[2] * (x.shape[3] if x.dim() == 5 else 1)


def hia_rope2d_tables(seg: Segments, D: int, base: float = 10000.0, out=None):
    """fp32 cos, sin [B, S, D] on the current CUDA device."""
    import torch
    if out is None:
        out = (torch.empty(seg.B, seg.S, D, device="cuda", dtype=torch.float32),
               torch.empty(seg.B, seg.S, D, device="cuda", dtype=torch.float32))
    c, s = out
    _check(lib().hia_rope2d_tables(seg.handle, int(D), float(base), c.data_ptr(), s.data_ptr(), _stream()),
           "hia_rope2d_tables")
    return c, s


def hia_attn_fwd_workspace_bytes(seg: Segments, Hq, Hkv, D):
    return int(lib().hia_attn_fwd_workspace_bytes(seg.handle, Hq, Hkv, D))


def hia_attn_bwd_workspace_bytes(seg: Segments, Hq, Hkv, D):
    return int(lib().hia_attn_bwd_workspace_bytes(seg.handle, Hq, Hkv, D))


def _ws(nbytes, workspace):
    import torch
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small")
        return workspace
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")


def _norm(qk_norm, D):
    """qk_norm = (wq, wk, eps) with fp32 [D] CUDA weights -> pointer to a
    hia_qk_norm (or None); the tensors are kept alive by the caller."""
    if qk_norm is None:
        return None
    wq, wk, eps = qk_norm
    for w in (wq, wk):
        if not w.is_cuda or w.dtype.itemsize != 4 or not w.dtype.is_floating_point or w.numel() != D \
                or not w.is_contiguous():
            raise ValueError("QK-norm weights must be contiguous fp32 CUDA tensors of D elements")
    return ctypes.pointer(_QkNorm(wq.data_ptr(), wk.data_ptr(), float(eps)))


def hia_attn_fwd(seg: Segments, q, k, v, cos, sin, scale=None, o=None, lse=None, workspace=None,
                 qk_norm=None):
    """Forward.  q [B,S,Hq,D], k, v [B,S,Hkv,D] bf16 CUDA tensors (or grouped
    5-D views).  Returns (o [B,S,Hq,D] bf16, lse [B,Hq,S] fp32).  qk_norm:
    optional (wq, wk, eps), fp32 [D] CUDA weights of the per-head RMSNorm
    applied after RoPE (hia_attn_fwd_ex)."""
    import torch
    Hq, Hkv, D = _heads(_view(seg, q)), _heads(_view(seg, k)), q.shape[-1]
    g = Hq // Hkv
    if scale is None:
        scale = D ** -0.5
    if o is None:
        shape = (seg.total_rows, Hq, D) if seg.packed else (seg.B, seg.S, Hq, D)
        o = torch.empty(shape, device=q.device, dtype=torch.bfloat16)
    if lse is None:
        shape = (Hq, seg.total_rows) if seg.packed else (seg.B, Hq, seg.S)
        lse = torch.empty(shape, device=q.device, dtype=torch.float32)
    o_ret = o
    q, k, v, o = (_view(seg, x) for x in (q, k, v, o))
    nb = hia_attn_fwd_workspace_bytes(seg, Hq, Hkv, D)
    ws = _ws(nb, workspace)
    if qk_norm is None:
        _check(lib().hia_attn_fwd(seg.handle, Hq, Hkv, D, _t(q, True, g), _t(k, False, 1), _t(v, False, 1),
                                  cos.data_ptr(), sin.data_ptr(), float(scale), _t(o, True, g), lse.data_ptr(),
                                  ws.data_ptr(), nb, _stream()), "hia_attn_fwd")
    else:
        _check(lib().hia_attn_fwd_ex(seg.handle, Hq, Hkv, D, _t(q, True, g), _t(k, False, 1), _t(v, False, 1),
                                     cos.data_ptr(), sin.data_ptr(), float(scale), _norm(qk_norm, D),
                                     _t(o, True, g), lse.data_ptr(), ws.data_ptr(), nb, _stream()),
               "hia_attn_fwd_ex")
    return o_ret, lse


def hia_attn_bwd(seg: Segments, q, k, v, cos, sin, o, lse, dout, scale=None, dq=None, dk=None, dv=None,
                 workspace=None, qk_norm=None, fwd_workspace=None):
    """Recompute backward.  Returns (dq, dk, dv) bf16; with qk_norm (the
    forward's (wq, wk, eps)) returns (dq, dk, dv, dwq, dwk), dwq/dwk fp32 [D]
    (hia_attn_bwd_ex).  fwd_workspace: the workspace tensor of the forward
    that produced o and lse, untouched since; its rotated q and k are reused
    (hia_attn_bwd_reuse_fwd)."""
    import torch
    Hq, Hkv, D = _heads(_view(seg, q)), _heads(_view(seg, k)), q.shape[-1]
    g = Hq // Hkv
    if scale is None:
        scale = D ** -0.5
    lead = (seg.total_rows,) if seg.packed else (seg.B, seg.S)
    if dq is None:
        dq = torch.empty(*lead, Hq, D, device=q.device, dtype=torch.bfloat16)
    if dk is None:
        dk = torch.empty(*lead, Hkv, D, device=q.device, dtype=torch.bfloat16)
    if dv is None:
        dv = torch.empty(*lead, Hkv, D, device=q.device, dtype=torch.bfloat16)
    ret = (dq, dk, dv)
    q, k, v, o, dout, dq, dk, dv = (_view(seg, x) for x in (q, k, v, o, dout, dq, dk, dv))
    nb = hia_attn_bwd_workspace_bytes(seg, Hq, Hkv, D)
    ws = _ws(nb, workspace)
    if fwd_workspace is not None:
        nf = hia_attn_fwd_workspace_bytes(seg, Hq, Hkv, D)
        if fwd_workspace.numel() * fwd_workspace.element_size() < nf:
            raise ValueError("forward workspace too small")
        dwq = dwk = None
        if qk_norm is not None:
            dwq = torch.empty(D, device=q.device, dtype=torch.float32)
            dwk = torch.empty(D, device=q.device, dtype=torch.float32)
        _check(lib().hia_attn_bwd_reuse_fwd(
            seg.handle, Hq, Hkv, D, _t(q, True, g), _t(k, False, 1), _t(v, False, 1), cos.data_ptr(),
            sin.data_ptr(), float(scale), _norm(qk_norm, D), _t(o, True, g), lse.data_ptr(), _t(dout, True, g),
            _t(dq, True, g), _t(dk, False, 1), _t(dv, False, 1), dwq.data_ptr() if dwq is not None else None,
            dwk.data_ptr() if dwk is not None else None, fwd_workspace.data_ptr(), nf, ws.data_ptr(), nb,
            _stream()), "hia_attn_bwd_reuse_fwd")
        return ret if qk_norm is None else (*ret, dwq, dwk)
    if qk_norm is None:
        _check(lib().hia_attn_bwd(seg.handle, Hq, Hkv, D, _t(q, True, g), _t(k, False, 1), _t(v, False, 1),
                                  cos.data_ptr(), sin.data_ptr(), float(scale), _t(o, True, g), lse.data_ptr(),
                                  _t(dout, True, g), _t(dq, True, g), _t(dk, False, 1), _t(dv, False, 1),
                                  ws.data_ptr(), nb, _stream()), "hia_attn_bwd")
        return ret
    dwq = torch.empty(D, device=q.device, dtype=torch.float32)
    dwk = torch.empty(D, device=q.device, dtype=torch.float32)
    _check(lib().hia_attn_bwd_ex(seg.handle, Hq, Hkv, D, _t(q, True, g), _t(k, False, 1), _t(v, False, 1),
                                 cos.data_ptr(), sin.data_ptr(), float(scale), _norm(qk_norm, D), _t(o, True, g),
                                 lse.data_ptr(), _t(dout, True, g), _t(dq, True, g), _t(dk, False, 1),
                                 _t(dv, False, 1), dwq.data_ptr(), dwk.data_ptr(), ws.data_ptr(), nb, _stream()),
           "hia_attn_bwd_ex")
    return (*ret, dwq, dwk)


class Step:
    """Owner of a library hia_step: device buffers, RoPE tables and workspaces
    for training steps fed from host memory (hia_attn_step_host)."""

    def __init__(self, seg: "Segments", Hq, Hkv, D, base=10000.0):
        self.seg, self.Hq, self.Hkv, self.D = seg, Hq, Hkv, D
        h = ctypes.c_void_p()
        _check(lib().hia_step_create(seg.handle, int(Hq), int(Hkv), int(D), float(base), ctypes.byref(h)),
               "hia_step_create")
        self.handle = h

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.hia_step_destroy(self.handle)
            self.handle = None


def hia_step_create(seg: "Segments", Hq, Hkv, D, base=10000.0) -> Step:
    return Step(seg, Hq, Hkv, D, base)


def hia_attn_step_host(step: Step, q, k, v, dout, o, lse, dq, dk, dv, scale=None, stream=None):
    """One forward + backward from host tensors (contiguous CPU tensors; pin
    them for asynchronous copies): q, dout [B,S,Hq,D], k, v [B,S,Hkv,D] bf16
    in; o, dq [B,S,Hq,D], dk, dv [B,S,Hkv,D] bf16 and lse [B,Hq,S] fp32 out.
    Enqueued on `stream` (default: the current CUDA stream)."""
    import torch
    B, S, Hq, Hkv, D = step.seg.B, step.seg.S, step.Hq, step.Hkv, step.D
    want = ((q, (B, S, Hq, D), torch.bfloat16), (k, (B, S, Hkv, D), torch.bfloat16),
            (v, (B, S, Hkv, D), torch.bfloat16), (dout, (B, S, Hq, D), torch.bfloat16),
            (o, (B, S, Hq, D), torch.bfloat16), (lse, (B, Hq, S), torch.float32),
            (dq, (B, S, Hq, D), torch.bfloat16), (dk, (B, S, Hkv, D), torch.bfloat16),
            (dv, (B, S, Hkv, D), torch.bfloat16))
    for t, shape, dt in want:
        if t.is_cuda or not t.is_contiguous() or tuple(t.shape) != shape or t.dtype != dt:
            raise ValueError(f"hia_attn_step_host takes contiguous host tensors {shape} {dt}")
    if scale is None:
        scale = step.D ** -0.5
    st = _stream() if stream is None else ctypes.c_void_p(stream.cuda_stream)
    _check(lib().hia_attn_step_host(step.handle, q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(),
                                    float(scale), o.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                    dv.data_ptr(), st), "hia_attn_step_host")


def hia_get_device_status():
    return int(lib().hia_get_device_status(_stream()))


def hia_debug_wait_timeout(timeout_ns: int):
    _check(lib().hia_debug_wait_timeout(int(timeout_ns), _stream()), "hia_debug_wait_timeout")


def hia_profile_begin():
    """Start per-kernel CUDA-event timing of every library launch."""
    _check(lib().hia_profile_begin(), "hia_profile_begin")


def hia_profile_end():
    """Stop timing; returns {kernel name: (launches, total_ms)}."""
    arr = (_KernelTime * 32)()
    n = ctypes.c_int(0)
    _check(lib().hia_profile_end(arr, 32, ctypes.byref(n)), "hia_profile_end")
    return {arr[i].name.decode(): (int(arr[i].launches), float(arr[i].total_ms)) for i in range(min(n.value, 32))}


def hia_moe_workspace_bytes(T, H, I, E, topk):
    return int(lib().hia_moe_workspace_bytes(ctypes.byref(_MoeDims(T, H, I, E, topk))))


def hia_moe_fwd(x, wg, w13, w2, topk, out=None, workspace=None):
    """MoE feed-forward of one block (jointmoe.h): x bf16 [T, H], wg fp32
    [E, H], w13 bf16 [E + 1, 2I, H] ([up; gate], index E the shared expert),
    w2 bf16 [E + 1, H, I], all contiguous CUDA tensors.  Returns (out bf16
    [T, H], topk_ids int32 [T, topk], topk_weights fp32 [T, topk])."""
    import torch
    T, H = x.shape
    E = wg.shape[0]
    I = w13.shape[1] // 2
    for t, dt in ((x, torch.bfloat16), (wg, torch.float32), (w13, torch.bfloat16), (w2, torch.bfloat16)):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != dt:
            raise ValueError("hia_moe_fwd takes contiguous CUDA tensors (x, w13, w2 bf16; wg fp32)")
    if tuple(w13.shape) != (E + 1, 2 * I, H) or tuple(w2.shape) != (E + 1, H, I) or wg.shape[1] != H:
        raise ValueError("inconsistent MoE weight shapes")
    dims = _MoeDims(T, H, I, E, int(topk))
    nb = int(lib().hia_moe_workspace_bytes(ctypes.byref(dims)))
    if nb == 0:
        raise HiaError(1, "hia_moe_workspace_bytes")
    ws = _ws(nb, workspace)
    if out is None:
        out = torch.empty(T, H, device=x.device, dtype=torch.bfloat16)
    ids = torch.empty(T, topk, device=x.device, dtype=torch.int32)
    w = torch.empty(T, topk, device=x.device, dtype=torch.float32)
    _check(lib().hia_moe_fwd(ctypes.byref(dims), x.data_ptr(), wg.data_ptr(), w13.data_ptr(), w2.data_ptr(),
                             out.data_ptr(), ids.data_ptr(), w.data_ptr(), ws.data_ptr(), nb, _stream()),
           "hia_moe_fwd")
    return out, ids, w


# ---------------------------------------------------------------- rotary positions with several axes
_NO_TENSOR = _Tensor(None, 0, 0, 0, 0)
_DTYPE_CODES = {}


def _dtype_code(dtype):
    if not _DTYPE_CODES:
        import torch
        _DTYPE_CODES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    code = _DTYPE_CODES.get(dtype)
    if code is None:
        raise ValueError(f"bf16, fp16 or fp32 tensors, not {dtype}")
    return code


def _on_device(*tensors):
    """Every tensor (None allowed) on the current CUDA device."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        d = t.get_device()  # -1 on the host
        if d < 0:
            raise ValueError("expected CUDA tensors")
        if dev is None:
            import torch
            dev = torch.cuda.current_device()
        if d != dev:
            raise ValueError("tensors on another device than the current one")


def _int32(t, shape, what, dev=None):
    """t a contiguous int32 tensor of that shape (and on that device)."""
    import torch
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous int32 {shape}")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{what} on another device")


def _q_heads(x):
    """Heads of a packed [T, H, D] tensor or [T, Hkv, g, D] view."""
    sh = x.shape
    if len(sh) == 3:
        return sh[1]
    if len(sh) == 4:
        return sh[1] * sh[2]
    raise ValueError("expected a packed [T, H, D] tensor or a [T, Hkv, g, D] view")


def _rows_q(x, T, Hq, Hkv, D, dtype, dev):
    """hia_tensor of a packed [T, Hq, D] tensor or [T, Hkv, g, D] view."""
    sh = x.shape
    if x.get_device() != dev or x.dtype is not dtype or sh[0] != T or sh[-1] != D:
        raise ValueError("tensors of different devices, types, rows or head dimensions")
    st = x.stride()
    if st[-1] != 1 and D != 1:
        raise ValueError("last dimension must be contiguous")
    if len(st) == 3:
        if sh[1] != Hq:
            raise ValueError("tensors of different heads")
        return _Tensor(x.data_ptr(), 0, st[0], st[1] * (Hq // Hkv), st[1])
    if len(st) != 4 or sh[1] != Hkv or sh[1] * sh[2] != Hq:
        raise ValueError("expected [T, Hq, D], or a grouped view [T, Hkv, Hq / Hkv, D]")
    return _Tensor(x.data_ptr(), 0, st[0], st[1], st[2])


def _rows_kv(x, T, Hkv, D, dtype, dev):
    """hia_tensor of a packed [T, Hkv, D] tensor."""
    sh = x.shape
    if len(sh) != 3 or sh[0] != T or sh[1] != Hkv or sh[2] != D or x.dtype is not dtype or x.get_device() != dev:
        raise ValueError("expected packed [T, Hkv, D] tensors of one device and type")
    st = x.stride()
    if st[2] != 1 and D != 1:
        raise ValueError("last dimension must be contiguous")
    return _Tensor(x.data_ptr(), 0, st[0], st[1], 0)


_devices = {}


def _empty(shape, dtype, dev):
    import torch
    d = _devices.get(dev)
    if d is None:
        d = _devices[dev] = torch.device("cuda", dev)
    return torch.empty(shape, dtype=dtype, device=d)


def _empty_rows(x, T, H, D, dtype, dev):
    """An uninitialised packed [T, H, D] tensor, the result for x."""
    if x.dim() == 3 and x.is_contiguous():
        import torch
        return torch.empty_like(x)  # half the host time of torch.empty
    return _empty((T, H, D), dtype, dev)


def _current_device(x):
    """The device of x, which has to be the current one."""
    dev = x.get_device()  # -1 on the host
    if dev < 0:
        raise ValueError("expected CUDA tensors")
    import torch
    if dev != torch.cuda.current_device():
        raise ValueError("tensors on another device than the current one")
    return dev


def hia_rope_plan(D, n_axes, sections=None, base=10000.0, per_axis=False) -> RopePlan:
    """Rotary plan for head dimension D and n_axes position axes
    (hia_rope_plan_init): sections = pairs of each axis (summing to D/2) or
    None to interleave them; per_axis: each axis its own frequency ladder."""
    plan = RopePlan()
    sec = None
    if sections is not None:
        if len(sections) != n_axes:
            raise ValueError("one section per axis")
        sec = (ctypes.c_int32 * len(sections))(*[int(x) for x in sections])
    _check(lib().hia_rope_plan_init(ctypes.byref(plan), int(D), int(n_axes), sec, float(base), int(bool(per_axis))),
           "hia_rope_plan_init")
    return plan


def hia_rope_axes_tables(plan: RopePlan, pos, out=None):
    """fp32 cos, sin [T, D] of positions pos int32 [T, n_axes]: the tables
    hia_attn_fwd / hia_attn_bwd take (viewed as [B, S, D])."""
    import torch
    T = pos.shape[0]
    _int32(pos, (T, plan.n_axes), "pos")
    if out is None:
        out = (torch.empty(T, plan.D, device=pos.device, dtype=torch.float32),
               torch.empty(T, plan.D, device=pos.device, dtype=torch.float32))
    _on_device(pos, *out)
    for t in out:
        if t.dtype != torch.float32 or t.numel() != T * plan.D or not t.is_contiguous():
            raise ValueError("cos, sin: contiguous fp32 tensors of T * D elements")
    _check(lib().hia_rope_axes_tables(plan, T, pos.data_ptr(), out[0].data_ptr(), out[1].data_ptr(),
                                      _stream()), "hia_rope_axes_tables")
    return out


def _rope_axes(fn, what, plan, pos, q, k, q_out, k_out):
    sh = q.shape
    Hq, T, D, dtype = _q_heads(q), sh[0], sh[-1], q.dtype
    Hkv = k.shape[1] if k is not None else sh[1] if len(sh) == 4 else Hq
    if D != plan.D:
        raise ValueError("the plan is for another head dimension")
    if Hkv == 0 or Hq % Hkv:
        raise HiaError(2, what)
    dev = _current_device(q)
    _int32(pos, (T, plan.n_axes), "pos", dev)
    qs = _rows_q(q, T, Hq, Hkv, D, dtype, dev)
    ks = ko = _NO_TENSOR
    if k is not None:
        ks = _rows_kv(k, T, Hkv, D, dtype, dev)
    if q_out is None:
        q_out = _empty_rows(q, T, Hq, D, dtype, dev)
        qo = _Tensor(q_out.data_ptr(), 0, Hq * D, Hq // Hkv * D, D)
    else:
        qo = _rows_q(q_out, T, Hq, Hkv, D, dtype, dev)
    if k is not None:
        if k_out is None:
            k_out = _empty_rows(k, T, Hkv, D, dtype, dev)
            ko = _Tensor(k_out.data_ptr(), 0, Hkv * D, D, 0)
        else:
            ko = _rows_kv(k_out, T, Hkv, D, dtype, dev)
    rc = fn(plan, T, pos.data_ptr(), _dtype_code(dtype), Hq, Hkv, qs, ks, qo, ko, _raw(dev))
    if rc:
        raise HiaError(rc, what)
    return q_out if k is None else (q_out, k_out)


def hia_rope_axes_fwd(plan: RopePlan, pos, q, k=None, q_out=None, k_out=None):
    """Rotate packed q [T, Hq, D] (or a [T, Hkv, g, D] view) and k [T, Hkv, D]
    by positions pos int32 [T, n_axes].  Returns q_out, or (q_out, k_out);
    passing q and k themselves as outputs rotates in place."""
    return _rope_axes(lib().hia_rope_axes_fwd, "hia_rope_axes_fwd", plan, pos, q, k, q_out, k_out)


def hia_rope_axes_bwd(plan: RopePlan, pos, dq_out, dk_out=None, dq=None, dk=None):
    """Gradient of hia_rope_axes_fwd: dq = R^T dq_out, dk = R^T dk_out."""
    return _rope_axes(lib().hia_rope_axes_bwd, "hia_rope_axes_bwd", plan, pos, dq_out, dk_out, dq, dk)


# ---------------------------------------------------------------- generation over a paged cache
class Cache:
    """A hia_cache over the caller's page tensors (kept alive here)."""

    def __init__(self, k_pages, v_pages):
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.stride() != v_pages.stride() \
                or k_pages.dtype != v_pages.dtype or k_pages.stride(3) != 1 \
                or k_pages.get_device() != v_pages.get_device():
            raise ValueError("k_pages, v_pages: [n_pages, page_size, Hkv, D] views of one shape, type and strides")
        self.k_pages, self.v_pages = k_pages, v_pages
        n, ps, h, d = k_pages.shape
        sp, ss, sh, _ = k_pages.stride()
        self.Hkv, self.D, self.dtype, self.device = h, d, k_pages.dtype, k_pages.get_device()
        self.struct = _Cache(k_pages.data_ptr(), v_pages.data_ptr(), sp, ss, sh, n, ps, h, d,
                             _dtype_code(k_pages.dtype))


def hia_cache(k_pages, v_pages) -> Cache:
    """The paged cache over two CUDA tensors viewed as [n_pages, page_size,
    Hkv, D] (token-major contiguous, or head-major pages [n_pages, Hkv,
    page_size, D] transposed)."""
    _on_device(k_pages, v_pages)
    return Cache(k_pages, v_pages)


class Chunk:
    """A hia_cache_chunk over the caller's device arrays (kept alive here; the
    kernels read their values when they run)."""

    def __init__(self, pages, past, rows):
        B = past.shape[0]
        _int32(past, (B,), "past")
        _int32(rows, (B + 1,), "rows")
        if pages.dim() != 2 or pages.shape[0] != B or str(pages.dtype) != "torch.int32" \
                or (pages.shape[1] > 1 and pages.stride(1) != 1):
            raise ValueError("pages: int32 [B, max_pages], rows contiguous")
        if not pages.get_device() == past.get_device() == rows.get_device():
            raise ValueError("pages, past and rows on one device")
        self.pages, self.past, self.rows, self.B, self.device = pages, past, rows, B, pages.get_device()
        self.struct = _Chunk(rows.data_ptr(), past.data_ptr(), pages.data_ptr(), pages.stride(0), B, pages.shape[1])


def hia_cache_chunk(pages, past, rows) -> Chunk:
    """The chunks of new tokens of B sequences: pages int32 [B, max_pages],
    past int32 [B] (tokens already in the cache), rows int32 [B + 1] (first
    row of each sequence's new tokens in the packed tensors, and the end)."""
    _on_device(pages, past, rows)
    return Chunk(pages, past, rows)


def hia_cache_append(cache: Cache, chunk: Chunk, q, k, v, plan=None, pos=None, qk_norm=None, q_out=None):
    """Rotate q [T, Hq, D] (or a [T, Hkv, g, D] view; None: keys and values
    only) and k [T, Hkv, D] of the new tokens by pos int32 [T, n_axes] (plan
    None: no rotation), apply the optional QK RMSNorm (wq, wk, eps), write k
    and v into their pages and q into q_out.  Returns q_out."""
    T, Hkv, D, dtype = k.shape[0], cache.Hkv, cache.D, cache.dtype
    dev = _current_device(k)
    if dev != cache.device or dev != chunk.device:
        raise ValueError("the cache or the chunk is on another device")
    ks, vs = _rows_kv(k, T, Hkv, D, dtype, dev), _rows_kv(v, T, Hkv, D, dtype, dev)
    if q is None:
        Hq, qs, qo, q_out = Hkv, _NO_TENSOR, _NO_TENSOR, None
    else:
        Hq = _q_heads(q)
        if Hq % Hkv:
            raise HiaError(2, "hia_cache_append")
        qs = _rows_q(q, T, Hq, Hkv, D, dtype, dev)
        if q_out is None:
            q_out = _empty_rows(q, T, Hq, D, dtype, dev)
            qo = _Tensor(q_out.data_ptr(), 0, Hq * D, Hq // Hkv * D, D)
        else:
            qo = _rows_q(q_out, T, Hq, Hkv, D, dtype, dev)
    pp = None
    if plan is not None:
        if pos is None:
            raise ValueError("a plan needs positions")
        _int32(pos, (T, plan.n_axes), "pos", dev)
        pp = pos.data_ptr()
    if qk_norm is not None and (qk_norm[0].get_device() != dev or qk_norm[1].get_device() != dev):
        raise ValueError("QK-norm weights on another device")
    rc = lib().hia_cache_append(cache.struct, chunk.struct, T, Hq, plan, pp, _norm(qk_norm, D), qs, ks, vs, qo, _raw(dev))
    if rc:
        raise HiaError(rc, "hia_cache_append")
    return q_out


def hia_attn_cache_workspace_bytes(cache: Cache, chunk: Chunk, T, Hq):
    return lib().hia_attn_cache_workspace_bytes(cache.struct, chunk.struct, T, Hq)


def hia_attn_cache_fwd(cache: Cache, chunk: Chunk, q, bound=None, scale=None, o=None, lse=None, workspace=None):
    """Attention of the chunks' rows q [T, Hq, D] (as hia_cache_append returns
    it) over the cache; bound int32 [T]: each row's last visible cache
    position (None: itself).  workspace: a contiguous CUDA tensor of at least
    hia_attn_cache_workspace_bytes bytes (None: allocated), for one call at a
    time.  Returns (o [T, Hq, D], lse fp32 [Hq, T])."""
    T, Hq, Hkv, D, dtype = q.shape[0], _q_heads(q), cache.Hkv, cache.D, cache.dtype
    if Hq % Hkv:
        raise HiaError(2, "hia_attn_cache_fwd")
    dev = _current_device(q)
    if dev != cache.device or dev != chunk.device:
        raise ValueError("the cache or the chunk is on another device")
    qs = _rows_q(q, T, Hq, Hkv, D, dtype, dev)
    if o is None:
        o = _empty_rows(q, T, Hq, D, dtype, dev)
        os_ = _Tensor(o.data_ptr(), 0, Hq * D, Hq // Hkv * D, D)
    else:
        os_ = _rows_q(o, T, Hq, Hkv, D, dtype, dev)
    fp32 = _fp32()
    if lse is None:
        lse = _empty((Hq, T), fp32, dev)
    elif lse.dtype is not fp32 or tuple(lse.shape) != (Hq, T) or not lse.is_contiguous() or lse.get_device() != dev:
        raise ValueError("lse: contiguous fp32 [Hq, T]")
    bp = None
    if bound is not None:
        _int32(bound, (T,), "bound", dev)
        bp = bound.data_ptr()
    L = lib()
    nb = L.hia_attn_cache_workspace_bytes(cache.struct, chunk.struct, T, Hq)
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError("workspace: a contiguous tensor on the current device")
    ws = _ws(nb, workspace)
    rc = L.hia_attn_cache_fwd(cache.struct, chunk.struct, T, Hq, qs, bp, D ** -0.5 if scale is None else scale, os_,
                              lse.data_ptr(), ws.data_ptr(), nb, _raw(dev))
    if rc:
        raise HiaError(rc, "hia_attn_cache_fwd")
    return o, lse


def _fp32():
    import torch
    return torch.float32
