"""ctypes binding of libvsa (argument marshalling only).

Every step of the layer runs in the CUDA library; this module checks tensor
types, shapes and devices, and passes raw pointers and the current CUDA stream.
PyTorch is used only to allocate device memory and to name streams. If the
library is missing the import fails: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libvsa.so")

MAX_HEADS = 64
MAX_SEGMENTS = 8
TILE = 64

VSA_OK = 0
STATUS_NAMES = {0: "VSA_OK", 1: "VSA_ERR_INVALID_ARG", 2: "VSA_ERR_UNSUPPORTED", 3: "VSA_ERR_CUDA",
                4: "VSA_ERR_DEVICE_TIMEOUT", 5: "VSA_ERR_BAD_INDEX", 6: "VSA_ERR_NO_MEMORY"}
SCORE_MODES = {"meanpool_gate": 0, "tripool": 1}

# every entry point declared in include/vsa.h
EXPORTS = ("vsa_plan_create", "vsa_plan_destroy", "vsa_plan_query", "vsa_plan_get_stats", "vsa_k_from_sparsity",
           "vsa_tile_pack", "vsa_tile_score", "vsa_topk_select", "vsa_sparse_attn", "vsa_tile_unpack",
           "vsa_layer_forward", "vsa_plan_check", "vsa_status_string", "vsa_tile_score_static",
           "vsa_tile_pack_pool", "vsa_tile_score_pooled", "vsa_teacher_tiles", "vsa_index_overlap",
           "vsa_ref_score", "vsa_topk_select_ref", "vsa_sparse_attn_ref", "vsa_tile_pack_pool_fp8",
           "vsa_sparse_attn_fp8", "vsa_plan_set_wait_limit", "vsa_plan_set_test_hold", "vsa_tile_pool",
           "vsa_sparse_attn_direct", "vsa_qk_norm_rope", "vsa_tile_norm_rope_pack_pool", "vsa_pooled_descriptors",
           "vsa_norm_bwd_workspace", "vsa_qk_norm_rope_bwd", "vsa_tile_norm_rope_bwd",
           "vsa_attn_bwd_workspace", "vsa_sparse_attn_bwd", "vsa_sparse_attn_ref_bwd",
           "vsa_linear_bwd_workspace", "vsa_linear", "vsa_linear_bwd")
ROPE_LAYOUTS = {"interleaved": 0, "halves": 1}
ACTIVATIONS = {"none": 0, "gelu_tanh": 1, "silu": 2}


class VsaDesc(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("W", ctypes.c_int32),
        ("n_segments", ctypes.c_int32), ("seg_len", ctypes.c_int32 * MAX_SEGMENTS),
        ("tile_shape", (ctypes.c_int32 * 3) * MAX_HEADS),
        ("k_per_head", ctypes.c_int32 * MAX_HEADS),
        ("score_mode", ctypes.c_int32), ("proj_dim", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
        ("seg_ref", ctypes.c_int32 * MAX_SEGMENTS), ("k_ref_per_head", ctypes.c_int32 * MAX_HEADS),
    ]


class VsaPlanInfo(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int64), ("n_prefix_tiles", ctypes.c_int32), ("nt_max", ctypes.c_int32),
        ("ntv_max", ctypes.c_int32), ("ntv", ctypes.c_int32 * MAX_HEADS), ("k_max", ctypes.c_int32),
        ("packed_elems", ctypes.c_int64), ("score_elems", ctypes.c_int64), ("index_elems", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_int64), ("lse_elems", ctypes.c_int64), ("attn_work_items", ctypes.c_int64),
        ("n_ref_tiles", ctypes.c_int32), ("k_ref_max", ctypes.c_int32),
        ("ref_score_elems", ctypes.c_int64), ("ref_index_elems", ctypes.c_int64),
        ("tile_scale_elems", ctypes.c_int64), ("direct_attn", ctypes.c_int32), ("reserved0", ctypes.c_int32),
    ]


class VsaPlanStats(ctypes.Structure):
    _fields_ = [
        ("calls_pack", ctypes.c_int64), ("calls_score", ctypes.c_int64), ("calls_select", ctypes.c_int64),
        ("calls_attn", ctypes.c_int64), ("calls_unpack", ctypes.c_int64), ("errors", ctypes.c_int64),
        ("computed_pairs", ctypes.c_int64), ("dense_pairs", ctypes.c_int64),
    ]


class VsaStrides(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("token", ctypes.c_int64)]


class VsaNormRope(ctypes.Structure):
    _fields_ = [
        ("w_q", ctypes.c_void_p), ("w_k", ctypes.c_void_p),
        ("cos_table", ctypes.c_void_p), ("sin_table", ctypes.c_void_p),
        ("per_head", ctypes.c_int32), ("layout", ctypes.c_int32), ("eps", ctypes.c_float),
    ]


class VsaLinearArgs(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("n_in", ctypes.c_int32), ("n_out", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("ld_x", ctypes.c_int64), ("w", ctypes.c_void_p), ("bias", ctypes.c_void_p),
        ("act", ctypes.c_int32), ("gate", ctypes.c_void_p), ("rows_per_gate", ctypes.c_int64),
        ("residual", ctypes.c_void_p), ("ld_residual", ctypes.c_int64), ("y", ctypes.c_void_p),
        ("ld_y", ctypes.c_int64), ("pre", ctypes.c_void_p), ("ld_pre", ctypes.c_int64),
    ]


class VsaLinearGradArgs(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("n_in", ctypes.c_int32), ("n_out", ctypes.c_int32),
        ("dy", ctypes.c_void_p), ("ld_dy", ctypes.c_int64), ("x", ctypes.c_void_p), ("ld_x", ctypes.c_int64),
        ("w", ctypes.c_void_p), ("act", ctypes.c_int32), ("pre", ctypes.c_void_p), ("ld_pre", ctypes.c_int64),
        ("gate", ctypes.c_void_p), ("rows_per_gate", ctypes.c_int64), ("dx", ctypes.c_void_p),
        ("ld_dx", ctypes.c_int64), ("dw", ctypes.c_void_p), ("dbias", ctypes.c_void_p), ("dgate", ctypes.c_void_p),
    ]


class VsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


_lib = None
_torch = _BF16 = _F32 = _I32T = _U8 = None      # torch and the dtypes the calls take, set when the library is loaded


def library() -> ctypes.CDLL:
    """The loaded libvsa (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libvsa.so not built ({LIB_PATH}); run python -m tile_sparse_video_pack_b200.build")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, D = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    sig = {
        "vsa_plan_create": (I32, [ctypes.POINTER(VsaDesc), ctypes.POINTER(P)]),
        "vsa_plan_destroy": (I32, [P]),
        "vsa_plan_query": (I32, [P, ctypes.POINTER(VsaPlanInfo)]),
        "vsa_plan_get_stats": (I32, [P, ctypes.POINTER(VsaPlanStats)]),
        "vsa_k_from_sparsity": (I32, [D, I32]),
        "vsa_tile_pack": (I32, [P, P, P, P, P, P, P, P]),
        "vsa_tile_score": (I32, [P, P, P, P, P, P, P, P]),
        "vsa_topk_select": (I32, [P, P, P, P, P]),
        "vsa_sparse_attn": (I32, [P, P, P, P, P, P, P, P, P]),
        "vsa_tile_unpack": (I32, [P, P, P, P]),
        "vsa_layer_forward": (I32, [P] + [P] * 15),
        "vsa_plan_check": (I32, [P]),
        "vsa_status_string": (ctypes.c_char_p, [I32]),
        "vsa_tile_score_static": (I32, [P, P, P, P, P, P, P]),
        "vsa_tile_pack_pool": (I32, [P] * 9),
        "vsa_tile_score_pooled": (I32, [P] * 6),
        "vsa_teacher_tiles": (I32, [P] * 6),
        "vsa_index_overlap": (I32, [P] * 6),
        "vsa_ref_score": (I32, [P] * 6),
        "vsa_topk_select_ref": (I32, [P] * 4),
        "vsa_sparse_attn_ref": (I32, [P] * 10),
        "vsa_tile_pack_pool_fp8": (I32, [P] * 13),
        "vsa_sparse_attn_fp8": (I32, [P] * 11),
        "vsa_plan_set_wait_limit": (I32, [P, ctypes.c_uint64]),
        "vsa_plan_set_test_hold": (I32, [P, I32]),
        "vsa_tile_pool": (I32, [P] * 5),
        "vsa_sparse_attn_direct": (I32, [P] * 9),
        "vsa_qk_norm_rope": (I32, [P] * 8),
        "vsa_tile_norm_rope_pack_pool": (I32, [P] * 11),
        "vsa_pooled_descriptors": (I32, [P] * 4),
        "vsa_norm_bwd_workspace": (I32, [P, ctypes.POINTER(I64)]),
        "vsa_qk_norm_rope_bwd": (I32, [P] * 13),
        "vsa_tile_norm_rope_bwd": (I32, [P] * 15),
        "vsa_attn_bwd_workspace": (I32, [P, ctypes.POINTER(I64)]),
        "vsa_sparse_attn_bwd": (I32, [P] * 14),
        "vsa_sparse_attn_ref_bwd": (I32, [P] * 15),
        "vsa_linear_bwd_workspace": (I32, [P, I64, I32, I32, I64, ctypes.POINTER(I64)]),
        "vsa_linear": (I32, [P, ctypes.POINTER(VsaLinearArgs), P]),
        "vsa_linear_bwd": (I32, [P, ctypes.POINTER(VsaLinearGradArgs), P, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    import torch
    global _torch, _BF16, _F32, _I32T, _U8
    _torch, _BF16, _F32, _I32T, _U8 = torch, torch.bfloat16, torch.float32, torch.int32, torch.uint8
    _lib = lib
    return lib


def k_from_sparsity(sparsity: float, n_tiles: int) -> int:
    return int(library().vsa_k_from_sparsity(float(sparsity), int(n_tiles)))


def _check(status: int, where: str):
    if status != VSA_OK:
        raise VsaError(status, where)


def make_desc(batch, heads, head_dim, T, H, W, segments, tile_shapes, k_per_head, score_mode="meanpool_gate",
              proj_dim=None, softmax_scale=0.0, seg_ref=(), k_ref_per_head=()) -> VsaDesc:
    d = VsaDesc()
    d.batch, d.heads, d.head_dim = batch, heads, head_dim
    d.T, d.H, d.W = T, H, W
    if len(segments) > MAX_SEGMENTS or heads > MAX_HEADS or len(tile_shapes) != heads or len(k_per_head) != heads:
        raise ValueError("descriptor does not fit vsa_desc")
    d.n_segments = len(segments)
    for i, s in enumerate(segments):
        d.seg_len[i] = s
    for h, shp in enumerate(tile_shapes):
        for a in range(3):
            d.tile_shape[h][a] = shp[a]
    for h, k in enumerate(k_per_head):
        d.k_per_head[h] = k
    d.score_mode = SCORE_MODES[score_mode] if isinstance(score_mode, str) else int(score_mode)
    d.proj_dim = head_dim if proj_dim is None else proj_dim
    d.softmax_scale = softmax_scale
    for i, f in enumerate(seg_ref):
        d.seg_ref[i] = int(f)
    for h, k in enumerate(k_ref_per_head):
        d.k_ref_per_head[h] = k
    return d


def _ptr(t, dtype, name, min_numel=0):
    """Device pointer of a contiguous CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        # the library launches on the current device, which must also be the plan's
        raise ValueError(f"{name} is on {t.device}, but cuda:{torch.cuda.current_device()} is the current device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < min_numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {min_numel}")
    return ctypes.c_void_p(t.data_ptr())


# The helpers below serve the calls around the layer, whose smallest sizes run in a few
# microseconds on the GPU: they check in one pass, pass addresses as plain integers and
# build the error message only once something is wrong.

def _addr(t, dtype, name, dev, min_numel=0):
    """Address of a contiguous tensor on device `dev`, the current one (None -> NULL)."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.numel() >= min_numel:
            return t.data_ptr()
    except AttributeError:
        pass
    return _ptr(t, dtype, name, min_numel).value     # raises what is wrong


def _strided_addr(t, dtype, name, dev):
    """Address of a tensor of any strides on device `dev`, the current one."""
    if not isinstance(t, _torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, but cuda:{dev} is the current device")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _matrix(t, cols, name, dev, rows=None):
    """(address, row stride, rows) of a bf16 [..., cols] tensor whose leading dimensions form one row axis."""
    try:
        ok = t.dtype is _BF16 and t.get_device() == dev
    except AttributeError:
        ok = False
    p = t.data_ptr() if ok else _strided_addr(t, _BF16, name, dev)
    shape = t.shape
    if not shape or shape[-1] != cols:
        raise ValueError(f"{name} must be [..., {cols}], got {tuple(shape)}")
    if len(shape) == 2:
        n, (ld, unit) = shape[0], t.stride()
    elif t.is_contiguous():
        n, ld, unit = t.numel() // cols, cols, 1
    else:
        try:
            m = t.view(-1, cols)
        except RuntimeError:
            raise ValueError(f"{name}'s leading dimensions {tuple(shape)} are not one row axis "
                             f"(strides {t.stride()})") from None
        n, (ld, unit) = m.shape[0], m.stride()
    if unit != 1 and n > 0 and cols > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    if rows is not None and n != rows:
        raise ValueError(f"{name} has {n} rows, needs {rows}")
    return p, (ld if n > 1 else cols), n


class NormRope:
    """RMS norm weights and rotation table of :meth:`Plan.qk_norm_rope` and its kin.

    ``w_q``, ``w_k``: fp32 ``[head_dim]`` or, one row per head, ``[heads, head_dim]`` (None: ones; both the
    same shape). ``cos``, ``sin``: fp32 ``[n_tokens, head_dim / 2]``, one angle per token and channel pair
    (both None: no rotation). ``layout``: "interleaved" turns channels (2i, 2i + 1) together, "halves"
    channels (i, i + head_dim / 2). :func:`axial_rope_table` makes a table for a (T, H, W) grid.
    """

    def __init__(self, w_q=None, w_k=None, cos=None, sin=None, layout="interleaved", eps=1e-6):
        if layout not in ROPE_LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}, got {layout!r}")
        if (cos is None) != (sin is None):
            raise ValueError("cos and sin come together")
        if w_q is not None and w_k is not None and w_q.shape != w_k.shape:
            raise ValueError(f"w_q {tuple(w_q.shape)} and w_k {tuple(w_k.shape)} differ in shape")
        self.w_q, self.w_k, self.cos, self.sin = w_q, w_k, cos, sin
        self.layout, self.eps = layout, float(eps)

        self._made = (None, None)      # the last struct, and the values it was made of

    @property
    def per_head(self):
        w = self.w_q if self.w_q is not None else self.w_k
        return w is not None and w.dim() == 2

    def _struct(self, plan, dev):
        per_head = self.per_head
        _, n, heads, d = plan._tokens
        want_w, want_t = ((heads, d) if per_head else (d,)), (n, d // 2)
        at = []
        for t, name, want in ((self.w_q, "w_q", want_w), (self.w_k, "w_k", want_w), (self.cos, "cos", want_t),
                              (self.sin, "sin", want_t)):
            if t is not None and t.shape != want:
                raise ValueError(f"{name} must be {want}, got {tuple(t.shape)}")
            at.append(_addr(t, _F32, name, dev))
        key = (*at, per_head, self.layout, self.eps)
        made = self._made
        if made[0] != key:
            made = (key, VsaNormRope(*at, int(per_head), ROPE_LAYOUTS[self.layout], self.eps))
            self._made = made
        return ctypes.byref(made[1])


def _karray(k_per_head, heads):
    """A host int32 array of the per-call k of each head (None -> NULL: the plan's own k)."""
    if k_per_head is None:
        return None
    ks = [int(x) for x in k_per_head]
    if len(ks) != heads:
        raise ValueError(f"k_per_head has {len(ks)} entries, the plan {heads} heads")
    return (ctypes.c_int32 * heads)(*ks)


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _here(stream):
    """(current device, raw stream) of a call."""
    c = _torch._C
    dev = c._cuda_getDevice()
    return dev, c._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


class Plan:
    """A vsa_plan: one layer's tiling tables and attention work list on the current device."""

    def __init__(self, desc: VsaDesc):
        lib = library()
        self.desc = desc
        h = ctypes.c_void_p()
        _check(lib.vsa_plan_create(ctypes.byref(desc), ctypes.byref(h)), "vsa_plan_create")
        self._h = h
        inf = VsaPlanInfo()
        _check(lib.vsa_plan_query(h, ctypes.byref(inf)), "vsa_plan_query")
        self.info = inf
        # what the calls around the layer check against, as plain numbers
        self._lib = lib
        self._tokens = (desc.batch, inf.n_tokens, desc.heads, desc.head_dim)
        self._pe, self._ws_bytes, self._lse, self._idx = (inf.packed_elems, inf.workspace_bytes, inf.lse_elems,
                                                          inf.index_elems)
        self._bytes = {}               # workspace sizes of this plan, by call and sizes

    @classmethod
    def from_config(cls, cfg, sparsity: float, k_per_head=None):
        """Plan for a :class:`vsa_synth.configs.LayerConfig` at one sparsity level."""
        ks = k_per_head
        if ks is None:
            ks = []
            for (pt, ph, pw) in cfg.tile_shapes:
                n = -(-cfg.T // pt) * -(-cfg.H // ph) * -(-cfg.W // pw)
                ks.append(k_from_sparsity(sparsity, n))
        seg_ref = tuple(getattr(cfg, "seg_ref", ()))
        k_ref = [int(cfg.k_ref)] * cfg.heads if any(seg_ref) else []
        return cls(make_desc(cfg.batch, cfg.heads, cfg.head_dim, cfg.T, cfg.H, cfg.W, cfg.segments,
                             cfg.tile_shapes, ks, cfg.score_mode, cfg.proj_dim, seg_ref=seg_ref,
                             k_ref_per_head=k_ref))

    def close(self):
        if getattr(self, "_h", None):
            library().vsa_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---- shapes ----------------------------------------------------------------
    @property
    def k_per_head(self):
        return [self.desc.k_per_head[h] for h in range(self.desc.heads)]

    def shapes(self):
        d, i = self.desc, self.info
        return {
            "tokens": (d.batch, i.n_tokens, d.heads, d.head_dim),
            "packed": (d.batch, d.heads, i.nt_max, TILE, d.head_dim),
            "scores": (d.batch, d.heads, i.ntv_max, i.ntv_max),
            "idx": (d.batch, d.heads, i.ntv_max, i.k_max),
            "lse": (d.batch, d.heads, i.nt_max, TILE),
            "workspace": (i.workspace_bytes,),
            "scores_ref": (d.batch, d.heads, i.ntv_max, i.n_ref_tiles),
            "idx_ref": (d.batch, d.heads, i.ntv_max, i.k_ref_max),
        }

    def allocate(self, device=None, with_lse=False, packed=True):
        """Device buffers for every intermediate of the layer (torch is only the allocator).

        packed=False leaves out the packed tiles (qp, kp, vp, op: None), which a plan with
        info.direct_attn does not need. Where heads differ in their number of tiles, the calls leave the
        entries past a head's own unwritten: they are zero here."""
        import torch
        dev = torch.device("cuda") if device is None else torch.device(device)
        s = self.shapes()
        ragged = any(self.info.ntv[h] != self.info.ntv_max for h in range(self.desc.heads))

        def new(name, dtype, written=False):
            return (torch.zeros if ragged and not written else torch.empty)(s[name], dtype=dtype, device=dev)

        bufs = {x: new("packed", torch.bfloat16, x != "op") if packed else None for x in ("qp", "kp", "vp", "op")}
        bufs.update({
            "scores": new("scores", torch.float32),
            "idx": new("idx", torch.int32),
            "workspace": new("workspace", torch.uint8, True),
            "lse": new("lse", torch.float32) if with_lse else None,
        })
        if self.info.n_ref_tiles:
            bufs["scores_ref"] = new("scores_ref", torch.float32)
            bufs["idx_ref"] = new("idx_ref", torch.int32)
        return bufs

    # ---- the five calls (same names as the C ABI) ------------------------------
    def tile_pack(self, q, k, v, qp, kp, vp, stream=None):
        import torch
        n_tok = self.desc.batch * self.info.n_tokens * self.desc.heads * self.desc.head_dim
        bf = torch.bfloat16
        args = [_ptr(x, bf, nm, n_tok) for x, nm in ((q, "q"), (k, "k"), (v, "v"))]
        outs = [_ptr(x, bf, nm, self.info.packed_elems) if src is not None else None
                for x, nm, src in ((qp, "qp", q), (kp, "kp", k), (vp, "vp", v))]
        _check(library().vsa_tile_pack(self._h, *args, *outs, _stream(stream)), "vsa_tile_pack")

    def tile_score(self, qp, kp, proj_q, proj_k, scores, workspace, stream=None):
        import torch
        pe = self.info.packed_elems
        _check(library().vsa_tile_score(
            self._h, _ptr(qp, torch.bfloat16, "qp", pe), _ptr(kp, torch.bfloat16, "kp", pe),
            _ptr(proj_q, torch.float32, "proj_q"), _ptr(proj_k, torch.float32, "proj_k"),
            _ptr(scores, torch.float32, "scores", self.info.score_elems),
            _ptr(workspace, torch.uint8, "workspace", self.info.workspace_bytes), _stream(stream)),
            "vsa_tile_score")

    def tile_pool(self, q, k, workspace, stream=None):
        """Pooling of the score stage straight from token-major q, k (plans with info.direct_attn)."""
        import torch
        n_tok = self.desc.batch * self.info.n_tokens * self.desc.heads * self.desc.head_dim
        bf = torch.bfloat16
        _check(library().vsa_tile_pool(
            self._h, _ptr(q, bf, "q", n_tok), _ptr(k, bf, "k", n_tok),
            _ptr(workspace, torch.uint8, "workspace", self.info.workspace_bytes), _stream(stream)),
            "vsa_tile_pool")

    def sparse_attn_direct(self, q, k, v, idx, o, lse=None, stream=None, k_per_head=None):
        """Attention from token-major q, k, v into token-major o (plans with info.direct_attn)."""
        import torch
        n_tok = self.desc.batch * self.info.n_tokens * self.desc.heads * self.desc.head_dim
        bf = torch.bfloat16
        _check(library().vsa_sparse_attn_direct(
            self._h, _ptr(q, bf, "q", n_tok), _ptr(k, bf, "k", n_tok), _ptr(v, bf, "v", n_tok),
            _ptr(idx, torch.int32, "idx", self.info.index_elems), _karray(k_per_head, self.desc.heads),
            _ptr(o, bf, "o", n_tok), _ptr(lse, torch.float32, "lse", self.info.lse_elems), _stream(stream)),
            "vsa_sparse_attn_direct")

    def tile_pack_pool(self, q, k, v, qp, kp, vp, workspace, stream=None):
        """tile_pack fused with the pooling of tile_score; follow with tile_score_pooled."""
        import torch
        n_tok = self.desc.batch * self.info.n_tokens * self.desc.heads * self.desc.head_dim
        pe, bf = self.info.packed_elems, torch.bfloat16
        _check(library().vsa_tile_pack_pool(
            self._h, _ptr(q, bf, "q", n_tok), _ptr(k, bf, "k", n_tok), _ptr(v, bf, "v", n_tok),
            _ptr(qp, bf, "qp", pe), _ptr(kp, bf, "kp", pe), _ptr(vp, bf, "vp", pe),
            _ptr(workspace, torch.uint8, "workspace", self.info.workspace_bytes), _stream(stream)),
            "vsa_tile_pack_pool")

    def tile_pack_pool_fp8(self, q, k, v, qp, kp, vp, qp8, kp8, q_scale, k_scale, workspace, stream=None):
        """tile_pack_pool plus e4m3 copies of Q and K with one fp32 scale per tile (head_dim 128)."""
        import torch
        n_tok = self.desc.batch * self.info.n_tokens * self.desc.heads * self.desc.head_dim
        pe, bf, u8, f32 = self.info.packed_elems, torch.bfloat16, torch.uint8, torch.float32
        ns = self.info.tile_scale_elems
        _check(library().vsa_tile_pack_pool_fp8(
            self._h, _ptr(q, bf, "q", n_tok), _ptr(k, bf, "k", n_tok), _ptr(v, bf, "v", n_tok),
            _ptr(qp, bf, "qp", pe), _ptr(kp, bf, "kp", pe), _ptr(vp, bf, "vp", pe),
            _ptr(qp8, u8, "qp8", pe), _ptr(kp8, u8, "kp8", pe), _ptr(q_scale, f32, "q_scale", ns),
            _ptr(k_scale, f32, "k_scale", ns),
            _ptr(workspace, u8, "workspace", self.info.workspace_bytes), _stream(stream)), "vsa_tile_pack_pool_fp8")

    def sparse_attn_fp8(self, qp8, kp8, q_scale, k_scale, vp, idx, op, lse=None, stream=None, k_per_head=None):
        """sparse_attn with Q K^T from the e4m3 tiles and their per-tile scales."""
        import torch
        pe, u8, f32, bf = self.info.packed_elems, torch.uint8, torch.float32, torch.bfloat16
        ns = self.info.tile_scale_elems
        _check(library().vsa_sparse_attn_fp8(
            self._h, _ptr(qp8, u8, "qp8", pe), _ptr(kp8, u8, "kp8", pe), _ptr(q_scale, f32, "q_scale", ns),
            _ptr(k_scale, f32, "k_scale", ns), _ptr(vp, bf, "vp", pe),
            _ptr(idx, torch.int32, "idx", self.info.index_elems), _karray(k_per_head, self.desc.heads),
            _ptr(op, bf, "op", pe),
            _ptr(lse, f32, "lse", self.info.lse_elems), _stream(stream)), "vsa_sparse_attn_fp8")

    def allocate_fp8(self, device=None):
        """The e4m3 Q, K tiles and their per-tile scales."""
        import torch
        dev = torch.device("cuda") if device is None else torch.device(device)
        pe, ns = self.info.packed_elems, self.info.tile_scale_elems
        return {"qp8": torch.empty(pe, dtype=torch.uint8, device=dev),
                "kp8": torch.empty(pe, dtype=torch.uint8, device=dev),
                "q_scale": torch.empty(ns, dtype=torch.float32, device=dev),
                "k_scale": torch.empty(ns, dtype=torch.float32, device=dev)}

    def tile_score_pooled(self, proj_q, proj_k, scores, workspace, stream=None):
        """Projection and scores from the descriptors tile_pack_pool left in the workspace."""
        import torch
        _check(library().vsa_tile_score_pooled(
            self._h, _ptr(proj_q, torch.float32, "proj_q"), _ptr(proj_k, torch.float32, "proj_k"),
            _ptr(scores, torch.float32, "scores", self.info.score_elems),
            _ptr(workspace, torch.uint8, "workspace", self.info.workspace_bytes), _stream(stream)),
            "vsa_tile_score_pooled")

    def teacher_tiles(self, qp, kp, lse, teacher, stream=None):
        """Max-pooled full-attention weights per video tile pair; lse from a dense sparse_attn."""
        import torch
        pe = self.info.packed_elems
        _check(library().vsa_teacher_tiles(
            self._h, _ptr(qp, torch.bfloat16, "qp", pe), _ptr(kp, torch.bfloat16, "kp", pe),
            _ptr(lse, torch.float32, "lse", self.info.lse_elems),
            _ptr(teacher, torch.float32, "teacher", self.info.score_elems), _stream(stream)), "vsa_teacher_tiles")

    def index_overlap(self, idx_a, idx_b, counts, stream=None, k_per_head=None):
        """Shared indices per row of two ascending top-k tables."""
        import torch
        n = self.desc.batch * self.desc.heads * self.info.ntv_max
        _check(library().vsa_index_overlap(
            self._h, _ptr(idx_a, torch.int32, "idx_a", self.info.index_elems),
            _ptr(idx_b, torch.int32, "idx_b", self.info.index_elems), _karray(k_per_head, self.desc.heads),
            _ptr(counts, torch.int32, "counts", n), _stream(stream)), "vsa_index_overlap")

    def tile_score_static(self, qp, kp, proj_q, proj_k, scores, stream=None):
        """tile_score with the library's fixed 32 MiB device scratch instead of a workspace.

        For callers that may not allocate device memory while the layer runs.
        Its first call on a device looks up the scratch address: make it before
        any stream capture. Calls that overlap on the GPU share the scratch and race.
        """
        import torch
        pe = self.info.packed_elems
        _check(library().vsa_tile_score_static(
            self._h, _ptr(qp, torch.bfloat16, "qp", pe), _ptr(kp, torch.bfloat16, "kp", pe),
            _ptr(proj_q, torch.float32, "proj_q"), _ptr(proj_k, torch.float32, "proj_k"),
            _ptr(scores, torch.float32, "scores", self.info.score_elems), _stream(stream)),
            "vsa_tile_score_static")

    def topk_select(self, scores, idx, stream=None, k_per_head=None):
        """k_per_head: this call's kept tiles per head (None: the plan's)."""
        import torch
        _check(library().vsa_topk_select(
            self._h, _ptr(scores, torch.float32, "scores", self.info.score_elems),
            _karray(k_per_head, self.desc.heads),
            _ptr(idx, torch.int32, "idx", self.info.index_elems), _stream(stream)), "vsa_topk_select")

    def sparse_attn(self, qp, kp, vp, idx, op, lse=None, stream=None, k_per_head=None):
        """k_per_head: this call's kept tiles per head (None: the plan's); as given to topk_select."""
        import torch
        pe, bf = self.info.packed_elems, torch.bfloat16
        _check(library().vsa_sparse_attn(
            self._h, _ptr(qp, bf, "qp", pe), _ptr(kp, bf, "kp", pe), _ptr(vp, bf, "vp", pe),
            _ptr(idx, torch.int32, "idx", self.info.index_elems), _karray(k_per_head, self.desc.heads),
            _ptr(op, bf, "op", pe),
            _ptr(lse, torch.float32, "lse", self.info.lse_elems), _stream(stream)), "vsa_sparse_attn")

    def ref_score(self, kp, proj_k, scores_ref, workspace, stream=None):
        """Scores of the reference tiles (R2VA budgets); after tile_score(_pooled) on the same workspace."""
        import torch
        _check(library().vsa_ref_score(
            self._h, _ptr(kp, torch.bfloat16, "kp", self.info.packed_elems), _ptr(proj_k, torch.float32, "proj_k"),
            _ptr(scores_ref, torch.float32, "scores_ref", self.info.ref_score_elems),
            _ptr(workspace, torch.uint8, "workspace", self.info.workspace_bytes), _stream(stream)), "vsa_ref_score")

    def topk_select_ref(self, scores_ref, idx_ref, stream=None):
        import torch
        _check(library().vsa_topk_select_ref(
            self._h, _ptr(scores_ref, torch.float32, "scores_ref", self.info.ref_score_elems),
            _ptr(idx_ref, torch.int32, "idx_ref", self.info.ref_index_elems), _stream(stream)),
            "vsa_topk_select_ref")

    def sparse_attn_ref(self, qp, kp, vp, idx, idx_ref, op, lse=None, stream=None, k_per_head=None):
        import torch
        pe, bf = self.info.packed_elems, torch.bfloat16
        _check(library().vsa_sparse_attn_ref(
            self._h, _ptr(qp, bf, "qp", pe), _ptr(kp, bf, "kp", pe), _ptr(vp, bf, "vp", pe),
            _ptr(idx, torch.int32, "idx", self.info.index_elems),
            _ptr(idx_ref, torch.int32, "idx_ref", self.info.ref_index_elems), _karray(k_per_head, self.desc.heads),
            _ptr(op, bf, "op", pe),
            _ptr(lse, torch.float32, "lse", self.info.lse_elems), _stream(stream)), "vsa_sparse_attn_ref")

    def tile_unpack(self, op, o, stream=None):
        import torch
        n_tok = self.desc.batch * self.info.n_tokens * self.desc.heads * self.desc.head_dim
        _check(library().vsa_tile_unpack(
            self._h, _ptr(op, torch.bfloat16, "op", self.info.packed_elems),
            _ptr(o, torch.bfloat16, "o", n_tok), _stream(stream)), "vsa_tile_unpack")

    def layer_forward(self, q, k, v, proj_q, proj_k, bufs, o, stream=None):
        """The layer's calls in one C-ABI call (vsa_layer_forward; the direct path when info.direct_attn)."""
        import torch
        pe, bf = self.info.packed_elems, torch.bfloat16
        n_tok = self.desc.batch * self.info.n_tokens * self.desc.heads * self.desc.head_dim
        _check(library().vsa_layer_forward(
            self._h, _ptr(q, bf, "q", n_tok), _ptr(k, bf, "k", n_tok), _ptr(v, bf, "v", n_tok),
            _ptr(proj_q, torch.float32, "proj_q"), _ptr(proj_k, torch.float32, "proj_k"),
            _ptr(bufs.get("qp"), bf, "qp", pe), _ptr(bufs.get("kp"), bf, "kp", pe), _ptr(bufs.get("vp"), bf, "vp", pe),
            _ptr(bufs["scores"], torch.float32, "scores", self.info.score_elems),
            _ptr(bufs["idx"], torch.int32, "idx", self.info.index_elems), _ptr(bufs.get("op"), bf, "op", pe),
            _ptr(bufs.get("lse"), torch.float32, "lse", self.info.lse_elems),
            _ptr(bufs["workspace"], torch.uint8, "workspace", self.info.workspace_bytes),
            _ptr(o, bf, "o", n_tok), _stream(stream)), "vsa_layer_forward")

    # ---- norm + rotation, and its gradient ------------------------------------------
    def _token_views(self, dev, *views):
        """(addresses, strides) of bf16 [B, N, heads, head_dim] views with contiguous heads and channels; strides
        None when all are contiguous."""
        want = self._tokens
        B, n, heads, d = want
        ptrs, strides, plain = [], [], True
        for name, t in views:
            try:
                ok = t.dtype is _BF16 and t.get_device() == dev and t.shape == want
            except AttributeError:
                ok = False
            if not ok:
                _strided_addr(t, _BF16, name, dev)
                raise ValueError(f"{name} must be {want}, got {tuple(t.shape)}")
            ptrs.append(t.data_ptr())
            if t.is_contiguous():
                strides += (n * heads * d, heads * d)
                continue
            plain = False
            sb, st, sh, sd = t.stride()
            if sd != 1 or (heads > 1 and sh != d):
                raise ValueError(f"{name}'s heads and channels must be contiguous (strides {t.stride()})")
            token = st if n > 1 else heads * d
            strides += (sb if B > 1 else token * n, token)
        return ptrs, (None if plain else (ctypes.c_int64 * len(strides))(*strides))

    def _workspace(self, call):
        """Bytes of a call's workspace, which the plan fixes."""
        n = self._bytes.get(call)
        if n is None:
            out = ctypes.c_int64()
            _check(getattr(self._lib, call)(self._h, ctypes.byref(out)), call)
            n = self._bytes[call] = out.value
        return n

    def qk_norm_rope(self, q, k, norm, q_out, k_out, stream=None):
        """RMS norm of every head's q and k row and the rotation, token-major views to token-major views
        (an output may be its own input)."""
        dev, s = _here(stream)
        ptrs, st = self._token_views(dev, ("q", q), ("k", k), ("q_out", q_out), ("k_out", k_out))
        status = self._lib.vsa_qk_norm_rope(self._h, norm._struct(self, dev), *ptrs, st, s)
        if status:
            _check(status, "vsa_qk_norm_rope")

    def tile_norm_rope_pack_pool(self, q, k, v, norm, qp, kp, vp, workspace, stream=None):
        """qk_norm_rope and tile_pack_pool in one pass; follow with tile_score_pooled."""
        dev, s = _here(stream)
        ptrs, st = self._token_views(dev, ("q", q), ("k", k), ("v", v))
        pe, bf = self._pe, _BF16
        _check(self._lib.vsa_tile_norm_rope_pack_pool(
            self._h, norm._struct(self, dev), *ptrs, st, _addr(qp, bf, "qp", dev, pe), _addr(kp, bf, "kp", dev, pe),
            _addr(vp, bf, "vp", dev, pe), _addr(workspace, _U8, "workspace", dev, self._ws_bytes),
            s), "vsa_tile_norm_rope_pack_pool")

    def pooled(self, workspace):
        """The descriptors that a pooling call left in the workspace: fp32 views [B, heads, ntv_max, w] of Q and K."""
        import torch
        base = _ptr(workspace, torch.uint8, "workspace", self.info.workspace_bytes)
        pq, pk = ctypes.c_void_p(), ctypes.c_void_p()
        _check(library().vsa_pooled_descriptors(self._h, base, ctypes.byref(pq), ctypes.byref(pk)),
               "vsa_pooled_descriptors")
        d, i = self.desc, self.info
        w = d.head_dim * (3 if d.score_mode == SCORE_MODES["tripool"] else 1)
        shape = (d.batch, d.heads, i.ntv_max, w)
        n = d.batch * d.heads * i.ntv_max * w * 4
        flat = workspace.view(-1)
        return tuple(flat[p.value - base.value:p.value - base.value + n].view(torch.float32).view(shape)
                     for p in (pq, pk))

    def norm_bwd_workspace_bytes(self):
        return self._workspace("vsa_norm_bwd_workspace")

    def _dw(self, norm, dw_q, dw_k, dev):
        _, _, heads, d = self._tokens
        want = (heads, d) if norm.per_head else (d,)
        for t, name in ((dw_q, "dw_q"), (dw_k, "dw_k")):
            if t is not None and t.shape != want:
                raise ValueError(f"{name} must be {want}, got {tuple(t.shape)}")
        return _addr(dw_q, _F32, "dw_q", dev), _addr(dw_k, _F32, "dw_k", dev)

    def qk_norm_rope_bwd(self, dq_out, dk_out, q, k, norm, dq, dk, dw_q, dw_k, workspace, stream=None):
        """Gradient of qk_norm_rope: dq, dk and (unless None) the weights' dw_q, dw_k."""
        dev, s = _here(stream)
        ptrs, st = self._token_views(dev, ("dq_out", dq_out), ("dk_out", dk_out), ("q", q), ("k", k), ("dq", dq),
                                     ("dk", dk))
        _check(self._lib.vsa_qk_norm_rope_bwd(
            self._h, norm._struct(self, dev), *ptrs, st, *self._dw(norm, dw_q, dw_k, dev),
            _addr(workspace, _U8, "workspace", dev, self.norm_bwd_workspace_bytes()), s),
            "vsa_qk_norm_rope_bwd")

    def tile_norm_rope_bwd(self, dqp, dkp, dvp, q, k, norm, dq, dk, dv, dw_q, dw_k, workspace, stream=None):
        """Gradient of tile_norm_rope_pack_pool: packed gradients back to token-major dq, dk, dv and to the weights."""
        dev, s = _here(stream)
        pe, bf = self._pe, _BF16
        ptrs, st = self._token_views(dev, ("q", q), ("k", k), ("dq", dq), ("dk", dk), ("dv", dv))
        _check(self._lib.vsa_tile_norm_rope_bwd(
            self._h, norm._struct(self, dev), _addr(dqp, bf, "dqp", dev, pe), _addr(dkp, bf, "dkp", dev, pe),
            _addr(dvp, bf, "dvp", dev, pe), *ptrs, st, *self._dw(norm, dw_q, dw_k, dev),
            _addr(workspace, _U8, "workspace", dev, self.norm_bwd_workspace_bytes()), s),
            "vsa_tile_norm_rope_bwd")

    # ---- gradient of the sparse attention --------------------------------------------
    def attn_bwd_workspace_bytes(self):
        return self._workspace("vsa_attn_bwd_workspace")

    def _attn_bwd_args(self, dev, qp, kp, vp, op, lse, dop, idx):
        pe, bf = self._pe, _BF16
        return (_addr(qp, bf, "qp", dev, pe), _addr(kp, bf, "kp", dev, pe), _addr(vp, bf, "vp", dev, pe),
                _addr(op, bf, "op", dev, pe), _addr(lse, _F32, "lse", dev, self._lse),
                _addr(dop, bf, "dop", dev, pe), _addr(idx, _I32T, "idx", dev, self._idx))

    def _attn_bwd_outs(self, dev, dqp, dkp, dvp, workspace):
        pe, bf = self._pe, _BF16
        return (_addr(dqp, bf, "dqp", dev, pe), _addr(dkp, bf, "dkp", dev, pe), _addr(dvp, bf, "dvp", dev, pe),
                _addr(workspace, _U8, "workspace", dev, self.attn_bwd_workspace_bytes()))

    def sparse_attn_bwd(self, qp, kp, vp, op, lse, dop, idx, dqp, dkp, dvp, workspace, stream=None, k_per_head=None):
        """Gradient of sparse_attn on packed tiles: dqp, dkp, dvp from dop, the forward's inputs and its op, lse."""
        dev, s = _here(stream)
        _check(self._lib.vsa_sparse_attn_bwd(
            self._h, *self._attn_bwd_args(dev, qp, kp, vp, op, lse, dop, idx), _karray(k_per_head, self.desc.heads),
            *self._attn_bwd_outs(dev, dqp, dkp, dvp, workspace), s), "vsa_sparse_attn_bwd")

    def sparse_attn_ref_bwd(self, qp, kp, vp, op, lse, dop, idx, idx_ref, dqp, dkp, dvp, workspace, stream=None,
                            k_per_head=None):
        """Gradient of sparse_attn_ref (R2VA budgets)."""
        dev, s = _here(stream)
        _check(self._lib.vsa_sparse_attn_ref_bwd(
            self._h, *self._attn_bwd_args(dev, qp, kp, vp, op, lse, dop, idx),
            _addr(idx_ref, _I32T, "idx_ref", dev, self.info.ref_index_elems),
            _karray(k_per_head, self.desc.heads), *self._attn_bwd_outs(dev, dqp, dkp, dvp, workspace), s),
            "vsa_sparse_attn_ref_bwd")

    # ---- linear layer with epilogue, and its gradient ---------------------------------
    @staticmethod
    def _gate(gate, rows, n_out, dev):
        if gate is None:
            return None, 0
        if gate.dim() != 2 or gate.shape[1] != n_out or gate.shape[0] < 1 or rows % gate.shape[0]:
            raise ValueError(f"gate must be [samples, {n_out}] with samples dividing {rows} rows, "
                             f"got {tuple(gate.shape)}")
        return _addr(gate, _F32, "gate", dev), rows // gate.shape[0] or 1

    @staticmethod
    def _act(act):
        if act not in ACTIVATIONS:
            raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
        return ACTIVATIONS[act]

    def linear(self, x, w, y, bias=None, act="none", gate=None, residual=None, pre=None, stream=None):
        """y = residual + gate * act(x w^T + bias): x [..., n_in], w [n_out, n_in], y [..., n_out] bf16, bias [n_out]
        and gate [samples, n_out] fp32. pre, if given, receives x w^T + bias for :meth:`linear_bwd`."""
        dev, s = _here(stream)
        if w.dim() != 2:
            raise ValueError(f"w must be [n_out, n_in], got {tuple(w.shape)}")
        n_out, n_in = w.shape
        px, ld_x, rows = _matrix(x, n_in, "x", dev)
        py, ld_y, _ = _matrix(y, n_out, "y", dev, rows)
        pr, ld_r, _ = _matrix(residual, n_out, "residual", dev, rows) if residual is not None else (None, 0, 0)
        pp, ld_p, _ = _matrix(pre, n_out, "pre", dev, rows) if pre is not None else (None, 0, 0)
        if bias is not None and bias.shape != (n_out,):
            raise ValueError(f"bias must be [{n_out}], got {tuple(bias.shape)}")
        pg, per = self._gate(gate, rows, n_out, dev)
        a = VsaLinearArgs(rows, n_in, n_out, px, ld_x, _addr(w, _BF16, "w", dev),
                          _addr(bias, _F32, "bias", dev), self._act(act), pg, per, pr, ld_r, py, ld_y, pp, ld_p)
        status = self._lib.vsa_linear(self._h, a, s)
        if status:
            _check(status, "vsa_linear")

    def linear_bwd_workspace_bytes(self, rows, n_in, n_out, samples=0):
        """Workspace of :meth:`linear_bwd`; samples: rows of the gate, 0 without one."""
        key = (rows, n_in, n_out, samples)
        n = self._bytes.get(key)
        if n is None:
            if samples and rows % samples:
                raise ValueError(f"{rows} rows do not divide into {samples} samples")
            out = ctypes.c_int64()
            _check(self._lib.vsa_linear_bwd_workspace(self._h, int(rows), int(n_in), int(n_out),
                                                      rows // samples if samples else 0, ctypes.byref(out)),
                   "vsa_linear_bwd_workspace")
            if len(self._bytes) > 256:           # sizes that keep changing: do not keep them all
                self._bytes.clear()
            n = self._bytes[key] = out.value
        return n

    def linear_bwd(self, dy, x, w, dx=None, dw=None, act="none", pre=None, gate=None, dbias=None, dgate=None,
                   workspace=None, stream=None):
        """Gradient of :meth:`linear`: any of dx [..., n_in], dw [n_out, n_in] (bf16), dbias [n_out] and dgate
        [samples, n_out] (fp32); that of the residual is dy itself."""
        dev, s = _here(stream)
        if w.dim() != 2:
            raise ValueError(f"w must be [n_out, n_in], got {tuple(w.shape)}")
        n_out, n_in = w.shape
        pdy, ld_dy, rows = _matrix(dy, n_out, "dy", dev)
        px, ld_x, _ = _matrix(x, n_in, "x", dev, rows) if x is not None else (None, 0, 0)
        pdx, ld_dx, _ = _matrix(dx, n_in, "dx", dev, rows) if dx is not None else (None, 0, 0)
        pp, ld_p, _ = _matrix(pre, n_out, "pre", dev, rows) if pre is not None else (None, 0, 0)
        if (act != "none" or dgate is not None) and pre is None:
            raise ValueError("an activation's or a gate's gradient needs pre")
        if dw is not None and x is None:
            raise ValueError("dw needs x")
        pg, per = self._gate(gate, rows, n_out, dev)
        if dgate is not None and (gate is None or dgate.shape != gate.shape):
            raise ValueError("dgate comes with a gate of its shape")
        if dw is not None and dw.shape != w.shape:
            raise ValueError(f"dw must be {tuple(w.shape)}, got {tuple(dw.shape)}")
        if dbias is not None and dbias.shape != (n_out,):
            raise ValueError(f"dbias must be [{n_out}], got {tuple(dbias.shape)}")
        need = self.linear_bwd_workspace_bytes(rows, n_in, n_out, gate.shape[0] if gate is not None else 0)
        if need and workspace is None:
            raise ValueError(f"this size needs a workspace of {need} bytes")
        bf, f32 = _BF16, _F32
        a = VsaLinearGradArgs(rows, n_in, n_out, pdy, ld_dy, px, ld_x, _addr(w, bf, "w", dev), self._act(act), pp, ld_p,
                              pg, per, pdx, ld_dx, _addr(dw, bf, "dw", dev), _addr(dbias, f32, "dbias", dev),
                              _addr(dgate, f32, "dgate", dev))
        _check(self._lib.vsa_linear_bwd(self._h, a, _addr(workspace, _U8, "workspace", dev, need), s),
               "vsa_linear_bwd")
        if rows == 0 and dgate is not None:      # samples without rows: the library sees none
            with _torch.cuda.stream(stream):
                dgate.zero_()

    def set_wait_limit(self, limit_ns: int = 0):
        """Bound of every device-side wait of the plan's tcgen05 kernels (0: the two-second default)."""
        _check(library().vsa_plan_set_wait_limit(self._h, int(limit_ns)), "vsa_plan_set_wait_limit")

    def set_test_hold(self, on: bool):
        """Test hook: attention, its gradient and linear wait for a release nothing gives, until the wait limit."""
        _check(library().vsa_plan_set_test_hold(self._h, 1 if on else 0), "vsa_plan_set_test_hold")

    def check(self):
        """Synchronise and raise if a kernel latched a device-side error."""
        _check(library().vsa_plan_check(self._h), "vsa_plan_check")

    def stats(self) -> dict:
        st = VsaPlanStats()
        _check(library().vsa_plan_get_stats(self._h, ctypes.byref(st)), "vsa_plan_get_stats")
        return {name: getattr(st, name) for name, _ in VsaPlanStats._fields_}
