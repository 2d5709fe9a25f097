"""ctypes binding of libedit_attn.so (include/edit_attn.h).

Argument marshalling only: torch tensors are passed as device pointers, the
stream as the current torch stream handle. Every step of the layer runs in the
library's CUDA kernels; there is no fallback. Loading raises if the library
has not been built.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libedit_attn.so")

EDIT_F32, EDIT_BF16 = 0, 1
WEIGHT_NAMES = ("cf3_w", "cf3_b", "gn_gamma", "gn_beta", "cf1_w", "cf1_b", "q_w", "q_b", "k_w", "k_b",
                "v_w", "v_b", "kdw_w", "kdw_b", "vdw_w", "vdw_b")
TEXT_NAMES = ("tq_w", "tq_b", "tk_w", "tk_b", "tv_w", "tv_b")
EXPORTS = ("edit_attn_workspace_bytes", "edit_attn_forward", "mmedit_workspace_bytes", "mmedit_hybrid_forward",
           "edit_attn_read_status", "edit_status_string", "edit_attn_workspace_layout",
           "edit_attn_set_stage_events", "edit_attn_kernel_launches", "edit_linear_attention_noalloc",
           "edit_attn_variant_workspace_bytes", "edit_attn_variant_forward", "edit_attn_variant_workspace_layout",
           "edit_attn_set_wait_drill", "edit_attn_band_workspace_bytes", "edit_attn_band_record_bytes",
           "edit_attn_band_partials", "edit_attn_band_finish", "edit_dit_block_workspace_bytes",
           "edit_dit_block_forward", "edit_packed_attention_workspace_bytes", "edit_packed_attention_forward",
           "edit_delta_rule_workspace_bytes", "edit_delta_rule_forward", "edit_delta_rule_step",
           "edit_block_norm_forward", "edit_dit_block_normed_forward")
STAGE_EVENTS_EDIT, STAGE_EVENTS_MM = 9, 12
PROC = {"none": 0, "cf": 1, "sc": 2}
VARIANT_NAMES = ("kcf3_w", "kcf3_b", "kgn_gamma", "kgn_beta", "kcf1_w", "kcf1_b", "o_w", "o_b")


SIDE_EVENTS = 4
_SIDE_FIELDS = [("side_stream", ctypes.c_void_p), ("side_events", ctypes.c_void_p * SIDE_EVENTS)]


class EditAttnWeights(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("c_red", ctypes.c_int), ("gn_groups", ctypes.c_int),
                ("gn_eps", ctypes.c_float), ("leaky_slope", ctypes.c_float), ("attn_eps", ctypes.c_float)] + \
               [(n, ctypes.c_void_p) for n in WEIGHT_NAMES] + \
               [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)] + _SIDE_FIELDS


EDIT_ETA_RATIO, EDIT_ETA_EXACT = 0, 1


class MMEditWeights(ctypes.Structure):
    _fields_ = [("img", EditAttnWeights)] + [(n, ctypes.c_void_p) for n in TEXT_NAMES] + \
               [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)] + _SIDE_FIELDS + \
               [("eta_mode", ctypes.c_int)]


DIT_NAMES = ("o_w", "o_b", "sst", "cq_w", "cq_b", "ck_w", "ck_b", "cv_w", "cv_b", "co_w", "co_b",
             "fc1_w", "fc1_b", "fc2_w", "fc2_b")


class DitBlockWeights(ctypes.Structure):
    _fields_ = [("attn", EditAttnWeights)] + [(n, ctypes.c_void_p) for n in DIT_NAMES] + \
               [("hidden", ctypes.c_int), ("ln_eps", ctypes.c_float), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)] + _SIDE_FIELDS


DIT_NORM_WEIGHTS = ("pre_attn_w", "pre_ffn_w", "post_attn_w", "post_cross_w", "post_ffn_w")


class DitBlockNorms(ctypes.Structure):
    _fields_ = [("norm_pre", ctypes.c_int), ("norm_post", ctypes.c_int)] + \
               [(n, ctypes.c_void_p) for n in DIT_NORM_WEIGHTS]


class EditAttnVariant(ctypes.Structure):
    _fields_ = [("q_proc", ctypes.c_int), ("k_proc", ctypes.c_int), ("v_proc", ctypes.c_int)] + \
               [(n, ctypes.c_void_p) for n in VARIANT_NAMES]


class WsLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("status", "U", "G", "Q", "KVp", "K", "V", "gn_stats", "Sz", "KT",
                                              "VTx", "Mp", "Wop", "NP")]


class PackedAttentionArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "heads", "kv_heads", "d", "nseq", "causal", "max_k")] + \
               [("scale", ctypes.c_float)] + \
               [(n, ctypes.c_int64) for n in ("rows_q", "rows_k", "ldq", "ldk", "ldv", "ldo")] + \
               [(n, ctypes.c_void_p) for n in ("q_offsets", "k_offsets", "k_lens", "workspace")] + \
               [("workspace_bytes", ctypes.c_size_t)]


class DeltaRuleArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "qk_heads", "heads", "d_k", "d_v", "nseq", "qk_norm")] + \
               [("scale", ctypes.c_float), ("qk_eps", ctypes.c_float)] + \
               [(n, ctypes.c_int64) for n in ("rows", "ldq", "ldk", "ldv", "ldo", "ldg", "ldb")] + \
               [("offsets", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


NORM = {"none": 0, "layer": 1, "rms": 2}
GATE_ACT = {"linear": 0, "tanh": 1}
NORM_VECTORS = ("post_w", "post_b", "pre_w", "pre_b", "gate0", "scale0", "shift0", "gate", "scale", "shift")


class BlockNormArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "norm_post", "norm_pre", "gate_act", "C", "samples")] + \
               [("eps", ctypes.c_float), ("res_scale", ctypes.c_float)] + \
               [(n, ctypes.c_int64) for n in ("rows", "rows_per_sample", "ldx", "ldy", "ldr", "ldh", "ld_mod")] + \
               [("offsets", ctypes.c_void_p)] + [(n, ctypes.c_void_p) for n in NORM_VECTORS]


_lib = None


def lib():
    """Load the shared library (raises RuntimeError if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                           "(python -m linear_compressed_attention_b200.build)")
    L = ctypes.CDLL(LIB_PATH)
    i, p, sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    W, MW = ctypes.POINTER(EditAttnWeights), ctypes.POINTER(MMEditWeights)
    L.edit_attn_workspace_bytes.argtypes = [i, i, i, i, i, W]
    L.edit_attn_workspace_bytes.restype = sz
    L.edit_attn_forward.argtypes = [p, i, i, i, i, i, W, p, p]
    L.edit_attn_forward.restype = i
    L.mmedit_workspace_bytes.argtypes = [i, i, i, i, i, i, MW]
    L.mmedit_workspace_bytes.restype = sz
    L.mmedit_hybrid_forward.argtypes = [p, p, i, i, i, i, i, i, MW, p, p, p]
    L.mmedit_hybrid_forward.restype = i
    L.edit_attn_read_status.argtypes = [p, p, ctypes.POINTER(ctypes.c_int)]
    L.edit_attn_read_status.restype = i
    L.edit_status_string.argtypes = [i]
    L.edit_status_string.restype = ctypes.c_char_p
    L.edit_attn_workspace_layout.argtypes = [i, i, i, i, i, W, ctypes.POINTER(WsLayout)]
    L.edit_attn_workspace_layout.restype = i
    L.edit_attn_set_stage_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), i]
    L.edit_attn_set_stage_events.restype = i
    L.edit_attn_kernel_launches.argtypes = []
    L.edit_attn_kernel_launches.restype = ctypes.c_uint64
    L.edit_attn_set_wait_drill.argtypes = [i, ctypes.c_uint64]
    L.edit_attn_set_wait_drill.restype = i
    L.edit_linear_attention_noalloc.argtypes = [p, p, p, i, i, i, i, i, i, ctypes.c_float, p, p]
    L.edit_linear_attention_noalloc.restype = i
    DW = ctypes.POINTER(DitBlockWeights)
    L.edit_dit_block_workspace_bytes.argtypes = [i, i, i, i, i, i, DW]
    L.edit_dit_block_workspace_bytes.restype = sz
    L.edit_dit_block_forward.argtypes = [p, p, p, i, i, i, i, i, i, DW, p, p]
    L.edit_dit_block_forward.restype = i
    L.edit_dit_block_normed_forward.argtypes = [p, p, p, i, i, i, i, i, i, DW, ctypes.POINTER(DitBlockNorms), p, p]
    L.edit_dit_block_normed_forward.restype = i
    V = ctypes.POINTER(EditAttnVariant)
    L.edit_attn_variant_workspace_bytes.argtypes = [i, i, i, i, i, W, V]
    L.edit_attn_variant_workspace_bytes.restype = sz
    L.edit_attn_variant_forward.argtypes = [p, i, i, i, i, i, W, V, p, p]
    L.edit_attn_variant_forward.restype = i
    L.edit_attn_variant_workspace_layout.argtypes = [i, i, i, i, i, W, V, ctypes.POINTER(WsLayout)]
    L.edit_attn_variant_workspace_layout.restype = i
    PA, DR, BN = (ctypes.POINTER(t) for t in (PackedAttentionArgs, DeltaRuleArgs, BlockNormArgs))
    L.edit_packed_attention_workspace_bytes.argtypes = [PA]
    L.edit_packed_attention_workspace_bytes.restype = sz
    L.edit_packed_attention_forward.argtypes = [p, p, p, PA, p, p]
    L.edit_packed_attention_forward.restype = i
    L.edit_delta_rule_workspace_bytes.argtypes = [DR]
    L.edit_delta_rule_workspace_bytes.restype = sz
    L.edit_delta_rule_forward.argtypes = [p, p, p, p, p, DR, p, p, p, p]
    L.edit_delta_rule_forward.restype = i
    L.edit_delta_rule_step.argtypes = [p, p, p, p, p, DR, p, p, p]
    L.edit_delta_rule_step.restype = i
    L.edit_block_norm_forward.argtypes = [p, p, BN, p, p, p]
    L.edit_block_norm_forward.restype = i
    _lib = L
    return L


class EditError(RuntimeError):
    def __init__(self, code):
        self.code = code
        super().__init__(f"edit_attn error {code}: {status_string(code)}")


def status_string(code: int) -> str:
    return lib().edit_status_string(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream(torch.cuda.current_device())  # (half the host time of the default argument)
    return ctypes.c_void_p(stream.cuda_stream)


def make_weights_struct(w: dict, dtype_code: int, c_red: int, gn_groups: int, gn_eps: float, leaky_slope: float,
                        attn_eps: float, workspace=None) -> EditAttnWeights:
    """Fill the C struct from a dict of device tensors named as in the header."""
    s = EditAttnWeights()
    s.dtype = dtype_code
    s.c_red, s.gn_groups = int(c_red), int(gn_groups)
    s.gn_eps, s.leaky_slope, s.attn_eps = float(gn_eps), float(leaky_slope), float(attn_eps)
    for n in WEIGHT_NAMES:
        t = w.get(n)
        setattr(s, n, None if t is None else t.data_ptr())
    if workspace is not None:
        s.workspace = workspace.data_ptr()
        s.workspace_bytes = workspace.numel() * workspace.element_size()
    return s


def make_mm_struct(img: EditAttnWeights, w: dict, workspace=None) -> MMEditWeights:
    s = MMEditWeights()
    s.img = img
    for n in TEXT_NAMES:
        t = w.get(n)
        setattr(s, n, None if t is None else t.data_ptr())
    if workspace is not None:
        s.workspace = workspace.data_ptr()
        s.workspace_bytes = workspace.numel() * workspace.element_size()
    return s


# ----------------------------------------------------------- C-ABI mirrors
def edit_attn_workspace_bytes(B, H, W, C, heads, weights: EditAttnWeights) -> int:
    return int(lib().edit_attn_workspace_bytes(B, H, W, C, heads, ctypes.byref(weights)))


def edit_attn_forward(x, B, H, W, C, heads, weights: EditAttnWeights, out, stream=None) -> int:
    """x, out: device tensors [B, H*W, C]; returns the status code (0 = OK)."""
    return int(lib().edit_attn_forward(_ptr(x), B, H, W, C, heads, ctypes.byref(weights), _ptr(out),
                                       _stream(stream)))


def mmedit_workspace_bytes(B, H, W, N_T, C, heads, weights: MMEditWeights) -> int:
    return int(lib().mmedit_workspace_bytes(B, H, W, N_T, C, heads, ctypes.byref(weights)))


def mmedit_hybrid_forward(x_img, x_txt, B, H, W, N_T, C, heads, weights: MMEditWeights, out_img, out_txt,
                          stream=None) -> int:
    return int(lib().mmedit_hybrid_forward(_ptr(x_img), _ptr(x_txt), B, H, W, N_T, C, heads,
                                           ctypes.byref(weights), _ptr(out_img), _ptr(out_txt), _stream(stream)))


def edit_attn_read_status(workspace, stream=None) -> int:
    st = ctypes.c_int(0)
    rc = lib().edit_attn_read_status(_ptr(workspace), _stream(stream), ctypes.byref(st))
    if rc != 0:
        raise EditError(rc)
    return int(st.value)


def edit_attn_workspace_layout(B, H, W, C, heads, weights: EditAttnWeights) -> dict:
    lay = WsLayout()
    rc = lib().edit_attn_workspace_layout(B, H, W, C, heads, ctypes.byref(weights), ctypes.byref(lay))
    if rc != 0:
        raise EditError(rc)
    return {n: int(getattr(lay, n)) for n, _ in WsLayout._fields_}


_stage_keepalive = None


def edit_attn_set_stage_events(handles) -> int:
    """handles: list of raw cudaEvent_t values (ints), or None to clear."""
    global _stage_keepalive
    if handles is None:
        _stage_keepalive = None
        return int(lib().edit_attn_set_stage_events(None, 0))
    arr = (ctypes.c_void_p * len(handles))(*handles)
    _stage_keepalive = arr
    return int(lib().edit_attn_set_stage_events(arr, len(handles)))


def edit_attn_kernel_launches() -> int:
    return int(lib().edit_attn_kernel_launches())


def edit_attn_set_wait_drill(gn_extra_arrivals: int, limit_ns: int) -> int:
    return int(lib().edit_attn_set_wait_drill(int(gn_extra_arrivals), int(limit_ns)))


def set_side(struct, side) -> None:
    """Lend a side stream to a weights struct: `side` is (stream, [4 events])
    of torch.cuda objects, or None for none."""
    if side is None:
        struct.side_stream = None
        for i in range(SIDE_EVENTS):
            struct.side_events[i] = None
        return
    stream, events = side
    struct.side_stream = stream.cuda_stream
    for i, e in enumerate(events):
        struct.side_events[i] = e.cuda_event


def make_side(device=None):
    """A side stream and its events for the library's concurrent branches,
    owned by the caller (kept alive by the returned tuple)."""
    import torch
    stream = torch.cuda.Stream(device=device)
    events = [torch.cuda.Event(enable_timing=False) for _ in range(SIDE_EVENTS)]
    with torch.cuda.stream(stream):
        for e in events:
            e.record(stream)  # torch creates the event handle at its first record
    return stream, events


def make_variant_struct(q_proc="cf", k_proc="sc", v_proc="sc", w: dict | None = None) -> EditAttnVariant:
    """Processing names 'cf' / 'sc' / 'none'; `w` holds the key ConvFusion
    weights and/or the output Linear (o_w, o_b) as device tensors, or None."""
    v = EditAttnVariant()
    v.q_proc, v.k_proc, v.v_proc = PROC[q_proc], PROC[k_proc], PROC[v_proc]
    for n in VARIANT_NAMES:
        t = (w or {}).get(n)
        setattr(v, n, None if t is None else t.data_ptr())
    return v


def edit_attn_variant_workspace_bytes(B, H, W, C, heads, weights: EditAttnWeights, variant: EditAttnVariant) -> int:
    return int(lib().edit_attn_variant_workspace_bytes(B, H, W, C, heads, ctypes.byref(weights),
                                                       ctypes.byref(variant)))


def edit_attn_variant_forward(x, B, H, W, C, heads, weights: EditAttnWeights, variant: EditAttnVariant, out,
                              stream=None) -> int:
    return int(lib().edit_attn_variant_forward(_ptr(x), B, H, W, C, heads, ctypes.byref(weights),
                                               ctypes.byref(variant), _ptr(out), _stream(stream)))


def edit_attn_variant_workspace_layout(B, H, W, C, heads, weights: EditAttnWeights, variant) -> dict:
    lay = WsLayout()
    vp = None if variant is None else ctypes.byref(variant)
    rc = lib().edit_attn_variant_workspace_layout(B, H, W, C, heads, ctypes.byref(weights), vp, ctypes.byref(lay))
    if rc != 0:
        raise EditError(rc)
    return {n: int(getattr(lay, n)) for n, _ in WsLayout._fields_}


def edit_linear_attention_noalloc(q, k, v, B, N, M, C, heads, dtype_code, attn_eps, out, stream=None) -> int:
    """Linear attention step with the library's static scratch (no workspace);
    q, out [B, N, C], k, v [B, M, C] device tensors. Returns the status code."""
    return int(lib().edit_linear_attention_noalloc(_ptr(q), _ptr(k), _ptr(v), B, N, M, C, heads, dtype_code,
                                                   float(attn_eps), _ptr(out), _stream(stream)))


# ----------------------------------------------------------- convenience
class EditAttention:
    """One EDiT (or MM-EDiT) layer with weights and workspace on a CUDA device.

    ``arrays`` is the dict the synthetic-input generator returns (numpy
    float32, bf16-exact for bf16); tensors are copied to the device once.
    """

    def __init__(self, arrays: dict, B: int, H: int, W: int, C: int, heads: int, dtype: str = "bf16",
                 n_txt: int = 0, mm: bool | None = None, device="cuda", variant: tuple | None = None,
                 out_proj: bool = False, side: bool = True, eta: str = "ratio"):
        """``variant`` = (q_proc, k_proc, v_proc) names ('cf', 'sc', 'none') and/or
        ``out_proj`` select edit_attn_variant_forward; weights a variant does
        not read are not copied to the device (NULL in the structs). With
        ``side`` the layer lends the library a side stream and its events
        (created here, owned by this object) for the concurrent branches.
        ``eta`` ('ratio' | 'exact') picks MM-EDiT's mixing weights."""
        import torch
        self.torch = torch
        self.B, self.H, self.W, self.C, self.heads, self.n_txt = B, H, W, C, heads, int(n_txt or 0)
        self.mm = bool(self.n_txt) if mm is None else bool(mm)
        self.tdtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.code = EDIT_BF16 if dtype == "bf16" else EDIT_F32
        self.is_variant = variant is not None or out_proj
        q, k, v = variant or ("cf", "sc", "sc")
        names = WEIGHT_NAMES + (TEXT_NAMES if self.mm else ())
        if self.is_variant:
            skip = set()
            if q != "cf":
                skip |= {"cf3_w", "cf3_b", "gn_gamma", "gn_beta", "cf1_w", "cf1_b"}
            if k != "sc":
                skip |= {"kdw_w", "kdw_b", "vdw_w", "vdw_b"}
            names = tuple(n for n in names if n not in skip)
            names += (("kcf3_w", "kcf3_b", "kgn_gamma", "kgn_beta", "kcf1_w", "kcf1_b") if k == "cf" else ())
            names += (("o_w", "o_b") if out_proj else ())
        self.w = {n: torch.from_numpy(np.ascontiguousarray(arrays[n])).to(device=device, dtype=self.tdtype)
                  for n in names}
        self.consts = dict(c_red=arrays["c_red"], gn_groups=arrays["gn_groups"], gn_eps=arrays["gn_eps"],
                           leaky_slope=arrays["leaky_slope"], attn_eps=arrays["attn_eps"])
        s = make_weights_struct(self.w, self.code, **self.consts)
        self.variant = make_variant_struct(q, k, v, self.w) if self.is_variant else None
        if self.mm:
            m = make_mm_struct(s, self.w)
            nbytes = mmedit_workspace_bytes(B, H, W, self.n_txt, C, heads, m)
        elif self.is_variant:
            nbytes = edit_attn_variant_workspace_bytes(B, H, W, C, heads, s, self.variant)
        else:
            nbytes = edit_attn_workspace_bytes(B, H, W, C, heads, s)
        if nbytes == 0:
            raise ValueError("shape/dtype rejected by the workspace query")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.struct = make_weights_struct(self.w, self.code, workspace=self.workspace, **self.consts)
        self.mm_struct = make_mm_struct(self.struct, self.w, self.workspace) if self.mm else None
        if self.mm_struct is not None:
            self.mm_struct.eta_mode = {"ratio": EDIT_ETA_RATIO, "exact": EDIT_ETA_EXACT}[eta]
        self.side = make_side(device) if side and self.code == EDIT_BF16 else None
        self.set_side(self.side)
        self.layout = edit_attn_variant_workspace_layout(B, H, W, C, heads, self.struct, self.variant)

    def set_side(self, side) -> None:
        """Lend (stream, events) to the library, or None to run every kernel
        on the call's stream."""
        set_side(self.struct, side)
        if self.mm_struct is not None:
            set_side(self.mm_struct, side)

    def forward(self, x, out=None, stream=None):
        if out is None:
            out = self.torch.empty_like(x)
        if self.is_variant:
            rc = edit_attn_variant_forward(x, self.B, self.H, self.W, self.C, self.heads, self.struct, self.variant,
                                           out, stream)
        else:
            rc = edit_attn_forward(x, self.B, self.H, self.W, self.C, self.heads, self.struct, out, stream)
        if rc != 0:
            raise EditError(rc)
        return out

    def forward_mm(self, x_img, x_txt, out_img=None, out_txt=None, stream=None):
        if out_img is None:
            out_img = self.torch.empty_like(x_img)
        if out_txt is None and x_txt is not None:
            out_txt = self.torch.empty_like(x_txt)
        rc = mmedit_hybrid_forward(x_img, x_txt, self.B, self.H, self.W, self.n_txt, self.C, self.heads,
                                   self.mm_struct, out_img, out_txt, stream)
        if rc != 0:
            raise EditError(rc)
        return out_img, out_txt

    def status(self, stream=None) -> int:
        return edit_attn_read_status(self.workspace, stream)

    def intermediate(self, name: str, shape, dtype=None):
        """View of an intermediate kept in the workspace (valid after the call completes)."""
        torch = self.torch
        off = self.layout[name]
        dt = dtype or self.tdtype
        n = int(np.prod(shape))
        es = torch.empty((), dtype=dt).element_size()
        return self.workspace[off:off + n * es].view(dt).view(*shape)


# ----------------------------------------------------------- DiT block
def edit_dit_block_workspace_bytes(B, H, W, N_T, C, heads, weights: DitBlockWeights) -> int:
    return int(lib().edit_dit_block_workspace_bytes(B, H, W, N_T, C, heads, ctypes.byref(weights)))


def edit_dit_block_forward(x, y, t6, B, H, W, N_T, C, heads, weights: DitBlockWeights, out, stream=None) -> int:
    return int(lib().edit_dit_block_forward(_ptr(x), _ptr(y), _ptr(t6), B, H, W, N_T, C, heads,
                                            ctypes.byref(weights), _ptr(out), _stream(stream)))


def edit_dit_block_normed_forward(x, y, t6, B, H, W, N_T, C, heads, weights: DitBlockWeights, norms: DitBlockNorms,
                                  out, stream=None) -> int:
    return int(lib().edit_dit_block_normed_forward(_ptr(x), _ptr(y), _ptr(t6), B, H, W, N_T, C, heads,
                                                   ctypes.byref(weights), ctypes.byref(norms), _ptr(out),
                                                   _stream(stream)))


class DitBlock:
    """One DiT block (EDiT self-attention, cross-attention over the caption
    tokens, MLP) with weights and workspace on a CUDA device; ``arrays`` is
    the synthetic-input dict drawn with ``dit_block=...``. ``norms`` = (pre,
    post[, weights]) names other norms before and after the branches ('none',
    'layer', 'rms') and a dict of their optional weights (pre_attn_w,
    pre_ffn_w, post_attn_w, post_cross_w, post_ffn_w: [C] arrays)."""

    def __init__(self, arrays: dict, B: int, H: int, W: int, N_T: int, C: int, heads: int, dtype: str = "bf16",
                 device="cuda", side: bool = True, norms: tuple | None = None):
        for n, a in (norms[2] if norms is not None and len(norms) > 2 else {}).items():
            if n not in DIT_NORM_WEIGHTS or np.shape(a) != (C,):
                raise ValueError(f"norm weight {n}: one of {DIT_NORM_WEIGHTS} of shape ({C},) expected")
        import torch
        self.torch = torch
        self.B, self.H, self.W, self.N_T, self.C, self.heads = B, H, W, N_T, C, heads
        self.tdtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        code = EDIT_BF16 if dtype == "bf16" else EDIT_F32
        names = WEIGHT_NAMES + DIT_NAMES
        self.w = {n: torch.from_numpy(np.ascontiguousarray(arrays[n])).to(device=device, dtype=self.tdtype)
                  for n in names}
        consts = dict(c_red=arrays["c_red"], gn_groups=arrays["gn_groups"], gn_eps=arrays["gn_eps"],
                      leaky_slope=arrays["leaky_slope"], attn_eps=arrays["attn_eps"])
        s = DitBlockWeights()
        s.attn = make_weights_struct(self.w, code, **consts)
        for n in DIT_NAMES:
            setattr(s, n, self.w[n].data_ptr())
        s.hidden = int(arrays["fc1_w"].shape[0])
        s.ln_eps = float(arrays["ln_eps"])
        nbytes = edit_dit_block_workspace_bytes(B, H, W, N_T, C, heads, s)
        if nbytes == 0:
            raise ValueError("shape/dtype rejected by the DiT block workspace query")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        s.workspace = self.workspace.data_ptr()
        s.workspace_bytes = nbytes
        self.struct = s
        self.side = make_side(device) if side and code == EDIT_BF16 else None
        set_side(self.struct, self.side)
        self.norms = None
        if norms is not None:
            self.norms = DitBlockNorms()
            self.norms.norm_pre, self.norms.norm_post = NORM[norms[0]], NORM[norms[1]]
            for n, a in (norms[2] if len(norms) > 2 else {}).items():
                self.w[n] = torch.from_numpy(np.ascontiguousarray(a)).to(device=device, dtype=self.tdtype)
                setattr(self.norms, n, self.w[n].data_ptr())

    def forward(self, x, y, t6, out=None, stream=None):
        if out is None:
            out = self.torch.empty_like(x)
        if self.norms is not None:
            rc = edit_dit_block_normed_forward(x, y, t6, self.B, self.H, self.W, self.N_T, self.C, self.heads,
                                               self.struct, self.norms, out, stream)
        else:
            rc = edit_dit_block_forward(x, y, t6, self.B, self.H, self.W, self.N_T, self.C, self.heads, self.struct,
                                        out, stream)
        if rc != 0:
            raise EditError(rc)
        return out

    def status(self, stream=None) -> int:
        return edit_attn_read_status(self.workspace, stream)


# ----------------------------------------------------------- packed sequences
def _addr(t):
    """A tensor's address for an argument of type void* (an int, as cheap as it gets: these calls may be short)."""
    return None if t is None else t.data_ptr()


def _handle(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream(torch.cuda.current_device())
    return stream.cuda_stream


def edit_packed_attention_workspace_bytes(args: PackedAttentionArgs) -> int:
    return int(lib().edit_packed_attention_workspace_bytes(ctypes.byref(args)))


def edit_packed_attention_forward(q, k, v, args: PackedAttentionArgs, out, stream=None) -> int:
    return int(lib().edit_packed_attention_forward(_addr(q), _addr(k), _addr(v), ctypes.byref(args), _addr(out),
                                                   _handle(stream)))


def edit_delta_rule_workspace_bytes(args: DeltaRuleArgs) -> int:
    return int(lib().edit_delta_rule_workspace_bytes(ctypes.byref(args)))


def edit_delta_rule_forward(q, k, v, g, beta, args: DeltaRuleArgs, state_in, state_out, out, stream=None) -> int:
    return int(lib().edit_delta_rule_forward(_addr(q), _addr(k), _addr(v), _addr(g), _addr(beta), ctypes.byref(args),
                                             _addr(state_in), _addr(state_out), _addr(out), _handle(stream)))


def edit_delta_rule_step(q, k, v, g, beta, args: DeltaRuleArgs, state, out, stream=None) -> int:
    return int(lib().edit_delta_rule_step(_addr(q), _addr(k), _addr(v), _addr(g), _addr(beta), ctypes.byref(args),
                                          _addr(state), _addr(out), _handle(stream)))


def edit_block_norm_forward(x, y, args: BlockNormArgs, r_out, h_out, stream=None) -> int:
    return int(lib().edit_block_norm_forward(_addr(x), _addr(y), ctypes.byref(args), _addr(r_out), _addr(h_out),
                                             _handle(stream)))


def _check_rows(name, t, dtype, shape, device):
    """A device tensor of rows whose other dimensions are contiguous; returns its row stride."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name}: {dtype} {shape} expected, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is not on the current device")
    width = shape[1] * shape[2] if len(shape) == 3 else shape[1]
    if shape[0] == 0:
        return width
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1 or (len(st) == 3 and st[1] != shape[2] and shape[1] > 1):
        raise ValueError(f"{name}: only the rows may be strided")
    return st[0] if shape[0] > 1 else width


def _check_ints(name, t, n, device):
    import torch
    if t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name}: {n} contiguous int32 on the current device expected")
    return t.data_ptr()


class _Packed:
    def __init__(self, dtype):
        import torch
        self.torch = torch
        self.tdtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.code = EDIT_BF16 if dtype == "bf16" else EDIT_F32
        self.ran = False

    def _workspace(self, nbytes, device):
        if nbytes == 0:
            raise ValueError("shape/dtype rejected by the workspace query")
        self.workspace = self.torch.empty(nbytes, dtype=self.torch.uint8, device=device)
        self.args.workspace, self.args.workspace_bytes = self.workspace.data_ptr(), nbytes
        self.device = self.workspace.get_device()

    def _current_device(self):
        dev = self.torch.cuda.current_device()
        if dev != self.device:
            raise ValueError(f"the workspace is on device {self.device}, the current device is {dev}")
        return dev

    def status(self, stream=None) -> int:
        """The last forward call's device-side status (EDIT_ERR_SHAPE: offsets or lengths out of range); waits for it.
        0 before the first one, which sets the word."""
        return edit_attn_read_status(self.workspace, stream) if self.ran else 0


class PackedAttention(_Packed):
    """Softmax attention over packed sequences, with its workspace: up to
    ``max_rows`` query rows of ``nseq`` sequences with at most ``max_k`` keys
    each. Calls that may overlap on the GPU need objects of their own."""

    def __init__(self, heads: int, kv_heads: int, d: int, nseq: int, max_rows: int, max_k: int, dtype: str = "bf16",
                 causal: bool = False, scale: float | None = None, device="cuda"):
        super().__init__(dtype)
        a = self.args = PackedAttentionArgs()
        a.dtype, a.heads, a.kv_heads, a.d, a.nseq, a.causal, a.max_k = \
            self.code, heads, kv_heads, d, nseq, int(causal), max_k
        a.scale = d ** -0.5 if scale is None else scale
        a.rows_q = max_rows
        self._workspace(edit_packed_attention_workspace_bytes(a), device)

    def forward(self, q, k, v, q_offsets, k_offsets, k_lens=None, out=None, stream=None):
        """q [rows, heads, d], k, v [rows, kv_heads, d]; int32 device offsets [nseq + 1] and lengths [nseq]."""
        a, dev = self.args, self._current_device()
        rk = k.shape[0]
        a.rows_q, a.rows_k = q.shape[0], rk
        a.ldq = _check_rows("q", q, self.tdtype, (a.rows_q, a.heads, a.d), dev)
        a.ldk = _check_rows("k", k, self.tdtype, (rk, a.kv_heads, a.d), dev)
        a.ldv = _check_rows("v", v, self.tdtype, (rk, a.kv_heads, a.d), dev)
        if out is None:
            out = self.torch.empty(q.shape, dtype=q.dtype, device=q.device)
        a.ldo = _check_rows("out", out, self.tdtype, (a.rows_q, a.heads, a.d), dev)
        a.q_offsets = _check_ints("q_offsets", q_offsets, a.nseq + 1, dev)
        a.k_offsets = _check_ints("k_offsets", k_offsets, a.nseq + 1, dev)
        a.k_lens = None if k_lens is None else _check_ints("k_lens", k_lens, a.nseq, dev)
        rc = edit_packed_attention_forward(q, k, v, a, out, stream)
        if rc != 0:
            raise EditError(rc)
        self.ran = True
        return out


class DeltaRule(_Packed):
    """The gated delta rule for ``nseq`` sequences, with the workspace of calls
    of up to ``max_rows`` packed rows (``forward``) and the single-token form
    (``step``). Calls that may overlap on the GPU need objects of their own."""

    def __init__(self, qk_heads: int, heads: int, d_k: int, d_v: int, nseq: int, max_rows: int, dtype: str = "bf16",
                 scale: float | None = None, qk_norm: bool = True, qk_eps: float = 1e-6, device="cuda"):
        super().__init__(dtype)
        a = self.args = DeltaRuleArgs()
        a.dtype, a.qk_heads, a.heads, a.d_k, a.d_v, a.nseq, a.qk_norm = \
            self.code, qk_heads, heads, d_k, d_v, nseq, int(qk_norm)
        a.scale, a.qk_eps = d_k ** -0.5 if scale is None else scale, qk_eps
        a.rows = max_rows
        self.state_shape = (nseq, heads, d_k, d_v)
        self._workspace(edit_delta_rule_workspace_bytes(a), device)

    def _inputs(self, q, k, v, g, beta, out):
        a, dev, f32 = self.args, self._current_device(), self.torch.float32
        n = q.shape[0]
        a.ldq = _check_rows("q", q, self.tdtype, (n, a.qk_heads, a.d_k), dev)
        a.ldk = _check_rows("k", k, self.tdtype, (n, a.qk_heads, a.d_k), dev)
        a.ldv = _check_rows("v", v, self.tdtype, (n, a.heads, a.d_v), dev)
        a.ldg = _check_rows("g", g, f32, (n, a.heads), dev)
        a.ldb = _check_rows("beta", beta, f32, (n, a.heads), dev)
        if out is None:
            out = self.torch.empty(v.shape, dtype=v.dtype, device=v.device)
        a.ldo = _check_rows("out", out, self.tdtype, (n, a.heads, a.d_v), dev)
        return n, dev, out

    def _state(self, name, t, dev):
        if t is not None and (t.dtype != self.torch.float32 or t.shape != self.state_shape or
                              not t.is_contiguous() or t.get_device() != dev):
            raise ValueError(f"{name}: contiguous float32 {self.state_shape} on the current device expected")

    def forward(self, q, k, v, g, beta, offsets, state_in=None, state_out=None, out=None, stream=None):
        """q, k [rows, qk_heads, d_k], v [rows, heads, d_v], fp32 g, beta [rows, heads]; int32 device offsets
        [nseq + 1]. state_out (which may be state_in) takes the final states. Returns out."""
        n, dev, out = self._inputs(q, k, v, g, beta, out)
        a = self.args
        a.rows = n
        a.offsets = _check_ints("offsets", offsets, a.nseq + 1, dev)
        self._state("state_in", state_in, dev)
        self._state("state_out", state_out, dev)
        rc = edit_delta_rule_forward(q, k, v, g, beta, a, state_in, state_out, out, stream)
        if rc != 0:
            raise EditError(rc)
        self.ran = True
        return out

    def step(self, q, k, v, g, beta, state, out=None, stream=None):
        """One token of each sequence (row s: sequence s); state is updated in place. Returns out. Has no part in
        ``status``, which is the last ``forward``'s."""
        n, dev, out = self._inputs(q, k, v, g, beta, out)
        a = self.args
        if n != a.nseq:
            raise ValueError(f"{a.nseq} rows expected, one a sequence")
        self._state("state", state, dev)
        rc = edit_delta_rule_step(q, k, v, g, beta, a, state, out, stream)
        if rc != 0:
            raise EditError(rc)
        return out


class BlockNorm:
    """The step between two branches of a block: r = x + res_scale act(gate)
    N_post(y), h = N_pre(r) (1 + scale) + shift, with the weights and common
    vectors ([C] device tensors, or None) that a layer keeps."""

    def __init__(self, C: int, dtype: str = "bf16", post: str = "none", pre: str = "layer", gate_act: str = "linear",
                 eps: float = 1e-6, res_scale: float = 1.0, post_w=None, post_b=None, pre_w=None, pre_b=None,
                 gate0=None, scale0=None, shift0=None):
        import torch
        self.torch = torch
        self.tdtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        a = self.args = BlockNormArgs()
        a.dtype = EDIT_BF16 if dtype == "bf16" else EDIT_F32
        a.norm_post, a.norm_pre, a.gate_act, a.C = NORM[post], NORM[pre], GATE_ACT[gate_act], C
        a.eps, a.res_scale = eps, res_scale
        self.kept = dict(post_w=post_w, post_b=post_b, pre_w=pre_w, pre_b=pre_b, gate0=gate0, scale0=scale0,
                         shift0=shift0)
        for n, t in self.kept.items():
            if t is not None:
                if t.dtype != self.tdtype or tuple(t.shape) != (C,) or not t.is_contiguous() or not t.is_cuda:
                    raise ValueError(f"{n}: contiguous {self.tdtype} ({C},) on the device expected")
                setattr(a, n, t.data_ptr())
        self.devices = {t.get_device() for t in self.kept.values() if t is not None}  # of the kept vectors

    def forward(self, x, y=None, gate=None, scale=None, shift=None, offsets=None, r_out=None, h_out=None,
                want_r: bool = True, want_h: bool = True, stream=None):
        """x, y [rows, C]; gate, scale, shift [samples, C] with one row stride; int32 device offsets [samples + 1],
        or equal shares of the rows without them. Returns (r, h), None for one that is not wanted."""
        a, dev = self.args, self.torch.cuda.current_device()
        if self.devices and self.devices != {dev}:
            raise ValueError(f"the kept vectors are on devices {self.devices}, the current device is {dev}")
        n, C = x.shape[0], a.C
        a.rows = n
        a.ldx = _check_rows("x", x, self.tdtype, (n, C), dev)
        if y is not None:
            a.ldy = _check_rows("y", y, self.tdtype, (n, C), dev)
        samples, strides = None, set()
        for name, t in (("gate", gate), ("scale", scale), ("shift", shift)):
            if t is None:
                setattr(a, name, None)
                continue
            samples = t.shape[0] if samples is None else samples
            strides.add(_check_rows(name, t, self.tdtype, (samples, C), dev))
            setattr(a, name, t.data_ptr())
        if len(strides) > 1:
            raise ValueError("gate, scale and shift: one row stride expected")
        if strides:
            a.ld_mod = strides.pop()
        if offsets is not None:
            samples = offsets.numel() - 1 if samples is None else samples
            a.offsets = _check_ints("offsets", offsets, samples + 1, dev)
        else:
            a.offsets = None
            samples = samples or 1
            if samples < 1 or n % samples:
                raise ValueError("rows do not divide into the samples: give offsets")
            a.rows_per_sample = max(1, n // samples)
        a.samples = samples
        if r_out is None and want_r:
            r_out = self.torch.empty((n, C), dtype=x.dtype, device=x.device)
        if h_out is None and want_h:
            h_out = self.torch.empty((n, C), dtype=x.dtype, device=x.device)
        if r_out is not None:
            a.ldr = _check_rows("r_out", r_out, self.tdtype, (n, C), dev)
        if h_out is not None:
            a.ldh = _check_rows("h_out", h_out, self.tdtype, (n, C), dev)
        rc = edit_block_norm_forward(x, y, a, r_out, h_out, stream)
        if rc != 0:
            raise EditError(rc)
        return r_out, h_out
