"""Python binding of the LazyFlash C ABI (include/lazyflash.h).

Argument marshalling only: every step of the path runs in the CUDA kernels of
liblazyflash.so.  PyTorch provides device memory and streams.  There is no CPU
fallback: importing the binding without the built library raises.

Functions keep the C names: lf_attn_fwd, lf_block_select, lf_attn_bwd,
lf_workspace_size, lf_attn_fwd_mod, lf_attn_bwd_mod, lf_qk_norm_rope, lf_qk_norm_rope_bwd, lf_qk_workspace_size,
lf_sync_status (alias lf_check_device_error), lf_status_string.  Tensors are torch
CUDA tensors in the layouts the header states; the stream defaults to torch's
current stream.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblazyflash.so")

LF_OK, LF_ERR_INVALID_ARG, LF_ERR_UNSUPPORTED, LF_ERR_WORKSPACE, LF_ERR_CUDA, LF_ERR_TIMEOUT = range(6)
LF_WS_FWD, LF_WS_SELECT, LF_WS_BWD = 0, 1, 2
LF_SELECT_NORMS_GIVEN = 0x1
LF_RULE_BUDGET, LF_RULE_FIXED_FRACTION, LF_RULE_TOPK = 0, 1, 2

EXPORTED = ("lf_workspace_size", "lf_attn_fwd", "lf_block_select", "lf_attn_bwd",
            "lf_attn_fwd_mod", "lf_attn_bwd_mod", "lf_qk_norm_rope", "lf_qk_norm_rope_bwd", "lf_qk_workspace_size",
            "lf_sync_status", "lf_check_device_error", "lf_status_string")
LF_ROPE_HALVES, LF_ROPE_PAIRS = 0, 1
LF_QK_NORM, LF_QK_ZERO_TAIL = 0x1, 0x2


class LfError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__("%s: %s" % (what, lf_status_string(code)))
        self.code = code


class lf_attn_desc(ctypes.Structure):
    _fields_ = [
        ("nseq", ctypes.c_int32),
        ("cu_seqlens", ctypes.c_void_p),
        ("max_seqlen", ctypes.c_int32),
        ("total_tokens", ctypes.c_int32),
        ("hq", ctypes.c_int32),
        ("hkv", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float),
        ("causal", ctypes.c_int32),
        ("block_q", ctypes.c_int32),
    ]


class lf_score_mod(ctypes.Structure):
    _fields_ = [
        ("softcap", ctypes.c_float),
        ("alibi_slopes", ctypes.c_void_p),
        ("prefix_len", ctypes.c_void_p),
        ("prefix_causal", ctypes.c_int32),
        ("row_start", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
    ]


class lf_qk_desc(ctypes.Structure):
    _fields_ = [
        ("total_tokens", ctypes.c_int32),
        ("hq", ctypes.c_int32),
        ("hkv", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("nseq", ctypes.c_int32),
        ("cu_seqlens", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
        ("cos_sin", ctypes.c_void_p),
        ("npos", ctypes.c_int32),
        ("rot", ctypes.c_int32),
        ("pairing", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("eps", ctypes.c_float),
        ("q_weight", ctypes.c_void_p),
        ("k_weight", ctypes.c_void_p),
        ("weights_bf16", ctypes.c_int32),
    ]


_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError("liblazyflash.so is not built (run __graft_entry__.build()); "
                          "there is no fallback path")
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, i32, u32, u64, dbl = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint32,
                                  ctypes.c_uint64, ctypes.c_double)
    dptr = ctypes.POINTER(lf_attn_desc)
    L.lf_status_string.argtypes = [i32]
    L.lf_status_string.restype = ctypes.c_char_p
    L.lf_workspace_size.argtypes = [dptr, i32, ctypes.POINTER(sz)]
    L.lf_workspace_size.restype = i32
    L.lf_attn_fwd.argtypes = [dptr, vp, vp, vp, vp, vp, vp, sz, vp]
    L.lf_attn_fwd.restype = i32
    L.lf_block_select.argtypes = [dptr, vp, vp, dbl, u64, u64, u32, vp, vp, vp, vp, vp, vp, vp,
                                  vp, sz, vp]
    L.lf_block_select.restype = i32
    L.lf_attn_bwd.argtypes = [dptr, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.lf_attn_bwd.restype = i32
    L.lf_check_device_error.argtypes = [vp]
    L.lf_check_device_error.restype = i32
    L.lf_sync_status.argtypes = [vp]
    L.lf_sync_status.restype = i32
    mptr = ctypes.POINTER(lf_score_mod)
    L.lf_attn_fwd_mod.argtypes = [dptr, mptr] + [vp] * 7
    L.lf_attn_fwd_mod.restype = i32
    L.lf_attn_bwd_mod.argtypes = [dptr, mptr] + [vp] * 15 + [sz, vp]
    L.lf_attn_bwd_mod.restype = i32
    i64, qptr = ctypes.c_int64, ctypes.POINTER(lf_qk_desc)
    L.lf_qk_norm_rope.argtypes = [qptr] + [vp, i64] * 4 + [vp]
    L.lf_qk_norm_rope.restype = i32
    L.lf_qk_workspace_size.argtypes = [qptr, ctypes.POINTER(sz)]
    L.lf_qk_workspace_size.restype = i32
    L.lf_qk_norm_rope_bwd.argtypes = [qptr] + [vp, i64] * 6 + [vp, vp, vp, sz, vp]
    L.lf_qk_norm_rope_bwd.restype = i32
    _lib = L
    return L


def lib():
    return _load()


def lf_status_string(code: int) -> str:
    return _load().lf_status_string(int(code)).decode()


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(code: int, what: str):
    if code != LF_OK:
        raise LfError(code, what)


def make_desc(cu_seqlens: torch.Tensor, max_seqlen: int, total_tokens: int, hq: int, hkv: int,
              d: int, softmax_scale: float, causal: bool = True, block_q: int = 128) -> lf_attn_desc:
    """cu_seqlens must be an int32 CUDA tensor that outlives every call using the desc."""
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
        raise ValueError("cu_seqlens must be an int32 CUDA tensor")
    desc = lf_attn_desc(cu_seqlens.numel() - 1, cu_seqlens.data_ptr(), int(max_seqlen),
                        int(total_tokens), hq, hkv, d, float(softmax_scale), int(bool(causal)),
                        block_q)
    desc._keepalive = cu_seqlens
    return desc


def lf_workspace_size(desc: lf_attn_desc, which: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_load().lf_workspace_size(ctypes.byref(desc), which, ctypes.byref(n)), "lf_workspace_size")
    return n.value


def lf_attn_fwd(desc, q, k, v, o, lse, ws=None, stream=None):
    _check(_load().lf_attn_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                               _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                               _stream(stream)), "lf_attn_fwd")


def lf_block_select(desc, dout, o, delta, seed, step, flags, block_norm, D, tau, block_weight,
                    keep, kept_idx, kept_cnt, ws=None, stream=None):
    _check(_load().lf_block_select(ctypes.byref(desc), _ptr(dout), _ptr(o), float(delta),
                                   int(seed) & (2**64 - 1), int(step) & (2**64 - 1), int(flags),
                                   _ptr(block_norm), _ptr(D), _ptr(tau), _ptr(block_weight),
                                   _ptr(keep), _ptr(kept_idx), _ptr(kept_cnt), _ptr(ws),
                                   0 if ws is None else ws.numel() * ws.element_size(),
                                   _stream(stream)), "lf_block_select")


def lf_block_select_rule(desc, dout, o, rule, param, seed, step, flags, block_norm, D, tau,
                         block_weight, keep, kept_idx, kept_cnt, ws=None, stream=None):
    L = _load()
    fn = L.lf_block_select_rule
    fn.argtypes = [ctypes.POINTER(lf_attn_desc), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                   ctypes.c_double, ctypes.c_uint64, ctypes.c_uint64, ctypes.c_uint32] + \
        [ctypes.c_void_p] * 8 + [ctypes.c_size_t, ctypes.c_void_p]
    fn.restype = ctypes.c_int
    _check(fn(ctypes.byref(desc), _ptr(dout), _ptr(o), int(rule), float(param),
              int(seed) & (2**64 - 1), int(step) & (2**64 - 1), int(flags), _ptr(block_norm),
              _ptr(D), _ptr(tau), _ptr(block_weight), _ptr(keep), _ptr(kept_idx), _ptr(kept_cnt),
              _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
           "lf_block_select_rule")


def lf_attn_bwd(desc, q, k, v, o, lse, dout, D, block_weight, kept_idx, kept_cnt, dq, dk, dv,
                ws, stream=None):
    _check(_load().lf_attn_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                               _ptr(dout), _ptr(D), _ptr(block_weight), _ptr(kept_idx),
                               _ptr(kept_cnt), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
                               0 if ws is None else ws.numel() * ws.element_size(),
                               _stream(stream)), "lf_attn_bwd")


def lf_watchdog_selftest(limit_log2=24, stream=None):
    L = _load()
    L.lf_watchdog_selftest.argtypes = [ctypes.c_uint32, ctypes.c_void_p]
    L.lf_watchdog_selftest.restype = ctypes.c_int
    _check(L.lf_watchdog_selftest(int(limit_log2), _stream(stream)), "lf_watchdog_selftest")


def lf_sync_status(stream=None):
    """Synchronizes the stream; raises LfError for a device-side failure of an
    earlier call (and clears it)."""
    _check(_load().lf_sync_status(_stream(stream)), "lf_sync_status")


def lf_check_device_error(stream=None):
    _check(_load().lf_check_device_error(_stream(stream)), "lf_check_device_error")


class Buffers:
    """Device buffers of one attention layer for one LazyFlash step (torch
    allocations: plumbing only).  With forward=False the forward's outputs (o, lse)
    are not allocated: the caller already holds them."""

    def __init__(self, desc: lf_attn_desc, device="cuda", forward: bool = True):
        T, hq, hkv, d = desc.total_tokens, desc.hq, desc.hkv, desc.d
        nbmax = (desc.max_seqlen + desc.block_q - 1) // desc.block_q
        bf = dict(dtype=torch.bfloat16, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.o = torch.empty(T, hq, d, **bf) if forward else None
        self.lse = torch.empty(hq, T, **f32) if forward else None
        self.norm = torch.empty(desc.nseq, hq, nbmax, **f32)
        self.D = torch.empty(hq, T, **f32)
        self.tau = torch.empty(desc.nseq, hq, dtype=torch.float64, device=device)
        self.w = torch.empty(desc.nseq, hq, nbmax, **f32)
        self.keep = torch.empty(desc.nseq, hq, nbmax, dtype=torch.uint8, device=device)
        self.kept_idx = torch.empty(desc.nseq, hq, nbmax, dtype=torch.int32, device=device)
        self.kept_cnt = torch.empty(desc.nseq, hq, dtype=torch.int32, device=device)
        self.dq = torch.empty(T, hq, d, **bf)
        self.dk = torch.empty(T, hkv, d, **bf)
        self.dv = torch.empty(T, hkv, d, **bf)
        nws = lf_workspace_size(desc, LF_WS_BWD)
        self.ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=device)


def lazyflash_step(desc, q, k, v, dout, delta, seed, step, bufs: Buffers, flags=0, stream=None):
    """Forward, selection and sparse backward of one layer (three C-ABI calls)."""
    lf_attn_fwd(desc, q, k, v, bufs.o, bufs.lse, stream=stream)
    lf_block_select(desc, dout, bufs.o, delta, seed, step, flags, bufs.norm, bufs.D, bufs.tau,
                    bufs.w, bufs.keep, bufs.kept_idx, bufs.kept_cnt, stream=stream)
    lf_attn_bwd(desc, q, k, v, bufs.o, bufs.lse, dout, bufs.D, bufs.w, bufs.kept_idx,
                bufs.kept_cnt, bufs.dq, bufs.dk, bufs.dv, bufs.ws, stream=stream)


def lf_attn_bwd_static_ws(desc, q, k, v, o, lse, dout, D, block_weight, kept_idx, kept_cnt, dq,
                          dk, dv, stream=None):
    """lf_attn_bwd with the library's static scratch array instead of a caller
    workspace (for callers that cannot allocate; see include/lazyflash.h)."""
    L = _load()
    fn = L.lf_attn_bwd_static_ws
    fn.argtypes = [ctypes.POINTER(lf_attn_desc)] + [ctypes.c_void_p] * 14
    fn.restype = ctypes.c_int
    _check(fn(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
              _ptr(D), _ptr(block_weight), _ptr(kept_idx), _ptr(kept_cnt), _ptr(dq), _ptr(dk),
              _ptr(dv), _stream(stream)), "lf_attn_bwd_static_ws")



def _on_device(device, call, stream):
    """call(stream pointer) with `device` current, on torch's current stream of that
    device unless a stream is given."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device.index)   # as an integer: no Stream object
    if torch.cuda.current_device() == device.index:
        return call(_stream(stream))
    with torch.cuda.device(device):
        return call(_stream(stream))


def _vector(t, name, device, dtypes, numel=None):
    """Checks a contiguous device array; returns its address (None for None)."""
    if t is None:
        return None
    if t.device != device or t.dtype not in dtypes or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor on %s" % (
            name, " or ".join(str(d).replace("torch.", "") for d in dtypes), device))
    if numel is not None and t.numel() != numel:
        raise ValueError("%s must have %d elements, not %d" % (name, numel, t.numel()))
    return t.data_ptr()


# --------------------------------------------------------------------------------------
# attention with modified scores
# --------------------------------------------------------------------------------------
def make_score_mod(softcap: float = 0.0, alibi_slopes=None, prefix_len=None, prefix_causal: bool = False,
                   row_start=None, positions=None) -> lf_score_mod:
    """Modifier of lf_attn_fwd_mod and lf_attn_bwd_mod (meaning: include/lazyflash.h).
    alibi_slopes fp32 [hq], prefix_len int32 [nseq], row_start and positions int32 [T]: CUDA
    tensors on one device, which the modifier keeps."""
    given = [t for t in (alibi_slopes, prefix_len, row_start, positions) if t is not None]
    dev = given[0].device if given else None
    if dev is not None and dev.type != "cuda":
        raise ValueError("the modifier's arrays must be CUDA tensors")
    i32 = (torch.int32,)
    mod = lf_score_mod(float(softcap), _vector(alibi_slopes, "alibi_slopes", dev, (torch.float32,)),
                       _vector(prefix_len, "prefix_len", dev, i32), int(bool(prefix_causal)),
                       _vector(row_start, "row_start", dev, i32), _vector(positions, "positions", dev, i32))
    mod._keepalive = (alibi_slopes, prefix_len, row_start, positions)
    mod._sizes = tuple(None if t is None else t.numel() for t in mod._keepalive)
    mod._device = dev
    return mod


def _check_attention(desc, mod, q, k, v, rest=()):
    """Types, shapes and devices of an attention call with modified scores; its device."""
    T, d, dev = desc.total_tokens, desc.d, q.device
    if dev.type != "cuda":
        raise ValueError("expected CUDA tensors")
    tokens = [("q", q, desc.hq), ("k", k, desc.hkv), ("v", v, desc.hkv)]
    for name, t, heads in tokens + [r for r in rest if r[1] is not None and isinstance(r[2], int)]:
        if t.dtype != torch.bfloat16 or t.device != dev or tuple(t.shape) != (T, heads, d) or not t.is_contiguous():
            raise ValueError("%s must be a contiguous bf16 [%d, %d, %d] tensor on %s" % (name, T, heads, d, dev))
    for name, t, want in rest:
        if t is not None and not isinstance(want, int):
            dtype, numel = want
            _vector(t, name, dev, (dtype,), numel)
    keep = getattr(desc, "_keepalive", None)
    if (keep is not None and keep.device != dev) or (mod._device is not None and mod._device != dev):
        raise ValueError("cu_seqlens and the modifier's arrays must be on %s" % dev)
    for name, n, want in zip(("alibi_slopes", "prefix_len", "row_start", "positions"), mod._sizes,
                             (desc.hq, desc.nseq, T, T)):
        if n is not None and n != want:
            raise ValueError("%s must have %d elements, not %d" % (name, want, n))
    return dev


def lf_attn_fwd_mod(desc, mod, q, k, v, o, lse, o_low=None, stream=None):
    dev = _check_attention(desc, mod, q, k, v, [
        ("o", o, desc.hq), ("o_low", o_low, desc.hq),
        ("lse", lse, (torch.float32, desc.hq * desc.total_tokens))])
    L = _load()
    args = [None if t is None else t.data_ptr() for t in (q, k, v, o, o_low, lse)]
    _check(_on_device(dev, lambda s: L.lf_attn_fwd_mod(ctypes.byref(desc), ctypes.byref(mod), *args, s), stream),
           "lf_attn_fwd_mod")


def lf_attn_bwd_mod(desc, mod, q, k, v, o, lse, dout, D, block_weight, kept_idx, kept_cnt, dq, dk, dv,
                    ws, o_low=None, stream=None):
    rows = (torch.float32, desc.hq * desc.total_tokens)
    heads = desc.nseq * desc.hq
    nb = heads * ((desc.max_seqlen + desc.block_q - 1) // desc.block_q)
    dev = _check_attention(desc, mod, q, k, v, [
        ("o", o, desc.hq), ("o_low", o_low, desc.hq), ("lse", lse, rows), ("dout", dout, desc.hq), ("D", D, rows),
        ("block_weight", block_weight, (torch.float32, nb)), ("kept_idx", kept_idx, (torch.int32, nb)),
        ("kept_cnt", kept_cnt, (torch.int32, heads)), ("dq", dq, desc.hq), ("dk", dk, desc.hkv),
        ("dv", dv, desc.hkv), ("ws", ws, (torch.uint8, None))])
    L = _load()
    args = [None if t is None else t.data_ptr()
            for t in (q, k, v, o, o_low, lse, dout, D, block_weight, kept_idx, kept_cnt, dq, dk, dv, ws)]
    args.append(0 if ws is None else ws.numel() * ws.element_size())
    _check(_on_device(dev, lambda s: L.lf_attn_bwd_mod(ctypes.byref(desc), ctypes.byref(mod), *args, s), stream),
           "lf_attn_bwd_mod")


def shared_prompt_tables(prompt_lens, answer_lens, device="cuda"):
    """Tables of a batch in which many answers share one prompt.  Segment s is packed as its
    prompt (prompt_lens[s] tokens) followed by its answers (answer_lens[s], a list of
    lengths).  Returns (cu_seqlens, prefix_len, row_start, positions), int32: the mask's
    arrays for make_score_mod(prefix_len=..., prefix_causal=True, row_start=...), and each
    token's position, every answer's continuing its prompt's, for qk_norm_rope and, where the
    scores have a distance bias, for make_score_mod(positions=...)."""
    cu, start, pos = [0], [], []
    for p, answers in zip(prompt_lens, answer_lens, strict=True):
        at = int(p)
        start.append(torch.zeros(at, dtype=torch.int32))
        pos.append(torch.arange(at, dtype=torch.int32))
        for n in answers:
            start.append(torch.full((int(n),), at, dtype=torch.int32))
            pos.append(torch.arange(int(p), int(p) + int(n), dtype=torch.int32))
            at += int(n)
        cu.append(cu[-1] + at)
    tables = (torch.tensor(cu, dtype=torch.int32), torch.tensor(list(prompt_lens), dtype=torch.int32),
              torch.cat(start), torch.cat(pos))
    return tuple(t.to(device) for t in tables)


# --------------------------------------------------------------------------------------
# norms of the query and key heads with the position rotation
# --------------------------------------------------------------------------------------
def rope_cos_sin(npos: int, rot: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """Table of lf_qk_norm_rope: fp32 [npos, rot], row p the cosines, then the sines, of
    p * theta^(-2i/rot), i < rot/2.  The angles are computed in 64 bits, so that far
    positions keep theirs."""
    inv = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(npos, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def make_qk_desc(q, k, q_weight=None, k_weight=None, cos_sin=None, cu_seqlens=None, positions=None,
                 eps: float = 1e-6, norm: bool = True, interleaved: bool = False,
                 zero_tail: bool = False) -> lf_qk_desc:
    """Descriptor of lf_qk_norm_rope for q [T, hq, d] and k [T, hkv, d] (only their sizes
    and device are taken).  Weights [d] bf16 or fp32, both of one type, or None for ones;
    cos_sin [npos, rot] fp32 (see rope_cos_sin) or None for no rotation; cu_seqlens and
    positions int32.  The descriptor keeps the tensors it points to."""
    if q.dim() != 3 or k.dim() != 3 or q.shape[0] != k.shape[0] or q.shape[2] != k.shape[2]:
        raise ValueError("q and k must be [T, heads, d] with the same T and d")
    if not q.is_cuda or k.device != q.device:
        raise ValueError("q and k must be CUDA tensors on one device")
    T, hq, d = q.shape
    ws = [w for w in (q_weight, k_weight) if w is not None]
    if len({w.dtype for w in ws}) > 1:
        raise ValueError("q_weight and k_weight must have one type")
    dev = q.device
    floats = (torch.bfloat16, torch.float32)
    if cos_sin is not None and cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [npos, rot]")
    desc = lf_qk_desc(
        T, hq, k.shape[1], d, 0 if cu_seqlens is None else cu_seqlens.numel() - 1,
        _vector(cu_seqlens, "cu_seqlens", dev, (torch.int32,)),
        _vector(positions, "positions", dev, (torch.int32,), T),
        _vector(cos_sin, "cos_sin", dev, (torch.float32,)),
        0 if cos_sin is None else cos_sin.shape[0], 0 if cos_sin is None else cos_sin.shape[1],
        LF_ROPE_PAIRS if interleaved else LF_ROPE_HALVES,
        (LF_QK_NORM if norm else 0) | (LF_QK_ZERO_TAIL if zero_tail else 0), float(eps),
        _vector(q_weight, "q_weight", dev, floats, d), _vector(k_weight, "k_weight", dev, floats, d),
        int(bool(ws) and ws[0].dtype == torch.bfloat16))
    desc._keepalive = (q_weight, k_weight, cos_sin, cu_seqlens, positions)
    desc._device, desc._index, desc._tokens_and_dim = dev, dev.index, (T, d)
    desc._heads = (hq, k.shape[1])
    return desc


def _rows(t, desc, heads, name):
    """Address and token stride of a [T, heads, d] bf16 operand whose heads are contiguous."""
    T, d = desc._tokens_and_dim
    if t.dtype is not torch.bfloat16 or t.get_device() != desc._index or t.shape != (T, heads, d):
        raise ValueError("%s must be a bf16 [%d, %d, %d] tensor on %s" % (name, T, heads, d, desc._device))
    token, head, one = t.stride()
    if T and (one != 1 or (heads > 1 and head != d)):
        raise ValueError("%s must have contiguous heads" % name)
    return t.data_ptr(), (token if T > 1 else heads * d)


def lf_qk_workspace_size(desc: lf_qk_desc) -> int:
    n = ctypes.c_size_t(0)
    _check(_load().lf_qk_workspace_size(ctypes.byref(desc), ctypes.byref(n)), "lf_qk_workspace_size")
    return n.value


def lf_qk_norm_rope(desc, q, k, q_out, k_out, stream=None):
    hq, hkv = desc._heads
    args = (*_rows(q, desc, hq, "q"), *_rows(k, desc, hkv, "k"),
            *_rows(q_out, desc, hq, "q_out"), *_rows(k_out, desc, hkv, "k_out"))
    _check(_on_device(desc._device, lambda s: _load().lf_qk_norm_rope(ctypes.byref(desc), *args, s),
                      stream), "lf_qk_norm_rope")


def lf_qk_norm_rope_bwd(desc, q, k, dq_out, dk_out, dq, dk, dqw=None, dkw=None, ws=None, stream=None):
    f32 = (torch.float32,)
    none = (None, 0)
    args = (*(none if q is None else _rows(q, desc, desc.hq, "q")),
            *(none if k is None else _rows(k, desc, desc.hkv, "k")),
            *_rows(dq_out, desc, desc.hq, "dq_out"), *_rows(dk_out, desc, desc.hkv, "dk_out"),
            *_rows(dq, desc, desc.hq, "dq"), *_rows(dk, desc, desc.hkv, "dk"),
            _vector(dqw, "dqw", desc._device, f32, desc.d), _vector(dkw, "dkw", desc._device, f32, desc.d),
            _vector(ws, "ws", desc._device, (torch.uint8,)), 0 if ws is None else ws.numel())
    _check(_on_device(desc._device, lambda s: _load().lf_qk_norm_rope_bwd(ctypes.byref(desc), *args, s),
                      stream), "lf_qk_norm_rope_bwd")
