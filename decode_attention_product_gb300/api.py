"""Torch-facing wrappers of the C ABI (device memory and streams from PyTorch).

Each function checks dtypes, devices and contiguity, passes raw pointers and
the current CUDA stream to libaqpq, and raises AQError on a non-OK status.  No
arithmetic of the method happens here.  Names follow include/aqpq.h.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib

HEAD_DIM = 128
CODEWORDS = 256
PAGE = 16


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _same_device(ref, **tensors) -> int:
    """ref's device index, once every given tensor is on that device (the
    library launches on the current device, which each wrapper sets to this
    one for the call)."""
    d = ref.get_device()
    for name, t in tensors.items():
        if t is not None and t.get_device() != d:
            raise ValueError(f"{name} is on {t.device}, the call's other tensors on {ref.device}")
    return d


def _need(t, dtype, name, ndim=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    return t


def new_status(device=None) -> torch.Tensor:
    """A zeroed int32 device_status word."""
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def fit_codebooks(samples: torch.Tensor, num_subspaces: int, iters: int = 10,
                  with_assign: bool = False):
    """Lloyd k-means codebooks from samples [U][N][D] fp16 -> fp16 [U][M][K][Dsub]."""
    _need(samples, torch.float16, "samples", 3)
    U, N, D = samples.shape
    M = num_subspaces
    cb = torch.empty((U, M, CODEWORDS, D // M), dtype=torch.float16, device=samples.device)
    asg = torch.empty((U, N, M), dtype=torch.int32, device=samples.device) if with_assign else None
    cfg = _lib.config(M, head_dim=D)
    dev = samples.get_device()
    with torch.cuda.device(dev):
        st = _lib.load().aq_fit_codebooks(ctypes.byref(cfg), U, N, iters, _ptr(samples), _ptr(cb),
                                          _ptr(asg), _stream(dev))
    _lib.check(st, "aq_fit_codebooks")
    return (cb, asg) if with_assign else cb


def refine_codebooks(samples: torch.Tensor, codebooks: torch.Tensor, iters: int = 3,
                     with_assign: bool = False):
    """Periodic codebook update in place: `iters` Lloyd steps on samples [U][N][D]
    fp16 starting from codebooks [U][M][K][Dsub] fp16 (returns the assignment
    [U][N][M] of the last step when asked)."""
    _need(samples, torch.float16, "samples", 3)
    _need(codebooks, torch.float16, "codebooks", 4)
    U, N, D = samples.shape
    M = codebooks.shape[1]
    if codebooks.shape[0] != U:
        raise ValueError("one codebook per sample unit")
    dev = _same_device(samples, codebooks=codebooks)
    asg = torch.empty((U, N, M), dtype=torch.int32, device=samples.device) if with_assign else None
    cfg = _lib.config(M, head_dim=D)
    with torch.cuda.device(dev):
        st = _lib.load().aq_refine_codebooks(ctypes.byref(cfg), U, N, iters, _ptr(samples), _ptr(codebooks),
                                             _ptr(asg), _stream(dev))
    _lib.check(st, "aq_refine_codebooks")
    return asg


def to_e4m3(x: torch.Tensor) -> torch.Tensor:
    """FP8 E4M3 codes (uint8, same shape) of an fp16 tensor (nearest, ties to
    even, saturating)."""
    _need(x, torch.float16, "x")
    out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    dev = x.get_device()
    with torch.cuda.device(dev):
        st = _lib.load().aq_codebooks_to_e4m3(x.numel(), _ptr(x), _ptr(out), _stream(dev))
    _lib.check(st, "aq_codebooks_to_e4m3")
    return out


def from_e4m3(codes: torch.Tensor) -> torch.Tensor:
    """The exact fp16 values (same shape) of FP8 E4M3 codes."""
    _need(codes, torch.uint8, "codes")
    out = torch.empty(codes.shape, dtype=torch.float16, device=codes.device)
    dev = codes.get_device()
    with torch.cuda.device(dev):
        st = _lib.load().aq_codebooks_from_e4m3(codes.numel(), _ptr(codes), _ptr(out), _stream(dev))
    _lib.check(st, "aq_codebooks_from_e4m3")
    return out


def kmeans_step(samples: torch.Tensor, centroids: torch.Tensor):
    """One Lloyd step from fp32 centroids [U][M][K][Dsub]: (centroids_out, assign)."""
    _need(samples, torch.float16, "samples", 3)
    _need(centroids, torch.float32, "centroids", 4)
    U, N, D = samples.shape
    M = centroids.shape[1]
    dev = _same_device(samples, centroids=centroids)
    out = torch.empty_like(centroids)
    asg = torch.empty((U, N, M), dtype=torch.int32, device=samples.device)
    cfg = _lib.config(M, head_dim=D)
    with torch.cuda.device(dev):
        st = _lib.load().aq_kmeans_step(ctypes.byref(cfg), U, N, _ptr(samples), _ptr(centroids),
                                        _ptr(out), _ptr(asg), _stream(dev))
    _lib.check(st, "aq_kmeans_step")
    return out, asg


def encode_append(kv: torch.Tensor, token_set: torch.Tensor, slot_mapping: torch.Tensor,
                  codebooks: torch.Tensor, code_pages: torch.Tensor,
                  status: torch.Tensor | None = None) -> None:
    """Encode kv [T][Hkv][2][D] fp16 into code_pages [NP][Hkv][P][2][M] uint8 (in place)."""
    _need(kv, torch.float16, "kv", 4)
    _need(token_set, torch.int32, "token_set", 1)
    _need(slot_mapping, torch.int64, "slot_mapping", 1)
    _need(codebooks, torch.float16, "codebooks", 6)
    _need(code_pages, torch.uint8, "code_pages", 5)
    T, Hkv, _, D = kv.shape
    M = codebooks.shape[3]
    dev = _same_device(kv, token_set=token_set, slot_mapping=slot_mapping, codebooks=codebooks,
                 code_pages=code_pages, status=status)
    cfg = _lib.config(M, head_dim=D, page_size=code_pages.shape[2])
    with torch.cuda.device(dev):
        st = _lib.load().aq_encode_append(
            ctypes.byref(cfg), T, Hkv, _ptr(kv), _ptr(token_set), _ptr(slot_mapping), _ptr(codebooks),
            codebooks.shape[0], _ptr(code_pages), code_pages.shape[0], _ptr(status), _stream(dev))
    _lib.check(st, "aq_encode_append")


def decode_plan(batch: int, num_q_heads: int, num_kv_heads: int, max_seq_len: int,
                num_subspaces: int = 4, num_splits: int = 0, fp16: bool = False):
    """(num_splits, cluster_size, workspace_bytes) a decode call will use."""
    cfg = _lib.config(num_subspaces)
    s, c, w = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_size_t()
    st = _lib.load().aq_decode_plan(ctypes.byref(cfg), batch, num_q_heads, num_kv_heads,
                                    max_seq_len, num_splits, int(fp16), ctypes.byref(s),
                                    ctypes.byref(c), ctypes.byref(w))
    _lib.check(st, "aq_decode_plan")
    return s.value, c.value, w.value


def workspace_for(batch, num_q_heads, num_kv_heads, max_seq_len, num_subspaces=4, num_splits=0,
                  fp16=False, device="cuda"):
    """A device workspace of the size the planned call needs (None when 0)."""
    _, _, w = decode_plan(batch, num_q_heads, num_kv_heads, max_seq_len, num_subspaces,
                          num_splits, fp16)
    return torch.empty(w, dtype=torch.uint8, device=device) if w else None


def decode_attention(q: torch.Tensor, code_pages: torch.Tensor, codebooks: torch.Tensor,
                     req_set: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                     max_seq_len: int, scale: float | None = None, num_splits: int = 0,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     status: torch.Tensor | None = None) -> torch.Tensor:
    """PQ decode attention; returns out [B][Hq][D] fp32."""
    _need(q, torch.float32, "q", 3)
    _need(code_pages, torch.uint8, "code_pages", 5)
    _need(codebooks, torch.float16, "codebooks", 6)
    _need(req_set, torch.int32, "req_set", 1)
    _need(block_table, torch.int32, "block_table", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    B, Hq, D = q.shape
    Hkv, M = codebooks.shape[1], codebooks.shape[3]
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = workspace_for(B, Hq, Hkv, max_seq_len, M, num_splits, device=q.device)
    dev = _same_device(q, code_pages=code_pages, codebooks=codebooks, req_set=req_set, block_table=block_table,
                 seq_lens=seq_lens, out=out, workspace=workspace, status=status)
    cfg = _lib.config(M, head_dim=D, page_size=code_pages.shape[2])
    with torch.cuda.device(dev):
        st = _lib.load().aq_decode_attention(
            ctypes.byref(cfg), B, Hq, Hkv, _ptr(q), _ptr(code_pages), code_pages.shape[0],
            _ptr(codebooks), codebooks.shape[0], _ptr(req_set), _ptr(block_table), block_table.shape[1],
            _ptr(seq_lens), max_seq_len, float(scale), num_splits, _ptr(out), _ptr(workspace),
            workspace.numel() if workspace is not None else 0, _ptr(status), _stream(dev))
    _lib.check(st, "aq_decode_attention")
    return out


def decode_step(q: torch.Tensor, kv_new: torch.Tensor, code_pages: torch.Tensor,
                codebooks: torch.Tensor, req_set: torch.Tensor, block_table: torch.Tensor,
                seq_lens: torch.Tensor, max_seq_len: int, scale: float | None = None,
                num_splits: int = 0, overlap: bool = False, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None,
                status: torch.Tensor | None = None) -> torch.Tensor:
    """Fused decode step: append kv_new [B][Hkv][2][D] fp16 (the token at
    position seq_lens[b]-1) to code_pages, then PQ decode attention over all
    seq_lens[b] tokens; returns out [B][Hq][D] fp32.  Codebooks are fp16, or
    uint8 FP8 E4M3 codes (to_e4m3) for half the codebook bytes."""
    _need(q, torch.float32, "q", 3)
    _need(kv_new, torch.float16, "kv_new", 4)
    _need(code_pages, torch.uint8, "code_pages", 5)
    e4m3 = codebooks.dtype == torch.uint8
    _need(codebooks, torch.uint8 if e4m3 else torch.float16, "codebooks", 6)
    _need(req_set, torch.int32, "req_set", 1)
    _need(block_table, torch.int32, "block_table", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    B, Hq, D = q.shape
    Hkv, M = codebooks.shape[1], codebooks.shape[3]
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = workspace_for(B, Hq, Hkv, max_seq_len, M, num_splits, device=q.device)
    dev = _same_device(q, kv_new=kv_new, code_pages=code_pages, codebooks=codebooks, req_set=req_set,
                 block_table=block_table, seq_lens=seq_lens, out=out, workspace=workspace, status=status)
    cfg = _lib.config(M, head_dim=D, page_size=code_pages.shape[2])
    with torch.cuda.device(dev):
        st = _lib.load().aq_decode_step(
            ctypes.byref(cfg), B, Hq, Hkv, _ptr(q), _ptr(kv_new), _ptr(code_pages), code_pages.shape[0],
            _ptr(codebooks), codebooks.shape[0], _ptr(req_set), _ptr(block_table), block_table.shape[1],
            _ptr(seq_lens), max_seq_len, float(scale), num_splits,
            (_lib.STEP_OVERLAP if overlap else 0) | (_lib.STEP_E4M3 if e4m3 else 0),
            _ptr(out), _ptr(workspace), workspace.numel() if workspace is not None else 0, _ptr(status),
            _stream(dev))
    _lib.check(st, "aq_decode_step")
    return out


def decode_step_mixed(q: torch.Tensor, kv_new: torch.Tensor, num_fp16_heads: int,
                      kv_pages_f16: torch.Tensor | None, code_pages: torch.Tensor | None,
                      codebooks: torch.Tensor | None, req_set: torch.Tensor | None,
                      block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                      num_subspaces: int = 4, scale: float | None = None, overlap: bool = False,
                      out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      status: torch.Tensor | None = None) -> torch.Tensor:
    """Mixed-precision decode step: kv heads [0, num_fp16_heads) append their
    new K/V to the fp16 cache kv_pages_f16 [NP16][n16][2][P][D] and attend over
    it, the other kv heads take the fused PQ step over code_pages / codebooks
    (pools of Hkv - n16 heads); returns out [B][Hq][D] fp32."""
    _need(q, torch.float32, "q", 3)
    _need(kv_new, torch.float16, "kv_new", 4)
    _need(block_table, torch.int32, "block_table", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    B, Hq, D = q.shape
    Hkv = kv_new.shape[1]
    n16 = int(num_fp16_heads)
    e4m3 = False
    if n16 > 0:
        _need(kv_pages_f16, torch.float16, "kv_pages_f16", 5)
    if n16 < Hkv:
        _need(code_pages, torch.uint8, "code_pages", 5)
        e4m3 = codebooks is not None and codebooks.dtype == torch.uint8
        _need(codebooks, torch.uint8 if e4m3 else torch.float16, "codebooks", 6)
        _need(req_set, torch.int32, "req_set", 1)
        num_subspaces = codebooks.shape[3]
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    cfg = _lib.config(num_subspaces, head_dim=D)
    if workspace is None:
        w = ctypes.c_size_t()
        st = _lib.load().aq_decode_step_mixed_workspace(ctypes.byref(cfg), B, Hq, Hkv, n16, max_seq_len,
                                                        ctypes.byref(w))
        _lib.check(st, "aq_decode_step_mixed_workspace")
        workspace = torch.empty(w.value, dtype=torch.uint8, device=q.device) if w.value else None
    dev = _same_device(q, kv_new=kv_new, kv_pages_f16=kv_pages_f16, code_pages=code_pages, codebooks=codebooks,
                 req_set=req_set, block_table=block_table, seq_lens=seq_lens, out=out, workspace=workspace,
                 status=status)
    with torch.cuda.device(dev):
        st = _lib.load().aq_decode_step_mixed(
            ctypes.byref(cfg), B, Hq, Hkv, n16, _ptr(q), _ptr(kv_new), _ptr(kv_pages_f16),
            kv_pages_f16.shape[0] if kv_pages_f16 is not None else 0, _ptr(code_pages),
            code_pages.shape[0] if code_pages is not None else 0, _ptr(codebooks),
            codebooks.shape[0] if codebooks is not None else 0, _ptr(req_set), _ptr(block_table),
            block_table.shape[1], _ptr(seq_lens), max_seq_len, float(scale),
            (_lib.STEP_OVERLAP if overlap else 0) | (_lib.STEP_E4M3 if e4m3 else 0), _ptr(out),
            _ptr(workspace), workspace.numel() if workspace is not None else 0, _ptr(status), _stream(dev))
    _lib.check(st, "aq_decode_step_mixed")
    return out


def decode_attention_fp16(q: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                          seq_lens: torch.Tensor, max_seq_len: int, scale: float | None = None,
                          num_splits: int = 0, out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None,
                          status: torch.Tensor | None = None) -> torch.Tensor:
    """fp16-cache decode attention (the comparison point); kv_pages [NP][Hkv][2][P][D]."""
    _need(q, torch.float32, "q", 3)
    _need(kv_pages, torch.float16, "kv_pages", 5)
    _need(block_table, torch.int32, "block_table", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    B, Hq, D = q.shape
    Hkv = kv_pages.shape[1]
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = workspace_for(B, Hq, Hkv, max_seq_len, 4, num_splits, fp16=True, device=q.device)
    dev = _same_device(q, kv_pages=kv_pages, block_table=block_table, seq_lens=seq_lens, out=out,
                 workspace=workspace, status=status)
    cfg = _lib.config(4, head_dim=D, page_size=kv_pages.shape[3])
    with torch.cuda.device(dev):
        st = _lib.load().aq_decode_attention_fp16(
            ctypes.byref(cfg), B, Hq, Hkv, _ptr(q), _ptr(kv_pages), kv_pages.shape[0],
            _ptr(block_table), block_table.shape[1], _ptr(seq_lens), max_seq_len, float(scale),
            num_splits, _ptr(out), _ptr(workspace), workspace.numel() if workspace is not None else 0,
            _ptr(status), _stream(dev))
    _lib.check(st, "aq_decode_attention_fp16")
    return out


# --------------------------------------------------------------------------
# rotary positions
# --------------------------------------------------------------------------
_functions = {}


def _launch(dev: int, name: str, *args) -> None:
    """Call the library's `name` with args and the stream, `dev` current."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(_lib.load(), name)
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st != _lib.AQ_OK:
        _lib.check(st, name)


def _addr(t):
    return t.data_ptr() if t is not None else None


@functools.lru_cache(maxsize=None)
def _cfg_ref(head_dim: int = HEAD_DIM, page_size: int = PAGE):
    return ctypes.byref(_lib.config(4, head_dim=head_dim, page_size=page_size))


def _shape(t, want, name):
    if t.shape != want:
        raise ValueError(f"{name} must have shape {tuple(want)}, got {tuple(t.shape)}")


def rope_frequencies(rot_dim: int = HEAD_DIM, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                     original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """(inv_freq float64 [rot_dim / 2] on `device`, mscale) for rope(); scaling
    is "plain", "linear", "ntk" or "yarn" (see aq_rope_frequencies)."""
    if scaling not in _lib.ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_lib.ROPE_SCALINGS)}, got {scaling!r}")
    w = (ctypes.c_double * (HEAD_DIM // 2))()
    m = ctypes.c_float()
    st = _lib.load().aq_rope_frequencies(rot_dim, base, _lib.ROPE_SCALINGS[scaling], factor, original_len, beta_fast,
                                         beta_slow, w, ctypes.byref(m))
    _lib.check(st, "aq_rope_frequencies")
    return torch.tensor(list(w)[:rot_dim // 2], dtype=torch.float64, device=device), m.value


def _out_of_place(t, out, name):
    """`out` is `t` itself or memory of its own."""
    a, b = t.data_ptr(), out.data_ptr()
    n = t.numel() * t.element_size()
    if a != b and a < b + n and b < a + n:
        raise ValueError(f"{name} overlaps its input without being it")


def rope(positions: torch.Tensor, inv_freq: torch.Tensor, q: torch.Tensor | None = None,
         kv: torch.Tensor | None = None, interleaved: bool = False, mscale: float = 1.0, transpose: bool = False,
         lengths: bool = False, q_out: torch.Tensor | None = None, kv_out: torch.Tensor | None = None):
    """Rotary positions of q [T][Hq][D] fp32 and of the keys of kv [T][Hkv][2][D]
    fp16 (either may be None): returns (q_out, kv_out), new tensors unless
    given (q_out=q, kv_out=kv work in place).  positions int32 [T], negative for
    padding; with lengths=True they are sequence lengths and token t stands at
    positions[t] - 1.  transpose=True is the gradient of the plain rotation."""
    _need(positions, torch.int32, "positions", 1)
    _need(inv_freq, torch.float64, "inv_freq", 1)
    T, D = positions.shape[0], HEAD_DIM
    if q is None and kv is None:
        raise ValueError("q or kv is required")
    Hq = Hkv = 0
    if q is not None:
        _need(q, torch.float32, "q", 3)
        Hq, D = q.shape[1], q.shape[2]
        _shape(q, (T, Hq, D), "q")
        if q_out is None:
            q_out = torch.empty_like(q)
        elif q_out is not q:
            _need(q_out, torch.float32, "q_out", 3)
            _shape(q_out, q.shape, "q_out")
            _out_of_place(q, q_out, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if kv is not None:
        _need(kv, torch.float16, "kv", 4)
        Hkv = kv.shape[1]
        D = kv.shape[3] if q is None else D
        _shape(kv, (T, Hkv, 2, D), "kv")
        if kv_out is None:
            kv_out = torch.empty_like(kv)
        elif kv_out is not kv:
            _need(kv_out, torch.float16, "kv_out", 4)
            _shape(kv_out, kv.shape, "kv_out")
            _out_of_place(kv, kv_out, "kv_out")
    elif kv_out is not None:
        raise ValueError("kv_out without kv")
    dev = _same_device(positions, inv_freq=inv_freq, q=q, kv=kv, q_out=q_out, kv_out=kv_out)
    _launch(dev, "aq_rope", _cfg_ref(D), T, Hq, Hkv, positions.data_ptr(), inv_freq.data_ptr(),
            2 * inv_freq.shape[0], mscale,
            (_lib.ROPE_INTERLEAVED if interleaved else 0) | (_lib.ROPE_TRANSPOSE if transpose else 0)
            | (_lib.ROPE_LENGTHS if lengths else 0), _addr(q), _addr(q_out), _addr(kv), _addr(kv_out))
    return q_out, kv_out


class Rope:
    """A model's rotary positions: the frequencies (rope_frequencies' arguments)
    and the pair layout, kept on the device.  `rope(positions, q, kv, ...)`."""

    def __init__(self, rot_dim: int = HEAD_DIM, base: float = 10000.0, interleaved: bool = False, device="cuda", **scaling):
        self.inv_freq, self.mscale = rope_frequencies(rot_dim, base, device=device, **scaling)
        self.interleaved = interleaved

    def __call__(self, positions, q=None, kv=None, **kw):
        return rope(positions, self.inv_freq, q, kv, interleaved=self.interleaved, mscale=self.mscale, **kw)


# --------------------------------------------------------------------------
# the 8-bit block-scaled cache
# --------------------------------------------------------------------------
def _need_q8(code_pages, page_scales) -> int:
    """The cache's checks; its format."""
    if code_pages is None or code_pages.dtype not in (torch.int8, torch.uint8):
        raise TypeError("code_pages must be torch.int8 (INT8) or torch.uint8 (E4M3 codes)")
    _need(code_pages, code_pages.dtype, "code_pages", 5)
    _need(page_scales, torch.float32, "page_scales", 3)
    NP, Hkv, two, P, D = code_pages.shape
    if two != 2:
        raise ValueError(f"code_pages must be [NP][Hkv][2][P][D], got {tuple(code_pages.shape)}")
    _shape(page_scales, (NP, Hkv, 2), "page_scales")
    return _lib.Q8_INT8 if code_pages.dtype == torch.int8 else _lib.Q8_E4M3


def _need_requests(block_table, seq_lens, cu_tokens=None):
    _need(block_table, torch.int32, "block_table", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    if block_table.shape[0] != seq_lens.shape[0]:
        raise ValueError("block_table and seq_lens must have one row per request")
    if cu_tokens is not None:
        _need(cu_tokens, torch.int32, "cu_tokens", 1)
        if cu_tokens.shape[0] != seq_lens.shape[0] + 1:
            raise ValueError("cu_tokens must have one entry more than seq_lens")


def new_q8_cache(num_pages: int, num_kv_heads: int, e4m3: bool = False, device="cuda"):
    """(code_pages, page_scales) of an empty 8-bit cache."""
    return (torch.zeros((num_pages, num_kv_heads, 2, PAGE, HEAD_DIM), dtype=torch.uint8 if e4m3 else torch.int8,
                        device=device),
            torch.zeros((num_pages, num_kv_heads, 2), dtype=torch.float32, device=device))


def _q8_cache_call(name, kv, code_pages, page_scales, block_table, seq_lens, cu_tokens, status):
    fmt = _need_q8(code_pages, page_scales)
    _need(kv, torch.float16, "kv", 4)
    _need_requests(block_table, seq_lens, cu_tokens)
    NP, Hkv, _, P, D = code_pages.shape
    T, B = kv.shape[0], seq_lens.shape[0]
    _shape(kv, (T, Hkv, 2, D), "kv")
    if cu_tokens is None and T != B:
        raise ValueError("kv holds one token per request unless cu_tokens is given")
    dev = _same_device(kv, code_pages=code_pages, page_scales=page_scales, block_table=block_table,
                       seq_lens=seq_lens, cu_tokens=cu_tokens, status=status)
    _launch(dev, name, _cfg_ref(D, P), fmt, B, T, Hkv, kv.data_ptr(), code_pages.data_ptr(), page_scales.data_ptr(),
            NP, block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(), _addr(cu_tokens), _addr(status))


def q8_append(kv: torch.Tensor, code_pages: torch.Tensor, page_scales: torch.Tensor, block_table: torch.Tensor,
              seq_lens: torch.Tensor, cu_tokens: torch.Tensor | None = None,
              status: torch.Tensor | None = None) -> None:
    """Append kv [T][Hkv][2][D] fp16 to the 8-bit cache code_pages
    [NP][Hkv][2][P][D] (int8, or uint8 E4M3 codes) with page_scales [NP][Hkv][2]
    fp32, in place: rows cu_tokens[b] .. cu_tokens[b + 1] - 1 are request b's last
    tokens, ending at position seq_lens[b] - 1 (one per request without
    cu_tokens)."""
    _q8_cache_call("aq_q8_append", kv, code_pages, page_scales, block_table, seq_lens, cu_tokens, status)


def q8_load(code_pages: torch.Tensor, page_scales: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
            cu_tokens: torch.Tensor | None = None, num_tokens: int | None = None,
            kv_out: torch.Tensor | None = None, status: torch.Tensor | None = None) -> torch.Tensor:
    """Read tokens back from the 8-bit cache as fp16 [T][Hkv][2][D]: each
    request's last cu_tokens[b + 1] - cu_tokens[b] tokens (its last one without
    cu_tokens).  num_tokens (T) is needed with cu_tokens unless kv_out is given."""
    if kv_out is None:
        if num_tokens is None:
            if cu_tokens is not None:
                raise ValueError("num_tokens is required with cu_tokens")
            num_tokens = seq_lens.shape[0]
        kv_out = torch.empty((num_tokens, code_pages.shape[1], 2, code_pages.shape[4]), dtype=torch.float16,
                             device=code_pages.device)
    _q8_cache_call("aq_q8_load", kv_out, code_pages, page_scales, block_table, seq_lens, cu_tokens, status)
    return kv_out


@functools.lru_cache(maxsize=4096)
def q8_decode_plan(batch: int, num_q_heads: int, num_kv_heads: int, max_seq_len: int, num_splits: int = 0):
    """(num_splits, workspace_bytes) a q8_decode_attention call will use."""
    s, w = ctypes.c_int32(), ctypes.c_size_t()
    st = _lib.load().aq_q8_decode_plan(_cfg_ref(), batch, num_q_heads, num_kv_heads, max_seq_len, num_splits,
                                       ctypes.byref(s), ctypes.byref(w))
    _lib.check(st, "aq_q8_decode_plan")
    return s.value, w.value


def q8_decode_attention(q: torch.Tensor, code_pages: torch.Tensor, page_scales: torch.Tensor,
                        block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                        scale: float | None = None, num_splits: int = 0, out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, status: torch.Tensor | None = None) -> torch.Tensor:
    """Decode attention over the 8-bit cache; q [B][Hq][D] fp32, returns out
    [B][Hq][D] fp32.  Any number of query heads per kv head."""
    _need(q, torch.float32, "q", 3)
    fmt = _need_q8(code_pages, page_scales)
    _need_requests(block_table, seq_lens)
    B, Hq, D = q.shape
    NP, Hkv, _, P, _ = code_pages.shape
    if seq_lens.shape[0] != B or code_pages.shape[4] != D:
        raise ValueError("q must be [B][Hq][D] with the requests and head_dim of the cache")
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, torch.float32, "out", 3)
        _shape(out, q.shape, "out")
    if max_seq_len > 0x7fffffff or num_splits > 0x7fffffff:
        raise ValueError("max_seq_len and num_splits are 32-bit numbers")
    need = q8_decode_plan(B, Hq, Hkv, max_seq_len, num_splits)[1]
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    dev = _same_device(q, code_pages=code_pages, page_scales=page_scales, block_table=block_table, seq_lens=seq_lens,
                       out=out, workspace=workspace, status=status)
    _launch(dev, "aq_q8_decode_attention", _cfg_ref(D, P), fmt, B, Hq, Hkv, q.data_ptr(), code_pages.data_ptr(),
            page_scales.data_ptr(), NP, block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(), max_seq_len,
            D ** -0.5 if scale is None else scale, num_splits, out.data_ptr(), _addr(workspace),
            workspace.numel() * workspace.element_size() if workspace is not None else 0, _addr(status))
    return out


# --------------------------------------------------------------------------
# pages
# --------------------------------------------------------------------------
def _need_table(block_table, seq_lens, refcount):
    _need_requests(block_table, seq_lens)
    _need(refcount, torch.int32, "refcount", 1)
    return block_table.shape[0], block_table.shape[1], refcount.shape[0]


def _need_rows(rows, other, name):
    _need(rows, torch.int32, "rows", 1)
    if other is not None:
        _need(other, torch.int32, name, 1)
        _shape(other, rows.shape, name)


def _pool_array(pools, num_pages, dev):
    """The pools as the library takes them."""
    if len(pools) > _lib.MAX_POOLS:
        raise ValueError(f"at most {_lib.MAX_POOLS} pools")
    arr = (_lib.PagePool * len(pools))()
    for i, t in enumerate(pools):
        if not t.is_cuda or not t.is_contiguous() or t.dim() < 2 or t.shape[0] != num_pages:
            raise ValueError(f"pool {i} must be a contiguous CUDA tensor of {num_pages} pages")
        if t.get_device() != dev:
            raise ValueError(f"pool {i} is on {t.device}, the call's other tensors on device {dev}")
        arr[i].data = t.data_ptr()
        arr[i].page_bytes = t.stride(0) * t.element_size()
    return arr


@functools.lru_cache(maxsize=1024)
def pages_workspace_bytes(num_rows: int, num_pages: int) -> int:
    """Workspace of the page calls over a table of num_rows rows and num_pages pages."""
    w = ctypes.c_size_t()
    _lib.check(_lib.load().aq_pages_workspace(num_rows, num_pages, ctypes.byref(w)), "aq_pages_workspace")
    return w.value


def _page_workspace(workspace, R, NP, device):
    if workspace is None:
        return torch.empty(pages_workspace_bytes(R, NP), dtype=torch.uint8, device=device)
    return workspace


def _bytes(t):
    return t.numel() * t.element_size()


def pages_extend(rows: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 refcount: torch.Tensor, pools, workspace: torch.Tensor | None = None,
                 status: torch.Tensor | None = None) -> None:
    """Rows (int32 [n]) of the table grow to new_lens: pages are allocated, and a
    shared, partly filled last page is copied (in every pool) before it is
    written.  block_table [R][max_pages], seq_lens [R] and refcount [NP] change
    in place; pools are the caches whose pages the table holds."""
    _need_rows(rows, new_lens, "new_lens")
    R, MP, NP = _need_table(block_table, seq_lens, refcount)
    ws = _page_workspace(workspace, R, NP, rows.device)
    dev = _same_device(rows, new_lens=new_lens, block_table=block_table, seq_lens=seq_lens, refcount=refcount,
                       workspace=ws, status=status)
    arr = pools if isinstance(pools, ctypes.Array) else _pool_array(pools, NP, dev)
    _launch(dev, "aq_pages_extend", rows.shape[0], rows.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(), R, MP,
            seq_lens.data_ptr(), refcount.data_ptr(), NP, arr, len(arr), ws.data_ptr(), _bytes(ws), _addr(status))


def pages_fork(src_rows: torch.Tensor, dst_rows: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
               refcount: torch.Tensor, status: torch.Tensor | None = None) -> None:
    """Empty rows dst_rows (int32 [n]) become copies of src_rows, sharing their pages."""
    _need_rows(src_rows, dst_rows, "dst_rows")
    R, MP, NP = _need_table(block_table, seq_lens, refcount)
    dev = _same_device(src_rows, dst_rows=dst_rows, block_table=block_table, seq_lens=seq_lens, refcount=refcount,
                       status=status)
    _launch(dev, "aq_pages_fork", src_rows.shape[0], src_rows.data_ptr(), dst_rows.data_ptr(), block_table.data_ptr(),
            R, MP, seq_lens.data_ptr(), refcount.data_ptr(), NP, _addr(status))


def pages_free(rows: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, refcount: torch.Tensor,
               keep_lens: torch.Tensor | None = None, status: torch.Tensor | None = None) -> None:
    """Rows (int32 [n]) keep their first keep_lens tokens (none by default); the
    pages behind them are given up."""
    _need_rows(rows, keep_lens, "keep_lens")
    R, MP, NP = _need_table(block_table, seq_lens, refcount)
    dev = _same_device(rows, keep_lens=keep_lens, block_table=block_table, seq_lens=seq_lens, refcount=refcount,
                       status=status)
    _launch(dev, "aq_pages_free", rows.shape[0], rows.data_ptr(), _addr(keep_lens), block_table.data_ptr(), R, MP,
            seq_lens.data_ptr(), refcount.data_ptr(), NP, _addr(status))


def pages_compact(block_table: torch.Tensor, seq_lens: torch.Tensor, refcount: torch.Tensor, pools,
                  workspace: torch.Tensor | None = None, status: torch.Tensor | None = None) -> None:
    """Live pages move to the lowest ids (in every pool); the table follows."""
    R, MP, NP = _need_table(block_table, seq_lens, refcount)
    ws = _page_workspace(workspace, R, NP, refcount.device)
    dev = _same_device(block_table, seq_lens=seq_lens, refcount=refcount, workspace=ws, status=status)
    arr = pools if isinstance(pools, ctypes.Array) else _pool_array(pools, NP, dev)
    _launch(dev, "aq_pages_compact", block_table.data_ptr(), R, MP, seq_lens.data_ptr(), refcount.data_ptr(), NP, arr,
            len(arr), ws.data_ptr(), _bytes(ws), _addr(status))


class PageTable:
    """A block table over the pages of some caches: `pools` are tensors of
    num_pages pages each (every layer's code_pages, page_scales, fp16 pages ...).
    Holds block_table, seq_lens, refcount, a workspace and a status word; the
    methods take int32 device tensors of rows."""

    def __init__(self, num_rows: int, max_pages: int, pools):
        self.pools = list(pools)
        if not self.pools:
            raise ValueError("at least one pool")
        dev, num_pages = self.pools[0].device, int(self.pools[0].shape[0])
        self._arr = _pool_array(self.pools, num_pages, self.pools[0].get_device())
        self.block_table = torch.full((num_rows, max_pages), -1, dtype=torch.int32, device=dev)
        self.seq_lens = torch.zeros(num_rows, dtype=torch.int32, device=dev)
        self.refcount = torch.zeros(num_pages, dtype=torch.int32, device=dev)
        self.workspace = torch.empty(pages_workspace_bytes(num_rows, num_pages), dtype=torch.uint8, device=dev)
        self.status = new_status(dev)

    def _state(self):
        return self.block_table, self.seq_lens, self.refcount

    def extend(self, rows, new_lens):
        pages_extend(rows, new_lens, *self._state(), self._arr, self.workspace, self.status)

    def fork(self, src_rows, dst_rows):
        pages_fork(src_rows, dst_rows, *self._state(), self.status)

    def free(self, rows, keep_lens=None):
        pages_free(rows, *self._state(), keep_lens, self.status)

    def compact(self):
        pages_compact(*self._state(), self._arr, self.workspace, self.status)

    def check_status(self):
        """Raise if a call flagged a data error (reads the status word)."""
        st = int(self.status.item())
        if st:
            raise RuntimeError(f"device status {st:#x}")


class Q8DecodeStep:
    """One decode step of a fixed batch over the 8-bit cache: the rotary
    positions (with a Rope), the append of each request's current token (at
    position seq_len - 1) and decode attention over all its tokens.  Holds the
    cache tensors, workspace, output and a status word; `run(q, new_kv)` works on
    the current stream and can be captured into a graph."""

    def __init__(self, code_pages, page_scales, block_table, seq_lens, max_seq_len, num_q_heads, scale=None,
                 num_splits=0, rope=None):
        _need_q8(code_pages, page_scales)
        self.code_pages, self.page_scales = code_pages, page_scales
        self.block_table, self.seq_lens = block_table, seq_lens
        self.max_seq_len, self.scale, self.num_splits = int(max_seq_len), scale, num_splits
        B, Hkv, dev = int(seq_lens.shape[0]), int(code_pages.shape[1]), code_pages.device
        need = q8_decode_plan(B, int(num_q_heads), Hkv, self.max_seq_len, num_splits)[1]
        self.workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        self.status = new_status(dev)
        self.out = torch.empty((B, int(num_q_heads), HEAD_DIM), dtype=torch.float32, device=dev)
        self.rope = rope
        if rope is not None:
            self._q = torch.empty_like(self.out)
            self._kv = torch.empty((B, Hkv, 2, HEAD_DIM), dtype=torch.float16, device=dev)

    def run(self, q, new_kv, out=None):
        if self.rope is not None:
            q, new_kv = self.rope(self.seq_lens, q, new_kv, lengths=True, q_out=self._q, kv_out=self._kv)
        q8_append(new_kv, self.code_pages, self.page_scales, self.block_table, self.seq_lens, status=self.status)
        return q8_decode_attention(q, self.code_pages, self.page_scales, self.block_table, self.seq_lens,
                                   self.max_seq_len, self.scale, self.num_splits,
                                   out=self.out if out is None else out, workspace=self.workspace, status=self.status)

    def check_status(self):
        """Raise if a kernel flagged a data error (reads the status word)."""
        st = int(self.status.item())
        if st:
            raise RuntimeError(f"device status {st:#x}")


class DecodeStep:
    """One decode step of a fixed batch: append each request's current K/V
    token (the one at position seq_len-1) into the PQ code cache, then PQ
    decode attention over the cache, as one aq_decode_step launch.

    Holds the cache tensors, the workspace, the output and a device status
    word.  `run(q, new_kv)` launches the step on the current stream.
    `capture_host(q_host, kv_host, out_host)` records the whole step -- copies
    of the pinned host inputs to the device, the step, the copy of the output
    back to pinned host memory -- into a CUDA graph; `replay()` launches it and,
    with wait=True, blocks until the output is on the host.  `launch()` /
    `wait()` split that in two, so that a caller keeping two sets of pinned
    buffers can launch step i before it waits for step i-1's output (the copies
    and the kernel of one step overlap the host's work on the other).
    `overlap=True` launches the step as a programmatic dependent of the
    preceding kernel (aq_decode_step's AQ_STEP_OVERLAP contract).  With a Rope,
    `run` first turns q and the new keys to position seq_len-1.
    """

    def __init__(self, code_pages, codebooks, req_set, block_table, seq_lens, max_seq_len,
                 new_slot, new_set, num_q_heads, scale=None, num_splits=0, overlap=False, rope=None):
        self.code_pages, self.codebooks = code_pages, codebooks
        self.req_set, self.block_table, self.seq_lens = req_set, block_table, seq_lens
        self.max_seq_len = int(max_seq_len)
        self.new_slot, self.new_set = new_slot, new_set
        self.B, self.Hq = int(seq_lens.shape[0]), int(num_q_heads)
        self.Hkv, self.M = int(codebooks.shape[1]), int(codebooks.shape[3])
        self.scale = scale
        self.num_splits = num_splits
        dev = code_pages.device
        self.workspace = workspace_for(self.B, self.Hq, self.Hkv, self.max_seq_len, self.M,
                                       num_splits, device=dev)
        self.status = new_status(dev)
        self.out = torch.empty((self.B, self.Hq, HEAD_DIM), dtype=torch.float32, device=dev)
        self.graph = None
        self._host = None
        self._done = None
        self._io = None
        self.overlap = overlap
        self.rope = rope
        if rope is not None:
            self._q = torch.empty_like(self.out)
            self._kv = torch.empty((self.B, self.Hkv, 2, HEAD_DIM), dtype=torch.float16, device=dev)

    def run(self, q, new_kv, out=None):
        if self.rope is not None:
            q, new_kv = self.rope(self.seq_lens, q, new_kv, lengths=True, q_out=self._q, kv_out=self._kv)
        return decode_step(q, new_kv, self.code_pages, self.codebooks, self.req_set,
                           self.block_table, self.seq_lens, self.max_seq_len, self.scale,
                           self.num_splits, overlap=self.overlap, out=self.out if out is None else out,
                           workspace=self.workspace, status=self.status)

    def pinned_io(self):
        """(q_host, kv_host, out_host): pinned host views of one input buffer
        (q [B][Hq][D] fp32 then the new K/V [B][Hkv][2][D] fp16) and an output
        buffer [B][Hq][D] fp32, for capture_host() without arguments: the inputs
        then reach the device in one copy."""
        if self._io is None:
            nq = self.B * self.Hq * HEAD_DIM * 4
            nkv = self.B * self.Hkv * 2 * HEAD_DIM * 2
            buf = torch.empty(nq + nkv, dtype=torch.uint8).pin_memory()
            q = buf[:nq].view(torch.float32).view(self.B, self.Hq, HEAD_DIM)
            kv = buf[nq:].view(torch.float16).view(self.B, self.Hkv, 2, HEAD_DIM)
            out = torch.empty((self.B, self.Hq, HEAD_DIM), dtype=torch.float32).pin_memory()
            self._io = (buf, q, kv, out)
        return self._io[1:]

    def capture_host(self, q_host=None, kv_host=None, out_host=None):
        """Capture copy-in, step, copy-out into a CUDA graph (pinned host
        tensors; none given: this object's pinned_io(), copied in one piece)."""
        dev = self.out.device
        if q_host is None:
            self.pinned_io()
            buf, q_host, kv_host, out_host = self._io
            buf_d = torch.empty(buf.shape, dtype=buf.dtype, device=dev)
            nq = q_host.numel() * 4
            q_d = buf_d[:nq].view(torch.float32).view(q_host.shape)
            kv_d = buf_d[nq:].view(torch.float16).view(kv_host.shape)
            copies = [(buf_d, buf)]
        else:
            for t, n in ((q_host, "q_host"), (kv_host, "kv_host"), (out_host, "out_host")):
                if t.is_cuda or not t.is_pinned():
                    raise ValueError(f"{n} must be a pinned host tensor")
            q_d = torch.empty(q_host.shape, dtype=q_host.dtype, device=dev)
            kv_d = torch.empty(kv_host.shape, dtype=kv_host.dtype, device=dev)
            copies = [(q_d, q_host), (kv_d, kv_host)]
        self._host = (q_host, kv_host, out_host, q_d, kv_d, copies)
        # one eager run sets kernel attributes outside the capture
        for d, h in copies:
            d.copy_(h)
        self.run(q_d, kv_d)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for d, h in copies:
                d.copy_(h, non_blocking=True)
            self.run(q_d, kv_d)
            out_host.copy_(self.out, non_blocking=True)
        self.graph = g
        return g

    def replay(self, wait=True):
        self.graph.replay()
        if wait:
            torch.cuda.current_stream().synchronize()

    def launch(self):
        """Replay the captured step on the current stream without waiting
        (replays on different streams may overlap: use distinct caches)."""
        self.graph.replay()
        if self._done is None:
            self._done = torch.cuda.Event()
        self._done.record()

    def wait(self):
        """Block until the last launch()'s output is in pinned host memory."""
        self._done.synchronize()

    def check_status(self):
        """Raise if a kernel flagged a data error (reads the status word)."""
        st = int(self.status.item())
        if st:
            raise RuntimeError(f"device status {st:#x}")


class HostDecodeStep:
    """aq_decode_step_host for a fixed batch and cache: one C call per step
    enqueues the copy of the query and the new K/V from pinned host memory, the
    fused step and the copy of the output back to pinned host memory, on
    `stream` (a torch.cuda.Stream; the current one if None).

    `q_host`, `kv_host`, `out_host` are the pinned tensors (write the next
    step's inputs into the first two, read the output from the last one after
    `sync()`); `launch()` enqueues one step.  The call's arguments are
    marshalled once, here; `launch()` itself does no device switch, so the
    cache's device must be the current one when it is called.
    """

    def __init__(self, code_pages, codebooks, req_set, block_table, seq_lens, max_seq_len,
                 num_q_heads, scale=None, num_splits=0, stream=None):
        _need(code_pages, torch.uint8, "code_pages", 5)
        e4m3 = codebooks.dtype == torch.uint8
        _need(codebooks, torch.uint8 if e4m3 else torch.float16, "codebooks", 6)
        for t, n in ((req_set, "req_set"), (seq_lens, "seq_lens")):
            _need(t, torch.int32, n, 1)
        _need(block_table, torch.int32, "block_table", 2)
        self.B, self.Hq = int(seq_lens.shape[0]), int(num_q_heads)
        self.Hkv, self.M = int(codebooks.shape[1]), int(codebooks.shape[3])
        dev = code_pages.device
        _same_device(code_pages, codebooks=codebooks, req_set=req_set, block_table=block_table,
                     seq_lens=seq_lens)
        self.stream = stream or torch.cuda.current_stream(dev)
        self.q_host = torch.empty((self.B, self.Hq, HEAD_DIM), dtype=torch.float32).pin_memory()
        self.kv_host = torch.empty((self.B, self.Hkv, 2, HEAD_DIM), dtype=torch.float16).pin_memory()
        self.out_host = torch.empty((self.B, self.Hq, HEAD_DIM), dtype=torch.float32).pin_memory()
        lib = _lib.load()
        n = lib.aq_decode_step_host_staging(self.B, self.Hq, self.Hkv)
        self.staging = torch.empty(n, dtype=torch.uint8, device=dev)
        self.workspace = workspace_for(self.B, self.Hq, self.Hkv, int(max_seq_len), self.M, num_splits,
                                       device=dev)
        self.status = new_status(dev)
        self._keep = (code_pages, codebooks, req_set, block_table, seq_lens)
        self._cfg = _lib.config(self.M, page_size=code_pages.shape[2])
        scale = HEAD_DIM ** -0.5 if scale is None else scale
        self._fn = lib.aq_decode_step_host
        self._args = (ctypes.byref(self._cfg), self.B, self.Hq, self.Hkv, _ptr(self.q_host), _ptr(self.kv_host),
                      _ptr(code_pages), code_pages.shape[0], _ptr(codebooks), codebooks.shape[0], _ptr(req_set),
                      _ptr(block_table), block_table.shape[1], _ptr(seq_lens), int(max_seq_len), float(scale),
                      num_splits, _lib.STEP_E4M3 if e4m3 else 0, _ptr(self.out_host), _ptr(self.staging),
                      self.staging.numel(), _ptr(self.workspace),
                      self.workspace.numel() if self.workspace is not None else 0, _ptr(self.status),
                      ctypes.c_void_p(self.stream.cuda_stream))

    def launch(self):
        """Enqueue one step (copies in, step, copy out) on the stream."""
        st = self._fn(*self._args)
        if st != _lib.AQ_OK:
            _lib.check(st, "aq_decode_step_host")

    def sync(self):
        """Wait until the last launched step's output is in out_host."""
        self.stream.synchronize()

    def check_status(self):
        """Raise if a kernel flagged a data error (reads the status word)."""
        st = int(self.status.item())
        if st:
            raise RuntimeError(f"device status {st:#x}")
