"""Local attention beside the sparse one: rotary positions, sliding-window
attention with sinks and its backward, and a paged cache of ragged sequences.

HSA reaches complete, strictly past chunks only and carries no positions; the
layers it is paired with attend to the recent tokens and a few first ones, with
rotary positions.  A query at position p sees key u iff u <= p, u is cached, and
window == 0, or p - u < window, or u < sinks.

Same manner as the rest of the package: torch supplies device memory and the
current stream, every step runs in the library's kernels.  The workspace's
status word is sticky for these calls (device_status() reads and clears it);
window_workspace and paged_workspace return one that starts clean.  It is the
only place for what the kernels find: a page number or length outside its
bounds, a wait that ran out.  A call that is given no workspace makes one for
itself, which nobody can ask: give one wherever that matters.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native
from ._native import hsa_paged_t, hsa_rope_t, hsa_window_t

__all__ = ["make_rope", "rope", "window_workspace", "window_attend", "window_backward", "paged_workspace",
           "paged_append", "paged_attend", "hsa_rope_t", "hsa_window_t", "hsa_paged_t"]

_DT = {torch.float32: _native.HSA_F32, torch.bfloat16: _native.HSA_BF16}
_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}
_byref = ctypes.byref
# torch.cuda.current_stream(index).cuda_stream and current_device() without the objects and checks around them; a
# torch without CUDA has neither, and no tensor that would get as far
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _dtype(t):
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"dtype {t.dtype} not supported (float32, bfloat16)") from None


def _check(like, *ts):
    """CUDA, contiguous, on one device, of one dtype (None is passed over)."""
    dev, dt = like.get_device(), like.dtype
    if dev >= 0 and like.is_contiguous():
        for t in ts:
            if t is not None and (t.get_device() != dev or t.dtype is not dt or not t.is_contiguous()):
                break
        else:
            return
    for t in (like,) + ts:      # something is wrong: say what
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
        if t.get_device() != dev:
            raise ValueError(f"tensors on {like.device} and {t.device}")
        if t.dtype != dt:
            raise TypeError(f"tensors of {dt} and {t.dtype}")


_I32 = torch.int32


def _ints(like, **tensors):
    dev = like.get_device()
    for t in tensors.values():
        if t.dtype is not _I32 or t.get_device() != dev or not t.is_contiguous():
            break
    else:
        return
    for name, t in tensors.items():
        if t.dtype is not _I32:
            raise TypeError(f"{name} must be int32, got {t.dtype}")
        if t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous and on {like.device}")


def _shape(name, t, want):
    if t is not None and t.shape != want:
        raise ValueError(f"{name} is {tuple(t.shape)}, expected {tuple(want)}")


def _wide(**ints):
    """An integer that its 32-bit (pos0, q_pos0: 64-bit) field would be cut to is refused here; a negative one is
    left to the library."""
    for name, x in ints.items():
        bits = 63 if name.endswith("pos0") else 31
        if x >> bits not in (0, -1):
            raise ValueError(f"{name}={x} does not fit {bits + 1} bits")


def _p(t):
    return None if t is None else t.data_ptr()


_fns = {}   # the library's functions by name


def _call(name, like, *args, ws=None):
    """One library call on the current stream of `like`'s device, with that device current."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(_native.lib(), name)
    index = like.get_device()
    if ws is not None:
        if ws.get_device() != index or not ws.is_contiguous():
            raise ValueError(f"ws must be contiguous and on {like.device}")
        args += (ws.data_ptr(), ws.numel())
    if _current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        _native.check(status, name)


def _workspace(fn, prob, device):
    n = ctypes.c_size_t(0)
    _native.check(getattr(_native.lib(), fn)(_byref(prob), _byref(n)), fn)
    ws = torch.empty(max(256, int(n.value)), dtype=torch.uint8, device=device)
    ws[:256].zero_()   # the sticky status word starts clean
    return ws


# ------------------------------------------------------------------------------------------------ rotary positions

def make_rope(rot: int, theta: float = 10000.0, interleaved: bool = False, scaling: str = "none", factor: float = 1.0,
              orig_len: int = 0, low: float = 0.0, high: float = 0.0, mscale: float = 0.0) -> hsa_rope_t:
    """A rotary embedding over the first `rot` elements of each head (hsa_rope_init).  scaling: "none", "linear",
    "ntk", "yarn" or "bands" (include/hsa.h gives each one's formula; orig_len, low and high belong to the last
    two).  Made once per model and kept."""
    if scaling not in _SCALING:
        raise ValueError(f"scaling {scaling!r}: one of {', '.join(_SCALING)}")
    if (rot | orig_len) >> 31:
        _wide(rot=rot, orig_len=orig_len)
    r = hsa_rope_t(rot, int(interleaved), _SCALING[scaling], orig_len, theta, factor, low, high, mscale)
    _native.check(_native.lib().hsa_rope_init(_byref(r)), "hsa_rope_init")
    return r


def rope(r: hsa_rope_t, Q=None, K=None, pos0: int = 0, pos=None, inverse: bool = False, Q_out=None, K_out=None):
    """Rotates Q [B,T,H,d] and/or K [B,T,Hkv,d] in one launch; token t sits at pos0 + t, or at pos[b,t] (int32).
    inverse: the transposed rotation, which takes the gradient of the rotated tensor to the gradient of the
    plain one.  Q_out may be Q (in place), K_out K.  Returns the rotated tensors that were given."""
    x = Q if Q is not None else K
    if x is None:
        raise ValueError("rope needs Q or K")
    _check(x, Q, K, Q_out, K_out)
    B, T, _, d = x.shape
    H, Hkv = x.shape[2], K.shape[2] if K is not None else x.shape[2]
    if Q is not None and K is not None:
        _shape("K", K, (B, T, Hkv, d))
        if H + Hkv > 16383:   # the most that one launch takes
            return (rope(r, Q, None, pos0, pos, inverse, Q_out), rope(r, None, K, pos0, pos, inverse, None, K_out))
    if pos is not None:
        _ints(x, pos=pos)
        _shape("pos", pos, (B, T))
    if Q is not None and Q_out is None:
        Q_out = torch.empty_like(Q)
    if K is not None and K_out is None:
        K_out = torch.empty_like(K)
    _shape("Q_out", Q_out, Q.shape if Q is not None else ())
    _shape("K_out", K_out, K.shape if K is not None else ())
    if pos0 >> 63:
        _wide(pos0=pos0)
    prob = hsa_window_t(B, T, 0, H, Hkv, d, pos0, 0, 0, 0.0, _dtype(x), 0, 0)
    _call("hsa_rope", x, _byref(r), _byref(prob), _p(pos), int(inverse), _p(Q), _p(K), _p(Q_out), _p(K_out))
    if Q is not None and K is not None:
        return Q_out, K_out
    return Q_out if Q is not None else K_out


# ------------------------------------------------------------------------------------------------ window

def _window(Q, K, window, sinks, q_pos0, kv_len, scale, force_simt):
    B, Tq, H, d = Q.shape
    if K.dim() != 4 or K.shape[0] != B or K.shape[3] != d:
        raise ValueError(f"K is {tuple(K.shape)}, expected ({B}, Tcap, Hkv, {d})")
    Tcap, Hkv = K.shape[1], K.shape[2]
    if kv_len is None:
        kv_len = Tcap
    if (window | sinks | kv_len) >> 31 or q_pos0 >> 63:
        _wide(window=window, sinks=sinks, kv_len=kv_len, q_pos0=q_pos0)
    return hsa_window_t(B, Tq, kv_len, H, Hkv, d, q_pos0, window, sinks, scale or 0.0,
                        _dtype(Q), _native.HSA_FLAG_SIMT if force_simt else 0, Tcap)


def window_workspace(Q, K, window, sinks=0, q_pos0=0, kv_len=None, backward=False, force_simt=False) -> torch.Tensor:
    """A workspace for window_attend on these shapes and on every smaller batch or length.  backward: for
    window_backward too, on these shapes alone."""
    prob = _window(Q, K, window, sinks, q_pos0, kv_len, 0.0, force_simt)
    ws = _workspace("hsa_window_workspace_size", prob, Q.device)
    if backward:
        wb = _workspace("hsa_window_backward_workspace_size", prob, Q.device)
        ws = wb if wb.numel() > ws.numel() else ws
    return ws


def window_attend(Q, K, V, window, sinks=0, q_pos0=0, kv_len=None, scale=None, O=None, ws=None, return_lse=False,
                  force_simt=False):
    """Sliding-window attention with sinks: Q [B,Tq,H,d] at positions q_pos0 .. over K, V [B,Tcap,Hkv,d], of which
    the first kv_len tokens are cached (default: all).  window 0: every past key.  scale None or 0: 1 / sqrt(d).
    Returns O, or (O, lse) with return_lse (lse [B,Tq,H] fp32, which window_backward takes).  Rows that see no key are
    zeros, lse -inf.  Without ws a wait that ran out goes unreported (device_status(ws))."""
    _check(Q, K, V, O)
    _shape("V", V, K.shape)
    _shape("O", O, Q.shape)
    prob = _window(Q, K, window, sinks, q_pos0, kv_len, scale, force_simt)
    if O is None:
        O = torch.empty_like(Q)
    if ws is None:
        ws = _workspace("hsa_window_workspace_size", prob, Q.device)
    lse = torch.empty(Q.shape[:3], dtype=torch.float32, device=Q.device) if return_lse else None
    _call("hsa_window_attend", Q, _byref(prob), _p(Q), _p(K), _p(V), _p(O), _p(lse), ws=ws)
    return (O, lse) if return_lse else O


def window_backward(Q, K, V, O, lse, dO, window, sinks=0, q_pos0=0, kv_len=None, scale=None, out=None, ws=None,
                    force_simt=False):
    """Gradients (dQ, dK, dV), in Q's dtype, of window_attend for the output gradient dO; O and lse as it
    returned them.  out: optional preallocated (dQ, dK, dV), overwritten.  Without ws a wait that ran out goes
    unreported (device_status(ws))."""
    dQ, dK, dV = out if out is not None else (torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V))
    _check(Q, K, V, O, dO, dQ, dK, dV)
    _shape("V", V, K.shape)
    for name, t, like in (("O", O, Q), ("dO", dO, Q), ("dQ", dQ, Q), ("dK", dK, K), ("dV", dV, K)):
        _shape(name, t, like.shape)
    _shape("lse", lse, Q.shape[:3])
    if lse.dtype != torch.float32 or lse.device != Q.device or not lse.is_contiguous():
        raise ValueError("lse must be the contiguous fp32 tensor that window_attend returned")
    prob = _window(Q, K, window, sinks, q_pos0, kv_len, scale, force_simt)
    if ws is None:
        ws = _workspace("hsa_window_backward_workspace_size", prob, Q.device)
    _call("hsa_window_backward", Q, _byref(prob), _p(Q), _p(K), _p(V), _p(O), _p(lse), _p(dO), _p(dQ), _p(dK), _p(dV),
          ws=ws)
    return dQ, dK, dV


# ------------------------------------------------------------------------------------------------ pages

def _paged(H, rows, Kp, table, max_q, max_kv, window, sinks, scale, force_simt):
    npages, page, Hkv, d = Kp.shape
    B, max_pages = table.shape
    if (max_q | max_kv | window | sinks) >> 31:
        _wide(max_q=max_q, max_kv=max_kv, window=window, sinks=sinks)
    return hsa_paged_t(B, rows, max_q, max_kv, H, Hkv, d, page, npages, max_pages, window, sinks, scale or 0.0,
                       _dtype(Kp), _native.HSA_FLAG_SIMT if force_simt else 0)


def paged_workspace(Q, K_pages, table, max_q=None, max_kv=0, window=0, sinks=0, force_simt=False) -> torch.Tensor:
    """A workspace for paged_append and paged_attend on these shapes and bounds and on all smaller ones: a server's
    largest batch's serves the others (one call at a time)."""
    prob = _paged(Q.shape[1], Q.shape[0], K_pages, table, Q.shape[0] if max_q is None else max_q, max_kv, window,
                  sinks, 0.0, force_simt)
    return _workspace("hsa_paged_workspace_size", prob, Q.device)


def paged_append(k_new, v_new, K_pages, V_pages, q_start, kv_len, table, Q=None, rope=None, Q_out=None, ws=None):
    """Writes the new tokens' k_new, v_new [rows,Hkv,d] into their pages of K_pages, V_pages [npages,page,Hkv,d]:
    sequence b owns rows q_start[b] .. q_start[b+1] - 1 and kv_len[b] counts its cached tokens with them; token u
    lies in page table[b, u // page] (q_start [B+1], kv_len [B], table [B,max_pages] int32 on the device).  With
    rope (make_rope) K is rotated to its position on the way, and Q [rows,H,d] too.  Returns Q_out (Q rotated; a
    new tensor unless given; rows behind the last sequence are not written), or None without Q.  Without ws a page number
    or length outside its bounds, whose write is skipped, goes unreported (device_status(ws))."""
    _check(k_new, v_new, K_pages, V_pages, Q, Q_out)
    _ints(k_new, q_start=q_start, kv_len=kv_len, table=table)
    rows, Hkv, d = k_new.shape
    if Q is None and Q_out is not None:
        raise ValueError("Q_out without Q")
    npages, page, B = K_pages.shape[0], K_pages.shape[1], table.shape[0]
    _shape("v_new", v_new, k_new.shape)
    _shape("K_pages", K_pages, (npages, page, Hkv, d))
    _shape("V_pages", V_pages, K_pages.shape)
    _shape("q_start", q_start, (B + 1,))
    _shape("kv_len", kv_len, (B,))
    H = Hkv
    if Q is not None:
        H = Q.shape[1]
        _shape("Q", Q, (rows, H, d))
        if Q_out is None:
            Q_out = torch.empty_like(Q)
        _shape("Q_out", Q_out, Q.shape)
    prob = _paged(H, rows, K_pages, table, rows, 0, 0, 0, 0.0, False)
    if ws is None:
        ws = torch.zeros(256, dtype=torch.uint8, device=k_new.device)
    _call("hsa_paged_append", k_new, _byref(prob), None if rope is None else _byref(rope), _p(k_new), _p(v_new), _p(Q),
          _p(Q_out), _p(q_start), _p(kv_len), _p(table), _p(K_pages), _p(V_pages), ws=ws)
    return Q_out if Q is not None else None


def paged_attend(Q, K_pages, V_pages, q_start, kv_len, table, max_q=None, max_kv=0, window=0, sinks=0, scale=None,
                 O=None, ws=None, force_simt=False):
    """Attention of the new tokens Q [rows,H,d] over the pages (which hold them already: paged_append first), with
    window and sinks as in window_attend.  max_q, max_kv: the most new and cached tokens of one sequence (defaults:
    rows, and what a table row can hold); the closer they are, the better the work is split.  scale None or 0:
    1 / sqrt(d).  Returns O; rows behind the last sequence are not written.  Without ws a page number outside the pool
    (zeros in its place), a length outside its bounds (cut to them) and a wait that ran out go unreported
    (device_status(ws))."""
    _check(Q, K_pages, V_pages, O)
    _ints(Q, q_start=q_start, kv_len=kv_len, table=table)
    rows, H, d = Q.shape
    B = table.shape[0]
    _shape("V_pages", V_pages, K_pages.shape)
    _shape("q_start", q_start, (B + 1,))
    _shape("kv_len", kv_len, (B,))
    _shape("O", O, Q.shape)
    if K_pages.shape[3] != d:
        raise ValueError(f"K_pages hold heads of {K_pages.shape[3]}, Q of {d}")
    prob = _paged(H, rows, K_pages, table, rows if max_q is None else max_q, max_kv, window, sinks, scale, force_simt)
    if O is None:
        O = torch.empty_like(Q)
    if ws is None:
        ws = _workspace("hsa_paged_workspace_size", prob, Q.device)
    _call("hsa_paged_attend", Q, _byref(prob), _p(Q), _p(K_pages), _p(V_pages), _p(q_start), _p(kv_len), _p(table),
          _p(O), ws=ws)
    return O
