"""Local attention on the host: hsa_rope_init against its formulas, and every refusal of the
entry points (an invalid call launches nothing, so no GPU is needed)."""
import ctypes
import math
import os
import random
import subprocess
import sys

import pytest
import torch

import landmark_guided_chunk_b200 as hsa
from landmark_guided_chunk_b200 import _native, local
from landmark_guided_chunk_b200._native import hsa_paged_t, hsa_rope_t, hsa_window_t
from tests.local_ref import inv_freq

INVALID, UNSUPPORTED, WORKSPACE = (_native.HSA_ERR_INVALID_ARG, _native.HSA_ERR_UNSUPPORTED,
                                   _native.HSA_ERR_WORKSPACE)
PTR = 1 << 20      # never followed: the calls below are refused first
BIG = 1 << 60


def _window(**kw):
    base = dict(B=2, Tq=100, Tkv=100, H=8, Hkv=2, d=128, q_pos0=0, window=10, sinks=2, scale=0.0, dtype=1, flags=0,
                kv_cap=0)
    base.update(kw)
    return hsa_window_t(**base)


def _paged(**kw):
    base = dict(B=2, rows=10, max_q=5, max_kv=0, H=8, Hkv=2, d=128, page=16, npages=9, max_pages=4, window=0, sinks=0,
                scale=0.0, dtype=1, flags=0)
    base.update(kw)
    return hsa_paged_t(**base)


COMMON = [(dict(H=7), INVALID), (dict(H=0), INVALID), (dict(Hkv=0), INVALID), (dict(B=-1), INVALID),
          (dict(dtype=2), INVALID), (dict(flags=1), INVALID), (dict(flags=64), INVALID),
          (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
          (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
          (dict(H=34), UNSUPPORTED), (dict(B=65536), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(Tq=-1), INVALID), (dict(Tkv=-1), INVALID), (dict(q_pos0=-1), INVALID), (dict(kv_cap=99), INVALID),
    (dict(q_pos0=1 << 30), UNSUPPORTED), (dict(q_pos0=1 << 40), UNSUPPORTED), (dict(kv_cap=(1 << 30) + 1), UNSUPPORTED),
    (dict(B=2048, kv_cap=1 << 20), UNSUPPORTED), (dict(B=2048, Tq=1 << 20), UNSUPPORTED)])
def test_window_refusals(kw, status):
    L = _native.lib()
    n = ctypes.c_size_t(77)
    p = ctypes.byref(_window(**kw))
    assert L.hsa_window_workspace_size(p, ctypes.byref(n)) == status
    assert L.hsa_window_backward_workspace_size(p, ctypes.byref(n)) == status
    assert n.value == 77 and L.hsa_last_error()
    assert L.hsa_window_attend(p, PTR, PTR, PTR, PTR, None, PTR, BIG, None) == status
    assert L.hsa_window_backward(p, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, BIG, None) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(rows=-1), INVALID), (dict(max_q=-1), INVALID), (dict(max_kv=-1), INVALID), (dict(max_kv=65), INVALID),
    (dict(npages=0), INVALID), (dict(max_pages=0), INVALID), (dict(page=0), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
    (dict(page=256), UNSUPPORTED), (dict(npages=1 << 28), UNSUPPORTED), (dict(max_pages=1 << 27), UNSUPPORTED)])
def test_paged_refusals(kw, status):
    L = _native.lib()
    n = ctypes.c_size_t(77)
    p = ctypes.byref(_paged(**kw))
    assert L.hsa_paged_workspace_size(p, ctypes.byref(n)) == status
    assert n.value == 77
    assert L.hsa_paged_attend(p, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, BIG, None) == status
    assert L.hsa_paged_append(p, None, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, BIG, None) == status


@pytest.mark.parametrize("q_pos0", [(1 << 30) - 99, 1 << 62, (1 << 63) - 1, (1 << 63) - 100])
def test_positions_up_to_the_last_64_bit_one_are_refused(q_pos0):
    """100 rows from q_pos0 pass 2^30, however their sum is stored (one row less at 2^30 - 99 would fit)."""
    L = _native.lib()
    n = ctypes.c_size_t(77)
    p = ctypes.byref(_window(q_pos0=q_pos0))
    assert L.hsa_window_workspace_size(p, ctypes.byref(n)) == UNSUPPORTED
    assert L.hsa_window_backward_workspace_size(p, ctypes.byref(n)) == UNSUPPORTED and n.value == 77
    assert L.hsa_window_attend(p, PTR, PTR, PTR, PTR, None, PTR, BIG, None) == UNSUPPORTED
    assert L.hsa_window_backward(p, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, BIG, None) == UNSUPPORTED
    r = hsa.make_rope(64)
    assert L.hsa_rope(ctypes.byref(r), p, None, 0, PTR, PTR, PTR, PTR, None) == UNSUPPORTED
    assert L.hsa_window_workspace_size(ctypes.byref(_window(q_pos0=(1 << 30) - 100)), ctypes.byref(n)) == 0


def _bytes(prob):
    n = ctypes.c_size_t()
    f = _native.lib().hsa_paged_workspace_size if isinstance(prob, hsa_paged_t) else _native.lib().hsa_window_workspace_size
    assert f(ctypes.byref(prob), ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("dtype,flags", [(1, 0), (0, 0), (1, _native.HSA_FLAG_SIMT)])
def test_a_workspace_serves_every_smaller_batch(dtype, flags):
    """A server sizes its workspace for the largest batch; smaller ones, which are split more, must fit it."""
    rng = random.Random(1)

    def size(hi):
        return min(hi, int(2 ** rng.uniform(0, math.log2(hi + 1))))

    partials = 0
    for _ in range(4000):
        Hkv, G, d = rng.choice([1, 2, 3, 8, 19, 32, 150, 300]), rng.choice([1, 3, 4, 5, 8, 16]), rng.choice([64, 128])
        win = rng.choice([0, 0, 100, 5000])
        same = dict(H=Hkv * G, Hkv=Hkv, d=d, dtype=dtype, flags=flags, window=win, sinks=rng.choice([0, 4, 3000]) if win else 0)
        big = dict(B=size(80), max_q=size(20000), max_kv=size(1 << 22))
        big["rows"] = big["max_q"] + size(100000)
        small = {k: rng.choice([v, size(v)]) for k, v in big.items()}
        paged = [_bytes(_paged(max_pages=1 << 19, **same, **x)) for x in (big, small)]
        window = [_bytes(_window(B=x["B"], Tq=x["max_q"], Tkv=x["max_kv"], q_pos0=0, **same)) for x in (big, small)]
        assert paged[1] <= paged[0], (same, big, small)
        assert window[1] <= window[0], (same, big, small)
        assert max(paged + window) < 64 << 20      # 148 CTAs' partials of two row tiles, or 296 blocks of 32 rows
        partials += paged[1] > 256
    assert partials > 400


def test_workspaces_of_batches_of_a_server():
    """32 + 8 heads of 128, pages of 64, up to 32768 keys: 32 sequences of up to 2048 new tokens down to single ones."""
    same = dict(H=32, Hkv=8, d=128, page=64, npages=20000, max_pages=512, max_kv=32768)
    n = [_bytes(_paged(B=B, rows=B * q, max_q=q, **same)) for B, q in ((32, 2048), (32, 512), (8, 512), (8, 1), (1, 1))]
    assert n == sorted(n, reverse=True)


def _each(fn, args, optional=()):
    """The call with each pointer missing, then misaligned, in turn."""
    for i, a in enumerate(args):
        if a != PTR:
            continue
        for bad in ((None,) if i not in optional else ()) + (PTR + 2,):
            yield i, bad, fn(*(bad if j == i else x for j, x in enumerate(args)))


def test_pointers_and_workspaces():
    L = _native.lib()
    p, g = ctypes.byref(_window()), ctypes.byref(_paged())
    r = hsa.make_rope(64)
    for i, bad, got in _each(L.hsa_window_attend, (p, PTR, PTR, PTR, PTR, PTR, None, BIG, None), optional=(5,)):
        assert got == INVALID, (i, bad)
    for i, bad, got in _each(L.hsa_window_backward, (p,) + (PTR,) * 9 + (None, BIG, None)):
        assert got == INVALID, (i, bad)
    for i, bad, got in _each(L.hsa_paged_attend, (g,) + (PTR,) * 7 + (None, BIG, None)):
        assert got == INVALID, (i, bad)
    args = (g, ctypes.byref(r), PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, None, BIG, None)
    for i, bad, got in _each(L.hsa_paged_append, args, optional=(4,)):
        assert got == INVALID, (i, bad)
    for i, bad, got in _each(L.hsa_rope, (ctypes.byref(r), p, PTR, 0, PTR, PTR, PTR, PTR, None), optional=(2, 4, 5)):
        assert got == INVALID, (i, bad)
    assert L.hsa_rope(ctypes.byref(r), p, None, 0, None, None, PTR, PTR, None) == INVALID
    n = ctypes.c_size_t()
    small = ctypes.byref(_window(B=1, Tq=1, Tkv=90000, q_pos0=89999, window=0))
    for call, prob, size in ((L.hsa_window_attend, small, L.hsa_window_workspace_size),
                             (L.hsa_window_backward, p, L.hsa_window_backward_workspace_size)):
        assert size(prob, ctypes.byref(n)) == 0 and n.value >= 256
        k = 5 if call is L.hsa_window_attend else 9
        assert call(prob, *(PTR,) * k, PTR, n.value - 1, None) == WORKSPACE
        assert call(prob, *(PTR,) * k, None, n.value, None) == WORKSPACE
        assert call(prob, *(PTR,) * k, PTR + 16, n.value, None) == WORKSPACE
    assert L.hsa_paged_append(g, None, *(PTR,) * 9, PTR, 255, None) == WORKSPACE
    for f in (L.hsa_window_workspace_size, L.hsa_window_backward_workspace_size):
        assert f(None, ctypes.byref(n)) == INVALID and f(p, None) == INVALID
    assert L.hsa_paged_workspace_size(None, ctypes.byref(n)) == INVALID
    assert L.hsa_paged_workspace_size(g, None) == INVALID


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=16.0, orig_len=4096),
                                dict(scaling="bands", factor=8.0, orig_len=8192, theta=5e5),
                                dict(scaling="yarn", factor=4.0, orig_len=2048, low=2.0, high=20.0)])
@pytest.mark.parametrize("rot", [4, 20, 64, 128])
def test_rope_frequencies(rot, kw):
    r = hsa.make_rope(rot, **kw)
    f, m = inv_freq(rot, **kw)
    got = torch.tensor(list(r.inv_freq), dtype=torch.float64)
    # a handful of 64-bit operations on each side
    assert float(((got[:rot // 2] - f) / f).abs().max()) < 64 * 2.0 ** -53
    assert not bool(got[rot // 2:].any())
    assert abs(r.mult - m) < 1e-14
    assert hsa.make_rope(rot, mscale=0.7, **kw).mult == 0.7


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=3), dict(rot=130), dict(theta=1.0), dict(theta=math.nan),
                                dict(theta=math.inf), dict(factor=0.5), dict(factor=math.nan), dict(factor=math.inf),
                                dict(scaling="yarn"), dict(scaling="bands"), dict(scaling="ntk", rot=2, factor=2.0),
                                dict(scaling="yarn", orig_len=64, low=3.0, high=3.0), dict(mscale=-1.0),
                                dict(scaling="bands", orig_len=64, low=-1.0, high=3.0), dict(mscale=math.inf)])
def test_rope_refusals(kw):
    with pytest.raises(hsa.HSAError) as e:
        hsa.make_rope(**{**dict(rot=64), **kw})
    assert e.value.status == INVALID


def test_rope_call_refusals():
    L = _native.lib()
    p = ctypes.byref(_window(d=64, H=4, Hkv=2))
    assert L.hsa_rope_init(None) == INVALID
    for r in (hsa.make_rope(128), hsa_rope_t()):       # wider than the head; never set up
        assert L.hsa_rope(ctypes.byref(r), p, None, 0, PTR, PTR, PTR, PTR, None) == INVALID
    r = ctypes.byref(hsa.make_rope(64))
    wide = ctypes.byref(_window(d=64, H=16000, Hkv=1000))
    assert L.hsa_rope(r, wide, None, 0, PTR, PTR, PTR, PTR, None) == UNSUPPORTED
    wide = ctypes.byref(_paged(d=64, H=16000, Hkv=1000))
    assert L.hsa_paged_append(wide, r, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, BIG, None) == UNSUPPORTED
    assert L.hsa_rope(None, p, None, 0, PTR, PTR, PTR, PTR, None) == INVALID
    assert L.hsa_rope(r, None, None, 0, PTR, PTR, PTR, PTR, None) == INVALID
    bad = hsa_rope_t(64, 0, 9, 0, 1e4, 1.0)
    assert L.hsa_rope_init(ctypes.byref(bad)) == INVALID
    bad = hsa_rope_t(64, 2, 0, 0, 1e4, 1.0)
    assert L.hsa_rope_init(ctypes.byref(bad)) == INVALID
    with pytest.raises(ValueError):
        hsa.make_rope(64, scaling="other")


def test_rope_takes_any_two_head_counts():
    """The rotation has no group: any H and Hkv, up to the heads of a launch (nothing is launched without rows)."""
    L = _native.lib()
    r = ctypes.byref(hsa.make_rope(64))
    for H, Hkv in ((32, 1), (5, 2), (2, 7), (1, 1), (16000, 383)):
        p = ctypes.byref(_window(H=H, Hkv=Hkv, Tq=0))
        assert L.hsa_rope(r, p, None, 0, PTR, PTR, PTR, PTR, None) == 0, (H, Hkv)
    top = 2 ** 31 - 1
    for H, Hkv, status in ((16000, 384, UNSUPPORTED), (top, top, UNSUPPORTED), (top, 1, UNSUPPORTED), (0, 4, INVALID),
                           (4, 0, INVALID), (-1, 4, INVALID)):
        p = ctypes.byref(_window(H=H, Hkv=Hkv, Tq=3))
        assert L.hsa_rope(r, p, None, 0, PTR, PTR, PTR, PTR, None) == status, (H, Hkv)


def test_binding_refusals():
    x = torch.zeros(1, 4, 2, 64)
    for call in (lambda: hsa.window_attend(x, x, x, 3), lambda: hsa.rope(hsa.make_rope(64), x),
                 lambda: hsa.window_backward(x, x, x, x, x, x, 3), lambda: hsa.rope(hsa.make_rope(64))):
        with pytest.raises(ValueError):
            call()
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        hsa.paged_attend(x[0], x, x, i, i[:1], i[None])
    with pytest.raises(ValueError):
        hsa.paged_append(x[0], x[0], x, x, i, i[:1], i[None])


@pytest.fixture
def calls(monkeypatch):
    """The binding with its device checks open to CPU tensors, and its library calls recorded in place of made."""
    made = []

    class Library(dict):
        def get(self, name):
            return lambda *a: made.append((name, a))

    monkeypatch.setattr(local, "_check", lambda *a: None)
    monkeypatch.setattr(local, "_fns", Library())
    monkeypatch.setattr(local, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(local, "_current_device", lambda: 0)
    return made


class _OnDevice(torch.Tensor):
    """A CPU tensor that says it is on device 0, for checks that must not follow its pointer."""

    def get_device(self):
        return 0


def _tensors():
    return (torch.zeros(s, dtype=t).as_subclass(_OnDevice) for s, t in (((1, 16, 2, 64), torch.float32), ((2,), torch.int32)))


def _five(x, i, ws=None, pos0=0, **kw):
    """The calls that take device data, on x as every tensor and i as every index array."""
    p, l = x[0], torch.zeros(x.shape[:3])
    ws = torch.zeros(1 << 20, dtype=torch.uint8).as_subclass(_OnDevice) if ws is None else ws
    w = {"window": 3, **{k: v for k, v in kw.items() if k in ("window", "sinks", "q_pos0", "kv_len")}}
    g = {k: v for k, v in kw.items() if k in ("window", "sinks", "max_q", "max_kv")}
    return {"window_attend": lambda: hsa.window_attend(x, x, x, ws=ws, **w),
            "window_backward": lambda: hsa.window_backward(x, x, x, x, l, x, ws=ws, **w),
            "paged_attend": lambda: hsa.paged_attend(p, x, x, i[:2], i[:1], i[None], ws=ws, **g),
            "paged_append": lambda: hsa.paged_append(p, p, x, x, i[:2], i[:1], i[None], ws=ws),
            "rope": lambda: hsa.rope(hsa.make_rope(64), x, pos0=pos0)}


@pytest.mark.parametrize("name,value", [(n, v) for n in ("window", "sinks", "kv_len", "max_q", "max_kv")
                                        for v in (2 ** 31, 2 ** 32 + 4, -2 ** 31 - 1)] +
                         [(n, v) for n in ("q_pos0", "pos0") for v in (2 ** 63, 2 ** 64 + 4, -2 ** 63 - 1)])
def test_binding_integers_are_not_cut_to_their_fields(calls, name, value):
    """2^32 + 4 in a 32-bit field would be 4: a window of four tokens in place of all."""
    x, i = _tensors()
    takes = {"window": 3, "sinks": 3, "kv_len": 2, "q_pos0": 2, "max_q": 1, "max_kv": 1, "pos0": 1}[name]
    refused = 0
    for call in _five(x, i, **{name: value}).values():
        try:
            call()
        except ValueError as e:
            assert name in str(e)
            refused += 1
    assert refused == takes and len(calls) == 5 - takes
    if name in ("window", "sinks", "kv_len", "q_pos0"):
        with pytest.raises(ValueError, match=name):
            hsa.window_workspace(x, x, **{"window": 3, name: value})
    if name in ("window", "sinks", "max_q", "max_kv"):
        with pytest.raises(ValueError, match=name):
            hsa.paged_workspace(x[0], x, i[None], **{name: value})


def test_binding_integers_at_the_ends_of_their_fields(calls):
    x, i = _tensors()
    for call in _five(x, i, window=2 ** 31 - 1, sinks=2 ** 31 - 1, pos0=2 ** 63 - 1).values():
        call()
    assert len(calls) == 5
    with pytest.raises(hsa.HSAError):       # negative ones are the library's to refuse
        hsa.window_workspace(x, x, -1)
    for kw in (dict(rot=2 ** 32 + 64), dict(rot=64, orig_len=2 ** 32 + 64)):
        with pytest.raises(ValueError):
            hsa.make_rope(**kw)


def test_binding_refuses_an_output_without_its_input(calls):
    x, i = _tensors()
    with pytest.raises(ValueError, match="Q_out"):
        hsa.paged_append(x[0], x[0], x, x, i[:2], i[:1], i[None], Q_out=x[0])
    for kw in (dict(Q=x, K_out=x), dict(K=x, Q_out=x)):
        with pytest.raises(ValueError, match="_out"):
            hsa.rope(hsa.make_rope(64), **kw)
    assert not calls


@pytest.mark.parametrize("ws", [torch.zeros(1 << 20, dtype=torch.uint8),
                                torch.zeros(1 << 21, dtype=torch.uint8)[::2].as_subclass(_OnDevice)], ids=["cpu", "strided"])
def test_binding_workspaces(calls, ws):
    """A workspace on the host, or a strided view, must not reach a kernel as a pointer."""
    x, i = _tensors()
    for name, call in _five(x, i, ws=ws).items():
        if name != "rope":
            with pytest.raises(ValueError, match="ws"):
                call()
    assert not calls
    for call in _five(x, i).values():
        call()
    assert len(calls) == 5


def test_the_package_imports_on_a_torch_without_cuda():
    """build.py, inputs, dp and sharded are for machines without a GPU as well."""
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import landmark_guided_chunk_b200 as hsa
from landmark_guided_chunk_b200 import build, dp, inputs, sharded
x = torch.zeros(1, 4, 2, 64)
try:
    hsa.window_attend(x, x, x, 3)
except ValueError as e:
    print("refused:", e)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused: all tensors must be CUDA tensors" in r.stdout, r.stderr[-2000:]


def test_nothing_to_do_needs_no_pointers():
    L = _native.lib()
    ws = (ctypes.c_char * 1024)()
    at = (ctypes.addressof(ws) + 255) & ~255
    for kw in (dict(B=0), dict(Tq=0)):
        p = ctypes.byref(_window(**kw))
        assert L.hsa_window_attend(p, None, None, None, None, None, at, 512, None) == 0
        assert L.hsa_rope(ctypes.byref(hsa.make_rope(64)), p, None, 0, None, None, None, None, None) == 0
    g = ctypes.byref(_paged(rows=0))
    assert L.hsa_paged_attend(g, *(None,) * 7, at, 512, None) == 0
    assert L.hsa_paged_append(g, None, *(None,) * 9, at, 512, None) == 0
