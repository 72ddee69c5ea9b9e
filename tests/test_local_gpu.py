"""Local attention on the GPU against its 64-bit restatement (tests/local_ref.py, which
derives the bounds): sliding window with sinks, its gradients, rotary positions, and the
paged cache, at the sizes and masks where they can go wrong."""
import math

import pytest
import torch

import landmark_guided_chunk_b200 as hsa
from tests.local_ref import Ref, check, seen, turn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _rand(seed, dt, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


def _clean(ws):
    hsa.device_status(ws)


def _forward(dt, d, H, Hkv, B, Tq, Tkv, cap, pos0, window, sinks, scale=None, simt=False, seed=0, poison=True):
    Q, K, V = _rand(seed, dt, B, Tq, H, d), _rand(seed + 1, dt, B, cap, Hkv, d), _rand(seed + 2, dt, B, cap, Hkv, d)
    p = torch.arange(pos0, pos0 + Tq, device="cuda")
    if poison and cap:      # what no query sees holds NaN and infinities
        live = seen(p, cap, Tkv, window, sinks).any(0) if Tq else torch.zeros(cap, dtype=torch.bool, device="cuda")
        K[:, ~live] = math.nan
        V[:, ~live] = math.inf
    ws = hsa.window_workspace(Q, K, window, sinks, q_pos0=pos0, kv_len=Tkv, force_simt=simt)
    ws[256:] = 0xFF         # NaN in every fp32 word: the scratch holds nothing that counts
    O = torch.full_like(Q, math.nan)
    O, lse = hsa.window_attend(Q, K, V, window, sinks, q_pos0=pos0, kv_len=Tkv, scale=scale, O=O, ws=ws,
                               return_lse=True, force_simt=simt)
    _clean(ws)
    for b in range(B):
        r = Ref(Q[b], K[b], V[b], p, Tkv, window, sinks, scale)
        check(f"O[{b}]", O[b], r.O, r.tO)
        check(f"lse[{b}]", lse[b], r.lse, r.tlse)
    O2 = hsa.window_attend(Q, K, V, window, sinks, q_pos0=pos0, kv_len=Tkv, scale=scale, ws=ws, force_simt=simt)
    assert torch.equal(O, O2), "equal calls differ"


# window, sinks: none, smallest, around the tile sizes, sinks that end inside and beyond a tile
MASKS = [(0, 0), (1, 0), (1, 3), (2, 1), (63, 64), (64, 5), (65, 0), (128, 4), (200, 130), (1000, 4)]


@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("dt,d", [(BF, 128), (BF, 64), (F32, 64), (F32, 128)])
def test_window_prompt(dt, d, window, sinks):
    _forward(dt, d, 8, 2, 2, 517, 517, 517, 0, window, sinks)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 300])
@pytest.mark.parametrize("dt", [BF, F32])
def test_window_lengths(dt, T):
    _forward(dt, 64, 4, 2, 2, T, T, T, 0, 50, 3)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 3), (6, 2), (5, 1), (7, 1), (16, 2), (16, 1), (11, 1), (48, 3)])
@pytest.mark.parametrize("Tq,past", [(200, 0), (1, 700), (9, 300)])
def test_window_heads(H, Hkv, Tq, past):
    _forward(BF, 128, H, Hkv, 1, Tq, past + Tq, past + Tq, past, 90, 2)
    _forward(F32, 64, H, Hkv, 1, Tq, past + Tq, past + Tq, past, 0, 0)


@pytest.mark.parametrize("Tq", [1, 2, 3, 4, 8, 31, 100])
@pytest.mark.parametrize("past", [0, 1, 63, 64, 127, 1000, 4321])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4), (700, 64), (1, 1)])
def test_window_tokens_over_a_cache(Tq, past, window, sinks):
    n = Tq + past
    _forward(BF, 128, 8, 2, 2, Tq, n, n + 5, past, window, sinks)
    _forward(F32 if Tq < 9 else BF, 64, 4, 1, 1, Tq, n, n + 70, past, window, sinks)


@pytest.mark.parametrize("B", [1, 9, 40, 160])
def test_window_many_items(B):
    """Several items per CTA, some with one row tile and some with two, shared between CTAs or whole."""
    _forward(BF, 64, 16, 8, B, 130, 130, 131, 0, 40, 2)
    _forward(BF, 128, 8, 8, B, 150, 450, 450, 300, 0, 0)


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
def test_window_rows_that_see_nothing(dt, simt):
    # the cache ends before the window begins: only sinks, or nothing, is left
    _forward(dt, 64, 4, 2, 1, 40, 30, 30, 45, 10, 0, simt=simt)
    _forward(dt, 64, 4, 2, 1, 40, 30, 30, 25, 10, 0, simt=simt)
    _forward(dt, 64, 4, 2, 1, 40, 30, 30, 400, 10, 3, simt=simt)
    _forward(dt, 128, 8, 1, 2, 1, 0, 0, 0, 0, 0, simt=simt)
    _forward(dt, 128, 8, 1, 2, 150, 0, 7, 3, 5, 2, simt=simt)


@pytest.mark.parametrize("dt", [BF, F32])
def test_window_simt_flag_and_scale(dt):
    _forward(dt, 128, 8, 2, 2, 333, 333, 340, 0, 77, 5, simt=True)
    _forward(dt, 64, 8, 2, 2, 130, 333, 340, 203, 77, 5, scale=0.31, simt=True)
    _forward(dt, 64, 8, 2, 1, 130, 333, 340, 203, 77, 5, scale=0.31)
    _forward(dt, 128, 8, 2, 1, 1, 333, 340, 332, 77, 5, scale=0.5)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("Tq", [1, 300])
def test_window_large_and_equal_scores(dt, Tq):
    """Scores of several hundred (a running maximum that moves far), and all-equal ones."""
    d, H, Hkv, n = 64, 4, 2, 300
    Q, K, V = _rand(1, dt, 1, Tq, H, d), _rand(2, dt, 1, n, Hkv, d), _rand(3, dt, 1, n, Hkv, d)
    p = torch.arange(n - Tq, n, device="cuda")
    for Qx, Kx in ((Q * 16, K * torch.linspace(0, 4, n, device="cuda")[None, :, None, None]), (Q * 0, K),
                   (Q.abs() * 8, -K.abs() * 8)):
        Qx, Kx = Qx.to(dt), Kx.to(dt)
        O, lse = hsa.window_attend(Qx, Kx, V, 120, 3, q_pos0=n - Tq, return_lse=True)
        r = Ref(Qx[0], Kx[0], V[0], p, n, 120, 3)
        check("O", O[0], r.O, r.tO)
        check("lse", lse[0], r.lse, r.tlse)


def test_window_far_rows():
    """Offsets beyond 2^31 elements in the cache: the last sequence of a cache of 2.6 G elements."""
    B, cap, Hkv, d = 5, 65536 * 8, 8, 128
    K = torch.empty(B, cap, Hkv, d, dtype=BF, device="cuda")
    V = torch.empty_like(K)
    assert K.numel() > 2 ** 31
    n = cap - 3
    w = 300
    K[:, n - w - 200:] = _rand(1, BF, B, w + 203, Hkv, d)
    V[:, n - w - 200:] = _rand(2, BF, B, w + 203, Hkv, d)
    K[:, :8], V[:, :8] = _rand(3, BF, B, 8, Hkv, d), _rand(4, BF, B, 8, Hkv, d)
    for Tq in (1, 150):
        Q = _rand(5, BF, B, Tq, 8, d)
        O = hsa.window_attend(Q, K, V, w, 5, q_pos0=n - Tq, kv_len=n)
        for b in (0, B - 1):
            # the same visible keys in a short cache: sinks, then the window, with positions moved down
            cut = n - Tq - w - 16
            Ks, Vs = torch.cat((K[b, :5], K[b, cut:n])), torch.cat((V[b, :5], V[b, cut:n]))
            p = torch.arange(n - Tq, n, device="cuda") - cut + 5
            r = Ref(Q[b], Ks, Vs, p, Ks.shape[0], w, 5)
            check(f"O[{b}]", O[b], r.O, r.tO)


# ------------------------------------------------------------------------------------------------ gradients

def _backward(dt, d, H, Hkv, B, Tq, Tkv, cap, pos0, window, sinks, scale=None, simt=False, seed=0):
    Q, K, V = _rand(seed, dt, B, Tq, H, d), _rand(seed + 1, dt, B, cap, Hkv, d), _rand(seed + 2, dt, B, cap, Hkv, d)
    dO = _rand(seed + 3, dt, B, Tq, H, d)
    p = torch.arange(pos0, pos0 + Tq, device="cuda")
    live = seen(p, cap, Tkv, window, sinks).any(0)
    K[:, ~live] = math.nan
    V[:, ~live] = math.nan
    ws = hsa.window_workspace(Q, K, window, sinks, q_pos0=pos0, kv_len=Tkv, backward=True, force_simt=simt)
    ws[256:] = 0xFF
    kw = dict(q_pos0=pos0, kv_len=Tkv, scale=scale, ws=ws, force_simt=simt)
    O, lse = hsa.window_attend(Q, K, V, window, sinks, return_lse=True, **kw)
    out = tuple(torch.full_like(x, math.nan) for x in (Q, K, V))
    dQ, dK, dV = hsa.window_backward(Q, K, V, O, lse, dO, window, sinks, out=out, **kw)
    _clean(ws)
    for b in range(B):
        r = Ref(Q[b], K[b], V[b], p, Tkv, window, sinks, scale, dO[b])
        check(f"dQ[{b}]", dQ[b], r.dQ, r.tdQ)
        check(f"dK[{b}]", dK[b], r.dK, r.tdK)
        check(f"dV[{b}]", dV[b], r.dV, r.tdV)
    again = hsa.window_backward(Q, K, V, O, lse, dO, window, sinks, **kw)
    assert all(torch.equal(x, y) for x, y in zip((dQ, dK, dV), again)), "equal calls differ"


@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("dt,d", [(BF, 128), (BF, 64), (F32, 64), (F32, 128)])
def test_window_backward(dt, d, window, sinks):
    _backward(dt, d, 8, 2, 2, 517, 517, 517, 0, window, sinks)


@pytest.mark.parametrize("T", [1, 2, 31, 64, 65, 127, 128, 129, 257])
@pytest.mark.parametrize("dt", [BF, F32])
def test_window_backward_lengths(dt, T):
    _backward(dt, 64, 4, 2, 2, T, T, T + 3, 0, 40, 3)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (6, 2), (5, 1), (7, 1), (16, 1), (22, 2)])
def test_window_backward_heads(H, Hkv):
    _backward(BF, 128, H, Hkv, 1, 260, 260, 260, 0, 90, 2)
    _backward(F32, 64, H, Hkv, 1, 130, 130, 130, 0, 0, 0)


@pytest.mark.parametrize("dt", [BF, F32])
def test_window_backward_of_a_chunk(dt):
    _backward(dt, 64, 4, 2, 1, 100, 400, 411, 300, 70, 5)      # keys behind the window and past the cache: zeros
    _backward(dt, 128, 4, 1, 2, 3, 200, 200, 197, 0, 0)
    _backward(dt, 64, 4, 2, 1, 40, 30, 30, 25, 10, 0)          # rows that see nothing
    _backward(dt, 64, 4, 2, 1, 40, 30, 33, 400, 10, 3)         # only sinks are seen
    _backward(dt, 128, 8, 2, 1, 300, 300, 300, 0, 50, 300)     # every key is a sink
    _backward(dt, 64, 8, 2, 2, 333, 333, 340, 0, 77, 5, scale=0.2, simt=True)


@pytest.mark.parametrize("B", [1, 9, 40])
def test_window_backward_many_items(B):
    _backward(BF, 64, 16, 8, B, 130, 130, 131, 0, 40, 2)
    _backward(BF, 128, 8, 8, B, 150, 150, 150, 0, 0, 0)


@pytest.mark.parametrize("dt", [BF, F32])
def test_window_backward_far_rows(dt):
    """Gradients of a cache of 2.3 G elements, 2^31 bytes and more per sequence: those of the window's and the sinks'
    tokens, and zeros in between and behind the cached ones."""
    B, cap, Hkv, d, w, S, Tq = 2, 1_100_000, 8, 128, 300, 5, 150
    K = torch.empty(B, cap, Hkv, d, dtype=dt, device="cuda")
    V, dK, dV = torch.empty_like(K), torch.empty_like(K), torch.empty_like(K)
    assert K.numel() > 2 ** 31 and K[0].numel() * K.element_size() > 2 ** 31
    n = cap - 7
    cut = n - Tq - w - 16
    for i, x in enumerate((K, V)):
        x[:, cut:], x[:, :8] = _rand(i, dt, B, cap - cut, Hkv, d), _rand(i + 2, dt, B, 8, Hkv, d)
    dK.fill_(math.nan)
    dV.fill_(math.nan)
    Q, dO = _rand(5, dt, B, Tq, 16, d), _rand(6, dt, B, Tq, 16, d)
    kw = dict(q_pos0=n - Tq, kv_len=n)
    O, lse = hsa.window_attend(Q, K, V, w, S, return_lse=True, **kw)
    dQ, _, _ = hsa.window_backward(Q, K, V, O, lse, dO, w, S, out=(torch.empty_like(Q), dK, dV), **kw)
    p = torch.arange(n - Tq, n, device="cuda") - cut + S
    for b in range(B):
        Ks, Vs = (torch.cat((x[b, :S], x[b, cut:n])) for x in (K, V))
        r = Ref(Q[b], Ks, Vs, p, Ks.shape[0], w, S, None, dO[b])
        check("dQ", dQ[b], r.dQ, r.tdQ)
        for x, want, tol in ((dK, r.dK, r.tdK), (dV, r.dV, r.tdV)):
            check("sinks", x[b, :S], want[:S], tol[:S])
            check("window", x[b, cut:n], want[S:], tol[S:])
            assert not bool(x[b, n:].any()) and not any(bool(y.any()) for y in x[b, S:cut].split(1 << 18))


@pytest.mark.parametrize("d,H,Hkv,T,Tkv,pos0,window,sinks,simt", [
    (64, 4, 2, 70, 70, 0, 1, 0, False), (128, 8, 2, 100, 100, 0, 1, 1, False), (128, 3, 1, 45, 45, 0, 0, 0, False),
    (64, 12, 4, 300, 300, 0, 7, 2, False), (64, 2, 2, 64, 64, 0, 64, 0, False), (128, 32, 2, 65, 200, 133, 33, 31, False),
    (64, 4, 4, 80, 60, 20, 30, 3, False), (64, 4, 2, 70, 70, 0, 5, 0, True)])
def test_window_backward_of_rows_that_see_few_keys(d, H, Hkv, T, Tkv, pos0, window, sinks, simt):
    """Where no row sees more than 64 keys, the bf16 gradients do not carry the rounding of O: D = sum P dP in fp32 is
    off by d 2^-24 sum P |dO||v| + e32 sum P |dP| (e32 as in local_ref, P being off by e32 relative), in place of
    sum |dO| bound(O).  One visible key: dS is nothing but such errors."""
    B = 2
    Q, dO = _rand(1, BF, B, T, H, d), _rand(4, BF, B, T, H, d)
    K, V = _rand(2, BF, B, Tkv, Hkv, d), _rand(3, BF, B, Tkv, Hkv, d)
    p = torch.arange(pos0, pos0 + T, device="cuda")
    assert int(seen(p, Tkv, Tkv, window, sinks).sum(1).max()) <= 64
    kw = dict(q_pos0=pos0, kv_len=Tkv, force_simt=simt)
    O, lse = hsa.window_attend(Q, K, V, window, sinks, return_lse=True, **kw)
    dQ, dK, _ = hsa.window_backward(Q, K, V, O, lse, dO, window, sinks, **kw)
    for b in range(B):
        r = Ref(Q[b], K[b], V[b], p, Tkv, window, sinks, None, dO[b], exact_d=True)
        check(f"dQ[{b}]", dQ[b], r.dQ, r.tdQ)
        check(f"dK[{b}]", dK[b], r.dK, r.tdK)


def test_window_backward_against_differences():
    """The fp32 gradients along random directions against central differences of the fp32 forward.  With step h a
    difference is off by h^2/6 of a third derivative (order 1 here times the sizes below) and by the forward's
    rounding over 2 h: h = 2^-6 keeps both under 2^-9 of sum |dO| |O| ~ 1e3 elements' random sum."""
    d, H, Hkv, T, W, s = 64, 4, 2, 90, 20, 3
    Q, K, V = _rand(1, F32, 1, T, H, d), _rand(2, F32, 1, T, Hkv, d), _rand(3, F32, 1, T, Hkv, d)
    dO = _rand(4, F32, 1, T, H, d)
    O, lse = hsa.window_attend(Q, K, V, W, s, return_lse=True)
    grads = hsa.window_backward(Q, K, V, O, lse, dO, W, s)
    h = 2.0 ** -6
    for i, (x, g) in enumerate(zip((Q, K, V), grads)):
        u = _rand(10 + i, F32, *x.shape)
        u /= u.double().norm()
        a, b = [[q if j != i else x + sg * h * u for j, q in enumerate((Q, K, V))] for sg in (1, -1)]
        fa, fb = (float((hsa.window_attend(*t, W, s).double() * dO.double()).sum()) for t in (a, b))
        want, got = (fa - fb) / (2 * h), float((g.double() * u.double()).sum())
        # forward rounding: each O within 2^-20 |O|-size, summed at random over T H d elements
        noise = 2.0 ** -20 * math.sqrt(T * H * d) / (2 * h) + h * h
        assert abs(want - got) <= noise + 1e-3 * abs(want), (i, want, got, noise)


def _far_tail(T):
    """Two sequences of T tokens, of which the last 300 see old keys at scores 512 below the others': what they bring
    is 2^-700, nothing, and a row's result is that over the last 300 keys alone."""
    Q, K, V = (_rand(i, BF, 2, T, 1, 64) for i in range(3))
    Q[..., 0] = 16
    K[:, :-300] = 0
    K[..., 0] = 0
    K[:, :-300, :, 0] = -256        # 16 (-256) / 8
    return Q, K, V


def _tail(b, n, *xs):
    return [x[b, -n:] for x in xs]


def test_a_call_of_seconds():
    """A helper warp that has no part in a sequence's whole tiles waits for the next ragged one, here for the whole
    first sequence: more than the limit of one second that a step has."""
    Q, K, V = _far_tail(3_000_007)
    ws = hsa.window_workspace(Q, K, 0)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    O, lse = hsa.window_attend(Q, K, V, 0, O=torch.full_like(Q, math.nan), ws=ws, return_lse=True)
    end.record()
    _clean(ws)
    assert start.elapsed_time(end) > 2400       # else the sizes above are too small to show it
    assert not bool(O.isnan().any())
    p = torch.arange(200, 300, device="cuda")
    for b in range(2):
        r = Ref(*_tail(b, 100, Q), *_tail(b, 300, K, V), p, 300, 0, 0)
        check(f"O[{b}]", O[b, -100:], r.O, r.tO)
        check(f"lse[{b}]", lse[b, -100:], r.lse, r.tlse)


def test_a_backward_of_seconds():
    """As above: the helper of dQ waits for the second sequence's ragged tile."""
    Q, K, V = _far_tail(2_200_007)
    dO = _rand(4, BF, *Q.shape)
    ws = hsa.window_workspace(Q, K, 0, backward=True)
    O, lse = hsa.window_attend(Q, K, V, 0, ws=ws, return_lse=True)
    out = tuple(torch.full_like(x, math.nan) for x in (Q, K, V))
    dQ, dK, dV = hsa.window_backward(Q, K, V, O, lse, dO, 0, out=out, ws=ws)
    _clean(ws)
    assert not any(bool(x.isnan().any()) for x in out)
    p = torch.arange(200, 300, device="cuda")
    for b in range(2):
        r = Ref(*_tail(b, 100, Q), *_tail(b, 300, K, V), p, 300, 0, 0, None, *_tail(b, 100, dO))
        check(f"dQ[{b}]", dQ[b, -100:], r.dQ, r.tdQ)


def test_window_without_queries_or_keys():
    K = torch.zeros(2, 5, 2, 64, device="cuda")
    Q = torch.zeros(2, 0, 4, 64, device="cuda")
    O, lse = hsa.window_attend(Q, K, K, 3, return_lse=True)
    dQ, dK, dV = hsa.window_backward(Q, K, K, O, lse, Q, 3, out=(Q.clone(), K + 1, K + 1))
    assert O.shape == Q.shape and not bool(dK.any()) and not bool(dV.any())
    Q, K = torch.ones(2, 3, 4, 64, device="cuda"), torch.zeros(2, 0, 2, 64, device="cuda")
    O, lse = hsa.window_attend(Q, K, K, 3, return_lse=True)
    assert not bool(O.any()) and bool((lse == -math.inf).all())
    dQ, dK, dV = hsa.window_backward(Q, K, K, O, lse, Q, 3)
    assert not bool(dQ.any())


# ------------------------------------------------------------------------------------------------ rotary

ROPES = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
         dict(scaling="yarn", factor=16.0, orig_len=4096), dict(scaling="bands", factor=8.0, orig_len=8192, theta=5e5),
         dict(scaling="yarn", factor=4.0, orig_len=2048, low=2.0, high=20.0),
         dict(scaling="bands", factor=4.0, orig_len=2048, low=0.5, high=9.0)]


@pytest.mark.parametrize("kw", ROPES, ids=lambda k: k.get("scaling", "none"))
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("rot,d", [(64, 64), (128, 128), (32, 128), (20, 64), (2, 64), (112, 128), (48, 64)])
def test_rope(rot, d, dt, kw):
    if rot == 2 and kw.get("scaling") == "ntk":
        pytest.skip("needs rot > 2")
    for inter in (False, True):
        r = hsa.make_rope(rot, interleaved=inter, **kw)
        Q, K = _rand(1, dt, 2, 37, 6, d), _rand(2, dt, 2, 37, 2, d)
        for pos0, inv in ((0, False), (16777000, True)):
            a, b = hsa.rope(r, Q, K, pos0=pos0, inverse=inv)
            pos = torch.arange(pos0, pos0 + 37, device="cuda").expand(2, 37)
            for x, y in ((Q, a), (K, b)):
                want, tol = turn(x, pos, rot, inter, inv, **kw)
                check("rope", y, want, tol)


def test_rope_forms():
    r = hsa.make_rope(64, theta=5e5)
    Q, K = _rand(1, BF, 3, 700, 5, 128), _rand(2, BF, 3, 700, 2, 128)    # 5 heads over 2: any two counts
    pos = torch.randint(0, 2 ** 24, (3, 700), device="cuda", dtype=torch.int32)
    a, b = hsa.rope(r, Q, K, pos=pos)
    for x, y in ((Q, a), (K, b)):
        want, tol = turn(x, pos, 64, theta=5e5)
        check("rope", y, want, tol)
    assert torch.equal(hsa.rope(r, Q, pos=pos), a) and torch.equal(hsa.rope(r, K=K, pos=pos), b)
    Qi, Ki = Q.clone(), K.clone()
    hsa.rope(r, Qi, Ki, pos=pos, Q_out=Qi, K_out=Ki)       # in place
    assert torch.equal(Qi, a) and torch.equal(Ki, b)
    assert hsa.rope(r, Q[:, :0].contiguous()).shape == (3, 0, 5, 128)
    big = _rand(3, BF, 1, 4099, 8, 128)                     # several tokens per block, a ragged last block
    want, tol = turn(big, torch.arange(9, 4108, device="cuda")[None], 64, theta=5e5)
    check("rope", hsa.rope(r, big, pos0=9), want, tol)


@pytest.mark.parametrize("H,Hkv", [(32, 1), (2, 7), (40, 2), (16380, 4)])
def test_rope_head_counts(H, Hkv):
    """Any two counts, more than 16 query heads to a kv head among them; above 16383 in all, in two launches."""
    r = hsa.make_rope(32)
    Q, K = _rand(1, BF, 2, 9, H, 64), _rand(2, BF, 2, 9, Hkv, 64)
    pos = torch.arange(5, 14, device="cuda").expand(2, 9)
    for x, y in zip((Q, K), hsa.rope(r, Q, K, pos0=5)):
        want, tol = turn(x, pos, 32)
        check("rope", y, want, tol)


def test_rope_gradient_is_the_transpose():
    """<rope(x), g> = <x, rope_inverse(g)> in fp32, each side's sum off by its roundings."""
    r = hsa.make_rope(48, scaling="yarn", factor=8.0, orig_len=4096, interleaved=True)
    x, g = _rand(1, F32, 2, 50, 4, 64), _rand(2, F32, 2, 50, 4, 64)
    y, z = hsa.rope(r, x, pos0=123456), hsa.rope(r, g, pos0=123456, inverse=True)
    a, b = (y.double() * g.double()).sum(), (x.double() * z.double()).sum()
    bound = 2.0 ** -21 * 2 * r.mult * float((x.abs().double() * g.abs().double()).sum() * 2)
    assert abs(float(a - b)) <= bound


# ------------------------------------------------------------------------------------------------ pages

class Pages:
    """A ragged batch over a pool of pages: shuffled page numbers, entries past a sequence's pages invalid."""

    def __init__(self, dt, d, H, Hkv, new, kv, page, pad=0, seed=0, spare=3):
        self.new, self.kv, self.page = new, kv, page
        B = len(new)
        need = [-(-m // page) for m in kv]
        n = sum(need) + spare
        order = torch.randperm(n, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        self.table = torch.full((B, max(max(need), 1)), -7, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.table = self.table.cuda()
        rows = sum(new) + pad
        self.Q, self.k, self.v = (_rand(seed + i, dt, rows, h, d) for i, h in enumerate((H, Hkv, Hkv)))
        self.K, self.V = (_rand(seed + 5 + i, dt, n, page, Hkv, d) for i in range(2))
        self.q_start = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32).cuda()
        self.kv_len = torch.tensor(kv, dtype=torch.int32).cuda()

    def cache(self, b, X):
        m = self.kv[b]
        u = torch.arange(m, device="cuda")
        return X[self.table[b].long()[u // self.page], u % self.page]

    def rows(self, b):
        a = sum(self.new[:b])
        return slice(a, a + self.new[b])

    def pos(self, b):
        return torch.arange(self.kv[b] - self.new[b], self.kv[b], device="cuda")


def _paged(dt, d, H, Hkv, new, kv, page, window, sinks, pad=2, simt=False, bounds=True, seed=0):
    P = Pages(dt, d, H, Hkv, new, kv, page, pad, seed)
    kw = dict(window=window, sinks=sinks, force_simt=simt)
    if bounds:
        kw.update(max_q=max(new), max_kv=max(kv))
    # page slots that no query sees: NaN; stale table entries behind every window
    live = torch.zeros(P.K.shape[:2], dtype=torch.bool, device="cuda")
    for b in range(len(new)):
        if new[b]:
            s = seen(P.pos(b), kv[b], kv[b], window, sinks).any(0).nonzero().flatten()
            live[P.table[b].long()[s // page], s % page] = True
    P.K[~live], P.V[~live] = math.nan, math.nan
    keep = P.table.clone()
    for b in range(len(new)):
        for i in range(P.table.shape[1]):
            if int(keep[b, i]) >= 0 and not bool(live[int(keep[b, i])].any()):
                P.table[b, i] = -1 if i % 2 else 2 ** 30
    ws = hsa.paged_workspace(P.Q, P.K, P.table, **kw)
    ws[256:] = 0xFF
    O = torch.full_like(P.Q, 7.0)
    hsa.paged_attend(P.Q, P.K, P.V, P.q_start, P.kv_len, P.table, O=O, ws=ws, **kw)
    _clean(ws)
    P.table = keep
    for b in range(len(new)):
        if new[b]:
            r = Ref(P.Q[P.rows(b)], P.cache(b, P.K), P.cache(b, P.V), P.pos(b), kv[b], window, sinks)
            check(f"O[{b}]", O[P.rows(b)], r.O, r.tO)
    assert bool((O[sum(new):] == 7.0).all()), "rows behind the last sequence were written"


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4), (17, 40), (1, 0)])
def test_paged_chunks(page, window, sinks):
    new, kv = [130, 1, 0, 64, 7, 300], [500, 77, 20, 64, 1029, 300]
    _paged(BF, 128, 8, 2, new, kv, page, window, sinks)
    _paged(BF, 64, 6, 2, new, kv, page, window, sinks)
    _paged(F32, 64, 4, 2, new, kv, page, window, sinks)
    _paged(BF, 128, 4, 2, new, kv, page, window, sinks, simt=True)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (5, 5), (16, 1), (7, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
def test_paged_single_tokens(page, H, Hkv, window, sinks):
    kv = [1, 2, 16, 17, 63, 64, 65, 128, 129, 700, 3001]
    _paged(BF, 128, H, Hkv, [1] * len(kv), kv, page, window, sinks)
    _paged(BF, 64, H, Hkv, [1] * len(kv), kv, page, window, sinks, bounds=False)
    _paged(F32, 128, H, Hkv, [1] * len(kv), kv, page, window, sinks)


@pytest.mark.parametrize("new,kv", [([1], [1]), ([1], [4000]), ([0, 0, 1], [0, 5, 9]), ([3, 2], [2, 1]), ([5], [3000]),
                                    ([40, 1], [9000, 9000]), ([0], [0])])
@pytest.mark.parametrize("dt", [BF, F32])
def test_paged_few_sequences(dt, new, kv):
    """One sequence, empty ones, and ones with fewer cached tokens than new ones (rows before position 0: zeros)."""
    _paged(dt, 64, 8, 2, new, kv, 32, 0, 0)
    _paged(dt, 128, 4, 2, new, kv, 16, 50, 2)


@pytest.mark.parametrize("dt,simt", [(BF, False), (BF, True), (F32, False)])
def test_paged_one_workspace_for_every_batch(dt, simt):
    """The workspace of the largest batch serves smaller ones, which are split more, one after another; rows behind the
    last sequence, more of them than the batch has, take no part."""
    d, H, Hkv, page = 64, 8, 2, 64
    big = Pages(dt, d, H, Hkv, [300] * 6, [20000] * 6, page)
    ws = hsa.paged_workspace(big.Q, big.K, big.table, max_q=300, max_kv=20000, force_simt=simt)
    ws[256:] = 0xFF
    for new, kv in (([300] * 6, [20000, 19000, 700, 301, 20000, 300]), ([1] * 6, [20000] * 6), ([1], [20000]), ([4], [17000]),
                    ([200, 1], [20000, 20000]), ([2, 0, 1], [16500, 9, 20000]), ([40], [4000])):
        P = Pages(dt, d, H, Hkv, new, kv, page, pad=400)
        O = torch.full_like(P.Q, 7.0)
        hsa.paged_attend(P.Q, P.K, P.V, P.q_start, P.kv_len, P.table, max_q=max(new), max_kv=max(kv), O=O, ws=ws, force_simt=simt)
        _clean(ws)
        for b in range(len(new)):
            if new[b]:
                r = Ref(P.Q[P.rows(b)], P.cache(b, P.K), P.cache(b, P.V), P.pos(b), kv[b], 0, 0)
                check(f"O[{b}]", O[P.rows(b)], r.O, r.tO)
        assert bool((O[sum(new):] == 7.0).all())


def _loose(dt, d, H, Hkv, new, kv, sample, **kw):
    """paged_attend without max_q: every sequence may hold all rows, as far as the call knows."""
    B, page = len(new), 16
    need = torch.tensor([-(-m // page) for m in kv])
    table = torch.full((B, int(need.max())), -1, dtype=torch.int32)
    at = torch.cat((torch.zeros(1, dtype=torch.long), need.cumsum(0)))
    for i in range(table.shape[1]):
        table[need > i, i] = (at[:-1][need > i] + i).to(torch.int32)
    q_start = torch.cat((torch.zeros(1, dtype=torch.long), torch.tensor(new).cumsum(0)))
    rows = int(q_start[-1])
    Q, K, V = _rand(1, dt, rows + 2, H, d), _rand(2, dt, int(at[-1]), page, Hkv, d), _rand(3, dt, int(at[-1]), page, Hkv, d)
    args = [x.to(torch.int32).cuda() for x in (q_start, torch.tensor(kv), table)]
    ws = hsa.paged_workspace(Q, K, args[2], **kw)
    O = torch.full_like(Q, 7.0)
    hsa.paged_attend(Q, K, V, *args, O=O, ws=ws, **kw)
    _clean(ws)
    assert bool((O[rows:] == 7.0).all())
    for b in sample:
        r0, m = int(q_start[b]), kv[b]
        k, v = (X[int(at[b]):int(at[b + 1])].reshape(-1, Hkv, d)[:m] for X in (K, V))
        if new[b]:
            r = Ref(Q[r0:r0 + new[b]], k, v, torch.arange(m - new[b], m, device="cuda"), m, 0, 0)
            check(f"O[{b}]", O[r0:r0 + new[b]], r.O, r.tO)
    return O[:rows]


@pytest.mark.parametrize("dt,simt", [(BF, False), (BF, True), (F32, False)])
def test_paged_many_sequences_without_a_bound(dt, simt):
    """20000 sequences of a token each, a few longer or empty: blocks without tokens by the million."""
    new, kv = [1] * 20000, [1 + i % 20 for i in range(20000)]
    for b, n in ((7, 300), (8, 0), (9, 0), (5000, 33), (19998, 0), (19999, 65)):
        new[b], kv[b] = n, n + 9
    O = _loose(dt, 64, 8, 2, new, kv, [0, 1, 6, 7, 10, 11, 4999, 5000, 5001, 13000, 19997, 19999], force_simt=simt)
    assert not bool((O == 7.0).flatten(1).all(1).any())


def test_paged_items_beyond_32_bits():
    """65535 sequences that may hold 65535 rows each, over 9 kv heads of 16: 2.4e9 pairs of row tiles."""
    O = _loose(BF, 64, 144, 9, [1] * 65535, [1 + i % 5 for i in range(65535)], [0, 1, 2, 30000, 65533, 65534])
    assert not bool((O == 7.0).flatten(1).all(1).any())


@pytest.mark.parametrize("H,Hkv", [(5, 1), (7, 1), (6, 2), (22, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_items_of_groups_that_do_not_divide_a_tile(d, H, Hkv):
    """Long items cut between CTAs and joined, rows of whole tokens that leave the end of a tile empty."""
    _paged(BF, d, H, Hkv, [200, 1, 300, 90], [9000, 9000, 300, 5001], 64, 0, 0)
    _paged(BF, d, H, Hkv, [200, 301], [9000, 6000], 16, 4000, 200)
    _forward(BF, d, H, Hkv, 1, 100, 9100, 9101, 9000, 0, 0)


def test_append_in_place():
    """Q rotated in place: what a Q_out of its own gets."""
    P = Pages(BF, 64, 6, 2, [30, 2], [100, 9], 16, pad=1)
    r = hsa.make_rope(64)
    K, V = P.K.clone(), P.V.clone()
    want = hsa.paged_append(P.k, P.v, K, V, P.q_start, P.kv_len, P.table, Q=P.Q, rope=r, Q_out=P.Q.clone())
    Q = P.Q.clone()
    assert hsa.paged_append(P.k, P.v, P.K, P.V, P.q_start, P.kv_len, P.table, Q=Q, rope=r, Q_out=Q) is Q
    assert torch.equal(Q, want) and torch.equal(P.K, K) and torch.equal(P.V, V)


def test_paged_bad_pages_and_lengths():
    """Page numbers outside the pool read as zeros and lengths are cut to their bounds; both are reported."""
    P = Pages(BF, 64, 4, 2, [4, 1], [100, 40], 32)
    good = P.table.clone()
    P.table[0, 1] = P.K.shape[0]
    caches = [[X[good[b].long()[torch.arange(P.kv[b], device="cuda") // 32], torch.arange(P.kv[b], device="cuda") % 32] for X in (P.K, P.V)]
              for b in range(2)]
    ws = hsa.paged_workspace(P.Q, P.K, P.table, max_q=4, max_kv=100)
    for simt in (False, True):
        O = hsa.paged_attend(P.Q, P.K, P.V, P.q_start, P.kv_len, P.table, max_q=4, max_kv=100, ws=ws, force_simt=simt)
        with pytest.raises(hsa.HSAError):
            hsa.device_status(ws)
        hsa.device_status(ws)    # read and cleared
        K, V = caches[0]
        K[32:64], V[32:64] = 0, 0
        r = Ref(P.Q[:4], K, V, P.pos(0), 100, 0, 0)
        check("O[0]", O[:4], r.O, r.tO)
        r = Ref(P.Q[4:], *caches[1], P.pos(1), 40, 0, 0)
        check("O[1]", O[4:], r.O, r.tO)
        bad = P.kv_len.clone()
        bad[1] = 2 ** 30
        hsa.paged_attend(P.Q, P.K, P.V, P.q_start, bad, P.table, max_q=4, max_kv=100, ws=ws, force_simt=simt)
        with pytest.raises(hsa.HSAError):
            hsa.device_status(ws)
    K0, V0 = P.K.clone(), P.V.clone()
    P.kv_len[0] = 66             # its new tokens sit at 62 .. 65: the first two in the bad page
    hsa.paged_append(P.k, P.v, P.K, P.V, P.q_start, P.kv_len, P.table, ws=ws)
    with pytest.raises(hsa.HSAError):
        hsa.device_status(ws)
    t = int(good[0, 2]), int(good[1, 1])
    K0[t[0], :2], V0[t[0], :2], K0[t[1], 39 % 32], V0[t[1], 39 % 32] = P.k[2:4], P.v[2:4], P.k[4], P.v[4]
    assert torch.equal(P.K, K0) and torch.equal(P.V, V0)


def test_a_call_needs_no_more_than_it_uses():
    """A prompt that is not split runs in the 256 bytes of the status word, whatever smaller ones would need."""
    Q, K = _rand(1, BF, 4, 4100, 32, 64), _rand(2, BF, 4, 4100, 8, 64)
    ws = hsa.window_workspace(Q, K, 0)
    assert ws.numel() > 1 << 20
    O = hsa.window_attend(Q, K, K, 0, ws=ws)
    assert torch.equal(hsa.window_attend(Q, K, K, 0, ws=ws[:256].clone()), O)
    with pytest.raises(hsa.HSAError):
        hsa.window_attend(Q, K, K, 0, ws=ws[:255].clone())


def test_workspaces_elsewhere_are_refused():
    P = Pages(BF, 64, 4, 2, [4, 1], [100, 40], 32)
    Q, K = _rand(1, BF, 1, 9, 4, 64), _rand(2, BF, 1, 9, 2, 64)
    O, lse = hsa.window_attend(Q, K, K, 3, return_lse=True)
    for ws in (torch.zeros(1 << 24, dtype=torch.uint8), torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")[::2]):
        for call in (lambda: hsa.window_attend(Q, K, K, 3, ws=ws),
                     lambda: hsa.window_backward(Q, K, K, O, lse, Q, 3, ws=ws),
                     lambda: hsa.paged_attend(P.Q, P.K, P.V, P.q_start, P.kv_len, P.table, ws=ws),
                     lambda: hsa.paged_append(P.k, P.v, P.K, P.V, P.q_start, P.kv_len, P.table, ws=ws)):
            with pytest.raises(ValueError, match="ws"):
                call()


def test_paged_shared_pages():
    """A forked prefix: two sequences whose tables name the same pages, one of them twice in a row of the table."""
    P = Pages(BF, 128, 8, 2, [1, 40, 1], [200, 200, 96], 32)
    P.table[1, :5] = P.table[0, :5]
    P.table[2, 1] = P.table[2, 0]
    for kw in (dict(max_q=40, max_kv=200), dict(window=70, sinks=5)):
        O = hsa.paged_attend(P.Q, P.K, P.V, P.q_start, P.kv_len, P.table, **kw)
        for b in range(3):
            r = Ref(P.Q[P.rows(b)], P.cache(b, P.K), P.cache(b, P.V), P.pos(b), P.kv[b], kw.get("window", 0), kw.get("sinks", 0))
            check(f"O[{b}]", O[P.rows(b)], r.O, r.tO)


def test_two_calls_at_once():
    """The same inputs read by calls on two streams, each with its own workspace and outputs."""
    T, W = 3000, 700
    Q, K, V, dO = (_rand(i, BF, 1, T, h, 128) for i, h in enumerate((8, 2, 2, 8)))
    O, lse = hsa.window_attend(Q, K, V, W, 4, return_lse=True)
    want = (O,) + tuple(hsa.window_backward(Q, K, V, O, lse, dO, W, 4))
    P = Pages(BF, 128, 8, 2, [300, 1], [9000, 9000], 64)
    wantP = hsa.paged_attend(P.Q, P.K, P.V, P.q_start, P.kv_len, P.table, max_q=300, max_kv=9000)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                if i < 2:
                    o, l = hsa.window_attend(Q, K, V, W, 4, return_lse=True)
                    got.append((o,) + tuple(hsa.window_backward(Q, K, V, o, l, dO, W, 4)))
                else:
                    got.append((hsa.paged_attend(P.Q, P.K, P.V, P.q_start, P.kv_len, P.table, max_q=300, max_kv=9000),))
    torch.cuda.synchronize()
    for g in got:
        w = want if len(g) > 1 else (wantP,)
        assert all(torch.equal(x, y) for x, y in zip(g, w))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("rot,inter,kw", [(64, False, dict()), (32, True, dict(scaling="linear", factor=2.0)),
                                          (20, False, dict(scaling="bands", factor=8.0, orig_len=64)), (0, False, dict())])
def test_paged_append(dt, rot, inter, kw):
    new, kv = [130, 1, 0, 64, 7, 2100], [500, 77, 20, 64, 1029, 2100]
    for page in (16, 128):
        P = Pages(dt, 64, 6, 2, new, kv, page, pad=3)
        K, V, Q = P.K.clone(), P.V.clone(), torch.full_like(P.Q, 7.0)
        r = hsa.make_rope(rot, interleaved=inter, **kw) if rot else None
        ws = hsa.paged_workspace(P.Q, P.K, P.table)
        assert hsa.paged_append(P.k, P.v, K, V, P.q_start, P.kv_len, P.table, Q=P.Q, rope=r, Q_out=Q, ws=ws) is Q
        _clean(ws)
        wantK, wantV, wantQ = P.K.double(), P.V.double(), torch.full_like(P.Q, 7.0).double()
        tolK, tolQ = torch.zeros_like(wantK), torch.zeros_like(wantQ)
        for b in range(len(new)):
            pos, rows = P.pos(b), P.rows(b)
            at = P.table[b].long()[pos // page], pos % page
            if rot:
                wantK[at], tolK[at] = turn(P.k[rows], pos, rot, inter, **kw)
                wantQ[rows], tolQ[rows] = turn(P.Q[rows], pos, rot, inter, **kw)
            else:
                wantK[at], wantQ[rows] = P.k[rows].double(), P.Q[rows].double()
            wantV[at] = P.v[rows].double()
        check("K", K, wantK, tolK)
        check("Q", Q, wantQ, tolQ)
        assert torch.equal(V.double(), wantV)
        K2, V2 = P.K.clone(), P.V.clone()
        assert hsa.paged_append(P.k, P.v, K2, V2, P.q_start, P.kv_len, P.table, rope=r) is None
        assert torch.equal(K, K2) and torch.equal(V, V2)


# ------------------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("dt", [BF, F32])
def test_a_served_batch_equals_whole_prompts(dt):
    """Two sequences served in chunks and single tokens (append with rotation, attention over the pages) against one
    call each on the whole contiguous sequence (rope, window_attend): same keys bit for bit, outputs within the
    two calls' bounds of the same 64-bit result."""
    d, H, Hkv, page, W, S = 64, 4, 2, 16, 40, 3
    r = hsa.make_rope(32, theta=1e4)
    n = [150, 90]
    Q, K, V = ([_rand(10 * i + j, dt, n[i], h, d) for i in range(2)] for j, h in enumerate((H, Hkv, Hkv)))
    table = torch.randperm(20, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(2, 10).cuda()
    Kp, Vp = torch.full((20, page, Hkv, d), math.nan, dtype=dt, device="cuda"), torch.full(
        (20, page, Hkv, d), math.nan, dtype=dt, device="cuda")
    done, outs = [0, 0], [[], []]
    ws = None
    while done != n:
        step = [min(n[i] - done[i], 64 if done[i] < 64 else 5 if done[i] % 2 else 1) for i in range(2)]
        rows = [torch.cat([X[i][done[i]:done[i] + step[i]] for i in range(2)]) for X in (Q, K, V)]
        q_start = torch.tensor([0, step[0], sum(step)], dtype=torch.int32).cuda()
        done = [done[i] + step[i] for i in range(2)]
        kv_len = torch.tensor(done, dtype=torch.int32).cuda()
        q = hsa.paged_append(rows[1], rows[2], Kp, Vp, q_start, kv_len, table, Q=rows[0], rope=r)
        o = hsa.paged_attend(q, Kp, Vp, q_start, kv_len, table, max_q=max(step), max_kv=max(done), window=W, sinks=S)
        for i, x in enumerate(o.split(step)):
            outs[i].append(x)
    for i in range(2):
        q, k = hsa.rope(r, Q[i][None], K[i][None])
        u = torch.arange(n[i], device="cuda")
        assert torch.equal(Kp[table[i].long()[u // page], u % page], k[0])
        O = hsa.window_attend(q, k, V[i][None], W, S)[0]
        ref = Ref(q[0], k[0], V[i], u, n[i], W, S)
        check("whole", O, ref.O, ref.tO)
        check("served", torch.cat(outs[i]), ref.O, ref.tO)


def test_a_training_step_of_a_local_layer():
    """rope -> window_attend -> window_backward -> rope (transposed) against differentiating the 64-bit formulas."""
    d, H, Hkv, T, W, S = 64, 4, 2, 140, 30, 2
    Q, K, V, dO = (_rand(i, F32, 1, T, h, d) for i, h in enumerate((H, Hkv, Hkv, H)))
    r = hsa.make_rope(64)
    q, k = hsa.rope(r, Q, K)
    O, lse = hsa.window_attend(q, k, V, W, S, return_lse=True)
    dq, dk, dV = hsa.window_backward(q, k, V, O, lse, dO, W, S)
    dQ, dK = hsa.rope(r, dq, dk, inverse=True)
    Qd, Kd, Vd = (x.double().requires_grad_() for x in (Q, K, V))
    pos = torch.arange(T, device="cuda")
    f = torch.arange(32, device="cuda").double().mul(-2 / 64 * math.log(1e4)).exp()
    a = pos.double()[:, None, None] * f

    def rot(x):
        x1, x2 = x[..., :32], x[..., 32:]
        return torch.cat((x1 * a.cos() - x2 * a.sin(), x2 * a.cos() + x1 * a.sin()), -1)

    qd, kd = rot(Qd)[0].transpose(0, 1), rot(Kd)[0].transpose(0, 1).repeat_interleave(2, 0)
    s = (qd @ kd.transpose(1, 2) / 8).masked_fill(~seen(pos, T, T, W, S), -math.inf)
    o = (torch.softmax(s, -1) @ Vd[0].transpose(0, 1).repeat_interleave(2, 0)).transpose(0, 1)[None]
    o.backward(dO.double())
    # every product and sum is fp32: 2^-24 (2 d S' + 2 n + 64) with S' < 16 and n < 2^9 stays below 2^-12 of the
    # tensors' size, through two such steps
    for got, want in ((O, o.detach()), (dQ, Qd.grad), (dK, Kd.grad), (dV, Vd.grad)):
        assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -11


def test_graph_replay_follows_the_lengths():
    """append + attend captured once; replayed as the lengths, tokens and pages on the device change, on another
    stream, with two graphs that have a workspace each."""
    d, H, Hkv, page = 128, 8, 2, 32
    P = Pages(BF, d, H, Hkv, [1, 1, 1], [400, 390, 7], page, spare=2)
    r = hsa.make_rope(64)
    graphs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for w in (0, 33):
            kw = dict(max_q=1, max_kv=400, window=w, sinks=4)
            ws, O, Qr = hsa.paged_workspace(P.Q, P.K, P.table, **kw), torch.empty_like(P.Q), torch.empty_like(P.Q)

            def step():
                hsa.paged_append(P.k, P.v, P.K, P.V, P.q_start, P.kv_len, P.table, Q=P.Q, rope=r, Q_out=Qr, ws=ws)
                hsa.paged_attend(Qr, P.K, P.V, P.q_start, P.kv_len, P.table, O=O, ws=ws, **kw)

            step()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                step()
            graphs.append((g, w, O, Qr, ws))
    torch.cuda.current_stream().wait_stream(s)
    for kv in ([100, 390, 7], [399, 1, 30]):
        P.kv = kv
        P.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        P.k.copy_(_rand(sum(kv), BF, *P.k.shape))
        for g, w, O, Qr, ws in graphs:
            g.replay()
            torch.cuda.synchronize()
            _clean(ws)
            for b in range(3):
                ref = Ref(Qr[P.rows(b)], P.cache(b, P.K), P.cache(b, P.V), P.pos(b), kv[b], w, 4)
                check("O", O[P.rows(b)], ref.O, ref.tO)
