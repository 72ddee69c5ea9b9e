"""Plain 64-bit restatement of the local attention, with a bound on what rounding
may do to each result.  No code of the library.

Rounding: to type t a value moves by at most half a step, eps(t)/2 relative (bf16
2^-8, fp32 2^-24).  The kernels
  * sum q.k over d products in fp32: |error of the scaled score| <= d 2^-24 S', with
    S' = scale max sum |q_x k_x| over the visible pairs; it enters exp once, and once more
    through the row's normalisation,
  * add at most n probabilities and products in fp32: n 2^-24 each for l and for O,
  * take exp2 and a division: 64 steps of 2^-24 cover them,
so a probability is off by e32 = 2^-24 (2 d S' + 2 n + 64) relative, plus, in bf16, the half
step of its rounding before the product.  With A = sum P |v|:
  |dO| <= (e_p + e32) A + (e_t + e32) |O|,   e_p = 2^-8 (bf16) or 0, e_t = half step of the output
  lse: 2^-24 (d S' + n + 8 + 8 |lse|)
Backward: D = sum dO o O of the stored O is off by dD = sum |dO| bound(O) + d 2^-24 sum |dO o O|;
dS = P (dP - D) by P (dD + d 2^-24 sum |dO||v|) + (e_p + e32) |dS|, then it is multiplied and summed
like P above:
  dV: (e_p + e32) sum P |dO| + (e_t + e32) |dV|
  dQ: scale sum bound(dS) |k| + e32 scale sum |dS||k| + (e_t + e32) |dQ|, dK alike.
"""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def seen(p, n_keys, kv, window, sinks):
    """[rows, keys] truth values: which keys the queries at positions p see."""
    u = torch.arange(n_keys, device=p.device)[None]
    p = p[:, None]
    v = (u <= p) & (u < kv)
    if window:
        v &= (p - u < window) | (u < sinks)
    return v


class Ref:
    """One sequence: Q [n,H,d], K, V [m,Hkv,d] as stored; p [n] positions; kv cached tokens (<= m)."""

    def __init__(self, Q, K, V, p, kv, window, sinks, scale=None, dO=None, exact_d=False):
        t = Q.dtype
        n, H, d = Q.shape
        Hkv = K.shape[1]
        G = H // Hkv
        sc = scale if scale else 1.0 / math.sqrt(d)
        vis = seen(p, K.shape[0], kv, window, sinks)
        live = vis.any(0)
        q = Q.double().transpose(0, 1)                                            # H, n, d
        # keys that no query sees may hold anything: they take no part
        k = torch.where(live[:, None, None], K.double(), 0).transpose(0, 1).repeat_interleave(G, 0)
        v = torch.where(live[:, None, None], V.double(), 0).transpose(0, 1).repeat_interleave(G, 0)
        s = sc * q @ k.transpose(1, 2)
        s = s.masked_fill(~vis, -math.inf)
        some = vis.any(1)
        self.lse = torch.logsumexp(s, -1)                                          # H, n
        P = torch.where(some[:, None], torch.exp(s - torch.where(some, self.lse, 0.0)[..., None]), 0.0)
        O = P @ v
        Sp = float((sc * (q.abs() @ k.abs().transpose(1, 2))).masked_fill(~vis, 0).max()) if vis.numel() else 0.0
        cnt = int(vis.sum(1).max()) if vis.numel() else 0
        u = 2.0 ** -24
        e32 = u * (2 * d * Sp + 2 * cnt + 64)
        ep, et = (HALF[t], HALF[t]) if t == torch.bfloat16 else (0.0, HALF[t])
        A = P @ v.abs()
        tO = (ep + e32) * A + (et + e32) * O.abs()
        self.O, self.tO = O.transpose(0, 1), tO.transpose(0, 1)
        self.lse, self.tlse = self.lse.transpose(0, 1), (u * (d * Sp + cnt + 8 + 8 * self.lse.abs().nan_to_num(0, 0, 0))).transpose(0, 1)
        if dO is None:
            return
        g = dO.double().transpose(0, 1)
        dP = g @ v.transpose(1, 2)
        D = (g * O).sum(-1, keepdim=True)
        dS = P * (dP - D)
        dD = (g.abs() * tO).sum(-1, keepdim=True) + d * u * (g * O).abs().sum(-1, keepdim=True)
        if exact_d:       # D = sum P dP in fp32
            dD = (P * (d * u * (g.abs() @ v.abs().transpose(1, 2)) + e32 * dP.abs())).sum(-1, keepdim=True)
        bS = P * (dD + d * u * (g.abs() @ v.abs().transpose(1, 2))) + (ep + e32) * dS.abs()

        def group(x):     # sums over the query heads of each kv head
            return x.reshape(Hkv, G, *x.shape[1:]).sum(1).transpose(0, 1)

        # dK, dV add over G n rows
        eg = u * (2 * G * n + 64) + e32
        dQ = sc * dS @ k
        self.dQ, self.tdQ = dQ.transpose(0, 1), (sc * bS @ k.abs() + e32 * sc * (dS.abs() @ k.abs())
                                                 + (et + e32) * dQ.abs()).transpose(0, 1)
        self.dK = group(sc * dS.transpose(1, 2) @ q)
        self.tdK = group(sc * bS.transpose(1, 2) @ q.abs() + eg * sc * (dS.abs().transpose(1, 2) @ q.abs()))
        self.dV = group(P.transpose(1, 2) @ g)
        self.tdV = group((ep + eg) * (P.transpose(1, 2) @ g.abs()))
        self.tdK = self.tdK + (et + eg) * self.dK.abs()
        self.tdV = self.tdV + (et + eg) * self.dV.abs()


def check(name, got, want, tol):
    """Every element within its bound; NaN nowhere."""
    got = got.double()
    assert not bool(got.isnan().any()), f"{name}: NaN"
    fin = want.isfinite()
    assert torch.equal(got[~fin], want[~fin]), f"{name}: infinities"
    over = ((got - want).abs() - tol)[fin]
    if over.numel() and float(over.max()) > 0:
        i = int(((got - want).abs() - tol).nan_to_num(-1).flatten().argmax())
        raise AssertionError(f"{name}: {int((over > 0).sum())} of {got.numel()} beyond their bound; element {i}: "
                             f"got {got.flatten()[i]:.6g}, want {want.flatten()[i]:.6g}, bound {tol.flatten()[i]:.3g}")


# ------------------------------------------------------------------------------------------------ rotary

def inv_freq(rot, theta=10000.0, scaling="none", factor=1.0, orig_len=0, low=0.0, high=0.0):
    """Frequencies and multiplier of a rotary embedding, in 64 bits, pair by pair."""
    f, mult = [], 1.0
    for i in range(rot // 2):
        x = theta ** (-2.0 * i / rot)
        if scaling == "linear":
            x /= factor
        elif scaling == "ntk":
            x = (theta * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
        elif scaling == "yarn":
            lo, hi = low or 1.0, high or 32.0
            a = max(0, math.floor(rot * math.log(orig_len / (hi * 2 * math.pi)) / (2 * math.log(theta))))
            b = min(rot - 1, math.ceil(rot * math.log(orig_len / (lo * 2 * math.pi)) / (2 * math.log(theta))))
            w = min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            x = w * x / factor + (1 - w) * x
            mult = 0.1 * math.log(factor) + 1.0
        elif scaling == "bands":
            lo, hi = low or 1.0, high or 4.0
            w = min(1.0, max(0.0, (orig_len * x / (2 * math.pi) - lo) / (hi - lo)))
            x = (1 - w) * x / factor + w * x
        f.append(x)
    return torch.tensor(f, dtype=torch.float64), mult


def turn(x, pos, rot, interleaved=False, inverse=False, **kw):
    """x [..., T, heads, d] rotated at pos [..., T], in 64 bits, and the bound of an fp32 computation that is
    rounded once: an angle's sine and cosine are off by 2^-22 (its reduction to one turn in fp64, then fp32), the
    two products and their sum by 3 half steps, the output by its own."""
    f, m = inv_freq(rot, **kw)
    a = pos.double()[..., None, None] * f.to(x.device)
    c, s = torch.cos(a) * m, torch.sin(a) * (-m if inverse else m)
    y = x.double().clone()
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    x1, x2 = x.double()[..., one], x.double()[..., two]
    y[..., one], y[..., two] = x1 * c - x2 * s, x2 * c + x1 * s
    tol = torch.zeros_like(y)
    b = m * (2.0 ** -22 + 4 * 2.0 ** -24) * (x1.abs() + x2.abs())
    tol[..., one], tol[..., two] = b, b
    tol[..., :rot] += HALF[x.dtype] * (y[..., :rot].abs() + tol[..., :rot])
    return y, tol
