"""Plain float64 forms of the operators around the fp8 cache, for the tests, with the error
bounds that a right kernel keeps (each derived from the roundings it makes)."""
import math

import numpy as np
import torch

import workloads as w

D_LAT, D_ROW = 512, 576
BF16_HALF = 2.0 ** -8              # half a step of bf16, relative: finfo(bfloat16).eps / 2
F32_HALF = 2.0 ** -24


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def e4m3_values() -> np.ndarray:
    v = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        a = math.nan if (e, m) == (15, 7) else (m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v.append(-a if code & 128 else a)
    return np.array(v)


# ------------------------------------------------------------------ norm and rotation
def norm_rope(x, weight, pos, inv_freq, eps, interleaved):
    """(y, bound): x [T, R, 576], pos [T], all float64."""
    y, tol = x.copy(), np.zeros_like(x)
    if weight is not None:
        lat = x[..., :D_LAT]
        y[..., :D_LAT] = lat / np.sqrt((lat ** 2).mean(-1, keepdims=True) + eps) * weight
        # sum of 512 squares (at most 21 roundings deep), rsqrt, two products, then bf16
        tol[..., :D_LAT] = np.abs(y[..., :D_LAT]) * (BF16_HALF + 32 * F32_HALF)
    ang = np.longdouble(pos)[:, None] * np.longdouble(inv_freq)[None, :]
    cs, sn = np.cos(ang).astype(np.float64)[:, None], np.sin(ang).astype(np.float64)[:, None]
    a_at = np.arange(32) * 2 if interleaved else np.arange(32)
    b_at = a_at + 1 if interleaved else a_at + 32
    a, b = x[..., D_LAT + a_at], x[..., D_LAT + b_at]
    ya, yb = a * cs - b * sn, b * cs + a * sn
    # the angle: half turns rounded to fp32 (pi 2^-24), the frequency in turns to 2^-53
    d_ang = math.pi * F32_HALF * 2 + 2 * math.pi * np.abs(pos)[:, None, None] * 2.0 ** -53
    for at, v in ((a_at, ya), (b_at, yb)):
        y[..., D_LAT + at] = v
        tol[..., D_LAT + at] = np.abs(v) * BF16_HALF + (np.abs(a) + np.abs(b)) * (d_ang + 8 * F32_HALF)
    return y, tol


# ------------------------------------------------------------------ the fp8 cache
def quantise(rows):
    """(codes uint8 [n, 512], scale float32 [n]) of float32 rows [n, >= 512], bit for bit."""
    x = np.asarray(rows, np.float32)[:, :D_LAT]
    fin = np.where(np.isfinite(x), np.abs(x), np.float32(0))
    scale = (fin.max(1) / np.float32(448.0)).astype(np.float32)
    with np.errstate(all="ignore"):
        ratio = np.where(scale[:, None] > 0, x / scale[:, None], x).astype(np.float32)
    nan = np.isnan(ratio)
    code = w.e4m3_encode(np.where(nan, 0.0, ratio).astype(np.float64))
    return np.where(nan, np.uint8(0x7F), code).astype(np.uint8), scale


def dequantise_rows(codes, scale, rope_f64):
    return np.concatenate([e4m3_values()[codes] * scale.astype(np.float64)[:, None], rope_f64], 1)


# ------------------------------------------------------------------ attention
def visible(mask, b, t, n, q_len):
    """bool [n]: the keys that draft t of stream b sees (mask: uint8 [B, q, q] or None)."""
    v = np.ones(n, bool)
    d = np.arange(q_len) <= t if mask is None else mask[b, t] != 0
    v[n - q_len:] = d
    return v


def attention(q, keys_of, seq, mask, scale):
    """(out, lse, out bound, lse bound).  q float64 [B, q_len, H, 576]; keys_of(b) float64 [n, 576]."""
    B, q_len, H, _ = q.shape
    out, lse = np.zeros((B, q_len, H, D_LAT)), np.full((B, q_len, H), -np.inf)
    t_out, t_lse = np.zeros_like(out), np.zeros_like(lse)
    for b in range(B):
        n = int(seq[b])
        k = keys_of(b)[:n]
        for t in range(q_len):
            v = visible(mask, b, t, n, q_len)
            if not v.any():
                continue
            kk = k[v]
            x = scale * (q[b, t] @ kk.T)                                  # [H, keys]
            m = x.max(1, keepdims=True)
            e = np.exp(x - m)
            lse[b, t] = m[:, 0] + np.log(e.sum(1))
            p = e / e.sum(1, keepdims=True)
            out[b, t] = p @ kk[:, :D_LAT]
            # scores: products of 16-bit queries and codes are exact in fp32, the sum of 576 rounds
            # (or truncates: a whole step) at each partial sum; scaling and exponent add a few steps
            ds = (600 * 2 * F32_HALF) * scale * (np.abs(q[b, t]) @ np.abs(kk).T) + 16 * F32_HALF * (np.abs(x) + np.abs(m))
            ds = ds.max(1)
            t_lse[b, t] = ds + (len(kk) + 64) * F32_HALF + 8 * F32_HALF * np.abs(lse[b, t])
            # probabilities rounded to 16 bits, each off by at most half a bf16 step; the output's own
            # rounding; a score's error is a relative error of its probability and of the sum
            size = p @ np.abs(kk[:, :D_LAT])
            t_out[b, t] = np.abs(out[b, t]) * BF16_HALF + size * (BF16_HALF * (1 + BF16_HALF) + 2 * ds[:, None]
                                                                 + 2 * (len(kk) + 64) * F32_HALF)
    return out, lse, t_out, t_lse


# ------------------------------------------------------------------ acceptance
def accept(p, q, tokens, parents, u, u_next):
    """(n_accepted, tokens, path) of one stream in float64; p, q [q_len, V] (q may be None)."""
    q_len, V = p.shape
    clean = lambda r: np.where(r > 0, np.minimum(r, 1.0), 0.0)
    par = list(range(-1, q_len - 1)) if parents is None else [int(x) for x in parents]
    node, went = 0, []
    while True:
        row = clean(p[node].astype(np.float64))
        R, S = row.copy(), 1.0
        for k in range(1, q_len):
            if par[k] != node or not 0 <= par[k] < k or not 0 <= tokens[k] < V:
                continue
            x = int(tokens[k])
            d = clean(q[node].astype(np.float64)) if q is not None else None
            if float(u[k]) * (1.0 if d is None else d[x]) * S < R[x]:
                went.append(k)
                node = k
                break
            if d is None:
                R[x] = 0.0
            else:
                R = np.maximum(R - S * d, 0.0)
            S = R.sum()
        else:
            break
    if R.sum() == 0:
        R = row
    cum = np.cumsum(R)
    nxt = int(np.argmax(cum > float(u_next) * cum[-1])) if cum[-1] > 0 else -1
    toks = [int(tokens[k]) for k in went] + [nxt]
    pad = lambda v: v + [-1] * (q_len - len(v))
    return len(went), pad(toks), pad(went)
