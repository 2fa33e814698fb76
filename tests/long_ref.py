"""Plain float64 forms of the long-context operators (attention under score rules, key weights, eviction),
with the error bounds that a right kernel keeps, and inputs for their tests."""
import numpy as np
import torch

import step_ref as ref
import workloads as w

F32_HALF = ref.F32_HALF


class Rules:
    """softcap, slopes [H], key_pos [B, stride], window, prefix_lens [B], key_doc [B, stride]: numpy or None."""

    def __init__(self, softcap=0.0, slopes=None, key_pos=None, window=0, prefix_lens=None, key_doc=None):
        self.softcap, self.slopes, self.key_pos, self.window = softcap, slopes, key_pos, window
        self.prefix_lens, self.key_doc = prefix_lens, key_doc

    def on(self, device):
        put = lambda a, t: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(t).to(device)
        return dict(softcap=self.softcap, slopes=put(self.slopes, torch.float32), key_pos=put(self.key_pos, torch.int32),
                    window=self.window, prefix_lens=put(self.prefix_lens, torch.int32),
                    key_doc=put(self.key_doc, torch.int32))

    def seen(self, mask, b, t, n, q_len):
        """(bool [n]: the keys that draft t sees, positions relative to the draft's own)."""
        pos = np.arange(n, dtype=np.int64) if self.key_pos is None else self.key_pos[b, :n].astype(np.int64)
        own = n - q_len + t
        v = ref.visible(mask, b, t, n, q_len)
        if self.window:
            v = v & (pos[own] - pos < self.window)
        if self.prefix_lens is not None:
            v = v | (pos < self.prefix_lens[b])
        if self.key_doc is not None:
            doc = self.key_doc[b, :n]
            v = v & ((doc == doc[own]) | (doc < 0))
        return v, pos - pos[own]

    def scores(self, q, k, away, scale):
        """(z [H, keys], bound) for queries q [H, 576] and key rows k."""
        z = scale * (q @ k.T)
        # products of 16-bit queries and keys are exact in fp32, the sum of 576 rounds (or truncates: a whole
        # step) at each partial sum; scaling adds a few steps
        tol = (600 * 2 * F32_HALF) * scale * (np.abs(q) @ np.abs(k).T) + 8 * F32_HALF * np.abs(z)
        if self.softcap > 0:
            z = self.softcap * np.tanh(z / self.softcap)
            tol = tol + np.abs(z) * (2.0 ** -19 + 4 * F32_HALF)   # tanh's slope is at most 1; its own error
        if self.slopes is not None:
            bias = self.slopes.astype(np.float64)[:, None] * away[None, :]
            z = z + bias
            tol = tol + 6 * F32_HALF * np.abs(bias)
        return z, tol


def attention(q, keys_of, seq, mask, scale, rules):
    """(out, lse, out bound, lse bound).  q float64 [B, q_len, H, 576]; keys_of(b) float64 [n, 576]."""
    B, q_len, H, _ = q.shape
    out, lse = np.zeros((B, q_len, H, 512)), np.full((B, q_len, H), -np.inf)
    t_out, t_lse = np.zeros_like(out), np.zeros_like(lse)
    for b in range(B):
        n = int(seq[b])
        k = keys_of(b)[:n]
        for t in range(q_len):
            v, away = rules.seen(mask, b, t, n, q_len)
            if not v.any():
                continue
            kk = k[v]
            x, tol = rules.scores(q[b, t], kk, away[v], scale)
            m = x.max(1, keepdims=True)
            e = np.exp(x - m)
            lse[b, t] = m[:, 0] + np.log(e.sum(1))
            p = e / e.sum(1, keepdims=True)
            out[b, t] = p @ kk[:, :512]
            # the exponent's argument in fp32; a score's error counts by its key's weight, once in the weight
            # and once in the sum
            ds = tol + 16 * F32_HALF * (np.abs(x) + np.abs(m))
            mean = (p * ds).sum(1)
            size = np.abs(kk[:, :512])
            t_lse[b, t] = mean * 1.01 + (len(kk) + 64) * F32_HALF + 8 * F32_HALF * np.abs(lse[b, t])
            # probabilities rounded to fp16 (2^-11 of each, and 2^-32 of the row's largest weight, probability
            # times key scale, where they are small: bounded here by the largest probability times the largest
            # value), the output's own rounding to bf16
            small = 2.0 ** -30 * size.max() * len(kk) * p.max(1)
            t_out[b, t] = np.abs(out[b, t]) * ref.BF16_HALF + (p * (ds + mean[:, None] + 2.0 ** -11 * 1.01)) @ size * (
                1 + ref.BF16_HALF) + (p @ size) * 2 * (len(kk) + 64) * F32_HALF + small[:, None]
    return out, lse, t_out, t_lse


def key_weights(q, keys_of, seq, mask, scale, rules, lse, counted, weights, decay, before):
    """(out [B, stride], bound): `before` is what out held; lse, weights float64 or None."""
    B, q_len, H, _ = q.shape
    out, tol = before.copy(), np.zeros_like(before)
    for b in range(B):
        n = int(seq[b])
        if not q_len <= n <= out.shape[1]:
            continue
        k, p = keys_of(b)[:n], n - q_len
        new, err = np.zeros(n), np.zeros(n)
        for t in range(q_len):
            v, away = rules.seen(mask, b, t, n, q_len)
            if (counted is not None and not counted[b, t]) or not v.any():
                continue
            z, ds = rules.scores(q[b, t], k[v], away[v], scale)
            with np.errstate(invalid="ignore"):
                e = np.where(np.isneginf(lse[b, t])[:, None], 0.0, np.exp(z - lse[b, t][:, None]))
                d = ds + 16 * F32_HALF * (np.abs(z) + np.abs(np.nan_to_num(lse[b, t], neginf=0.0))[:, None]) + 2.0 ** -21
            new[v] += e.sum(0)
            err[v] += (e * d).sum(0) * 1.01
        old = np.zeros(n)
        if weights is not None:
            old[:p] = decay * weights[b, :p]
        out[b, :n] = old + new
        # sums of q_len H numbers of one sign, in any order; results below 2^-126 may be 0
        tol[b, :n] = err + new * (q_len * H + 8) * F32_HALF + (np.abs(old) + new) * 4 * F32_HALF + q_len * H * 2.0 ** -125
    return out, tol


def evict(table, seq, weights, budget, sink, recent, key_pos, key_doc, outs):
    """What the outputs (a dict of numpy arrays, some None) hold afterwards, bit for bit."""
    o = {k: None if v is None else v.copy() for k, v in outs.items()}
    for b, n in enumerate(int(x) for x in seq):
        o["lens_out"][b], o["n_freed"][b] = n, 0
        if not 0 <= n <= table.shape[1]:
            continue
        want = int(budget if np.isscalar(budget) else budget[b])
        left = min(n, max(want, sink + recent, 0))
        lo, hi = min(sink, n), max(min(sink, n), n - recent)
        wt = weights[b, :n].astype(np.float64)
        # NaN first, then by weight, then by index
        by_weight = sorted(range(lo, hi), key=lambda j: (not np.isnan(wt[j]), -wt[j] if not np.isnan(wt[j]) else 0.0, j))
        keep = sorted(list(range(lo)) + by_weight[:left - lo - (n - hi)] + list(range(hi, n)))
        gone = sorted(set(range(n)) - set(keep))
        for name, src in (("table_out", table), ("weights_out", weights),
                          ("pos_out", np.broadcast_to(np.arange(table.shape[1], dtype=np.int32), table.shape)
                           if key_pos is None else key_pos), ("doc_out", key_doc)):
            if o.get(name) is not None:
                o[name][b, :left] = src[b][keep]
        if o["freed"] is not None:
            o["freed"][b, :n - left] = table[b][gone]
        o["lens_out"][b], o["n_freed"][b] = left, n - left
    return o


# ------------------------------------------------------------------ inputs
class Step:
    """A step's queries, cache and tables: numpy where the reference wants them, device tensors on call."""

    def __init__(self, seed, lens, q_len, H, *, mask="chain", cache="fp8", stride=None, extra=5, q_size=1.0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.q_len, self.H = len(lens), q_len, H
        self.seq = np.array(lens, np.int32)
        self.stride = stride or max(int(self.seq.max()), q_len)
        pool = int(self.seq.sum()) + extra
        rows = torch.randn((pool, 576), generator=g).to(torch.bfloat16)
        self.table = torch.randint(0, pool, (self.B, self.stride), generator=g, dtype=torch.int32)
        perm, at = torch.randperm(pool, generator=g).to(torch.int32), 0
        for b, n in enumerate(lens):
            n = min(n, self.stride)
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.cache = cache
        if cache == "fp8":
            codes, scale = ref.quantise(rows.float().numpy())
            self.lat, self.scale, self.rope = torch.from_numpy(codes), torch.from_numpy(scale), rows[:, 512:].contiguous()
        else:
            self.kv = rows
        self.q = (torch.randn((self.B, q_len, H, 576), generator=g) * q_size).to(torch.bfloat16)
        self.mask = None
        if mask != "chain":
            par = w.tree_parents(seed + 1, self.B, q_len)
            self.mask = w.tree_mask_from_parents(np.asarray(par).astype(np.int64)).astype(np.uint8)
        self.packed = mask == "packed"

    def keys_of(self, b):
        at = self.table[b].numpy()
        if self.cache == "fp8":
            return ref.dequantise_rows(self.lat.numpy()[at], self.scale.numpy()[at], ref.f64(self.rope)[at])
        return ref.f64(self.kv)[at]

    def on(self, device):
        """(q, cache tensors .., table, seq, mask) as the calls take them."""
        cache = (self.lat, self.scale, self.rope) if self.cache == "fp8" else (self.kv,)
        mask = None
        if self.mask is not None:
            mask = torch.from_numpy(self.mask)
            if self.packed:
                bits = (self.mask.astype(np.uint64) << np.arange(self.q_len, dtype=np.uint64)).sum(2, dtype=np.uint64)
                mask = torch.from_numpy(bits.view(np.int64))
            mask = mask.to(device)
        return (self.q.to(device), *(t.to(device) for t in cache), self.table.to(device),
                torch.from_numpy(self.seq).to(device), mask)


def gaps(seed, B, stride, chance=0.5, start=0):
    """Ascending positions with gaps, as evictions leave them."""
    r = np.random.default_rng(seed)
    return (np.cumsum(1 + (r.random((B, stride)) < chance), 1) - 1 + start).astype(np.int32)


def slopes(H):
    return (2.0 ** (-8.0 * np.arange(1, H + 1) / H)).astype(np.float32)
