"""What is measured of the operators around the fp8 latent cache of one speculative-verify step.

The step, in order: the queries' and the new key rows' norm and position rotation
(``qk_norm_rope``), the quantising append of the rows to the fp8 cache
(``kv_append_quant``), the verify attention over that cache (``verify_attn_fp8``), and the
acceptance of the drafted tokens against the target's probabilities (``draft_verify``);
``kv_read_fp8`` reads cached rows back as bf16 (a prefix that another pass needs dense).

``own`` False computes each operator in elementary torch operations, True calls the
framework.  Both take the same state from ``prepare``.
"""
import math

import torch

own = False

D_LAT, D_ROPE, D_ROW = 512, 64, 576
E4M3_MAX = 448.0
SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6
DEV = "cuda"


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one stream's verify step, nine drafts on a rank with eight heads: latency
        {"name": "rope-step", "op": "norm_rope", "T": 9, "H": 8, "q_norm": False, "interleaved": True, "pos": 65545},
        # a full decode batch, 128 streams of nine drafts with all 64 heads: bandwidth
        {"name": "rope-batch", "op": "norm_rope", "T": 1152, "H": 64, "q_norm": True, "interleaved": False, "pos": 1 << 20},
        # the draft rows of eight streams entering the cache before a verify call
        {"name": "append-drafts", "op": "append", "rows": 72, "pool": 16384},
        # a prompt's rows entering the cache after its prefill
        {"name": "append-prompt", "op": "append", "rows": 46080, "pool": 131072},
        # a short prefix read back
        {"name": "read-4k", "op": "read", "rows": 4105, "pool": 16384},
        # all keys of a mixed batch read back from scattered slots
        {"name": "read-batch", "op": "read", "rows": 169817, "pool": 262144},
        # the smallest verify call: one stream, prefix 256
        {"name": "attn-256", "op": "attn", "B": 1, "q_len": 9, "H": 8, "lo": 256, "hi": 256, "mask": "chain", "pool": 512},
        # one stream with every head on the GPU: bound by the matrix products
        {"name": "attn-4k-h64", "op": "attn", "B": 1, "q_len": 9, "H": 64, "lo": 4096, "hi": 4096, "mask": "tree", "pool": 8192},
        # eight streams of mixed prefixes up to 46080 keys, draft trees: bound by the cache's bytes
        {"name": "attn-mixed", "op": "attn", "B": 8, "q_len": 9, "H": 8, "lo": 1024, "hi": 46080, "mask": "packed", "pool": 262144},
        # plain decode (one token a stream), 32 streams with 64 heads
        {"name": "attn-decode", "op": "attn", "B": 32, "q_len": 1, "H": 64, "lo": 1500, "hi": 2047, "mask": "chain", "pool": 65536},
        # one stream's chain of eight drafts, a small vocabulary: latency
        {"name": "accept-chain", "op": "accept", "B": 1, "q_len": 9, "V": 32000, "tree": False, "drafter": True},
        # a batch of draft trees over a large vocabulary: bandwidth
        {"name": "accept-trees", "op": "accept", "B": 64, "q_len": 16, "V": 131072, "tree": True, "drafter": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


HEADS = (1, 2, 3, 4, 5, 8, 12, 16, 20, 24, 32, 48, 64, 96, 128)


def draw(rng):
    op = rng.choice(("norm_rope", "append", "read", "attn", "attn", "accept"))
    if op == "norm_rope":
        H = rng.choice(HEADS)
        return {"op": op, "T": _log_int(rng, 1, 73728 // max(H, 16)), "H": H, "q_norm": rng.random() < 0.5,
                "interleaved": rng.random() < 0.5, "pos": _log_int(rng, 64, 1 << 20)}
    if op == "append":
        n = _log_int(rng, 1, 46080)
        return {"op": op, "rows": n, "pool": min(131072, n + _log_int(rng, 16, 65536))}
    if op == "read":
        n = _log_int(rng, 1, 169817)
        return {"op": op, "rows": n, "pool": min(262144, n + _log_int(rng, 16, 65536))}
    if op == "attn":
        while True:
            B, q_len, H = _log_int(rng, 1, 32), rng.choice((1, 1, 2, 5, 9, 9, 12, 17, 33, 64)), rng.choice(HEADS)
            hi = _log_int(rng, 1, 46080)
            # cost bounds: the cache's bytes and the products of the largest listed cases
            if B * (hi + q_len) <= 170000 and B * (hi + q_len) * q_len * H <= 9000000 and q_len * H <= 1152:
                break
        return {"op": op, "B": B, "q_len": q_len, "H": H, "lo": rng.randint(max(0, hi // 4), hi), "hi": hi,
                "mask": rng.choice(("chain", "tree", "packed")), "pool": B * (hi + q_len) + rng.randint(1, 4096)}
    while True:
        B, q_len, V = _log_int(rng, 1, 64), rng.randint(1, 17), _log_int(rng, 500, 131072)
        if B * q_len * V <= 64 * 16 * 131072 // 2:
            break
    return {"op": op, "B": B, "q_len": q_len, "V": V, "tree": rng.random() < 0.5, "drafter": rng.random() < 0.75}


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _host_gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _token_rows(g, n):
    """bf16 rows [n, 576]: token norms that differ, as a projection gives them."""
    size = torch.exp(0.5 * _normal(g, n, 1))
    return (_normal(g, n, D_ROW) * size).to(torch.bfloat16)


def _quantised_pool(g, n):
    """An fp8 cache as the quantising append leaves it: codes, per-token scales, bf16 ropes."""
    rows = _token_rows(g, n).float()
    lat = rows[:, :D_LAT] / rows[:, :D_LAT].square().mean(1, keepdim=True).sqrt() * torch.exp(0.2 * _normal(g, n, 1))
    scale = lat.abs().amax(1) / E4M3_MAX
    codes = (lat / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    rope = _normal(g, n, D_ROPE).to(torch.bfloat16)
    return codes, scale.contiguous(), rope


def _parents(h, B, q_len, tree):
    """parent[b, i] of draft node i (node 0 is the root): a chain, or U{0..i-1}."""
    i = torch.arange(q_len)
    if not tree:
        return (i - 1).expand(B, q_len).contiguous()
    u = torch.rand((B, q_len), generator=h, dtype=torch.float64)
    par = torch.minimum((u * i).long(), (i - 1).clamp(min=0))
    par[:, :1] = -1
    return par


def _tree_mask(par):
    """mask[b, t, i] = 1 where draft i is t or an ancestor of t."""
    B, q = par.shape
    m = torch.zeros((B, q, q), dtype=torch.uint8)
    b = torch.arange(B)
    for t in range(q):
        if t:
            m[:, t] = m[b, par[:, t]]
        m[:, t, t] = 1
    return m


def _prepare_attn(c, g, h):
    B, q_len, H = c["B"], c["q_len"], c["H"]
    pre = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=h)
    if B > 1:
        pre[0], pre[-1] = c["hi"], c["lo"]
    seq = pre + q_len
    stride = int(seq.max())
    lat, scale, rope = _quantised_pool(g, c["pool"])
    perm = torch.randperm(c["pool"], generator=h).to(torch.int32)
    first = torch.cumsum(seq, 0) - seq
    j = torch.arange(stride)
    at = first[:, None] + torch.minimum(j[None], seq[:, None] - 1)
    s = {"q": _normal(g, B, q_len, H, D_ROW).to(torch.bfloat16), "lat": lat, "scale": scale, "rope": rope,
         "table": perm[at].to(DEV), "seq": seq.to(torch.int32).to(DEV), "mask": None,
         # the static buffers that a serving loop keeps
         "out": torch.empty((B, q_len, H, D_LAT), dtype=torch.bfloat16, device=DEV),
         "lse": torch.empty((B, q_len, H), dtype=torch.float32, device=DEV),
         "workspace": torch.empty(96 << 20, dtype=torch.uint8, device=DEV)}
    if c["mask"] != "chain":
        m = _tree_mask(_parents(h, B, q_len, True))
        if c["mask"] == "packed":
            m = (m.long() << torch.arange(q_len)).sum(2)   # bit i of word (b, t): draft t sees draft i
        s["mask"] = m.to(DEV)
    return s


def _prepare_accept(c, g, h):
    B, q_len, V = c["B"], c["q_len"], c["V"]
    par = _parents(h, B, q_len, c["tree"])
    # rank of each node among its parent's children: each child is a draw of its own
    same = (par[:, :, None] == par[:, None, :]) & (torch.arange(q_len)[None, :] < torch.arange(q_len)[:, None])
    rank = same.sum(2)
    z = 4.0 * _normal(g, B, q_len, V)
    p = torch.softmax(z, -1)
    q = torch.softmax(z + 0.8 * _normal(g, B, q_len, V), -1)
    del z
    draws = torch.multinomial(q.view(B * q_len, V), int(rank.max()) + 1, replacement=True, generator=g).view(B, q_len, -1)
    b = torch.arange(B, device=DEV)[:, None]
    tok = draws[b, par.clamp(min=0).to(DEV), rank.to(DEV)]
    return {"p": p, "q": q if c["drafter"] else None, "tokens": tok.to(torch.int32).contiguous(),
            "parents": par.to(torch.int32).to(DEV) if c["tree"] else None,
            "u": torch.rand((B, q_len), generator=g, device=DEV), "u_next": torch.rand((B,), generator=g, device=DEV)}


def prepare(case, seed):
    c = dict(case)
    g, h = _gen(seed), _host_gen(seed)
    if c["op"] == "norm_rope":
        T, H = c["T"], c["H"]
        freq = 10000.0 ** (-torch.arange(0, D_ROPE, 2, dtype=torch.float64) / D_ROPE)
        s = {"x_q": _normal(g, T, H, D_ROW).to(torch.bfloat16), "x_kv": _token_rows(g, T),
             "positions": torch.randint(0, c["pos"], (T,), generator=g, device=DEV, dtype=torch.int32),
             "inv_freq": freq.float().to(DEV),
             "q_weight": (1 + 0.1 * _normal(g, D_LAT)).to(torch.bfloat16) if c["q_norm"] else None,
             "kv_weight": (1 + 0.1 * _normal(g, D_LAT)).to(torch.bfloat16),
             "q_out": torch.empty((T, H, D_ROW), dtype=torch.bfloat16, device=DEV),
             "kv_out": torch.empty((T, D_ROW), dtype=torch.bfloat16, device=DEV)}
    elif c["op"] in ("append", "read"):
        lat, scale, rope = _quantised_pool(g, c["pool"])
        s = {"lat": lat, "scale": scale, "rope": rope,
             "slots": torch.randperm(c["pool"], generator=g, device=DEV)[:c["rows"]].to(torch.int32)}
        if c["op"] == "append":
            s["rows"] = _token_rows(g, c["rows"])
        else:
            s["out"] = torch.empty((c["rows"], D_ROW), dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "attn":
        s = _prepare_attn(c, g, h)
    else:
        s = _prepare_accept(c, g, h)
    s["case"] = c
    return s


# ----------------------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    a, b = x[..., :D_ROPE // 2], x[..., D_ROPE // 2:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _norm_rope_plain(x, weight, positions, inv_freq, interleaved):
    y = x.float()
    lat, rope = y[..., :D_LAT], y[..., D_LAT:]
    if weight is not None:
        lat = lat * torch.rsqrt(lat.square().mean(-1, keepdim=True) + EPS) * weight.float()
    angle = positions.double()[:, None] * inv_freq.double()
    angle = angle.view((angle.shape[0],) + (1,) * (x.dim() - 2) + (D_ROPE // 2,))
    rope = _rotate(rope, torch.cos(angle).float(), torch.sin(angle).float(), interleaved)
    return torch.cat((lat, rope), -1).to(torch.bfloat16)


def _append_plain(s):
    x = s["rows"].float()
    lat, slots = x[:, :D_LAT], s["slots"].long()
    peak = lat.abs().amax(1)
    scale = peak / torch.full_like(peak, E4M3_MAX)         # a true division: by a number it is a product
    ratio = torch.where(scale[:, None] > 0, lat / scale[:, None], lat * 0)
    s["lat"][slots] = ratio.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    s["scale"][slots] = scale
    s["rope"][slots] = s["rows"][:, D_LAT:]


def _dequantised(s, slots):
    """fp32 rows [..., 576] of the cache."""
    lat = s["lat"][slots].view(torch.float8_e4m3fn).float()
    return torch.cat((lat * s["scale"][slots].unsqueeze(-1), s["rope"][slots].float()), -1)


def _seen(s, B, q_len, n_max):
    """[B, q_len, n_max]: whether draft t of stream b sees key j."""
    j = torch.arange(n_max, device=DEV)
    t = torch.arange(q_len, device=DEV)
    i = j - (s["seq"].long()[:, None] - q_len)             # [B, n_max]: draft index of key j, < 0: prefix
    m = s["mask"]
    if m is None:
        draft = (t[:, None] >= t).expand(B, q_len, q_len)
    elif m.dtype == torch.int64:
        draft = ((m[:, :, None] >> t) & 1) != 0
    else:
        draft = m != 0
    at = i.clamp(0, q_len - 1)[:, None, :].expand(B, q_len, n_max)
    return ((i < 0)[:, None, :] | torch.gather(draft, 2, at)) & (i < q_len)[:, None, :]


def _attn_plain(s):
    B, q_len, H, _ = s["q"].shape
    n_max = s["table"].shape[1]
    k = _dequantised(s, s["table"].long())                 # [B, n_max, 576]
    x = torch.matmul(s["q"].float().view(B, q_len * H, D_ROW), k.transpose(1, 2)).mul_(SCALE)
    x = x.view(B, q_len, H, n_max).masked_fill_(~_seen(s, B, q_len, n_max)[:, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = x.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, q_len * H, n_max), k[:, :, :D_LAT]).view(B, q_len, H, D_LAT)
    out = torch.where(total > 0, o / total, torch.zeros_like(o))
    return {"out": out.to(torch.bfloat16), "lse": (top + total.log()).squeeze(-1)}


def _accept_plain(s):
    """The walk down the draft tree, node after node; at the current node R = max(p - A q, 0) is what
    the rejections among its children have left of the target's distribution, S its sum."""
    p, q, tok = s["p"], s["q"], s["tokens"].long()
    B, q_len, V = p.shape
    b = torch.arange(B, device=DEV)
    par = s["parents"].long() if s["parents"] is not None else (torch.arange(q_len, device=DEV) - 1).expand(B, q_len)
    cur = torch.zeros(B, dtype=torch.long, device=DEV)
    n_acc = torch.zeros_like(cur)
    left = p[:, 0].double()                                # R
    total = torch.ones(B, dtype=torch.float64, device=DEV) # S: one before any rejection
    tokens = torch.full((B, q_len), -1, dtype=torch.long, device=DEV)
    path = tokens.clone()
    for i in range(1, q_len):
        x, here = tok[:, i], par[:, i] == cur
        qx = q[b, cur, x].double() if q is not None else torch.ones(B, dtype=torch.float64, device=DEV)
        yes = here & (s["u"][:, i].double() * qx * total < left[b, x])
        no = here & ~yes
        if q is not None:
            rest = (left - total[:, None] * q[b, cur].double()).clamp(min=0)
        else:
            rest = left.clone()
            rest[b, x] = 0
        left = torch.where(yes[:, None], p[:, i].double(), torch.where(no[:, None], rest, left))
        total = torch.where(yes, torch.ones_like(total), torch.where(no, rest.sum(1), total))
        tokens[b, n_acc] = torch.where(yes, x, tokens[b, n_acc])
        path[b, n_acc] = torch.where(yes, torch.full_like(x, i), path[b, n_acc])
        n_acc = n_acc + yes.long()
        cur = torch.where(yes, torch.full_like(cur, i), cur)
    whole = left.sum(1)
    left = torch.where((whole > 0)[:, None], left, p[b, cur].double())
    cdf = torch.cumsum(left, 1)
    hit = cdf > s["u_next"].double()[:, None] * cdf[:, -1:]
    nxt = torch.argmax(hit.to(torch.uint8), 1)
    tokens[b, n_acc] = nxt
    return {"accepted": n_acc.to(torch.int32), "tokens": tokens.to(torch.int32), "path": path.to(torch.int32)}


def run(s):
    op = s["case"]["op"]
    if own:
        import mla_speculative_verify_attention_gb300 as mv
    if op == "norm_rope":
        c = s["case"]
        if own:
            q, kv = mv.qk_norm_rope(s["x_q"], s["x_kv"], s["positions"], s["inv_freq"], q_weight=s["q_weight"],
                                    kv_weight=s["kv_weight"], eps=EPS, interleaved=c["interleaved"], q_out=s["q_out"],
                                    kv_out=s["kv_out"])
        else:
            q = _norm_rope_plain(s["x_q"], s["q_weight"], s["positions"], s["inv_freq"], c["interleaved"])
            kv = _norm_rope_plain(s["x_kv"], s["kv_weight"], s["positions"], s["inv_freq"], c["interleaved"])
        return {"q": q, "kv": kv}
    if op == "append":
        if own:
            mv.kv_append_quant(s["lat"], s["scale"], s["rope"], s["slots"], s["rows"])
        else:
            _append_plain(s)
        return {"lat": s["lat"].view(torch.float8_e4m3fn), "scale": s["scale"], "rope": s["rope"]}
    if op == "read":
        if own:
            return {"rows": mv.kv_read_fp8(s["lat"], s["scale"], s["rope"], s["slots"], out=s["out"])}
        return {"rows": _dequantised(s, s["slots"].long()).to(torch.bfloat16)}
    if op == "attn":
        if own:
            out, lse = mv.verify_attn_fp8(s["q"], s["lat"], s["scale"], s["rope"], s["table"], s["seq"], s["mask"],
                                          SCALE, out=s["out"], lse=s["lse"], workspace=s["workspace"])
            return {"out": out, "lse": lse}
        return _attn_plain(s)
    if own:
        n, tokens, path = mv.draft_verify(s["p"], s["q"], s["tokens"], s["parents"], s["u"], s["u_next"])
        return {"accepted": n, "tokens": tokens, "path": path}
    return _accept_plain(s)


# ----------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "norm_rope":
        return {"bytes": 2 * c["T"] * (c["H"] + 1) * D_ROW * 2 + c["T"] * 4, "flops": c["T"] * (c["H"] + 1) * 4 * D_ROW}
    if c["op"] in ("append", "read"):
        # one bf16 row, one quantised row (codes, scale, rope) and its slot index
        return {"bytes": c["rows"] * (2 * D_ROW + D_LAT + 4 + 2 * D_ROPE + 4), "flops": c["rows"] * 3 * D_LAT}
    if c["op"] == "attn":
        rows = c["B"] * c["q_len"] * c["H"]
        keys = c["B"] * ((c["lo"] + c["hi"]) / 2 + c["q_len"])
        return {"bytes": keys * (D_LAT + 4 + 2 * D_ROPE + 4) + rows * (2 * D_ROW + 2 * D_LAT + 4),
                "flops": 2 * (D_ROW + D_LAT) * keys * c["q_len"] * c["H"]}
    # the rows that the next token is drawn from: the target's, and the drafter's where a draft was rejected
    return {"bytes": c["B"] * c["V"] * (8 if c["drafter"] else 4), "flops": c["B"] * c["V"] * 4}


# ----------------------------------------------------------------------------- 64 bits
def _e4m3_values():
    """The 256 codes' values: sign, four exponent bits of bias 7, three mantissa bits."""
    v = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        a = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v.append(-a if code & 128 else a)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _exact_norm_rope(s):
    c, got = s["case"], {}
    turn = s["positions"].double()[:, None] * s["inv_freq"].double()[None]
    z = torch.complex(torch.cos(turn), torch.sin(turn))     # one complex factor a pair
    for name, x, w in (("q", s["x_q"], s["q_weight"]), ("kv", s["x_kv"][:, None], s["kv_weight"])):
        y = x.double().clone()
        if w is not None:
            y[..., :D_LAT] *= w.double() / (y[..., :D_LAT].pow(2).sum(-1, keepdim=True) / D_LAT + EPS).sqrt()
        r = y[..., D_LAT:]
        pair = r.unflatten(-1, (32, 2)) if c["interleaved"] else r.unflatten(-1, (2, 32)).transpose(-1, -2)
        turned = torch.view_as_real(torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous()) * z[:, None])
        y[..., D_LAT:] = turned.flatten(-2) if c["interleaved"] else turned.transpose(-1, -2).flatten(-2)
        got[name] = y if name == "q" else y[:, 0]
    return got


def _exact_append(s):
    values = _e4m3_values()
    lat, scale, rope = values[s["lat"].long()], s["scale"].double(), s["rope"].double()
    at, x = s["slots"].long(), s["rows"].double()
    peak = x[:, :D_LAT].abs().max(1).values
    sc = (peak / E4M3_MAX).float().double()
    ratio = torch.where(sc[:, None] > 0, x[:, :D_LAT] / sc[:, None], torch.zeros_like(x[:, :D_LAT]))
    grid = values[:127]                                     # the non-negative finite values, ascending
    size = ratio.abs().clamp(max=E4M3_MAX)
    up = torch.searchsorted(grid, size).clamp(max=126)
    low = (up - 1).clamp(min=0)
    d_up, d_low = grid[up] - size, size - grid[low]
    code = torch.where((d_up < d_low) | ((d_up == d_low) & (up % 2 == 0)), up, low)
    lat[at], scale[at], rope[at] = torch.copysign(grid[code], ratio), sc, x[:, D_LAT:]
    return {"lat": lat, "scale": scale, "rope": rope}


def _exact_rows(s, at):
    return torch.cat((_e4m3_values()[s["lat"][at].long()] * s["scale"][at].double()[:, None], s["rope"][at].double()), 1)


def _exact_attn(s):
    B, q_len, H, _ = s["q"].shape
    out = torch.zeros((B, q_len, H, D_LAT), dtype=torch.float64, device=DEV)
    lse = torch.full((B, q_len, H), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        n = int(s["seq"][b])
        k = _exact_rows(s, s["table"][b, :n].long())
        for t in range(q_len):
            keys = list(range(q_len))
            if s["mask"] is None:
                keys = keys[:t + 1]
            elif s["mask"].dim() == 2:
                keys = [i for i in keys if (int(s["mask"][b, t]) >> i) & 1]
            else:
                keys = [i for i, seen in enumerate(s["mask"][b, t].tolist()) if seen]
            kk = torch.cat((k[:n - q_len], k[n - q_len:][keys]))
            x = SCALE * (s["q"][b, t].double() @ kk.T)
            lse[b, t] = torch.logsumexp(x, 1)
            out[b, t] = torch.exp(x - lse[b, t][:, None]) @ kk[:, :D_LAT]
    return {"out": out, "lse": lse}


def _exact_accept(s):
    B, q_len, V = s["p"].shape
    n_acc, tokens, path = [], [], []
    tok, u, u_next = s["tokens"].tolist(), s["u"].double().tolist(), s["u_next"].double().tolist()
    par = s["parents"].tolist() if s["parents"] is not None else [list(range(-1, q_len - 1))] * B
    for b in range(B):
        node, went, said = 0, [], []
        while True:
            p = s["p"][b, node].double()
            r, norm, stop = p, 1.0, True
            for k in [k for k in range(1, q_len) if par[b][k] == node]:
                q = s["q"][b, node].double() if s["q"] is not None else torch.nn.functional.one_hot(
                    torch.tensor(tok[b][k], device=DEV), V).double()
                if u[b][k] * float(q[tok[b][k]]) < float(r[tok[b][k]]) / norm:
                    went.append(k)
                    said.append(tok[b][k])
                    node, stop = k, False
                    break
                r = torch.clamp(r / norm - q, min=0) if s["q"] is not None else (r / norm) * (1 - q)
                norm = float(r.sum())
                if norm == 0:
                    r, norm = p * 0, 1.0
            if stop:
                break
        if float(r.sum()) == 0:
            r = p
        cdf = torch.cumsum(r, 0)
        nxt = int((cdf <= u_next[b] * float(cdf[-1])).sum())
        n_acc.append(len(went))
        tokens.append(said + [nxt] + [-1] * (q_len - 1 - len(said)))
        path.append(went + [-1] * (q_len - len(went)))
    as_int = lambda v: torch.tensor(v, dtype=torch.int32)
    return {"accepted": as_int(n_acc), "tokens": as_int(tokens), "path": as_int(path)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        return _exact_norm_rope(s)
    if op == "append":
        return _exact_append(s)
    if op == "read":
        return {"rows": _exact_rows(s, s["slots"].long())}
    return _exact_attn(s) if op == "attn" else _exact_accept(s)
