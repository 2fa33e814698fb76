"""What is measured of the operators for long contexts over the latent cache.

``verify_attn_fp8_rules`` is the verify attention under score rules (a tanh cap, a bias by
distance, a sliding window, a prefix that everyone sees, documents); ``key_weights_fp8`` and
``key_weights`` add up what weight each cached key got from a step's queries; ``kv_evict``
keeps each stream's heaviest keys and compacts its slot table.

``own`` False computes each operator in elementary torch operations, True calls the
framework.  Both take the same state from ``prepare``.
"""
import math

import torch

own = False

D_LAT, D_ROPE, D_ROW = 512, 64, 576
E4M3_MAX = 448.0
SCALE = 1.0 / math.sqrt(192.0)
DEV = "cuda"


# ----------------------------------------------------------------------------- cases
def listed():
    rules = {"cap": 0.0, "bias": False, "pos": False, "window": 0, "prefix": 0, "docs": 0}
    return [
        # one stream with a short prefix, capped scores with a bias by distance: latency
        {**rules, "name": "attn-256-capped", "op": "attn", "B": 1, "q_len": 9, "H": 8, "lo": 256, "hi": 256, "mask": "chain",
         "cap": 30.0, "bias": True},
        # eight streams whose caches were thinned by evictions, draft trees: the keys' positions have gaps
        {**rules, "name": "attn-mixed-evicted", "op": "attn", "B": 8, "q_len": 9, "H": 8, "lo": 1024, "hi": 46080,
         "mask": "packed", "cap": 50.0, "bias": True, "pos": True},
        # long streams under a sliding window beside a prefix that stays visible
        {**rules, "name": "attn-window", "op": "attn", "B": 16, "q_len": 9, "H": 8, "lo": 1024, "hi": 46080, "mask": "chain",
         "window": 4096, "prefix": 64},
        # plain decode, several documents packed into each stream
        {**rules, "name": "attn-decode-docs", "op": "attn", "B": 32, "q_len": 1, "H": 64, "lo": 1500, "hi": 2047,
         "mask": "chain", "docs": 3},
        # the keys' weights of one stream's verify step: latency
        {**rules, "name": "weights-256", "op": "weights", "B": 1, "q_len": 9, "H": 8, "lo": 256, "hi": 256, "mask": "chain",
         "cache": "fp8", "part": True},
        # a mixed batch of verify steps: bound by the cache's bytes
        {**rules, "name": "weights-mixed", "op": "weights", "B": 8, "q_len": 9, "H": 8, "lo": 1024, "hi": 46080,
         "mask": "packed", "cache": "fp8", "part": False},
        # the last 64 queries of a prompt look back over it, all heads: bound by the products
        {**rules, "name": "weights-prompt", "op": "weights", "B": 1, "q_len": 64, "H": 64, "lo": 4096, "hi": 4096,
         "mask": "chain", "cache": "fp8", "part": False},
        # decode over the bf16 cache, keys thinned before, capped scores
        {**rules, "name": "weights-decode-bf16", "op": "weights", "B": 32, "q_len": 1, "H": 64, "lo": 1500, "hi": 4095,
         "mask": "chain", "cache": "bf16", "part": False, "cap": 50.0, "pos": True, "bias": True},
        # one stream brought back to 2048 keys
        {"name": "evict-4k", "op": "evict", "B": 1, "lo": 4105, "hi": 4105, "budget": 2048, "sink": 4, "recent": 64,
         "docs": 0, "pos": False, "each": False},
        # a batch of long streams, positions and documents carried along
        {"name": "evict-batch", "op": "evict", "B": 64, "lo": 1024, "hi": 46089, "budget": 4096, "sink": 4, "recent": 256,
         "docs": 5, "pos": True, "each": True},
        # two streams of a million keys
        {"name": "evict-1m", "op": "evict", "B": 2, "lo": 1000003, "hi": 1 << 20, "budget": 131072, "sink": 16,
         "recent": 1024, "docs": 0, "pos": True, "each": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


HEADS = (1, 2, 3, 4, 5, 8, 12, 16, 20, 24, 32, 48, 64, 96, 128)


def draw(rng):
    op = rng.choice(("attn", "attn", "weights", "weights", "evict"))
    if op == "evict":
        while True:
            B, hi = _log_int(rng, 1, 64), _log_int(rng, 1, 1 << 20)
            if B * hi <= 1 << 21:
                break
        budget = _log_int(rng, 1, hi)
        sink = rng.randint(0, min(16, budget))
        return {"op": op, "B": B, "lo": rng.randint(max(0, hi // 8), hi), "hi": hi, "budget": budget, "sink": sink,
                "recent": rng.randint(0, min(1024, budget - sink)), "docs": rng.choice((0, 5)), "pos": rng.random() < 0.5,
                "each": rng.random() < 0.5}
    most = 9000000 if op == "attn" else 64 * 64 * 4160       # row and key pairs of the largest listed cases
    while True:
        B, q_len, H = _log_int(rng, 1, 32), rng.choice((1, 1, 2, 5, 9, 9, 12, 17, 33, 64)), rng.choice(HEADS)
        hi = _log_int(rng, 1, 46080)
        # cost bounds: the cache's bytes and the products of the largest listed cases
        if B * (hi + q_len) <= 170000 and B * (hi + q_len) * q_len * H <= most and (op == "weights" or q_len * H <= 1152):
            break
    c = {"op": op, "B": B, "q_len": q_len, "H": H, "lo": rng.randint(max(0, hi // 4), hi), "hi": hi,
         "mask": rng.choice(("chain", "tree", "packed")),
         "cap": rng.choice((0.0, 0.0, 10.0, 30.0, 50.0)), "bias": rng.random() < 0.5, "pos": rng.random() < 0.5,
         "window": rng.choice((0, 0, _log_int(rng, 16, 16384))), "prefix": rng.choice((0, rng.randint(1, 512))),
         "docs": rng.choice((0, 0, 4))}
    if op == "attn":
        if not (c["cap"] or c["bias"] or c["window"] or c["prefix"] or c["docs"]):
            c["cap"] = 20.0
    else:
        c.update(cache=rng.choice(("fp8", "bf16")), part=rng.random() < 0.3)
    return c


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


def _pool_rows(g, n):
    """fp32 key rows [n, 576]: normalised latents with a learned gain, rotated dims."""
    x = _normal(g, n, D_ROW)
    x[:, :D_LAT] *= torch.exp(0.2 * _normal(g, n, 1))
    return x


def _parents(h, B, q_len):
    """parent[b, i] of draft node i (node 0 is the root): U{0..i-1}."""
    i = torch.arange(q_len)
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


def _lengths(c, h):
    n = torch.randint(c["lo"], c["hi"] + 1, (c["B"],), generator=h)
    if c["B"] > 1:
        n[0], n[-1] = c["hi"], c["lo"]
    return n


def _docs_of(h, B, stride, docs):
    """Documents one after the other, the first keys shared by all (-1)."""
    at = torch.sort(torch.rand((B, docs), generator=h), 1).values * stride
    doc = (torch.arange(stride)[None, :, None] >= at[:, None, :]).sum(2) - 1
    return doc.to(torch.int32).to(DEV)


def _prepare_step(c, g, h):
    """A step's queries, cache, lengths, masks and rules."""
    B, q_len, H = c["B"], c["q_len"], c["H"]
    seq = _lengths(c, h) + q_len
    stride = int(seq.max())
    pool = int(seq.sum()) + 37
    rows = _pool_rows(g, pool)
    s = {}
    if c["op"] == "attn" or c["cache"] == "fp8":
        scale = rows[:, :D_LAT].abs().amax(1) / E4M3_MAX
        s["lat"] = (rows[:, :D_LAT] / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        s["scale"], s["rope"] = scale.contiguous(), rows[:, D_LAT:].to(torch.bfloat16)
    else:
        s["kv"] = rows.to(torch.bfloat16)
    del rows
    perm = torch.randperm(pool, generator=h).to(torch.int32)
    first = torch.cumsum(seq, 0) - seq
    at = first[:, None] + torch.minimum(torch.arange(stride)[None], seq[:, None] - 1)
    s.update(q=_normal(g, B, q_len, H, D_ROW).to(torch.bfloat16), table=perm[at].to(DEV), seq=seq.to(torch.int32).to(DEV),
             mask=None)
    if c["mask"] != "chain":
        m = _tree_mask(_parents(h, B, q_len))
        if c["mask"] == "packed":
            m = (m.long() << torch.arange(q_len)).sum(2)   # bit i of word (b, t): draft t sees draft i
        s["mask"] = m.to(DEV)
    s["rules"] = {"softcap": c["cap"], "window": c["window"],
                  # the usual geometric slopes of a bias by distance
                  "slopes": 2.0 ** (-8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H).to(DEV) if c["bias"] else None,
                  "key_pos": None, "prefix_lens": None, "key_doc": None}
    if c["pos"]:                                           # every key kept with a chance of a half
        gap = 1 + (torch.rand((B, stride), generator=h) < 0.5).long()
        s["rules"]["key_pos"] = (torch.cumsum(gap, 1) - 1).to(torch.int32).to(DEV)
    if c["prefix"]:
        s["rules"]["prefix_lens"] = torch.randint((c["prefix"] + 1) // 2, c["prefix"] + 1, (B,), generator=h).to(
            torch.int32).to(DEV)
    if c["docs"]:
        s["rules"]["key_doc"] = _docs_of(h, B, stride, c["docs"])
    return s


def prepare(case, seed):
    c = dict(case)
    g, h = _gen(seed), _host_gen(seed)
    B = c["B"]
    if c["op"] == "evict":
        seq = _lengths(c, h)
        stride = int(seq.max()) + 9
        # accumulated weights: spread over orders of magnitude, a tenth of the keys never seen
        wt = torch.exp(2.5 * _normal(g, B, stride) - 6) * (torch.rand((B, stride), generator=g, device=DEV) > 0.1)
        wt[:, :4] += 1
        s = {"table": torch.stack([torch.randperm(stride, generator=h) + b * stride for b in range(B)]).to(torch.int32).to(DEV),
             "seq": seq.to(torch.int32).to(DEV), "weights": wt, "pos": None, "doc": None, "budget": c["budget"]}
        if c["pos"]:
            gap = 1 + (torch.rand((B, stride), generator=h) < 0.5).long()
            s["pos"] = (torch.cumsum(gap, 1) - 1).to(torch.int32).to(DEV)
        if c["docs"]:
            s["doc"] = _docs_of(h, B, stride, c["docs"])
        if c["each"]:
            least = max(c["sink"] + c["recent"], c["budget"] // 2)
            s["budget"] = torch.randint(least, c["budget"] + 1, (B,), generator=h).to(torch.int32).to(DEV)
        # the second set of tables that a serving loop changes over to
        new = lambda t: torch.zeros_like(t)
        s["out"] = {"table_out": new(s["table"]), "lens_out": new(s["seq"]), "weights_out": new(wt),
                    "pos_out": new(s["table"]), "doc_out": new(s["table"]) if c["docs"] else None,
                    "freed": new(s["table"]), "n_freed": new(s["seq"])}
    else:
        s = _prepare_step(c, g, h)
        q_len, H, stride = c["q_len"], c["H"], s["table"].shape[1]
        if c["op"] == "attn":
            # the static buffers that a serving loop keeps
            s["out"] = torch.empty((B, q_len, H, D_LAT), dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.empty((B, q_len, H), dtype=torch.float32, device=DEV)
            s["workspace"] = torch.empty(96 << 20, dtype=torch.uint8, device=DEV)
        else:
            s["lse"] = _log_sums(_scores_plain(s, _keys_plain(s)))          # of the attention before
            s["weights"] = torch.exp(2.0 * _normal(g, B, stride) - 4)
            s["decay"] = 0.98
            s["counted"] = (torch.rand((B, q_len), generator=g, device=DEV) < 0.5).to(torch.uint8) if c["part"] else None
            s["out"] = torch.zeros((B, stride), dtype=torch.float32, device=DEV)
    s["case"] = c
    return s


# ----------------------------------------------------------------------------- plain forms
def _keys_plain(s):
    """fp32 key rows [B, n_max, 576]."""
    at = s["table"].long()
    if "kv" in s:
        return s["kv"][at].float()
    lat = s["lat"][at].view(torch.float8_e4m3fn).float()
    return torch.cat((lat * s["scale"][at].unsqueeze(-1), s["rope"][at].float()), -1)


def _seen(s, B, q_len, n_max):
    """[B, q_len, n_max]: whether draft t of stream b sees key j."""
    r = s["rules"]
    j = torch.arange(n_max, device=DEV)
    t = torch.arange(q_len, device=DEV)
    start = s["seq"].long()[:, None] - q_len               # [B, 1]: key of draft 0
    i = j - start                                          # [B, n_max]: draft index of key j, < 0: before the drafts
    m = s["mask"]
    if m is None:
        draft = (t[:, None] >= t).expand(B, q_len, q_len)
    elif m.dtype == torch.int64:
        draft = ((m[:, :, None] >> t) & 1) != 0
    else:
        draft = m != 0
    at = i.clamp(0, q_len - 1)[:, None, :].expand(B, q_len, n_max)
    ok = (i < 0)[:, None, :] | torch.gather(draft, 2, at)
    pos = j.expand(B, n_max) if r["key_pos"] is None else r["key_pos"].long()
    mine = torch.gather(pos, 1, start + t)                 # [B, q_len]
    if r["window"]:
        ok = ok & (mine[:, :, None] - pos[:, None, :] < r["window"])
    if r["prefix_lens"] is not None:
        ok = ok | (pos < r["prefix_lens"].long()[:, None])[:, None, :]
    if r["key_doc"] is not None:
        doc = r["key_doc"]
        ok = ok & ((doc[:, None, :] == torch.gather(doc, 1, start + t)[:, :, None]) | (doc < 0)[:, None, :])
    return ok & (i < q_len)[:, None, :], (pos[:, None, :] - mine[:, :, None]).float()


def _scores_plain(s, k):
    """fp32 scores [B, q_len, H, n_max] under the rules, -inf where a key is not seen."""
    B, q_len, H, _ = s["q"].shape
    n_max, r = s["table"].shape[1], s["rules"]
    x = torch.matmul(s["q"].float().view(B, q_len * H, D_ROW), k.transpose(1, 2)).mul_(SCALE).view(B, q_len, H, n_max)
    if r["softcap"]:
        x = x.div_(r["softcap"]).tanh_().mul_(r["softcap"])
    ok, away = _seen(s, B, q_len, n_max)
    if r["slopes"] is not None:
        x += r["slopes"][None, None, :, None] * away[:, :, None, :]
    return x.masked_fill_(~ok[:, :, None, :], -math.inf)


def _log_sums(x):
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    return (top + (x - top).exp_().sum(-1, keepdim=True).log()).squeeze(-1)


def _attn_plain(s):
    B, q_len, H, _ = s["q"].shape
    k = _keys_plain(s)
    x = _scores_plain(s, k)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = x.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, q_len * H, -1), k[:, :, :D_LAT]).view(B, q_len, H, D_LAT)
    out = torch.where(total > 0, o / total, torch.zeros_like(o))
    return {"out": out.to(torch.bfloat16), "lse": (top + total.log()).squeeze(-1)}


def _weights_plain(s):
    B, q_len, H, _ = s["q"].shape
    x = _scores_plain(s, _keys_plain(s))
    some = torch.isfinite(s["lse"])
    if s["counted"] is not None:
        some = some & (s["counted"] != 0)[:, :, None]
    lse = torch.where(some, s["lse"], torch.full_like(s["lse"], math.inf))
    new = x.sub_(lse.unsqueeze(-1)).exp_().sum((1, 2))
    j = torch.arange(new.shape[1], device=DEV)
    old = torch.where(j < s["seq"][:, None] - q_len, s["weights"] * s["decay"], torch.zeros_like(new))
    out = s["out"]
    out.copy_(torch.where(j < s["seq"][:, None], old + new, out))
    return {"weights": out}


def _evict_plain(s):
    c, o = s["case"], s["out"]
    B, stride = s["table"].shape
    n = s["seq"].long()[:, None]
    j = torch.arange(stride, device=DEV).expand(B, stride)
    budget = s["budget"].long()[:, None] if torch.is_tensor(s["budget"]) else torch.full_like(n, s["budget"])
    left = torch.minimum(n, budget.clamp(min=c["sink"] + c["recent"]))
    rank = s["weights"].masked_fill((j < c["sink"]) | (j >= n - c["recent"]), math.inf).masked_fill(j >= n, -math.inf)
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices
    place = torch.empty_like(order)
    place.scatter_(1, order, j)
    keep = (place < left) & (j < n)
    b = torch.arange(B, device=DEV)[:, None].expand(B, stride)
    to = torch.cumsum(keep, 1) - 1
    arrays = [(s["table"], o["table_out"]), (s["weights"], o["weights_out"]),
              (j.to(torch.int32) if s["pos"] is None else s["pos"], o["pos_out"]), (s["doc"], o["doc_out"])]
    for src, dst in arrays:
        if src is not None:
            dst[b[keep], to[keep]] = src[keep]
    gone = ~keep & (j < n)
    o["freed"][b[gone], (torch.cumsum(gone, 1) - 1)[gone]] = s["table"][gone]
    o["lens_out"].copy_(left[:, 0])
    o["n_freed"].copy_((n - left)[:, 0])
    return {k: v for k, v in o.items() if v is not None}


def run(s):
    op = s["case"]["op"]
    if own:
        import mla_speculative_verify_attention_gb300 as mv
    if op == "attn":
        if own:
            out, lse = mv.verify_attn_fp8_rules(s["q"], s["lat"], s["scale"], s["rope"], s["table"], s["seq"], s["mask"],
                                                SCALE, **s["rules"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
            return {"out": out, "lse": lse}
        return _attn_plain(s)
    if op == "weights":
        if not own:
            return _weights_plain(s)
        more = dict(s["rules"], weights=s["weights"], decay=s["decay"], counted=s["counted"], out=s["out"])
        if "kv" in s:
            return {"weights": mv.key_weights(s["q"], s["kv"], s["table"], s["seq"], s["mask"], SCALE, s["lse"], **more)}
        return {"weights": mv.key_weights_fp8(s["q"], s["lat"], s["scale"], s["rope"], s["table"], s["seq"], s["mask"], SCALE,
                                              s["lse"], **more)}
    if own:
        c = s["case"]
        mv.kv_evict(s["table"], s["seq"], s["weights"], s["budget"], sink=c["sink"], recent=c["recent"], key_pos=s["pos"],
                    key_doc=s["doc"], **s["out"])
        return {k: v for k, v in s["out"].items() if v is not None}
    return _evict_plain(s)


# ----------------------------------------------------------------------------- work
def work(case):
    c = case
    mean = (c["lo"] + c["hi"]) / 2
    if c["op"] == "evict":
        kept = min(mean, c["budget"] * (0.75 if c["each"] else 1))
        arrays = 3 + (c["docs"] > 0)                        # slots, weights, positions, documents
        return {"bytes": c["B"] * (4 * mean + kept * (8 * arrays - 4 - 4 * (not c["pos"])) + (mean - kept) * 8 + 16),
                "flops": c["B"] * mean}
    rows = c["B"] * c["q_len"] * c["H"]
    if c["window"] and not c["pos"]:                        # keys that no draft sees are not read
        n = c["B"]
        lens = [c["lo"] + (c["hi"] - c["lo"]) * (i + 0.5) / n for i in range(n)]
        keys = sum(min(x, c["window"] + min(c["prefix"] * 0.75, max(0, x - c["window"]))) + c["q_len"] for x in lens)
    else:
        keys = c["B"] * (mean + c["q_len"])
    marks = 4 * c["pos"] + 4 * (c["docs"] > 0)
    if c["op"] == "attn":
        return {"bytes": keys * (D_LAT + 4 + 2 * D_ROPE + 4 + marks) + rows * (2 * D_ROW + 2 * D_LAT + 4),
                "flops": 2 * (D_ROW + D_LAT) * keys * c["q_len"] * c["H"]}
    row = D_LAT + 4 + 2 * D_ROPE if c["cache"] == "fp8" else 2 * D_ROW
    return {"bytes": keys * (row + 4 + marks) + 8 * c["B"] * (mean + c["q_len"]) + rows * (2 * D_ROW + 4),
            "flops": 2 * D_ROW * keys * c["q_len"] * c["H"]}


# ----------------------------------------------------------------------------- 64 bits
def _e4m3_values():
    """The 256 codes' values: sign, four exponent bits of bias 7, three mantissa bits."""
    v = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        a = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v.append(-a if code & 128 else a)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _exact_step(s):
    """For each stream and draft: (b, t, key rows, the keys' indices, scores [H, keys]) over the keys it sees."""
    B, q_len, H, _ = s["q"].shape
    r, values = s["rules"], _e4m3_values()
    seq = s["seq"].tolist()
    prefix = None if r["prefix_lens"] is None else r["prefix_lens"].tolist()
    packed = s["mask"] is not None and s["mask"].dim() == 2
    for b in range(B):
        n = seq[b]
        p, at = n - q_len, s["table"][b, :n].long()
        if "kv" in s:
            k = s["kv"][at].double()
        else:
            k = torch.cat((values[s["lat"][at].long()] * s["scale"][at].double()[:, None], s["rope"][at].double()), 1)
        pos = torch.arange(n, device=DEV) if r["key_pos"] is None else r["key_pos"][b, :n].long()
        doc = None if r["key_doc"] is None else r["key_doc"][b, :n]
        for t in range(q_len):
            see = torch.ones(n, dtype=torch.bool, device=DEV)
            if s["mask"] is None:
                see[p + t + 1:] = False
            elif packed:
                word = int(s["mask"][b, t])
                see[p:] = torch.tensor([(word >> i) & 1 == 1 for i in range(q_len)], device=DEV)
            else:
                see[p:] = s["mask"][b, t].bool()
            if r["window"] > 0:
                see &= pos > pos[p + t] - r["window"]
            if prefix is not None:
                see |= pos < prefix[b]
            if doc is not None:
                see &= (doc < 0) | (doc == doc[p + t])
            idx = see.nonzero()[:, 0]
            x = (s["q"][b, t].double() @ k[idx].T) * SCALE
            if r["softcap"] > 0:
                x = r["softcap"] * torch.tanh(x / r["softcap"])
            if r["slopes"] is not None:
                x = x + torch.outer(r["slopes"].double(), (pos[idx] - pos[p + t]).double())
            yield b, t, k, idx, x


def _exact_attn(s):
    B, q_len, H, _ = s["q"].shape
    out = torch.zeros((B, q_len, H, D_LAT), dtype=torch.float64, device=DEV)
    lse = torch.full((B, q_len, H), -math.inf, dtype=torch.float64, device=DEV)
    for b, t, k, idx, x in _exact_step(s):
        if idx.numel():
            lse[b, t] = torch.logsumexp(x, 1)
            out[b, t] = torch.exp(x - lse[b, t][:, None]) @ k[idx][:, :D_LAT]
    return {"out": out, "lse": lse}


def _exact_weights(s):
    B, q_len, H, _ = s["q"].shape
    out = s["out"].double().clone()
    for b, n in enumerate(s["seq"].tolist()):
        out[b, :n - q_len] = s["decay"] * s["weights"][b, :n - q_len].double()
        out[b, n - q_len:n] = 0
    lse = s["lse"].double()
    for b, t, _, idx, x in _exact_step(s):
        if s["counted"] is None or int(s["counted"][b, t]):
            part = torch.exp(x - lse[b, t][:, None])
            out[b, idx] += part[torch.isfinite(lse[b, t])].sum(0)
    return {"weights": out}


def _exact_evict(s):
    c = s["case"]
    o = {k: v.cpu().clone() for k, v in s["out"].items() if v is not None}
    table, wt = s["table"].cpu(), s["weights"].cpu()
    for b, n in enumerate(s["seq"].tolist()):
        budget = int(s["budget"][b]) if torch.is_tensor(s["budget"]) else s["budget"]
        left = min(n, max(budget, c["sink"] + c["recent"]))
        if left == n:
            keep = torch.arange(n)
        else:
            lo, hi = c["sink"], n - c["recent"]
            w = wt[b, lo:hi].double()
            k = left - c["sink"] - c["recent"]
            border = torch.sort(w, descending=True).values[k - 1] if k else math.inf
            above = (w > border).nonzero()[:, 0]
            ties = (w == border).nonzero()[:, 0][:k - above.numel()]
            mid = torch.sort(torch.cat((above, ties))).values + lo
            keep = torch.cat((torch.arange(lo), mid, torch.arange(hi, n)))
        rest = torch.ones(n, dtype=torch.bool)
        rest[keep] = False
        o["table_out"][b, :left] = table[b, keep]
        o["weights_out"][b, :left] = wt[b, keep]
        o["pos_out"][b, :left] = keep.to(torch.int32) if s["pos"] is None else s["pos"][b].cpu()[keep]
        if "doc_out" in o:
            o["doc_out"][b, :left] = s["doc"][b].cpu()[keep]
        o["freed"][b, :n - left] = table[b, :n][rest]
        o["lens_out"][b], o["n_freed"][b] = left, n - left
    o["weights_out"] = o["weights_out"].double()
    return o


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](s)
