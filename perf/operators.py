"""Cases of the paged-cache operators: what each computes in plain tensor operations, and the calls a user makes.

Four operators that one serving step runs around the MLA cache (pages of 64 tokens, one KV head, rows of
512 latent values and 64 RoPE values):

  pages   give every request the pages its new tokens need and name the cache slot of each new token
  store   write the new tokens' latents through those slots: bf16 rows, FP8 rows with four scales, FP8
          rows with one scale per token
  window  decode attention over the first `sinks` and the last `window` tokens of every request
  prefix  decode attention of a batch whose requests share a long prefix, read once for all of them

``own`` selects the framework's kernels in ``run``; otherwise ``run`` computes the same values with
elementary torch operations in 32 bits.  ``exact`` computes them in 64 bits.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
D_QK = 576
D_V = 512
ROW_BYTES = {"bf16": 1152, "fp8": 656, "fp8_token": 640}
DEV = "cuda"


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a mid-size batch: every request appends one token
        {"name": "pages_decode", "kind": "pages", "batch": 64, "cached": 32768, "new_lo": 1, "new_hi": 1, "pad": 0},
        # a chunked-prefill step: ragged chunks, some requests idle, a padded slot map
        {"name": "pages_prefill", "kind": "pages", "batch": 256, "cached": 16384, "new_lo": 0, "new_hi": 2047,
         "pad": 1000},
        # a decode step's new tokens into the FP8 cache, read from separate latent and RoPE tensors
        {"name": "store_fp8_decode", "kind": "store", "fmt": "fp8", "tokens": 128, "width": 0, "pad": 8},
        # a prefill's tokens into the bf16 cache
        {"name": "store_bf16_prefill", "kind": "store", "fmt": "bf16", "tokens": 65535, "width": 0, "pad": 1},
        # a prefill's tokens, a slice of a wider fused projection, into the per-token-scale cache
        {"name": "store_token_prefill", "kind": "store", "fmt": "fp8_token", "tokens": 30001, "width": 2112, "pad": 63},
        # few requests, a short window: latency counts
        {"name": "window_small", "kind": "window", "fmt": "bf16", "batch": 4, "h_q": 16, "s_q": 1, "len_lo": 300,
         "len_hi": 5000, "window": 512, "sinks": 4},
        # a tensor-parallel shard of the heads over the bf16 cache: bound by memory
        {"name": "window_bf16", "kind": "window", "fmt": "bf16", "batch": 128, "h_q": 16, "s_q": 1, "len_lo": 1024,
         "len_hi": 16384, "window": 4096, "sinks": 64},
        # the same over the FP8 cache
        {"name": "window_fp8", "kind": "window", "fmt": "fp8", "batch": 128, "h_q": 16, "s_q": 1, "len_lo": 1024,
         "len_hi": 16384, "window": 4096, "sinks": 100},
        # all heads and two query tokens (speculative decoding): many rows share a short key set
        {"name": "window_heads", "kind": "window", "fmt": "bf16", "batch": 48, "h_q": 128, "s_q": 2, "len_lo": 50,
         "len_hi": 9000, "window": 1000, "sinks": 16},
        # a few requests behind a system prompt
        {"name": "prefix_small", "kind": "prefix", "fmt": "bf16", "batch": 6, "h_q": 16, "s_q": 1, "prefix": 1999,
         "own_lo": 1, "own_hi": 200},
        # a data-parallel rank: all heads, one long document, short answers
        {"name": "prefix_bf16", "kind": "prefix", "fmt": "bf16", "batch": 64, "h_q": 128, "s_q": 1, "prefix": 8192,
         "own_lo": 1, "own_hi": 512},
        # a tensor-parallel shard over the FP8 cache, a longer document
        {"name": "prefix_fp8", "kind": "prefix", "fmt": "fp8", "batch": 100, "h_q": 16, "s_q": 1, "prefix": 20001,
         "own_lo": 100, "own_hi": 700},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["pages", "store", "window", "window", "prefix", "prefix"])
    if kind == "pages":
        new_hi = _log(rng, 1, 2048)
        return {"kind": kind, "batch": _log(rng, 1, 256), "cached": _log(rng, 100, 32768),
                "new_lo": rng.choice([0, 1, new_hi]), "new_hi": new_hi, "pad": rng.choice([0, 1, 1000])}
    fmt = rng.choice(["bf16", "fp8", "fp8_token"])
    if kind == "store":
        return {"kind": kind, "fmt": fmt, "tokens": _log(rng, 1, 65536), "width": rng.choice([0, 0, 576, 2112]),
                "pad": rng.choice([0, 1, 50])}
    h_q = rng.choice([1, 8, 16, 16, 20, 32, 64, 128, 128])
    s_q = rng.choice([1, 1, 1, 2, 3])
    rows = h_q * s_q
    if kind == "window":
        window = _log(rng, 1, 8192)
        # no more keys in reach than the listed cases read, and no more products
        batch = max(1, min(_log(rng, 1, 128), 500000 // (window + 300), int(2.5e7) // (rows * (window + 300))))
        return {"kind": kind, "fmt": fmt, "batch": batch, "h_q": h_q, "s_q": s_q, "len_lo": rng.choice([0, 1, 500]),
                "len_hi": _log(rng, 500, 16384), "window": window, "sinks": rng.choice([0, 1, 4, 64, 200])}
    prefix = _log(rng, 1, 32768)
    batch = max(1, min(_log(rng, 1, 128), int(6e7) // (rows * (prefix + 600))))
    return {"kind": kind, "fmt": fmt, "batch": batch, "h_q": h_q, "s_q": s_q, "prefix": prefix, "own_lo": s_q,
            "own_hi": _log(rng, max(2, s_q), 600)}


# --------------------------------------------------------------------------- inputs
def _host(seed, *more):
    return np.random.default_rng([int(seed), *more])


def _dev_rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _lens(rng, lo, hi, n):
    return rng.integers(lo, hi + 1, n).astype(np.int64)


def _tables(rng, pages_of, spare=3):
    """Block table over a shuffled pool; rows are as wide as the longest, unused entries are 0."""
    total = int(pages_of.sum())
    pool = rng.permutation(total + spare).astype(np.int32)
    width = max(1, int(pages_of.max()))
    bt = np.zeros((len(pages_of), width), np.int32)
    at = np.concatenate([[0], np.cumsum(pages_of)])
    for b in range(len(pages_of)):
        bt[b, :pages_of[b]] = pool[at[b]:at[b + 1]]
    return bt, total + spare


def _cache(fmt, pages, g):
    """A filled cache: latents of unit scale whose magnitude differs from token to token, as a layer's do."""
    rows = pages * PAGE
    if fmt == "bf16":
        x = torch.randn(rows, D_QK, device=DEV, generator=g, dtype=torch.bfloat16)
        return x.view(pages, PAGE, 1, D_QK), None
    kv = torch.empty(rows, ROW_BYTES[fmt], dtype=torch.uint8, device=DEV)
    sc = torch.empty(rows, 1, dtype=torch.float32, device=DEV)
    for a in range(0, rows, 1 << 18):
        n = min(1 << 18, rows - a)
        x = torch.randn(n, D_V, device=DEV, generator=g)
        x *= torch.rand(n, 1, device=DEV, generator=g) + 0.5
        t = x.view(n, 4, 128) if fmt == "fp8" else x.view(n, 1, D_V)
        s = t.abs().amax(-1, keepdim=True) / 448.0
        codes = (t / s).to(torch.float8_e4m3fn).view(n, D_V).view(torch.uint8)
        kv[a:a + n, :D_V] = codes
        if fmt == "fp8":
            kv[a:a + n, 512:528] = s.view(n, 4).contiguous().view(torch.uint8)
        else:
            sc[a:a + n] = s.view(n, 1)
        rope = torch.randn(n, 64, device=DEV, generator=g, dtype=torch.bfloat16)
        kv[a:a + n, ROW_BYTES[fmt] - 128:] = rope.view(torch.uint8)
    return kv.view(pages, PAGE, 1, -1), sc.view(pages, PAGE) if fmt == "fp8_token" else None


def _t(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV, dtype)


def prepare(case, seed):
    rng, g = _host(seed, 17), _dev_rng(seed)
    c, kind = case, case["kind"]
    if kind == "pages":
        old = _lens(rng, 0, c["cached"], c["batch"])
        new = _lens(rng, c["new_lo"], c["new_hi"], c["batch"])
        budget = c["batch"] * (c["new_lo"] + c["new_hi"]) // 2  # a step's new tokens, whatever their split
        for b in rng.permutation(c["batch"]):
            new[b] = min(c["new_hi"], max(c["new_lo"], new[b] + budget - new.sum()))
        have, want = -(-old // PAGE), -(-(old + new) // PAGE)
        need = int((want - have).sum())
        pool = rng.permutation(int(want.sum()) + 100).astype(np.int32)
        width = -(-(c["cached"] + c["new_hi"]) // PAGE) + 1
        bt = np.full((c["batch"], width), -1, np.int32)
        at = np.concatenate([[0], np.cumsum(have)])
        for b in range(c["batch"]):
            bt[b, :have[b]] = pool[at[b]:at[b + 1]]
        start = int(rng.integers(0, 20))  # pages that earlier steps took from the front of the list
        free = np.concatenate([rng.integers(0, len(pool), start).astype(np.int32), pool[at[-1]:]])
        assert len(free) >= start + need
        return {"case": c, "old": _t(old), "new": _t(new), "free": _t(free), "cursor": _t(np.array([start])),
                "table": _t(bt), "tokens": budget + c["pad"]}
    if kind == "store":
        n, pages = c["tokens"], -(-c["tokens"] // PAGE) + 40
        x = torch.randn(n, max(c["width"], D_QK), device=DEV, generator=g, dtype=torch.bfloat16)
        x *= (torch.rand(n, 1, device=DEV, generator=g) * 3 + 0.1).to(torch.bfloat16)
        if c["width"]:
            latent, rope = x[:, -D_QK:-64], x[:, -64:]
        else:
            latent, rope = x[:, :D_V].contiguous(), x[:, D_V:].contiguous()
        order = rng.permutation(pages)[: -(-n // PAGE)]
        slots = (order[:, None] * PAGE + np.arange(PAGE)).reshape(-1)[:n]
        slots[max(0, n - c["pad"]):] = -1  # padding at the end of the batch
        kv = torch.randint(0, 64, (pages, PAGE, 1, ROW_BYTES[c["fmt"]]), device=DEV, generator=g, dtype=torch.uint8)
        sc = torch.rand(pages, PAGE, device=DEV, generator=g) if c["fmt"] == "fp8_token" else None
        if c["fmt"] == "bf16":
            kv = kv.view(torch.bfloat16)
        return {"case": c, "latent": latent, "rope": rope, "slots": _t(slots), "kv": kv, "scales": sc}
    b, h, s = c["batch"], c["h_q"], c["s_q"]
    q = torch.randn(b, s, h, D_QK, device=DEV, generator=g, dtype=torch.bfloat16)
    st = {"case": c, "q": q, "scale": 1.0 / math.sqrt(D_QK)}
    if kind == "window":
        lens = _lens(rng, c["len_lo"], max(c["len_lo"], c["len_hi"]), b)
        bt, pages = _tables(rng, -(-lens // PAGE))
        st |= {"lens": _t(lens), "table": _t(bt)}
        reach = min(int(lens.max()), c["window"] + s - 1 + c["sinks"])
    else:
        lens = _lens(rng, c["own_lo"], max(c["own_lo"], c["own_hi"]), b)
        pp = -(-c["prefix"] // PAGE)
        bt, pages = _tables(rng, np.concatenate([[pp], -(-lens // PAGE)]))
        own_width = max(1, int((-(-lens // PAGE)).max()))
        st |= {"lens": _t(lens), "table": _t(bt[1:, :own_width]), "prefix_table": _t(bt[0, :pp]),
               "prefix_len": _t(np.array([c["prefix"]]))}
        reach = int(lens.max())
    st["reach"] = max(1, reach)
    st["kv"], st["scales"] = _cache(c["fmt"], pages, g)
    return st


# --------------------------------------------------------------------------- one pass
def run(state):
    kind = state["case"]["kind"]
    if own:
        import paged_mla_decode_07_gb300 as mla

        if kind == "pages":
            lens, offsets, slots, cursor = mla.assign_pages(state["old"], state["new"], state["free"],
                                                            state["cursor"], state["table"], state["tokens"])
            return {"table": state["table"], "lens": lens, "offsets": offsets, "slots": slots, "cursor": cursor}
        if kind == "store":
            mla.cache_store(state["latent"], state["rope"], state["slots"], state["kv"], kv_scales=state["scales"])
            return _stored(state)
        if kind == "window":
            out, lse = mla.window_decode(state["q"], state["kv"], state["table"], state["lens"], state["scale"],
                                         window=state["case"]["window"], sinks=state["case"]["sinks"],
                                         kv_scales=state["scales"])
        else:
            out, lse = mla.shared_prefix_decode(state["q"], state["kv"], state["prefix_table"], state["prefix_len"],
                                                state["table"], state["lens"], state["scale"], is_causal=True,
                                                kv_scales=state["scales"])
        return {"out": out, "lse": lse}
    if kind == "pages":
        return _plain_pages(state)
    if kind == "store":
        _plain_store(state)
        return _stored(state)
    return _plain_window(state) if kind == "window" else _plain_prefix(state)


def _stored(state):
    """The cache as the values it holds (views of the state's own buffers)."""
    kv, fmt = state["kv"], state["case"]["fmt"]
    if fmt == "bf16":
        return {"rows": kv}
    r = ROW_BYTES[fmt]
    got = {"codes": kv[..., :D_V].view(torch.float8_e4m3fn), "rope": kv[..., r - 128:].view(torch.bfloat16)}
    got["scales"] = kv[..., 512:528].view(torch.float32) if fmt == "fp8" else state["scales"]
    return got


def _plain_pages(st):
    old, new, table = st["old"].clamp(min=0).long(), st["new"].clamp(min=0).long(), st["table"]
    total = old + new
    ends = new.cumsum(0)
    have = (old + PAGE - 1) // PAGE
    need = (total + PAGE - 1) // PAGE - have
    first = st["cursor"].long() + need.cumsum(0) - need
    j = torch.arange(table.shape[1], device=DEV)
    fresh = (j >= have[:, None]) & (j < (have + need)[:, None])
    take = (first[:, None] + j - have[:, None]).clamp(0, st["free"].shape[0] - 1)
    table = torch.where(fresh, st["free"][take], table)
    t = torch.arange(st["tokens"], device=DEV)
    b = torch.searchsorted(ends, t, right=True).clamp(max=len(new) - 1)
    pos = old[b] + t - (ends - new)[b]
    page = table[b, (pos // PAGE).clamp(0, table.shape[1] - 1)].long()
    slots = torch.where(t < ends[-1], page * PAGE + pos % PAGE, -1)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), ends])
    return {"table": table, "lens": total.int(), "offsets": offsets.int(), "slots": slots.int(),
            "cursor": (st["cursor"] + need.sum()).int()}


def _plain_store(st):
    kv, fmt = st["kv"], st["case"]["fmt"]
    rows = kv.view(-1, kv.shape[-1])
    keep = st["slots"] >= 0
    at = st["slots"][keep].long()
    latent, rope = st["latent"][keep], st["rope"][keep]
    if fmt == "bf16":
        rows[at] = torch.cat([latent, rope], 1)
        return
    n = latent.shape[0]
    x = latent.float().view(n, 4 if fmt == "fp8" else 1, -1)
    amax = x.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    codes = (x / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).view(n, D_V)
    tail = rope.contiguous().view(torch.uint8)
    if fmt == "fp8":
        rows[at] = torch.cat([codes, s.view(n, 4).view(torch.uint8), tail], 1)
    else:
        rows[at] = torch.cat([codes, tail], 1)
        st["scales"].view(-1)[at] = s.view(n)


def _values(rows, scales, fmt):
    """Cache rows as the float32 values the attention uses: bf16 values, or bf16 of code x scale."""
    if fmt == "bf16":
        return rows.float()
    n = rows.shape[:-1]
    codes = rows[..., :D_V].contiguous().view(torch.float8_e4m3fn).float()
    if fmt == "fp8":
        s = rows[..., 512:528].contiguous().view(torch.float32)[..., None]
        lat = (codes.view(*n, 4, 128) * s).view(*n, D_V)
    else:
        lat = codes * scales[..., None]
    rope = rows[..., ROW_BYTES[fmt] - 128:].contiguous().view(torch.bfloat16).float()
    return torch.cat([lat.to(torch.bfloat16).float(), rope], -1)


def _gather(st, table, pos):
    """Values of the tokens at logical positions `pos` (any value; masked later) of each table row."""
    kv, fmt = st["kv"], st["case"]["fmt"]
    pos = pos.clamp(0, table.shape[-1] * PAGE - 1)
    at = table.gather(-1, pos // PAGE).long() * PAGE + pos % PAGE
    rows = kv.view(-1, kv.shape[-1])[at]
    return _values(rows, st["scales"].view(-1)[at] if st["scales"] is not None else None, fmt)


def _softmax_v(logits, v):
    """(out, base-2 log-sum-exp) of natural logits [.., rows, keys] (-inf: masked) over values [.., keys, 512]."""
    m = logits.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    e = torch.exp(logits - m)
    z = e.sum(-1, keepdim=True)
    out = (e @ v) / torch.where(z > 0, z, torch.ones_like(z))
    return out, (torch.log(z) + m)[..., 0] / math.log(2.0)


def _plain_window(st):
    c, q, lens = st["case"], st["q"], st["lens"].long()
    b, s, h = q.shape[:3]
    # the keys any query token sees: the sinks, then the last `window + s - 1` tokens
    tail = max(1, min(st["reach"], c["window"] + s - 1))
    n_sink = min(c["sinks"], st["reach"])
    begin = (lens - tail).clamp(min=0)
    t = torch.arange(tail, device=DEV)
    pos = torch.cat([torch.arange(n_sink, device=DEV).expand(b, -1), begin[:, None] + t], 1)
    twice = torch.cat([torch.zeros(b, n_sink, dtype=torch.bool, device=DEV), begin[:, None] + t < n_sink], 1)
    k = _gather(st, st["table"], pos)
    logits = (q.float().view(b, s * h, D_QK) @ k.transpose(1, 2)) * st["scale"]
    at = lens[:, None] - s + torch.arange(s, device=DEV)  # position of each query token
    seen = (pos[:, None] <= at[..., None]) & ((pos[:, None] < c["sinks"]) | (pos[:, None] > at[..., None] - c["window"]))
    seen = seen & (pos < lens[:, None])[:, None] & ~twice[:, None]
    logits = logits.view(b, s, h, -1).masked_fill(~seen[:, :, None], -math.inf).view(b, s * h, -1)
    out, lse = _softmax_v(logits, k[..., :D_V])
    return {"out": out.view(b, s, h, D_V).to(torch.bfloat16), "lse": lse.view(b, s, h)}


def _plain_prefix(st):
    c, q, lens = st["case"], st["q"], st["lens"].long()
    b, s, h = q.shape[:3]
    qf = q.float()
    pos = torch.arange(c["prefix"], device=DEV)
    k0 = _gather(st, st["prefix_table"], pos)
    l0 = (qf.view(-1, D_QK) @ k0.t()) * st["scale"]
    own_pos = torch.arange(st["reach"], device=DEV).expand(b, -1)
    k1 = _gather(st, st["table"], own_pos)
    l1 = (qf.view(b, s * h, D_QK) @ k1.transpose(1, 2)) * st["scale"]
    at = lens[:, None] - s + torch.arange(s, device=DEV)
    seen = own_pos[:, None] <= at[..., None]
    l1 = l1.view(b, s, h, -1).masked_fill(~seen[:, :, None], -math.inf).view(b * s * h, -1)
    m = torch.maximum(l0.amax(-1, keepdim=True), l1.amax(-1, keepdim=True))
    e0, e1 = torch.exp(l0 - m), torch.exp(l1 - m)
    z = e0.sum(-1, keepdim=True) + e1.sum(-1, keepdim=True)
    o = e0 @ k0[:, :D_V] + (e1.view(b, s * h, -1) @ k1[..., :D_V]).view(-1, D_V)
    lse = (torch.log(z) + m)[:, 0] / math.log(2.0)
    return {"out": (o / z).view(b, s, h, D_V).to(torch.bfloat16), "lse": lse.view(b, s, h)}


# --------------------------------------------------------------------------- work
def work(case):
    c, kind = case, case["kind"]
    if kind == "pages":
        new = c["batch"] * (c["new_lo"] + c["new_hi"]) // 2
        # lengths in and out, offsets, one slot per token; pages taken from the list and put into the table
        return {"bytes": c["batch"] * 16 + 4 * (new + c["pad"]) + 8 * (new / PAGE), "flops": 0}
    if kind == "store":
        n = max(0, c["tokens"] - c["pad"])
        extra = 4 if c["fmt"] == "fp8_token" else 0
        return {"bytes": c["tokens"] * 4 + n * (D_QK * 2 + ROW_BYTES[c["fmt"]] + extra), "flops": 0}
    row = ROW_BYTES[c["fmt"]] + (4 if c["fmt"] == "fp8_token" else 0)
    rows = c["batch"] * c["s_q"] * c["h_q"]
    io = rows * (D_QK * 2 + D_V * 2 + 4)
    if kind == "window":
        lo, hi = c["len_lo"], max(c["len_lo"], c["len_hi"])
        n = np.linspace(lo, hi, 257)  # lengths are uniform
        keys = float(np.minimum(n, c["window"] + c["s_q"] - 1 + np.minimum(c["sinks"], n)).mean())
        seen = float(np.minimum(n, c["window"] + c["sinks"]).mean())
        return {"bytes": io + c["batch"] * keys * (row + 4 / PAGE), "flops": 2 * rows * seen * (D_QK + D_V)}
    mean = (c["own_lo"] + max(c["own_lo"], c["own_hi"])) / 2
    return {"bytes": io + (c["prefix"] + c["batch"] * mean) * (row + 4 / PAGE),
            "flops": 2 * rows * (c["prefix"] + mean) * (D_QK + D_V)}


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "pages":
        return _exact_pages(st)
    if kind == "store":
        return _exact_store(st)
    q, lens = st["q"], st["lens"].tolist()
    b, s, h = q.shape[:3]
    out = torch.zeros(b, s, h, D_V, dtype=torch.float64, device=DEV)
    lse = torch.full((b, s, h), -math.inf, dtype=torch.float64, device=DEV)
    prefix = None
    if kind == "prefix":
        prefix = _rows64(st, st["prefix_table"], torch.arange(case["prefix"], device=DEV))
    for e in range(b):
        for i in range(s):
            last = lens[e] - s + i
            if kind == "window":
                see = sorted({*range(0, min(case["sinks"], last + 1)), *range(max(0, last - case["window"] + 1), last + 1)})
            else:
                see = list(range(last + 1))
            keys = []
            if prefix is not None:
                keys.append(prefix)
            if see:
                keys.append(_rows64(st, st["table"][e], torch.tensor(see, device=DEV)))
            if not keys:
                continue
            k = torch.cat(keys)
            z = (q[e, i].double() @ k.t()) * st["scale"]
            total = torch.logsumexp(z, -1)
            out[e, i] = torch.softmax(z, -1) @ k[:, :D_V]
            lse[e, i] = total / math.log(2.0)
    return {"out": out, "lse": lse}


def _rows64(st, table_row, pos):
    kv, fmt = st["kv"], st["case"]["fmt"]
    at = table_row.long()[pos // PAGE] * PAGE + pos % PAGE
    r = kv.reshape(-1, kv.shape[-1])[at]
    if fmt == "bf16":
        return r.double()
    code = r[:, :D_V].contiguous().view(torch.float8_e4m3fn).double()
    if fmt == "fp8":
        scale = r[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
    else:
        scale = st["scales"].reshape(-1)[at].double()[:, None]
    # a stored FP8 value stands for bf16(code x scale): part of the format's definition (the product of a
    # 4-bit and a 24-bit mantissa, rounded once)
    lat = (code * scale).to(torch.bfloat16).double()
    return torch.cat([lat, r[:, -128:].contiguous().view(torch.bfloat16).double()], 1)


def _exact_pages(st):
    old, new = st["old"].tolist(), st["new"].tolist()
    free, table, cur = st["free"].tolist(), st["table"].cpu().numpy().copy(), int(st["cursor"][0])
    slots, offsets, lens = [], [0], []
    for b in range(len(old)):
        page = -(-old[b] // PAGE)
        while page * PAGE < old[b] + new[b]:
            table[b, page] = free[cur]
            cur, page = cur + 1, page + 1
        p = np.arange(old[b], old[b] + new[b])
        slots.append(table[b, p // PAGE].astype(np.int64) * PAGE + p % PAGE)
        offsets.append(offsets[-1] + new[b])
        lens.append(old[b] + new[b])
    slots = np.concatenate(slots) if slots else np.zeros(0, np.int64)
    slots = np.concatenate([slots, np.full(st["tokens"] - len(slots), -1)])
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32)  # noqa: E731
    return {"table": i32(table), "lens": i32(lens), "offsets": i32(offsets), "slots": i32(slots), "cursor": i32([cur])}


def _exact_store(st):
    fmt = st["case"]["fmt"]
    want = {k: (v.double() if v.is_floating_point() or "float8" in str(v.dtype) else v).clone()
            for k, v in _stored(st).items()}
    keep = st["slots"] >= 0
    at = st["slots"][keep].long()
    x, rope = st["latent"][keep].double(), st["rope"][keep].double()
    if fmt == "bf16":
        want["rows"].view(-1, D_QK)[at] = torch.cat([x, rope], 1)
        return want
    t = x.view(len(x), 4 if fmt == "fp8" else 1, -1)
    s = t.abs().amax(-1, keepdim=True) / 448.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    v = (t / s).view(len(x), D_V).abs()
    # nearest E4M3 magnitude: steps of 2^(e - 3) in [2^e, 2^(e + 1)), e >= -6 (below: the subnormal step 2^-9)
    step = torch.exp2(torch.floor(torch.log2(v.clamp(min=2.0 ** -6))) - 3)
    code = (torch.round(v / step) * step).clamp(max=448.0) * torch.sign(x)
    want["codes"].view(-1, D_V)[at] = code
    want["rope"].view(-1, 64)[at] = rope
    want["scales"].view(-1, s.shape[1])[at] = s.view(len(x), -1)
    return want
