"""Cases of the 4-bit cache and of attention over whole prompts: what each computes in plain tensor
operations, and the calls a user makes.

Four operators that serving runs around an MLA cache (pages of 64 tokens, one KV head, tokens of 512 latent
and 64 RoPE values):

  store   write new tokens into FP4 cache rows through their slots, and read them back as bf16 rows
  load    read cached tokens of a batch back as packed bf16 rows, as a chunked prefill does
  decode  decode attention over an FP4 cache, over everything or over a window with sinks
  prompt  causal attention over packed prompts, 192-wide queries and keys (128 per head and 64 RoPE values
          that the heads share), 128-wide values

An FP4 row is 400 bytes: 64 words of eight 4-bit codes (E2M1), 16 scale bytes, 64 bf16 RoPE values.  Word w
holds latent values 8 w .. 8 w + 7: bits 4 i .. 4 i + 2 are the magnitude of value i, bit 8 i + 7 the sign of
value i and bit 8 i + 3 that of value 4 + i (i < 4).  Scale byte s stands for 2^(s - 127) and serves 32 values.

``own`` selects the framework's kernels in ``run``; otherwise ``run`` computes the same values with elementary
torch operations in 32 bits.  ``exact`` computes them in 64 bits.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
D_QK, D_V, D_ROPE = 576, 512, 64
HEAD_QK, HEAD_V = 192, 128
ROW_BYTES = {"bf16": 1152, "fp8": 656, "fp8_token": 640, "fp4": 400}
DEV = "cuda"
ALL = 1 << 30  # a window over everything


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's new tokens, one per request, read back
        {"name": "store4_decode", "kind": "store", "batch": 128, "new_lo": 1, "new_hi": 1, "cached": 8192, "width": 0},
        # a prefill's ragged chunks, slices of a wider fused projection
        {"name": "store4_prefill", "kind": "store", "batch": 17, "new_lo": 501, "new_hi": 3029, "cached": 16384,
         "width": 2112},
        # the context of a few requests ahead of their next chunk, from the 4-bit cache
        {"name": "load4_context", "kind": "load", "fmt": "fp4", "batch": 9, "len_lo": 30, "len_hi": 3001, "from": 0},
        # many long contexts behind a shared prefix that is already there, from the FP8 cache
        {"name": "load_fp8_long", "kind": "load", "fmt": "fp8", "batch": 24, "len_lo": 1000, "len_hi": 8192, "from": 999},
        # few requests: latency counts
        {"name": "decode4_small", "kind": "decode", "batch": 4, "h_q": 16, "s_q": 1, "len_lo": 300, "len_hi": 5000,
         "window": 512, "sinks": 4},
        # a tensor-parallel shard of the heads over long contexts: bound by memory
        {"name": "decode4_long", "kind": "decode", "batch": 64, "h_q": 16, "s_q": 1, "len_lo": 2048, "len_hi": 16384,
         "window": ALL, "sinks": 0},
        # all heads of a data-parallel rank
        {"name": "decode4_heads", "kind": "decode", "batch": 32, "h_q": 128, "s_q": 1, "len_lo": 1001, "len_hi": 8191,
         "window": ALL, "sinks": 0},
        # all heads, two query tokens (speculative decoding), a window
        {"name": "decode4_window", "kind": "decode", "batch": 48, "h_q": 128, "s_q": 2, "len_lo": 50, "len_hi": 9000,
         "window": 1000, "sinks": 16},
        # a few short prompts, a shard of the heads: latency counts
        {"name": "prompt_small", "kind": "prompt", "batch": 3, "h_q": 16, "h_kv": 16, "new_lo": 50, "new_hi": 401,
         "ctx_lo": 0, "ctx_hi": 0},
        # chunks behind cached context
        {"name": "prompt_chunk", "kind": "prompt", "batch": 8, "h_q": 16, "h_kv": 16, "new_lo": 256, "new_hi": 1023,
         "ctx_lo": 0, "ctx_hi": 8192},
        # all heads of a data-parallel rank, ragged prompts
        {"name": "prompt_heads", "kind": "prompt", "batch": 5, "h_q": 128, "h_kv": 128, "new_lo": 333, "new_hi": 4096,
         "ctx_lo": 0, "ctx_hi": 0},
        # one long document, grouped heads
        {"name": "prompt_long", "kind": "prompt", "batch": 1, "h_q": 16, "h_kv": 4, "new_lo": 16384, "new_hi": 16384,
         "ctx_lo": 0, "ctx_hi": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["store", "load", "decode", "decode", "prompt", "prompt"])
    if kind == "store":
        batch = _log(rng, 1, 128)
        hi = _log(rng, 1, max(1, min(16384, 30000 // batch)))
        return {"kind": kind, "batch": batch, "new_lo": rng.choice([0, 1, hi]), "new_hi": hi, "cached": _log(rng, 1, 16384),
                "width": rng.choice([0, 0, 576, 2112])}
    if kind == "load":
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, min(32768, 200000 // batch))
        return {"kind": kind, "fmt": rng.choice(["bf16", "fp8", "fp8_token", "fp4", "fp4"]), "batch": batch,
                "len_lo": rng.choice([0, 1, hi]), "len_hi": hi, "from": rng.choice([0, 0, 1, 64, 500])}
    if kind == "decode":
        h_q, s_q = rng.choice([1, 8, 16, 16, 20, 32, 64, 128, 128]), rng.choice([1, 1, 1, 2, 3])
        window = rng.choice([ALL, ALL, _log(rng, 1, 8192)])
        hi = _log(rng, 100, 16384)
        batch = max(1, min(_log(rng, 1, 128), 500000 // hi, int(3e7) // (h_q * s_q * hi)))
        return {"kind": kind, "batch": batch, "h_q": h_q, "s_q": s_q, "len_lo": rng.choice([0, 1, 50, hi]), "len_hi": hi,
                "window": window, "sinks": rng.choice([0, 1, 4, 64, 200])}
    h_q = rng.choice([1, 4, 8, 16, 16, 32, 128])
    h_kv = rng.choice([g for g in (h_q, h_q, h_q // 2, h_q // 4) if g >= 1])
    new_hi, ctx_hi = _log(rng, 1, 8192), rng.choice([0, 0, _log(rng, 1, 8192)])
    batch = max(1, min(_log(rng, 1, 32), int(1.5e9) // (h_q * new_hi * (new_hi + ctx_hi)), 20000 // (new_hi + ctx_hi)))
    return {"kind": kind, "batch": batch, "h_q": h_q, "h_kv": h_kv, "new_lo": rng.choice([0, 1, new_hi]), "new_hi": new_hi,
            "ctx_lo": 0, "ctx_hi": ctx_hi}


# --------------------------------------------------------------------------- inputs
def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly spread."""
    return np.rint(np.linspace(lo, max(lo, hi), n)).astype(np.int64) if n > 1 else np.array([max(lo, hi)], np.int64)


def _t(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV, dtype)


def _offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def _tables(rng, pages_of, spare=3):
    """Block table over a shuffled pool of pages; rows are as wide as the longest."""
    pool = rng.permutation(int(pages_of.sum()) + spare).astype(np.int32)
    bt = np.zeros((len(pages_of), max(1, int(pages_of.max()))), np.int32)
    at = _offsets(pages_of)
    for b in range(len(pages_of)):
        bt[b, :pages_of[b]] = pool[at[b]:at[b + 1]]
    return bt, len(pool)


def _cache(fmt, pages, g):
    """A filled cache: latents of unit scale whose magnitude differs from token to token, as a layer's do."""
    rows = pages * PAGE
    if fmt == "bf16":
        return torch.randn(rows, D_QK, device=DEV, generator=g, dtype=torch.bfloat16).view(pages, PAGE, 1, D_QK), None
    kv = torch.empty(rows, ROW_BYTES[fmt], dtype=torch.uint8, device=DEV)
    sc = torch.empty(rows, 1, dtype=torch.float32, device=DEV)
    for a in range(0, rows, 1 << 18):
        n = min(1 << 18, rows - a)
        x = torch.randn(n, D_V, device=DEV, generator=g)
        x *= torch.rand(n, 1, device=DEV, generator=g) + 0.5
        rope = torch.randn(n, D_ROPE, device=DEV, generator=g, dtype=torch.bfloat16).view(torch.uint8)
        if fmt == "fp4":
            kv[a:a + n] = _fp4_rows(x, rope)
            continue
        t = x.view(n, 4, 128) if fmt == "fp8" else x.view(n, 1, D_V)
        s = t.abs().amax(-1, keepdim=True) / 448.0
        kv[a:a + n, :D_V] = (t / s).to(torch.float8_e4m3fn).view(n, D_V).view(torch.uint8)
        if fmt == "fp8":
            kv[a:a + n, 512:528] = s.view(n, 4).contiguous().view(torch.uint8)
        else:
            sc[a:a + n] = s.view(n, 1)
        kv[a:a + n, ROW_BYTES[fmt] - 128:] = rope
    return kv.view(pages, PAGE, 1, -1), sc.view(pages, PAGE) if fmt == "fp8_token" else None


def prepare(case, seed):
    rng = np.random.default_rng([int(seed), 23])
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    c, kind = case, case["kind"]
    st = {"case": c}
    if kind == "prompt":
        new = rng.permutation(_spread(c["new_lo"], c["new_hi"], c["batch"]))
        keys = new + rng.permutation(_spread(c["ctx_lo"], c["ctx_hi"], c["batch"]))
        qo, ko = _offsets(new), _offsets(keys)
        q = torch.randn(int(qo[-1]), c["h_q"], HEAD_QK, device=DEV, generator=g, dtype=torch.bfloat16)
        up = torch.randn(int(ko[-1]), c["h_kv"], HEAD_QK - D_ROPE + HEAD_V, device=DEV, generator=g, dtype=torch.bfloat16)
        rows = torch.randn(int(ko[-1]), D_QK, device=DEV, generator=g, dtype=torch.bfloat16)
        # keys and values are the two halves of one up-projection; the RoPE values come with the latent rows
        return st | {"q": q, "k_nope": up[..., :128], "v": up[..., 128:], "k_rope": rows[:, D_V:], "qo": _t(qo),
                     "ko": _t(ko), "scale": HEAD_QK ** -0.5, "new": new.tolist(), "keys": keys.tolist()}
    if kind in ("store", "load"):
        if kind == "store":
            starts = rng.integers(0, c["cached"] + 1, c["batch"])
            lens = rng.permutation(_spread(c["new_lo"], c["new_hi"], c["batch"]))
        else:
            starts = np.full(c["batch"], c["from"])
            lens = rng.permutation(_spread(c["len_lo"], c["len_hi"], c["batch"]))
        bt, pages = _tables(rng, -(-(starts + lens) // PAGE))
        off = _offsets(lens)
        st |= {"table": _t(bt), "starts": _t(starts), "offsets": _t(off), "tokens": int(off[-1])}
        if kind == "load":
            st["kv"], st["scales"] = _cache(c["fmt"], pages, g)
            return st
        n = st["tokens"]
        x = torch.randn(n, max(c["width"], D_QK), device=DEV, generator=g, dtype=torch.bfloat16)
        x *= (torch.rand(n, 1, device=DEV, generator=g) * 3 + 0.1).to(torch.bfloat16)
        if c["width"]:
            st["latent"], st["rope"] = x[:, -D_QK:-D_ROPE], x[:, -D_ROPE:]
        else:
            st["latent"], st["rope"] = x[:, :D_V].contiguous(), x[:, D_V:].contiguous()
        b = np.repeat(np.arange(c["batch"]), lens)
        pos = np.arange(n) - off[b] + starts[b]
        st["slots"] = _t(bt[b, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE)
        st["kv"] = torch.randint(0, 100, (pages, PAGE, 1, ROW_BYTES["fp4"]), device=DEV, generator=g, dtype=torch.uint8)
        st["scales"] = None
        return st
    b, h, s = c["batch"], c["h_q"], c["s_q"]
    lens = rng.permutation(_spread(c["len_lo"], c["len_hi"], b))
    bt, pages = _tables(rng, -(-lens // PAGE))
    st |= {"q": torch.randn(b, s, h, D_QK, device=DEV, generator=g, dtype=torch.bfloat16), "scale": D_QK ** -0.5,
           "lens": _t(lens), "table": _t(bt), "longest": max(1, int(lens.max()))}
    st["kv"], st["scales"] = _cache("fp4", pages, g)
    return st


# --------------------------------------------------------------------------- one pass
def run(state):
    kind, st = state["case"]["kind"], state
    if own:
        import paged_mla_decode_07_gb300 as mla

        if kind == "store":
            mla.cache_store(st["latent"], st["rope"], st["slots"], st["kv"])
            return mla.cache_load(st["kv"], st["table"], st["offsets"], st["tokens"], starts=st["starts"])
        if kind == "load":
            return mla.cache_load(st["kv"], st["table"], st["offsets"], st["tokens"], starts=st["starts"],
                                  kv_scales=st["scales"])
        if kind == "decode":
            out, lse = mla.window_decode(st["q"], st["kv"], st["table"], st["lens"], st["scale"],
                                         window=st["case"]["window"], sinks=st["case"]["sinks"])
        else:
            out, lse = mla.prompt_attention(st["q"], st["k_nope"], st["k_rope"], st["v"], st["qo"], st["ko"], st["scale"])
        return {"out": out, "lse": lse}
    if kind == "store":
        rows = st["kv"].view(-1, ROW_BYTES["fp4"])
        rows[st["slots"].long()] = _fp4_rows(st["latent"].float(), st["rope"].contiguous().view(torch.uint8))
        return _plain_load(st, "fp4")
    if kind == "load":
        return _plain_load(st, st["case"]["fmt"])
    return _plain_decode(st) if kind == "decode" else _plain_prompt(st)


def _fp4_rows(x, rope_bytes):
    """fp32 latents [n, 512] and RoPE bytes [n, 128] as FP4 rows."""
    n = x.shape[0]
    t = x.view(n, 16, 32)
    amax = t.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1): at most 6 2^(e - 3) where m <= 3/4
    e = torch.where(amax > 0, e - 3 + (m > 0.75), -13).clamp(-13, 13)
    y = torch.ldexp(t, -e).abs()
    # nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6; ties go to the even code
    mag = (y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)
    sign = torch.signbit(t).int()
    mag, sign = mag.view(n, 64, 8), sign.view(n, 64, 8)
    i = torch.arange(8, device=x.device)
    at = torch.where(i < 4, 8 * i + 7, 8 * (i - 4) + 3)
    words = ((mag.long() << (4 * i)) + (sign.long() << at)).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()
    scales = (e + 127).view(n, 16).to(torch.uint8)
    return torch.cat([words.view(torch.uint8), scales, rope_bytes], 1)


def _fp4_latents(rows):
    """FP4 rows [.., 400] as float32 latents [.., 512]."""
    n = rows.shape[:-1]
    w = rows[..., :256].contiguous().view(torch.int32)[..., None]
    i = torch.arange(8, device=rows.device)
    mag = (w >> (4 * i)) & 7
    sign = (w >> torch.where(i < 4, 8 * i + 7, 8 * (i - 4) + 3)) & 1
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=rows.device)[mag]
    v = torch.where(sign == 1, -v, v).view(*n, 16, 32)
    return torch.ldexp(v, rows[..., 256:272].int()[..., None] - 127).view(*n, D_V)


def _values(rows, scales, fmt):
    """Cache rows as the float32 values they stand for (an FP8 latent: bf16 of code x scale)."""
    if fmt == "bf16":
        return rows.float()
    rope = rows[..., ROW_BYTES[fmt] - 128:].contiguous().view(torch.bfloat16).float()
    if fmt == "fp4":
        return torch.cat([_fp4_latents(rows), rope], -1)
    n = rows.shape[:-1]
    codes = rows[..., :D_V].contiguous().view(torch.float8_e4m3fn).float()
    if fmt == "fp8":
        s = rows[..., 512:528].contiguous().view(torch.float32)[..., None]
        lat = (codes.view(*n, 4, 128) * s).view(*n, D_V)
    else:
        lat = codes * scales[..., None]
    return torch.cat([lat.to(torch.bfloat16).float(), rope], -1)


def _plain_load(st, fmt):
    t = torch.arange(st["tokens"], device=DEV)
    b = torch.searchsorted(st["offsets"][1:].long(), t, right=True)
    pos = st["starts"][b].long() + t - st["offsets"][b]
    at = st["table"][b, pos // PAGE].long() * PAGE + pos % PAGE
    kv = st["kv"].view(-1, st["kv"].shape[-1])
    return _values(kv[at], st["scales"].view(-1)[at] if st["scales"] is not None else None, fmt).to(torch.bfloat16)


def _softmax_v(logits, v):
    """(out, base-2 log-sum-exp) of natural logits [.., rows, keys] (-inf: masked) over values [.., keys, d]."""
    m = logits.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    e = torch.exp(logits - m)
    z = e.sum(-1, keepdim=True)
    out = (e @ v) / torch.where(z > 0, z, torch.ones_like(z))
    return out, (torch.log(z) + m)[..., 0] / math.log(2.0)


def _plain_decode(st):
    c, q, lens = st["case"], st["q"], st["lens"].long()
    b, s, h = q.shape[:3]
    pos = torch.arange(st["longest"], device=DEV).expand(b, -1)
    at = st["table"].gather(1, pos // PAGE).long() * PAGE + pos % PAGE
    k = _values(st["kv"].view(-1, ROW_BYTES["fp4"])[at], None, "fp4")
    logits = (q.float().view(b, s * h, D_QK) @ k.transpose(1, 2)) * st["scale"]
    last = lens[:, None] - s + torch.arange(s, device=DEV)  # position of each query token
    seen = (pos[:, None] <= last[..., None]) & ((pos[:, None] < c["sinks"]) | (pos[:, None] > last[..., None] - c["window"]))
    logits = logits.view(b, s, h, -1).masked_fill(~seen[:, :, None], -math.inf).view(b, s * h, -1)
    out, lse = _softmax_v(logits, k[..., :D_V])
    return {"out": out.view(b, s, h, D_V).to(torch.bfloat16), "lse": lse.view(b, s, h)}


def _prompt(st, dtype):
    """(out, lse) of each sequence in `dtype`, some queries at a time."""
    q, group = st["q"], st["q"].shape[1] // st["v"].shape[1]
    out = torch.empty(*q.shape[:2], HEAD_V, dtype=torch.bfloat16 if dtype == torch.float32 else dtype, device=DEV)
    lse = torch.empty(q.shape[:2], dtype=dtype, device=DEV)
    q0 = k0 = 0
    for n, m in zip(st["new"], st["keys"]):
        if n:
            heads = st["v"].shape[1]
            rope = st["k_rope"][k0:k0 + m].to(dtype)[:, None].expand(-1, heads, -1)
            k = torch.cat([st["k_nope"][k0:k0 + m].to(dtype), rope], -1).permute(1, 2, 0)  # [heads, 192, keys]
            v = st["v"][k0:k0 + m].to(dtype).transpose(0, 1)
            step = max(1, (1 << 28) // (q.shape[1] * max(m, 1)))
            for a in range(0, n, step):
                e = min(n, a + step)
                see = m - n + e  # keys that the last of these queries sees
                if see <= 0:
                    out[q0 + a:q0 + e], lse[q0 + a:q0 + e] = 0, -math.inf
                    continue
                x = q[q0 + a:q0 + e].to(dtype).view(e - a, heads, group, HEAD_QK).permute(1, 2, 0, 3)
                z = x.reshape(heads, -1, HEAD_QK) @ k[:, :, :see] * st["scale"]
                last = m - n + torch.arange(a, e, device=DEV)
                hide = torch.arange(see, device=DEV) > last[:, None]
                z = z.view(heads, group, e - a, see).masked_fill(hide, -math.inf).view(heads, -1, see)
                o, l = _softmax_v(z, v[:, :see])
                out[q0 + a:q0 + e] = o.view(heads, group, e - a, HEAD_V).permute(2, 0, 1, 3).reshape(e - a, -1, HEAD_V)
                lse[q0 + a:q0 + e] = l.view(heads, group, e - a).permute(2, 0, 1).reshape(e - a, -1)
        q0, k0 = q0 + n, k0 + m
    return out, lse


def _plain_prompt(st):
    out, lse = _prompt(st, torch.float32)
    return {"out": out, "lse": lse}


# --------------------------------------------------------------------------- work
def work(case):
    c, kind = case, case["kind"]
    if kind == "store":  # read, write rows; read them, write bf16
        n = int(_spread(c["new_lo"], c["new_hi"], c["batch"]).sum())
        return {"bytes": n * (D_QK * 2 + 4 + 2 * ROW_BYTES["fp4"] + D_QK * 2) + c["batch"] * 8, "flops": 0}
    if kind == "load":
        n = int(_spread(c["len_lo"], c["len_hi"], c["batch"]).sum())
        extra = 4 if c["fmt"] == "fp8_token" else 0
        return {"bytes": n * (ROW_BYTES[c["fmt"]] + extra + D_QK * 2 + 4 / PAGE) + c["batch"] * 8, "flops": 0}
    if kind == "decode":
        lens, rows = _spread(c["len_lo"], c["len_hi"], c["batch"]), c["s_q"] * c["h_q"]
        keys = np.minimum(lens, c["window"] + c["s_q"] - 1 + np.minimum(c["sinks"], lens)).sum()
        seen = np.minimum(lens, c["window"] + c["sinks"]).sum()
        io = c["batch"] * rows * (D_QK * 2 + D_V * 2 + 4)
        return {"bytes": float(io + keys * (ROW_BYTES["fp4"] + 4 / PAGE)), "flops": float(2 * rows * seen * (D_QK + D_V))}
    new, ctx = _spread(c["new_lo"], c["new_hi"], c["batch"]), _spread(c["ctx_lo"], c["ctx_hi"], c["batch"])
    # (which context goes with which chunk differs from seed to seed: on average the mean one)
    pairs = float((new * (new + 1) / 2).sum() + new.sum() * ctx.mean())
    nbytes = new.sum() * c["h_q"] * (2 * HEAD_QK + 2 * HEAD_V + 4) + \
        (new.sum() + ctx.sum()) * (c["h_kv"] * 2 * (HEAD_QK - D_ROPE + HEAD_V) + 2 * D_ROPE)
    return {"bytes": float(nbytes), "flops": 2 * pairs * c["h_q"] * (HEAD_QK + HEAD_V)}


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "store":
        return torch.cat([_nearest_fp4(st["latent"].double()), st["rope"].double()], 1)
    if kind == "load":
        off, out = st["offsets"].tolist(), []
        for b in range(case["batch"]):
            pos = st["starts"][b].long() + torch.arange(off[b + 1] - off[b], device=DEV)
            out.append(_rows64(st, case["fmt"], b, pos))
        return torch.cat(out)
    if kind == "prompt":
        return _exact_prompt(st)
    q, lens = st["q"], st["lens"].tolist()
    b, s, h = q.shape[:3]
    out = torch.zeros(b, s, h, D_V, dtype=torch.float64, device=DEV)
    lse = torch.full((b, s, h), -math.inf, dtype=torch.float64, device=DEV)
    for e in range(b):
        keys = _rows64(st, "fp4", e, torch.arange(lens[e], device=DEV))
        for i in range(s):
            last = lens[e] - s + i
            see = sorted({*range(0, min(case["sinks"], last + 1)), *range(max(0, last - case["window"] + 1), last + 1)})
            if see:
                k = keys[torch.tensor(see, device=DEV)]
                z = (q[e, i].double() @ k.t()) * st["scale"]
                out[e, i] = torch.softmax(z, -1) @ k[:, :D_V]
                lse[e, i] = torch.logsumexp(z, -1) / math.log(2.0)
    return {"out": out, "lse": lse}


def _nearest_fp4(x):
    """What 4 bits hold of x [n, 512]: the nearest multiple of the step that each value's binade has."""
    t = x.view(len(x), 16, 32)
    top = t.abs().amax(-1, keepdim=True) / 6.0
    half, power = torch.frexp(top.clamp(min=2.0 ** -20))  # (log2 of a power of two may come out beside it)
    unit = torch.exp2((power - (half == 0.5).int()).clamp(-13, 13).double())
    y = (t / unit).clamp(-6.0, 6.0)
    step = torch.where(y.abs() >= 4, 2.0, torch.where(y.abs() >= 2, 1.0, 0.5))
    return (torch.round(y / step) * step * unit).view_as(x)


def _rows64(st, fmt, b, pos):
    at = st["table"][b].long()[pos // PAGE] * PAGE + pos % PAGE
    r = st["kv"].reshape(-1, st["kv"].shape[-1])[at]
    if fmt == "bf16":
        return r.double()
    rope = r[:, -128:].contiguous().view(torch.bfloat16).double()
    if fmt == "fp4":
        # value 8 w + i of word w: E2M1 bits e e m, exponent 0 without the leading one
        byte = r[:, :256].long().view(-1, 64, 4)
        low, high = byte & 15, byte >> 4
        nib = torch.stack([low, high], -1).view(-1, 64, 8)  # nibble i of each word
        m3 = nib & 7
        bit = nib >> 3
        sign = torch.cat([bit[..., 1::2], bit[..., 0::2]], -1)  # signs of values 0..3 lie in the odd nibbles
        mag = torch.where(m3 < 2, m3 * 0.5, (1 + (m3 & 1) * 0.5) * torch.exp2((m3 >> 1).double() - 1))
        lat = mag.double() * (1 - 2 * sign)
        scale = torch.exp2(r[:, 256:272].double() - 127)
        lat = (lat.view(-1, 16, 32) * scale[..., None]).view(-1, D_V)
    else:
        code = r[:, :D_V].contiguous().view(torch.float8_e4m3fn).double()
        if fmt == "fp8":
            scale = r[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
        else:
            scale = st["scales"].reshape(-1)[at].double()[:, None]
        lat = (code * scale).to(torch.bfloat16).double()  # part of the format's definition
    return torch.cat([lat, rope], 1)


def _exact_prompt(st):
    q, v = st["q"], st["v"]
    group = q.shape[1] // v.shape[1]
    out = torch.zeros(*q.shape[:2], HEAD_V, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    q0 = k0 = 0
    for n, m in zip(st["new"], st["keys"]):
        rope = st["k_rope"][k0:k0 + m].double()
        for h in range(q.shape[1]):
            nope, val = st["k_nope"][k0:k0 + m, h // group].double(), v[k0:k0 + m, h // group].double()
            for a in range(0, n, 4096):
                e = min(n, a + 4096)
                see = m - n + e
                if see <= 0:
                    continue
                x = q[q0 + a:q0 + e, h].double()
                z = (x[:, :128] @ nope[:see].t() + x[:, 128:] @ rope[:see].t()) * st["scale"]
                z.masked_fill_(torch.ones_like(z, dtype=torch.bool).triu(m - n + a + 1), -math.inf)
                total = torch.logsumexp(z, -1, keepdim=True)
                w = torch.exp(z - torch.where(torch.isfinite(total), total, 0.0))
                out[q0 + a:q0 + e, h] = w @ val[:see]
                lse[q0 + a:q0 + e, h] = total[:, 0] / math.log(2.0)
        q0, k0 = q0 + n, k0 + m
    return {"out": out, "lse": lse}
