"""Cases of block-sparse decode attention and of cache compaction: inputs, plain forms in elementary torch, the calls.

A key summary holds, for each (block, KV head), a box around the block's keys: per channel the least and the greatest K
of its tokens, as 8-bit integers with one power-of-two scale.  summaries [NB, H_kv, 2, D] int8 (lower, upper) and
sum_scales [NB, H_kv] uint8, byte b = 2^(b - 127).  Four operators:

  summarize  rebuilds the summaries of the blocks that hold each sequence's newest tokens
  select     scores every block of a sequence by the largest product its box allows with any query head of the KV head,
             and lists the top_k blocks of each (sequence, KV head), ascending
  decode     single-token attention over the listed blocks alone
  compact    moves a sequence's kept tokens together, in place (accepted drafts, evicted prefixes)

over a 16-bit pool [NB, B, 2, H_kv, D] or a quantised cache (e4m3 qpool [NB, H_kv, 2, B, D] with scale bytes [NB, H_kv, 2,
B]).
"""
import math

import numpy as np
import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E_MIN, E_MAX = -40, 40      # exponents a scale can take
K_TOP, Q_TOP = 127, 511     # integer magnitudes of summaries and of queries in the score


# ------------------------------------------------------------------------------------------------ cases

def listed():
    llama = {"H_q": 32, "H_kv": 8, "D": 128, "B": 16, "dtype": "bf16", "quant": False}
    return [
        # after a decode step of a serving batch: every sequence's last block has one token more
        {"name": "summarize 64 x 1 token", "op": "summarize", **llama, "N": 64, "lens": "lognormal", "ctx": 4096,
         "chunk": 1},
        # after the prefill of long prompts: 268 MB of K
        {"name": "summarize 8 x 16384", "op": "summarize", **llama, "N": 8, "lens": "fixed", "ctx": 16384,
         "chunk": 16384},
        # the same over a quantised cache, ragged chunks that start inside a block
        {"name": "summarize 32 chunks quant", "op": "summarize", **llama, "quant": True, "N": 32, "lens": "uniform",
         "ctx": 8192, "chunk": 4001},
        # one chat with a long document: latency
        {"name": "select 1 x 16384", "op": "select", **llama, "N": 1, "lens": "fixed", "ctx": 16384, "top_k": 64},
        # a serving batch; the short ones keep every block
        {"name": "select 64 uniform", "op": "select", **llama, "N": 64, "lens": "uniform", "ctx": 16384, "top_k": 64},
        # long documents, 7 query heads per KV head
        {"name": "select 16 x 32768", "op": "select", "H_q": 56, "H_kv": 8, "D": 128, "B": 16, "dtype": "f16",
         "quant": False, "N": 16, "lens": "fixed", "ctx": 32768, "top_k": 128},
        # one chat, 1024 tokens of its context
        {"name": "decode 1 x 64 blocks", "op": "decode", **llama, "N": 1, "lens": "fixed", "ctx": 16384, "top_k": 64},
        # a serving batch
        {"name": "decode 64 x 128 blocks", "op": "decode", **llama, "N": 64, "lens": "uniform", "ctx": 16384,
         "top_k": 128},
        # long documents over a quantised cache, 7 query heads per KV head
        {"name": "decode 16 x 256 quant", "op": "decode", "H_q": 56, "H_kv": 8, "D": 128, "B": 16, "dtype": "bf16",
         "quant": True, "N": 16, "lens": "fixed", "ctx": 32768, "top_k": 256},
        # after a step of speculative decoding: the accepted ones of 24 drafted tokens
        {"name": "compact 64 x 24 drafts", "op": "compact", **llama, "N": 64, "lens": "lognormal", "ctx": 4096,
         "span": 24, "keep": 0.25},
        # half of each long context evicted
        {"name": "compact 8 x 16384", "op": "compact", **llama, "N": 8, "lens": "fixed", "ctx": 16384, "span": 16384,
         "keep": 0.5},
        # the same for a few ragged ones over a quantised cache
        {"name": "compact 5 x 8192 quant", "op": "compact", **llama, "quant": True, "N": 5, "lens": "uniform",
         "ctx": 8192, "span": 8192, "keep": 0.7},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["summarize", "select", "select", "decode", "decode", "compact"])
    H_kv = rng.choice([1, 2, 3, 4, 8, 8, 10, 16])
    N = _log_int(rng, 1, 128)
    # the cached K and V stay within a listed case's
    ctx = _log_int(rng, 20, max(21, min(32768, 1000000 // (N * H_kv))))
    c = {"op": op, "H_q": rng.choice([1, 2, 3, 4, 4, 5, 7, 8]) * H_kv, "H_kv": H_kv, "D": rng.choice([64, 128, 128]),
         "B": rng.choice([8, 16, 32]), "dtype": rng.choice(["f16", "bf16"]), "quant": rng.random() < 0.5, "N": N,
         "lens": rng.choice(["fixed", "uniform", "lognormal"]), "ctx": ctx}
    if op == "summarize":
        return {**c, "chunk": _log_int(rng, 1, ctx)}
    if op == "compact":
        return {**c, "span": _log_int(rng, 2, ctx), "keep": round(rng.uniform(0.1, 0.95), 2)}
    return {**c, "top_k": _log_int(rng, 2, max(3, min(256, ctx // c["B"])))}


def _lengths(c):
    """Context lengths [N]: a property of the case, not of the seed."""
    r = np.random.Generator(np.random.PCG64([c["N"], c["ctx"], c["B"]]))
    N, top = c["N"], c["ctx"]
    if c["lens"] == "fixed":
        ctx = np.full(N, top)
    elif c["lens"] == "uniform":
        ctx = r.integers(max(1, top // 16), top + 1, size=N)
    else:
        ctx = np.clip(np.rint(r.lognormal(math.log(max(2.0, min(1000.0, top / 4))), 1.0, size=N)), 1, top)
    return ctx.astype(np.int64)


def _chunks(c, ctx):
    """Newest tokens of each sequence whose summaries are rebuilt [N]; a large chunk is ragged over the batch."""
    n = np.minimum(ctx, c["chunk"])
    if c["lens"] != "fixed" and c["chunk"] > 1:
        r = np.random.Generator(np.random.PCG64([c["N"], c["chunk"], 3]))
        n = np.maximum(1, n - r.integers(0, max(1, c["chunk"] // 2), size=c["N"]))
    return n


def _keeps(c, ctx, seed):
    """First position that may change [N], and the ascending kept positions from there on, one list per sequence."""
    r = np.random.Generator(np.random.PCG64([seed, 5]))
    base = np.maximum(0, ctx - c["span"])
    keep = []
    for b, L in zip(base.tolist(), ctx.tolist()):
        m = max(1, round((L - b) * c["keep"]))
        keep.append(np.sort(r.choice(L - b, size=m, replace=False)) + b)
    return base, keep


def _moved(c, ctx):
    """Tokens that a compaction of this case moves, on average over the seeds (those kept where they are stay)."""
    base, keep = _keeps(c, ctx, 0)
    return sum(int((k != b + np.arange(len(k))).sum()) for b, k in zip(base.tolist(), keep))


def work(case):
    c = case
    ctx = _lengths(c)
    B, H, D = c["B"], c["H_kv"], c["D"]
    nb = -(-ctx // B)
    half = H * (D + 1) if c["quant"] else H * D * 2       # bytes of one token's K (or V)
    box = H * (2 * D + 1)
    if c["op"] == "summarize":
        first = (ctx - _chunks(c, ctx)) // B
        tok, blocks = int((ctx - first * B).sum()), int((nb - first).sum())
        return {"bytes": tok * half + blocks * box, "flops": 2 * tok * H * D}
    if c["op"] == "select":
        scored = int(nb[nb > c["top_k"]].sum())
        return {"bytes": scored * box + 2 * c["N"] * c["H_q"] * D + 4 * c["N"] * H * c["top_k"],
                "flops": 2 * scored * c["H_q"] * D}
    if c["op"] == "decode":
        tok = 0
        for L, n in zip(ctx.tolist(), nb.tolist()):       # the last block, which may be ragged, is always listed
            tok += (min(c["top_k"], n) - 1) * B + L - (n - 1) * B
        return {"bytes": tok * 2 * half + 2 * 2 * c["N"] * c["H_q"] * D, "flops": 4 * tok * c["H_q"] * D}
    m = _moved(c, ctx)
    return {"bytes": 2 * m * 2 * half, "flops": m}


# ------------------------------------------------------------------------------------------------ inputs

def _pow2(e):
    """2^e in fp32 for an integer tensor e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(a, top):
    """The least e in [E_MIN, E_MAX] with a <= top * 2^e for fp32 a >= 0 (E_MAX where none is); top is 2^b - 1."""
    bits = top.bit_length()
    f, e = torch.frexp(a)                                 # a = f 2^e, f in [0.5, 1)
    e = e - bits + (f > top / (1 << bits))
    e = torch.where(a > 0, e, torch.full_like(e, E_MIN))
    return torch.where(torch.isinf(a), torch.full_like(e, E_MAX), e).clamp(E_MIN, E_MAX)


def _rows(g, shape, dtype):
    """K or V rows [..., H, D] as a model produces them: channels of different size, tokens of different norm."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= 0.8 * torch.exp(0.5 * torch.randn(shape[-2:], generator=g, device="cuda"))
    x *= torch.exp(0.3 * torch.randn(shape[:-1], generator=g, device="cuda"))[..., None]
    return x.to(dtype)


def _cache(s, g, NB, c):
    """The filled cache: a pool, or qpool and scales quantised from one (the least scale that holds the row in 448)."""
    x = _rows(g, (NB, c["B"], 2, c["H_kv"], c["D"]), DT[c["dtype"]])
    if not c["quant"]:
        s["pool"] = x
        return
    x = x.permute(0, 3, 2, 1, 4).float()
    a = x.abs().amax(-1)
    f, e = torch.frexp(a)
    e = torch.where(a > 0, e - 9 + (f > 0.875), torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    s["qpool"] = (x * _pow2(-e)[..., None]).to(torch.float8_e4m3fn).contiguous()
    s["scales"] = (e + 127).to(torch.uint8).contiguous()


def _boxes(g, NB, c):
    """Summaries [NB, H_kv, 2, D] and sum_scales [NB, H_kv] of rows like _rows', by the definition."""
    ch = torch.exp(0.5 * torch.randn((c["H_kv"], c["D"]), generator=g, device="cuda"))
    mid = torch.randn((NB, c["H_kv"], c["D"]), generator=g, device="cuda")
    wide = 1.0 + torch.rand((NB, c["H_kv"], c["D"]), generator=g, device="cuda")
    lo, hi = (mid - wide) * ch, (mid + wide) * ch
    e = _exponent(torch.maximum(lo.abs(), hi.abs()).amax(-1), K_TOP)
    box = torch.stack([torch.floor(lo * _pow2(-e)[..., None]), torch.ceil(hi * _pow2(-e)[..., None])], 2)
    return box.clamp(-K_TOP, K_TOP).to(torch.int8), (e + 127).to(torch.uint8)


def prepare(case, seed):
    c, dt = case, DT[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": dict(c)}
    ctx = _lengths(c)
    N, B = c["N"], c["B"]
    used = -(-ctx // B)
    MB, NB = int(used.max()), int(used.sum()) + 8
    perm = torch.randperm(NB, generator=g, device="cuda").to(torch.int32)
    start = torch.from_numpy(np.concatenate([[0], np.cumsum(used)[:-1]])).cuda()
    at = start[:, None] + torch.arange(MB, device="cuda")
    valid = torch.arange(MB, device="cuda") < torch.from_numpy(used).cuda()[:, None]
    s["tables"] = torch.where(valid, perm[at.clamp(max=NB - 1)], torch.full_like(perm[:1], 0)).contiguous()
    s["ctx"] = torch.from_numpy(ctx.astype(np.int32)).cuda()
    s["max_ctx"] = int(ctx.max())
    if c["op"] != "select":
        _cache(s, g, NB, c)
    if c["op"] == "summarize":
        n = _chunks(c, ctx)
        s["summaries"], s["sum_scales"] = _boxes(g, NB, c)
        s["q_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
        s["max_q_len"] = int(n.max())
    elif c["op"] == "compact":
        base, keep = _keeps(c, ctx, int(seed))
        s["base"] = torch.from_numpy(base.astype(np.int32)).cuda()
        s["keep"] = torch.from_numpy(np.concatenate(keep).astype(np.int32)).cuda()
        s["keep_start"] = torch.from_numpy(np.cumsum([0] + [len(k) for k in keep]).astype(np.int32)).cuda()
    else:
        s["q"] = torch.randn(N, c["H_q"], c["D"], generator=g, device="cuda").to(dt)
        if c["op"] == "select":
            s["summaries"], s["sum_scales"] = _boxes(g, NB, c)
            s["selected"] = torch.empty(N, c["H_kv"], c["top_k"], dtype=torch.int32, device="cuda")
        else:
            # a random choice of blocks per KV head, the first and the last among them
            r = torch.rand(N, c["H_kv"], MB, generator=g, device="cuda")
            b = torch.arange(MB, device="cuda")
            last = torch.from_numpy(used).cuda()[:, None, None] - 1
            s["selected"] = _lowest(r.masked_fill((b == 0) | (b == last), -1.0).masked_fill(b > last, 2.0),
                                    last + 1, c["top_k"])
            s["out"] = torch.empty_like(s["q"])
    return s


def _lowest(r, nb, k):
    """Ascending indices of the k least of r [N, H, MB] among the first nb, ties to the lower index, then -1."""
    MB = r.shape[-1]
    first = torch.sort(r, dim=-1, stable=True).indices[..., :k]
    first = torch.where(first < nb, first, torch.full_like(first, MB)).sort(-1).values
    out = torch.full(r.shape[:-1] + (k,), -1, dtype=torch.int32, device=r.device)
    out[..., : first.shape[-1]] = torch.where(first < MB, first, torch.full_like(first, -1)).to(torch.int32)
    return out


# ------------------------------------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_summarize(s):
    import paged_kv_cache_302_gb300 as pa
    pa.pa_summarize_blocks(s["summaries"], s["sum_scales"], s["qpool"] if "qpool" in s else s["pool"], s["tables"],
                           s["ctx"], s["max_q_len"], q_start=s["q_start"], scales=s.get("scales"))
    return s["summaries"], s["sum_scales"]


def _own_select(s):
    import paged_kv_cache_302_gb300 as pa
    c = s["case"]
    if "workspace" not in s:
        nbytes = pa.pa_select_workspace_bytes(c["N"], c["H_kv"], s["max_ctx"], c["B"])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return pa.pa_select_blocks(s["selected"], s["q"], s["summaries"], s["sum_scales"], s["tables"], s["ctx"],
                               s["max_ctx"], c["B"], sink_blocks=1, recent_blocks=1, workspace=s["workspace"])


def _own_decode(s):
    import paged_kv_cache_302_gb300 as pa
    c = s["case"]
    if "workspace" not in s:
        nbytes = pa.pa_decode_sparse_workspace_bytes(c["N"], c["H_q"], c["H_kv"], c["D"], c["B"], c["top_k"])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return pa.pa_decode_sparse(s["out"], s["q"], s["qpool"] if c["quant"] else s["pool"], s["tables"], s["ctx"],
                               s["selected"], scales=s.get("scales"), workspace=s["workspace"])


def _own_compact(s):
    import paged_kv_cache_302_gb300 as pa
    pa.pa_compact_tokens(s["qpool"] if "qpool" in s else s["pool"], s["tables"], s["ctx"], s["base"], s["keep"],
                         s["keep_start"], scales=s.get("scales"))
    return (s["qpool"], s["scales"]) if "qpool" in s else s["pool"]


def _values(qpool, scales):
    """fp32 values of quantised rows."""
    return qpool.float() * _pow2(scales.to(torch.int32) - 127)[..., None]


def _plain_summarize(s):
    c = s["case"]
    B, ctx = c["B"], s["ctx"].long()
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    first = (ctx - n) // B
    b = first[:, None] + torch.arange((s["max_q_len"] + B - 2) // B + 1, device="cuda")
    seq, i = torch.nonzero(b * B < ctx[:, None], as_tuple=True)
    b = b[seq, i]
    phys = s["tables"][seq, b].long()
    if "qpool" in s:
        k = _values(s["qpool"].view(torch.uint8)[phys, :, 0].view(torch.float8_e4m3fn), s["scales"][phys, :, 0])
    else:
        k = s["pool"][phys, :, 0].float().transpose(1, 2)              # [n, H, B, D]
    seen = (b[:, None] * B + torch.arange(B, device="cuda") < ctx[seq][:, None])[:, None, :, None]
    seen = seen & ~torch.isnan(k)
    lo = k.masked_fill(~seen, math.inf).amin(2)
    hi = k.masked_fill(~seen, -math.inf).amax(2)
    none = ~seen.any(2)
    lo, hi = lo.masked_fill(none, 0.0), hi.masked_fill(none, 0.0)
    e = _exponent(torch.maximum(lo.abs(), hi.abs()).amax(-1), K_TOP)
    inv = _pow2(-e)[..., None]
    s["summaries"][phys, :, 0] = torch.floor(lo * inv).clamp(-K_TOP, K_TOP).to(torch.int8)
    s["summaries"][phys, :, 1] = torch.ceil(hi * inv).clamp(-K_TOP, K_TOP).to(torch.int8)
    s["sum_scales"][phys] = (e + 127).to(torch.uint8)
    return s["summaries"], s["sum_scales"]


def _plain_select(s):
    c = s["case"]
    N, H, D = c["N"], c["H_kv"], c["D"]
    q = s["q"].float()
    f = _exponent(q.abs().amax(-1), Q_TOP)
    q = torch.round(q * _pow2(-f)[..., None]).clamp(-Q_TOP, Q_TOP).view(N, H, -1, D)
    t = s["tables"].long()
    box = s["summaries"][t].float().permute(0, 2, 3, 1, 4)             # [N, H, 2, MB, D]
    # the greater of q lo and q hi is q hi for q >= 0, q lo below; sums of integers under 2^24 are exact
    x = torch.matmul(q.clamp(min=0), box[:, :, 1].transpose(-1, -2))
    x += torch.matmul(q.clamp(max=0), box[:, :, 0].transpose(-1, -2))
    x = (x * _pow2(f).view(N, H, -1, 1)).amax(2)
    x = x * _pow2(s["sum_scales"][t].to(torch.int32) - 127).permute(0, 2, 1)
    nb = ((s["ctx"].long() + c["B"] - 1) // c["B"])[:, None, None]
    b = torch.arange(t.shape[1], device="cuda")
    x = x.masked_fill((b == 0) | (b == nb - 1), math.inf).masked_fill(b >= nb, -math.inf)
    s["selected"].copy_(_lowest(-x, nb, c["top_k"]))
    return s["selected"]


def _plain_decode(s):
    c = s["case"]
    N, H, D, B = c["N"], c["H_kv"], c["D"], c["B"]
    sel = s["selected"].long()
    phys = torch.gather(s["tables"].long()[:, None].expand(N, H, -1), 2, sel.clamp(min=0))
    h = torch.arange(H, device="cuda")[None, :, None]
    if "qpool" in s:
        x = _values(s["qpool"].view(torch.uint8)[phys, h].view(torch.float8_e4m3fn), s["scales"][phys, h])
        k, v = (x[:, :, :, i].reshape(N, H, -1, D) for i in (0, 1))    # [N, H, k, 2, B, D]
    else:
        x = s["pool"][phys, :, :, h].float()                           # [N, H, k, B, 2, D]
        k, v = (x[:, :, :, :, i].reshape(N, H, -1, D) for i in (0, 1))
    pos = sel[..., None] * B + torch.arange(B, device="cuda")
    seen = ((sel[..., None] >= 0) & (pos < s["ctx"][:, None, None, None])).view(N, H, 1, -1)
    x = torch.matmul(s["q"].float().view(N, H, -1, D), k.transpose(-1, -2)) / math.sqrt(D)
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - m.masked_fill(m == -math.inf, 0.0))
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / l.masked_fill(l == 0, 1.0)
    return o.reshape(N, c["H_q"], D).to(s["q"].dtype)


def _plain_compact(s):
    c = s["case"]
    B = c["B"]
    ks = s["keep_start"].long()
    j = torch.arange(s["keep"].numel(), device="cuda")
    seq = torch.searchsorted(ks[1:], j, right=True)
    src, dst = s["keep"].long(), s["base"].long()[seq] + j - ks[seq]
    sb, db = s["tables"][seq, src // B].long(), s["tables"][seq, dst // B].long()
    if "qpool" in s:
        q = s["qpool"].view(torch.uint8)
        q[db, :, :, dst % B] = q[sb, :, :, src % B]                    # (the right side is gathered whole before the write)
        s["scales"][db, :, :, dst % B] = s["scales"][sb, :, :, src % B]
        return s["qpool"], s["scales"]
    s["pool"][db, dst % B] = s["pool"][sb, src % B]
    return s["pool"]


_PLAIN = {"summarize": _plain_summarize, "select": _plain_select, "decode": _plain_decode, "compact": _plain_compact}
_OWN = {"summarize": _own_summarize, "select": _own_select, "decode": _own_decode, "compact": _own_compact}


# ------------------------------------------------------------------------------------------------ in 64 bits

def _least_exponent(a, top):
    """The least e in [E_MIN, E_MAX] with a <= top * 2^e, by comparison with every bound (float64 a)."""
    bounds = top * torch.exp2(torch.arange(E_MIN, E_MAX, device=a.device, dtype=torch.float64))
    return E_MIN + (a[..., None] > bounds).sum(-1)


def _tokens(s, b, L):
    """K and V [H, L, D] in float64 of sequence b's first L tokens."""
    c = s["case"]
    blocks = s["tables"][b, : -(-L // c["B"])].long()
    if "qpool" in s:
        x = s["qpool"].view(torch.uint8)[blocks].view(torch.float8_e4m3fn).double()
        x = x * torch.exp2(s["scales"][blocks].double() - 127)[..., None]      # [nb, H, 2, B, D]
        return tuple(x[:, :, i].transpose(0, 1).reshape(c["H_kv"], -1, c["D"])[:, :L] for i in (0, 1))
    x = s["pool"][blocks].flatten(0, 1)[:L].double()                           # [L, 2, H, D]
    return x[:, 0].transpose(0, 1), x[:, 1].transpose(0, 1)


def exact(case, seed):
    s, c = prepare(case, seed), case
    B, D, H, G = c["B"], c["D"], c["H_kv"], c["H_q"] // c["H_kv"]
    ctx = s["ctx"].tolist()
    if c["op"] == "summarize":
        qs = s["q_start"].tolist()
        for b, L in enumerate(ctx):
            first = (L - (qs[b + 1] - qs[b])) // B
            k, _ = _tokens(s, b, L)
            k = torch.nn.functional.pad(k[:, first * B:], (0, 0, 0, -L % B), value=math.nan)
            k = k.reshape(H, -1, B, D)                                         # [H, blocks, B, D]
            lo, hi = k.nan_to_num(nan=math.inf).amin(2), k.nan_to_num(nan=-math.inf).amax(2)
            e = _least_exponent(torch.maximum(lo.abs(), hi.abs()).amax(-1), K_TOP)
            unit = torch.exp2(e.double())[..., None]
            at = s["tables"][b, first: -(-L // B)].long()
            for i, x in enumerate((torch.floor(lo / unit), torch.ceil(hi / unit))):
                s["summaries"][at, :, i] = x.clamp(-K_TOP, K_TOP).to(torch.int8).transpose(0, 1)
            s["sum_scales"][at] = (e + 127).to(torch.uint8).transpose(0, 1)
        return s["summaries"], s["sum_scales"]
    if c["op"] == "select":
        sel = torch.full((c["N"], H, c["top_k"]), -1, dtype=torch.int32)
        for b, L in enumerate(ctx):
            nb = -(-L // B)
            at = s["tables"][b, :nb].long()
            for h in range(H):
                q = s["q"][b, h * G: (h + 1) * G].double()
                f = _least_exponent(q.abs().amax(-1), Q_TOP).double()
                q = torch.round(q / torch.exp2(f)[:, None]).clamp(-Q_TOP, Q_TOP)
                box = s["summaries"][at, h].double() * torch.exp2(s["sum_scales"][at, h].double() - 127)[:, None, None]
                top = torch.full((nb,), -math.inf, dtype=torch.float64, device="cuda")
                for i in range(G):
                    x = torch.maximum(q[i] * box[:, 0], q[i] * box[:, 1]).sum(-1) * torch.exp2(f[i])
                    top = torch.maximum(top, x)
                x = top.cpu().numpy()
                x[[0, nb - 1]] = math.inf
                pick = np.sort(np.lexsort((np.arange(nb), -x))[: c["top_k"]])
                sel[b, h, : len(pick)] = torch.from_numpy(pick.astype(np.int32))
        return sel.cuda()
    if c["op"] == "decode":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, L in enumerate(ctx):
            k, v = _tokens(s, b, L)
            for h in range(H):
                pick = s["selected"][b, h]
                t = (pick[pick >= 0].long()[:, None] * B + torch.arange(B, device="cuda")).flatten()
                t = t[t < L]
                x = s["q"][b, h * G: (h + 1) * G].double() @ k[h, t].T / math.sqrt(D)
                out[b, h * G: (h + 1) * G] = torch.softmax(x, -1) @ v[h, t]
        return out
    keep, ks, base = s["keep"].tolist(), s["keep_start"].tolist(), s["base"].tolist()
    tab = s["tables"].tolist()
    src, dst = [], []
    for b in range(c["N"]):
        for j, t in enumerate(keep[ks[b]: ks[b + 1]]):
            to = base[b] + j
            src.append(tab[b][t // B] * B + t % B)
            dst.append(tab[b][to // B] * B + to % B)
    src, dst = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
    if not c["quant"]:
        x = s["pool"].flatten(0, 1).double()
        x.index_copy_(0, dst, x[src])
        return x.view(s["pool"].shape)
    both = []
    for x in (s["qpool"].double(), s["scales"].clone()):
        y = x.movedim(3, 1).flatten(0, 1)                                      # [NB B, H, 2, (D)]
        y = y.index_copy(0, dst, y[src]).view((-1, B) + y.shape[1:])
        both.append(y.movedim(1, 3).contiguous())
    return tuple(both)
