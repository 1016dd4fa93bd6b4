"""Cases of the quantised cache and of tree attention: inputs, plain forms in elementary torch, and the library's calls.

A quantised cache holds e4m3 values, qpool [NB, H_kv, 2, B, D], and one power-of-two scale per (token, KV head, K or
V) row, scales [NB, H_kv, 2, B] uint8: byte b stands for 2^(b - 127).  Four operators work on it: the write that
quantises, the read that restores 16-bit blocks, single-token decode attention, and attention for a tree of drafted
tokens (the last over a 16-bit pool [NB, B, 2, H_kv, D] as well).
"""
import math

import numpy as np
import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E_MIN, E_MAX = -40, 40      # exponents a scale can take
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of four short sequences into a small pool: latency only
        {"name": "write 4 tokens", "op": "write", "T": 4, "H_kv": 2, "D": 64, "B": 8, "dtype": "f16", "NB": 64},
        # the chunked prefill of a few long prompts, 8 KV heads: 134 MB of K and V quantised in one call
        {"name": "write 16387 tokens", "op": "write", "T": 16387, "H_kv": 8, "D": 128, "B": 16, "dtype": "bf16",
         "NB": 1100},
        # a sequence's prefix brought back to 16 bits before a chunk of prefill over it
        {"name": "read 37 blocks", "op": "read", "n": 37, "H_kv": 8, "D": 128, "B": 16, "dtype": "bf16", "NB": 128},
        # many prefixes at once
        {"name": "read 4001 blocks", "op": "read", "n": 4001, "H_kv": 8, "D": 128, "B": 16, "dtype": "bf16",
         "NB": 4200},
        # one chat sequence, one token
        {"name": "decode 1 x 1000", "op": "decode", "N": 1, "H_q": 32, "H_kv": 8, "D": 128, "B": 16, "dtype": "bf16",
         "lens": "fixed", "ctx": 1000},
        # a serving batch with chat-like lengths
        {"name": "decode 256 chats", "op": "decode", "N": 256, "H_q": 32, "H_kv": 8, "D": 128, "B": 16,
         "dtype": "bf16", "lens": "lognormal", "ctx": 4096},
        # long documents, 7 query heads per KV head
        {"name": "decode 8 x 32768", "op": "decode", "N": 8, "H_q": 56, "H_kv": 8, "D": 128, "B": 32, "dtype": "bf16",
         "lens": "fixed", "ctx": 32768},
        # one KV head per query head, uniform lengths
        {"name": "decode 64 mha", "op": "decode", "N": 64, "H_q": 40, "H_kv": 40, "D": 128, "B": 16, "dtype": "f16",
         "lens": "uniform", "ctx": 2048},
        # a single user's drafted chain and branches: latency
        {"name": "tree 1 x 8 over 500", "op": "tree", "N": 1, "n": 8, "H_q": 32, "H_kv": 8, "D": 128, "B": 16,
         "dtype": "bf16", "quant": False, "lens": "fixed", "ctx": 500},
        # a serving batch, every sequence with its own tree of up to 24 tokens
        {"name": "tree 64 x 24 chats", "op": "tree", "N": 64, "n": 24, "H_q": 32, "H_kv": 8, "D": 128, "B": 16,
         "dtype": "bf16", "quant": False, "lens": "lognormal", "ctx": 4096},
        # wide trees over a quantised cache
        {"name": "tree 16 x 63 quantised", "op": "tree", "N": 16, "n": 63, "H_q": 32, "H_kv": 8, "D": 128, "B": 16,
         "dtype": "bf16", "quant": True, "lens": "uniform", "ctx": 8000},
        # long documents, 7 query heads per KV head, quantised
        {"name": "tree 4 x 18 over 16384", "op": "tree", "N": 4, "n": 18, "H_q": 56, "H_kv": 8, "D": 128, "B": 32,
         "dtype": "f16", "quant": True, "lens": "fixed", "ctx": 16384},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "tree", "tree", "tree"])
    H_kv = rng.choice([1, 2, 3, 4, 8, 8, 10, 16])
    c = {"op": op, "H_kv": H_kv, "D": rng.choice([64, 128, 128]), "B": rng.choice([8, 16, 32]),
         "dtype": rng.choice(["f16", "bf16"])}
    if op == "write":
        T = _log_int(rng, 1, 131000 // H_kv)
        return {**c, "T": T, "NB": -(-T // c["B"]) + rng.randint(1, 40)}
    if op == "read":
        n = _log_int(rng, 1, 512000 // (H_kv * c["B"]))
        return {**c, "n": n, "NB": n + rng.randint(1, 200)}
    G = rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    N = _log_int(rng, 1, 128)
    n = _log_int(rng, 1, 64) if op == "tree" else 1
    # the K and V bytes, and the products of a tree, stay below the largest listed case's
    top = min(16384, 1000000 // (N * H_kv), 45_000_000_000 // (4 * c["D"] * N * n * G * H_kv))
    c = {**c, "N": N, "H_q": G * H_kv, "lens": rng.choice(["fixed", "uniform", "lognormal"]),
         "ctx": _log_int(rng, 70, max(71, top))}
    if op == "decode":
        return c
    return {**c, "n": n, "quant": rng.random() < 0.5}


def _lengths(c):
    """Context lengths [N] (drafted tokens included): a property of the case, not of the seed."""
    r = np.random.Generator(np.random.PCG64([c["N"], c["ctx"], c["B"]]))
    N, top = c["N"], c["ctx"]
    if c["lens"] == "fixed":
        ctx = np.full(N, top)
    elif c["lens"] == "uniform":
        ctx = r.integers(max(1, top // 16), top + 1, size=N)
    else:
        ctx = np.clip(np.rint(r.lognormal(math.log(max(2.0, min(1000.0, top / 4))), 1.0, size=N)), 1, top)
    return ctx.astype(np.int64)


def _drafts(c, ctx):
    """Drafted tokens per sequence [N], at most the context; the last of several sequences has nothing but its draft."""
    r = np.random.Generator(np.random.PCG64([c["N"], c["n"], 7]))
    n = r.integers(max(1, c["n"] // 2), c["n"] + 1, size=c["N"])
    n[0] = c["n"]
    n = np.minimum(n, ctx)
    if c["N"] > 1:
        ctx = ctx.copy()
        ctx[-1] = n[-1]
    return n, ctx


def work(case):
    c = case
    row = c["H_kv"] * c["D"]
    if c["op"] == "write":
        return {"bytes": c["T"] * (2 * row * 2 + 2 * row + 2 * c["H_kv"] + 8), "flops": 4 * c["T"] * row}
    if c["op"] == "read":
        t = c["n"] * c["B"]
        return {"bytes": t * (2 * row + 2 * c["H_kv"] + 2 * row * 2) + 16 * c["n"], "flops": 2 * t * row}
    ctx = _lengths(c)
    if c["op"] == "decode":
        tok = int(ctx.sum())
        kv = tok * (2 * row + 2 * c["H_kv"])
        return {"bytes": kv + 2 * c["N"] * c["H_q"] * c["D"] * 2, "flops": 4 * tok * c["H_q"] * c["D"]}
    n, ctx = _drafts(c, ctx)
    tok = int(ctx.sum())
    kv = tok * (2 * row + 2 * c["H_kv"]) if c["quant"] else tok * 2 * row * 2
    T = int(n.sum())
    return {"bytes": kv + 2 * T * c["H_q"] * c["D"] * 2 + T * ((c["n"] + 31) // 32) * 4,
            "flops": 4 * c["H_q"] * c["D"] * int((n * (ctx - n)).sum() + n.sum() * 1)}


# ------------------------------------------------------------------------------------------------ inputs

def _pow2(e):
    """2^e in fp32 for an integer tensor e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """(e4m3 values, scale bytes) of rows x [..., D]: the smallest power of two that brings the row below 448."""
    a = x.float().abs().amax(-1)
    f, e = torch.frexp(a)                            # a = f 2^e, f in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(a > 0, e - 9 + (f > 0.875), torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    return (x.float() * _pow2(-e)[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _rows(g, shape, dtype):
    """K or V rows [..., H, D] as a model produces them: channels of different size, tokens of different norm."""
    x = torch.randn(shape, generator=g, device="cuda")
    ch = torch.exp(0.5 * torch.randn(shape[-2:], generator=g, device="cuda"))
    tok = torch.exp(0.3 * torch.randn(shape[:-1], generator=g, device="cuda"))[..., None]
    return (0.8 * x * ch * tok).to(dtype)


def _pool(g, NB, c):
    """A filled 16-bit pool [NB, B, 2, H_kv, D]."""
    return _rows(g, (NB, c["B"], 2, c["H_kv"], c["D"]), DT[c["dtype"]])


def _quant_pool(g, NB, c):
    """A filled quantised pool: qpool [NB, H_kv, 2, B, D] and its scale bytes [NB, H_kv, 2, B]."""
    x = _pool(g, NB, c).permute(0, 3, 2, 1, 4)
    q, e = _quantise(x)
    return q.contiguous(), e.contiguous()


def prepare(case, seed):
    c, dt = case, DT[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": dict(c)}
    if c["op"] == "write":
        s["k"] = _rows(g, (c["T"], c["H_kv"], c["D"]), dt)
        s["v"] = _rows(g, (c["T"], c["H_kv"], c["D"]), dt)
        s["qpool"], s["scales"] = _quant_pool(g, c["NB"], c)
        s["slots"] = torch.randperm(c["NB"] * c["B"], generator=g, device="cuda")[: c["T"]].contiguous()
        return s
    if c["op"] == "read":
        s["qpool"], s["scales"] = _quant_pool(g, c["NB"], c)
        src = torch.randperm(c["NB"], generator=g, device="cuda")[: c["n"]]
        dst = torch.randperm(c["n"], generator=g, device="cuda")
        s["pairs"] = torch.stack([src, dst], 1).contiguous()
        s["pool"] = torch.zeros(c["n"], c["B"], 2, c["H_kv"], c["D"], dtype=dt, device="cuda")
        return s
    ctx = _lengths(c)
    n = None
    if c["op"] == "tree":
        n, ctx = _drafts(c, ctx)
    MB = int(-(-ctx.max() // c["B"]))
    used = -(-ctx // c["B"])
    NB = int(used.sum()) + 8
    perm = torch.randperm(NB, generator=g, device="cuda").to(torch.int32)
    start = torch.from_numpy(np.concatenate([[0], np.cumsum(used)[:-1]])).cuda()
    at = start[:, None] + torch.arange(MB, device="cuda")
    valid = torch.arange(MB, device="cuda") < torch.from_numpy(used).cuda()[:, None]
    s["tables"] = torch.where(valid, perm[at.clamp(max=NB - 1)], torch.full_like(perm[:1], 0)).contiguous()
    s["ctx"] = torch.from_numpy(ctx.astype(np.int32)).cuda()
    s["max_ctx"] = int(ctx.max())
    if c["op"] == "decode" or c["quant"]:
        s["qpool"], s["scales"] = _quant_pool(g, NB, c)
    else:
        s["pool"] = _pool(g, NB, c)
    if c["op"] == "decode":
        s["q"] = torch.randn(c["N"], c["H_q"], c["D"], generator=g, device="cuda").to(dt)
        s["out"] = torch.empty_like(s["q"])
        return s
    T = int(n.sum())
    s["q"] = torch.randn(T, c["H_q"], c["D"], generator=g, device="cuda").to(dt)
    s["out"] = torch.empty_like(s["q"])
    s["q_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
    s["max_q_len"] = int(n.max())
    s["mask"] = torch.from_numpy(_tree_masks(n, c["n"], int(seed)).view(np.int32)).cuda()
    return s


def _tree_masks(n, top, seed):
    """Packed ancestor masks [T, W] uint32 of random trees: token i's parent is an earlier token or the prefix; in a
    sequence that has no prefix the last token is padding and sees nothing."""
    r = np.random.Generator(np.random.PCG64([seed, 11]))
    N, W = len(n), (top + 31) // 32
    m = np.zeros((N, top, W), dtype=np.uint32)
    for i in range(top):
        par = np.maximum(r.integers(-1, i, size=N), r.integers(-1, i, size=N)) if i else np.full(N, -1)
        if i:
            m[:, i] = np.where((par >= 0)[:, None], m[np.arange(N), np.maximum(par, 0)], 0)
        m[:, i, i // 32] |= np.uint32(1 << (i % 32))
    if N > 1 and n[-1] > 1:
        m[-1, n[-1] - 1] = 0
    return np.concatenate([m[s, : n[s]] for s in range(N)])


# ------------------------------------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_write(s):
    import paged_kv_cache_302_gb300 as pa
    pa.pa_reshape_and_cache_quant(s["k"], s["v"], s["qpool"], s["scales"], s["slots"])
    return s["qpool"], s["scales"]


def _own_read(s):
    import paged_kv_cache_302_gb300 as pa
    pa.pa_dequant_blocks(s["pool"], s["qpool"], s["scales"], s["pairs"])
    return s["pool"]


def _own_decode(s):
    import paged_kv_cache_302_gb300 as pa
    c = s["case"]
    if "workspace" not in s:
        nbytes = pa.pa_decode_workspace_bytes(c["N"], c["H_q"], c["H_kv"], c["D"], s["max_ctx"])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return pa.pa_decode_quant(s["out"], s["q"], s["qpool"], s["scales"], s["tables"], s["ctx"], s["max_ctx"],
                              workspace=s["workspace"])


def _own_tree(s):
    import paged_kv_cache_302_gb300 as pa
    c = s["case"]
    if "workspace" not in s:
        nbytes = pa.pa_decode_tree_workspace_bytes(c["N"], c["H_q"], c["H_kv"], c["D"], s["max_q_len"])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return pa.pa_decode_tree(s["out"], s["q"], s["qpool"] if c["quant"] else s["pool"], s["tables"], s["ctx"],
                             s["q_start"], s["mask"], s["max_q_len"], scales=s["scales"] if c["quant"] else None,
                             workspace=s["workspace"])


def _plain_write(s):
    B = s["case"]["B"]
    blk, off = s["slots"] // B, s["slots"] % B
    q, e = _quantise(torch.stack([s["k"], s["v"]], 2))       # [T, H_kv, 2, D]
    s["qpool"].view(torch.uint8)[blk, :, :, off] = q.view(torch.uint8)
    s["scales"][blk, :, :, off] = e
    return s["qpool"], s["scales"]


def _values(qpool, scales):
    """fp32 values of quantised rows."""
    return qpool.float() * _pow2(scales.to(torch.int32) - 127)[..., None]


def _plain_read(s):
    src, dst = s["pairs"][:, 0], s["pairs"][:, 1]
    x = _values(s["qpool"].view(torch.uint8)[src].view(torch.float8_e4m3fn), s["scales"][src])
    x = x.permute(0, 3, 2, 1, 4)
    if s["pool"].dtype == torch.float16:
        x = x.clamp(-65504.0, 65504.0)
    s["pool"][dst] = x.to(s["pool"].dtype)
    return s["pool"]


def _gathered(s):
    """fp32 K and V [N, H_kv, MB*B, D] through the block tables."""
    t = s["tables"].long()
    N, MB = t.shape
    if "qpool" in s:
        x = _values(s["qpool"].view(torch.uint8)[t].view(torch.float8_e4m3fn), s["scales"][t])
        x = x.permute(3, 0, 2, 1, 4, 5)              # [N, MB, H, 2, B, D] -> [2, N, H, MB, B, D]
    else:
        x = s["pool"][t].float().permute(3, 0, 4, 1, 2, 5)   # [N, MB, B, 2, H, D]
    x = x.reshape(2, N, x.shape[2], -1, x.shape[-1])
    return x[0], x[1]


def _plain_decode(s):
    c = s["case"]
    k, v = _gathered(s)
    N, H, S, D = k.shape
    q = s["q"].float().view(N, H, -1, D)
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)
    seen = torch.arange(S, device="cuda") < s["ctx"][:, None]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(x, v) / x.sum(-1, keepdim=True)
    return o.reshape(N, c["H_q"], D).to(s["q"].dtype)


def _plain_tree(s):
    c = s["case"]
    k, v = _gathered(s)
    N, H, S, D = k.shape
    n, T = s["max_q_len"], s["q"].shape[0]
    qs = s["q_start"].long()
    n_s = qs[1:] - qs[:-1]
    i = torch.arange(n, device="cuda")
    row = (qs[:-1, None] + i).clamp(max=T - 1)       # [N, n] row of q, clamped past the sequence's last
    q = s["q"].float()[row].view(N, n, H, -1, D).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(N, H, -1, D), k.transpose(-1, -2)) / math.sqrt(D)
    x = x.view(N, H, -1, n, S)                       # [N, H, G, n, S]
    t = torch.arange(S, device="cuda")
    base = s["ctx"].long() - n_s                     # tokens before the draft
    j = t - base[:, None]                            # [N, S] index among the drafted tokens
    W = s["mask"].shape[1]
    word = s["mask"][row].gather(2, (j >> 5).clamp(0, W - 1)[:, None].expand(N, n, S))
    bit = ((word >> (j & 31)[:, None]) & 1).bool() & (j < n_s[:, None])[:, None]
    seen = torch.where((j < 0)[:, None], torch.ones_like(bit), bit)[:, None, None]
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - m.masked_fill(m == -math.inf, 0.0))
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(N, H, -1, S), v).view(N, H, -1, n, D) / l.masked_fill(l == 0, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(N * n, c["H_q"], D)
    at = torch.arange(T, device="cuda")
    sq = torch.searchsorted(qs[1:], at, right=True)  # the sequence of each row
    return o[sq * n + at - qs[sq]].to(s["q"].dtype)


_PLAIN = {"write": _plain_write, "read": _plain_read, "decode": _plain_decode, "tree": _plain_tree}
_OWN = {"write": _own_write, "read": _own_read, "decode": _own_decode, "tree": _own_tree}


# ------------------------------------------------------------------------------------------------ in 64 bits

def _e4m3_64(y):
    """Nearest e4m3 value (ties to even) of float64 |y| <= 448."""
    _, e = torch.frexp(y)
    step = torch.exp2((e.clamp(min=-5) - 4).double())
    return torch.round(y / step) * step


def exact(case, seed):
    s, c = prepare(case, seed), case
    D = c["D"]
    if c["op"] == "write":
        vals, by = s["qpool"].double(), s["scales"].clone()
        for i, x in enumerate((s["k"].double(), s["v"].double())):
            a = x.abs().amax(-1)
            e = torch.ceil(torch.log2(a / E4M3_MAX))
            e = torch.where(a > E4M3_MAX * torch.exp2(e), e + 1, e)
            e = torch.where(a <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)
            e = torch.where(a == 0, torch.full_like(e, E_MIN), e).clamp(E_MIN, E_MAX)
            y = _e4m3_64((x / torch.exp2(e)[..., None]).clamp(-E4M3_MAX, E4M3_MAX))
            vals[s["slots"] // c["B"], :, i, s["slots"] % c["B"]] = y
            by[s["slots"] // c["B"], :, i, s["slots"] % c["B"]] = (e + 127).to(torch.uint8)
        return vals, by
    if c["op"] == "read":
        out = torch.zeros(s["pool"].shape, dtype=torch.float64, device="cuda")
        for a in range(0, c["n"], 512):
            p = s["pairs"][a: a + 512]
            x = torch.stack([s["qpool"][i].double() for i in p[:, 0].tolist()])
            x = x * torch.exp2(s["scales"][p[:, 0]].double() - 127)[..., None]
            out[p[:, 1]] = x.permute(0, 3, 2, 1, 4)
        return out
    ctx = s["ctx"].tolist()
    qs = s["q_start"].tolist() if c["op"] == "tree" else list(range(c["N"] + 1))
    G = c["H_q"] // c["H_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(c["N"]):
        L, n = ctx[b], qs[b + 1] - qs[b]
        blocks = s["tables"][b, : -(-L // c["B"])].tolist()
        if "qpool" in s:
            x = torch.stack([s["qpool"][i] .double() * torch.exp2(s["scales"][i].double() - 127)[..., None]
                             for i in blocks])                       # [nb, H, 2, B, D]
            k, v = (x[:, :, i].transpose(0, 1).reshape(c["H_kv"], -1, D)[:, :L] for i in (0, 1))
        else:
            x = torch.cat([s["pool"][i] for i in blocks])[:L].double()   # [L, 2, H, D]
            k, v = x[:, 0].transpose(0, 1), x[:, 1].transpose(0, 1)
        see = torch.ones(n, L, dtype=torch.bool, device="cuda")
        if c["op"] == "tree":
            words = s["mask"][qs[b]: qs[b + 1]].cpu().numpy().view(np.uint32)
            bits = np.unpackbits(words.view(np.uint8), axis=1, bitorder="little")[:, :n]
            see[:, L - n:] = torch.from_numpy(bits.astype(bool)).cuda()
        for h in range(c["H_q"]):
            x = s["q"][qs[b]: qs[b + 1], h].double() @ k[h // G].T / math.sqrt(D)
            x = torch.where(see, x, torch.full_like(x, -math.inf))
            top = x.amax(1, keepdim=True)
            p = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
            tot = p.sum(1, keepdim=True)
            out[qs[b]: qs[b + 1], h] = (p @ v[h // G]) / torch.where(tot == 0, torch.ones_like(tot), tot)
    return out
