"""Cases of the cache-eviction and differential-attention operators: their inputs, plain forms and exact values.

Four operators over the paged quantized KV cache, as a serving loop uses them:

  weights  decode attention of one new token per sequence that also accumulates, per KV head and cached position,
           the attention weight the position received (INT4 and INT8 pools)
  select   the positions each KV head keeps when its cache is cut to a budget: the first ones, the last ones and the
           ones of largest accumulated weight
  compact  the kept rows moved to the front of the sequence's pages, in place or into other pages
  diff     decode attention with the difference of two softmax maps, normalised per head

With ``own`` false, ``run`` computes them in elementary torch operations (fp32); with ``own`` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-5


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # the first replies of a chat: one sequence, half a thousand tokens; the call's latency is what counts
        dict(name="weights mha short", op="weights", codec="int4", B=1, Hq=8, Hkv=8, d=128, P=16, Gk=64, Gv=128,
             lo=513, hi=513, decay=1.0),
        # a served batch at one query head per KV head, the benchmark's shape
        dict(name="weights mha 8k", op="weights", codec="int4", B=8, Hq=32, Hkv=32, d=128, P=16, Gk=64, Gv=128,
             lo=8193, hi=8193, decay=1.0),
        # long documents with grouped query heads
        dict(name="weights gqa 32k", op="weights", codec="int4", B=4, Hq=32, Hkv=8, d=128, P=16, Gk=64, Gv=128,
             lo=32769, hi=32769, decay=1.0),
        # a continuous batch of uneven sequences, older weight fading
        dict(name="weights gqa ragged", op="weights", codec="int4", B=32, Hq=32, Hkv=8, d=128, P=32, Gk=32, Gv=64,
             lo=1, hi=4096, decay=0.98),
        # the same over the INT8 cache, only the last step's weight kept
        dict(name="weights int8 ragged", op="weights", codec="int8", B=8, Hq=40, Hkv=8, d=128, P=64, Gk=128, Gv=128,
             lo=300, hi=8191, decay=0.0),
        # small budgets, many heads: a chat batch cut back to 512 positions
        dict(name="select short", op="select", codec="int4", B=8, Hkv=32, lo=400, hi=1025, keep=512, sinks=4,
             recent=64),
        # long documents cut to an eighth
        dict(name="select 32k", op="select", codec="int4", B=4, Hkv=8, lo=32768, hi=32768, keep=4096, sinks=4,
             recent=512),
        # the served batch cut to a quarter, within its own pages
        dict(name="compact mha in place", op="compact", codec="int4", B=8, Hkv=32, d=128, P=16, Gk=64, Gv=128,
             lo=8192, hi=8192, keep=2048, sinks=4, recent=256, in_place=True),
        # uneven INT8 sequences, some below the budget, moved to fresh pages (the old ones are shared)
        dict(name="compact int8 moved", op="compact", codec="int8", B=4, Hkv=8, d=128, P=64, Gk=128, Gv=128,
             lo=1000, hi=32768, keep=4095, sinks=4, recent=255, in_place=False),
        # one short sequence: latency
        dict(name="diff short", op="diff", codec="int4", B=1, Hq=8, Hkv=8, d=128, P=16, Gk=64, Gv=128, lo=513, hi=513,
             norm=True),
        # full heads of 2 x 128, a batch of a few thousand tokens
        dict(name="diff mha 4k", op="diff", codec="int4", B=8, Hq=16, Hkv=16, d=256, P=16, Gk=64, Gv=128, lo=4097,
             hi=4097, norm=True),
        # long documents, grouped query heads
        dict(name="diff gqa 32k", op="diff", codec="int4", B=4, Hq=32, Hkv=8, d=128, P=16, Gk=64, Gv=128, lo=32769,
             hi=32769, norm=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("weights", "weights", "select", "compact", "diff"))
    codec = rng.choice(("int4", "int4", "int8")) if op in ("weights", "compact") else "int4"
    d = 128 if codec == "int8" else rng.choice((64, 128, 128, 256))
    Hkv = rng.choice((1, 2, 3, 4, 5, 8, 12, 16, 32))
    B = _log(rng, 1, 32)
    # at most about the positions of the largest listed case of the same operator
    most = (8 * 32 * 8192 * 128) // ({"weights": 4, "diff": 4}.get(op, 1) * Hkv * d * B)
    hi = _log(rng, 1, max(2, min(32768, most)))
    lo = rng.choice((hi, 0, 1, hi // 2))
    case = dict(op=op, codec=codec, B=B, Hkv=Hkv, lo=min(lo, hi), hi=hi)
    if op != "select":
        groups = [g for g in (32, 64, 128) if g <= (d // 2 if op == "diff" else d) and (d < 256 or g >= 64)]
        case.update(d=d, P=rng.choice((16, 32, 64)), Gk=rng.choice(groups),
                    Gv=rng.choice([g for g in (32, 64, 128) if g <= d]))
    if op in ("select", "compact"):
        keep = max(1, int(hi * rng.uniform(0.05, 1.1)))
        sinks = rng.randint(0, min(8, keep))
        case.update(keep=keep, sinks=sinks, recent=rng.randint(0, keep - sinks))
    if op == "compact":
        case.update(in_place=rng.random() < 0.5)
    if op == "weights":
        case.update(Hq=Hkv * rng.randint(1, 4 if d == 256 else 8), decay=rng.choice((1.0, 0.0, 0.9)))
    if op == "diff":
        case.update(Hq=Hkv * rng.randint(1, 2 if d == 256 else 4), norm=rng.random() < 0.7)
    return case


def _lens(c):
    """Sequence lengths from lo to hi in even steps; the last one is hi."""
    return [c["hi"] if c["B"] == 1 else c["lo"] + (c["hi"] - c["lo"]) * b // (c["B"] - 1) for b in range(c["B"])]


def _max_len(c):
    return max(1, c["hi"])


def _sections(c):
    """(offset, bytes per token row) of a block's K codes, V codes, K scales, V scales, and the block's bytes."""
    d, P = c["d"], c["P"]
    if c["codec"] == "int8":
        rows = (d, d, 4, 4)
    else:
        rows = (d // 2, d // 2, 2 * (d // c["Gk"]), 2 * (d // c["Gv"]))
    offs = [P * sum(rows[:i]) for i in range(4)]
    return list(zip(offs, rows)), (P * sum(rows) + 15) // 16 * 16


def work(case):
    c, lens = case, _lens(case)
    tokens = c["Hkv"] * sum(lens)
    kept = c["Hkv"] * sum(min(n, c["keep"]) for n in lens) if "keep" in c else 0
    if c["op"] == "select":
        return {"bytes": 4 * tokens + 4 * c["B"] * c["Hkv"] * c["keep"] + 8 * c["B"], "flops": 0}
    row = sum(r for _, r in _sections(c)[0])
    if c["op"] == "compact":
        return {"bytes": 2 * kept * row + 4 * (kept + tokens) + 4 * kept, "flops": 0}
    io = c["B"] * c["Hq"] * c["d"] * 6
    heads = c["Hq"] // c["Hkv"]
    if c["op"] == "weights":
        wbytes = 4 * tokens * (1 if c["decay"] == 0.0 else 2)
        return {"bytes": tokens * row + wbytes + io, "flops": 4 * heads * tokens * c["d"]}
    return {"bytes": tokens * row + io, "flops": 6 * heads * tokens * c["d"]}


# ---- inputs --------------------------------------------------------------------------------------

def _pack_rows(x, c, group):
    """Rows x [.., d] fp16 as stored bytes: (codes, scales), each uint8 [.., bytes]."""
    x = x.float()
    if c["codec"] == "int8":
        s = (x.abs().amax(-1, keepdim=True) / 127.0).clamp(min=1e-8)
        codes = torch.round(x / s).clamp(-128, 127).to(torch.int8)
        return codes.view(torch.uint8), s.contiguous().view(torch.uint8)
    g = x.unflatten(-1, (-1, group))
    s = (g.abs().amax(-1, keepdim=True) / 7.0).half()
    s = torch.where(s == 0, torch.ones_like(s), s)
    n = (torch.round(g / s.float()).clamp(-7, 7) + 8).to(torch.uint8).flatten(-2)
    return n[..., 0::2] | (n[..., 1::2] << 4), s.flatten(-2).contiguous().view(torch.uint8)


def _pool(c, gen, pages):
    """A pool of `pages` full pages: unit-normal rows, four channels of each KV head's keys 20 times larger."""
    H, P, d = c["Hkv"], c["P"], c["d"]
    k = torch.randn((pages, H, P, d), generator=gen, device=DEV)
    big = torch.rand((H, d), generator=gen, device=DEV).topk(4, dim=-1).indices
    k = (k * torch.ones((H, d), device=DEV).scatter_(1, big, 20.0)[:, None, :]).half()
    kc, ks = _pack_rows(k, c, c["Gk"])
    del k
    vc, vs = _pack_rows(torch.randn((pages, H, P, d), generator=gen, device=DEV).half(), c, c["Gv"])
    block = torch.cat([t.flatten(2) for t in (kc, vc, ks, vs)], dim=-1)
    pad = _sections(c)[1] - block.shape[-1]
    return torch.nn.functional.pad(block, (0, pad)).flatten()


def _weights(c, gen):
    """Accumulated weights [B, Hkv, max_len]: heavy-tailed, a quarter of them equal to others."""
    w = torch.exp(1.5 * torch.randn((c["B"], c["Hkv"], _max_len(c)), generator=gen, device=DEV))
    tied = torch.rand(w.shape, generator=gen, device=DEV) < 0.25
    return torch.where(tied, (w * 4).floor() / 4, w).contiguous()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    lens = _lens(c)
    s = dict(case=c, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), max_len=_max_len(c))
    if c["op"] in ("weights", "select", "compact"):
        s["weights"] = _weights(c, gen)
    if c["op"] == "weights":  # a few steps' weight, nothing yet behind each sequence
        step = (8.0 / 3.0) * (c["Hq"] // c["Hkv"]) / s["lens"].clamp(min=1)[:, None, None]
        behind = torch.arange(s["max_len"], device=DEV) >= s["lens"][:, None, None]
        s["weights"] = (s["weights"] * step).masked_fill_(behind, 0.0)
    if c["op"] == "select":
        s["kept"] = torch.empty((c["B"], c["Hkv"], c["keep"]), dtype=torch.int32, device=DEV)
        s["new_lens"] = torch.empty(c["B"], dtype=torch.int32, device=DEV)
        return s
    P, nb = c["P"], (s["max_len"] + c["P"] - 1) // c["P"]
    used = (s["lens"][:, None].long() + P - 1) // P > torch.arange(nb, device=DEV)
    pages = sum((n + P - 1) // P for n in lens)
    fresh = 0
    if c["op"] == "compact" and not c["in_place"]:
        nd = (c["keep"] + P - 1) // P
        fresh = c["B"] * nd
    total = pages + fresh + 1
    s["pool"] = _pool(c, gen, total)
    order = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    s["table"] = torch.full((c["B"], nb), -1, dtype=torch.int32, device=DEV)
    s["table"][used] = order[:pages]
    s["pages"] = total
    if c["op"] == "compact":
        s["dst"] = s["table"] if c["in_place"] else order[pages:pages + fresh].view(c["B"], nd).contiguous()
        s["kept"] = _plain_select(s["weights"], s["lens"], c["keep"], c["sinks"], c["recent"])[0]
        return s
    s["q"] = torch.randn((c["B"], c["Hq"], c["d"]), generator=gen, device=DEV).half()
    s["out"] = torch.empty((c["B"], c["Hq"], c["d"]), dtype=torch.float32, device=DEV)
    s["scale"] = (c["d"] if c["op"] == "weights" else c["d"] // 2) ** -0.5
    if c["op"] == "diff":
        s["lam"] = 0.2 + 0.6 * torch.rand(c["Hq"], generator=gen, device=DEV)
        s["gain"] = 1.0 + 0.1 * torch.randn(c["d"], generator=gen, device=DEV) if c["norm"] else None
    return s


# ---- plain forms ---------------------------------------------------------------------------------

def _plain_rows(s):
    """K and V of every table position in fp32, [B, Hkv, positions, d] each."""
    c = s["case"]
    d, P, H = c["d"], c["P"], c["Hkv"]
    sec, block = _sections(c)
    x = s["pool"].view(-1, H, block)[s["table"].clamp(min=0).long()].transpose(1, 2)  # [B, H, pages, block]
    part = [x[..., o:o + P * r].unflatten(-1, (P, r)).contiguous() for o, r in sec]

    def rows(codes, scales, group):
        if c["codec"] == "int8":
            return (codes.view(torch.int8).float() * scales.view(torch.float32)).flatten(2, 3)
        n = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
        g = (n.float() - 8.0).unflatten(-1, (-1, group))
        return (g * scales.view(torch.float16).float().unsqueeze(-1)).flatten(-2).flatten(2, 3)

    return rows(part[0], part[2], c["Gk"]), rows(part[1], part[3], c["Gv"])


def _plain_softmax(z, valid):
    z = z.masked_fill(~valid, -math.inf)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _plain_weights(s):
    c = s["case"]
    K, V = _plain_rows(s)
    q = s["q"].float().unflatten(1, (c["Hkv"], -1))
    valid = torch.arange(K.shape[2], device=DEV) < s["lens"][:, None, None, None]
    p = _plain_softmax(torch.matmul(q, K.transpose(-1, -2)) * s["scale"], valid)
    s["out"].copy_(torch.matmul(p, V).flatten(1, 2))
    n = s["weights"].shape[2]
    mass, old = p.sum(2)[..., :n], s["weights"]
    s["weights"].copy_(torch.where(valid[:, 0, :, :n], mass if c["decay"] == 0.0 else c["decay"] * old + mass, old))
    return [s["out"], s["weights"]]


def _plain_select(weights, lens, keep, sinks, recent):
    n = lens[:, None, None].long()
    at = torch.arange(weights.shape[2], device=DEV)
    w = torch.where(weights.isnan(), torch.full_like(weights, -math.inf), weights)
    kind = torch.where((at < sinks) | (at >= n - recent), 0, 1)
    kind = torch.where(at >= n, 2, kind).expand(w.shape)
    by_w = torch.sort(w, dim=-1, descending=True, stable=True).indices
    by_kind = torch.sort(kind.gather(-1, by_w), dim=-1, stable=True).indices
    order = by_w.gather(-1, by_kind)[..., :keep]
    order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]), value=weights.shape[2])
    order = torch.where(order < n, order, weights.shape[2]).sort(dim=-1).values
    kept = torch.where(order < n, order, -1).to(torch.int32)
    return kept, lens.clamp(max=keep)


def _plain_compact(s):
    c = s["case"]
    P, H, kept = c["P"], c["Hkv"], s["kept"].long()
    sec, block = _sections(c)
    b, h, i = torch.nonzero(kept >= 0, as_tuple=True)
    t = kept[b, h, i]
    src, dst = s["table"][b, t // P].long(), s["dst"][b, i // P].long()
    blocks = s["pool"].view(-1, H, block)
    views = [blocks[..., o:o + P * r].unflatten(-1, (P, r)) for o, r in sec]
    taken = [v[src, h, t % P] for v in views]
    [v.index_put_((dst, h, i % P), x) for v, x in zip(views, taken)]
    w = s["weights"][b, h, t]
    freed = torch.arange(s["weights"].shape[2], device=DEV) < s["lens"][:, None, None]
    s["weights"].masked_fill_(freed, 0.0)
    s["weights"][b, h, i] = w
    # rows move as they are stored, codes and scales unread: the pool's bytes are the answer, every one of them equal
    return [s["pool"], s["weights"]]


def _plain_diff(s):
    c = s["case"]
    K, V = _plain_rows(s)
    half = c["d"] // 2
    q = s["q"].float().unflatten(1, (c["Hkv"], -1))
    valid = torch.arange(K.shape[2], device=DEV) < s["lens"][:, None, None, None]
    p1 = _plain_softmax(torch.matmul(q[..., :half], K[..., :half].transpose(-1, -2)) * s["scale"], valid)
    p2 = _plain_softmax(torch.matmul(q[..., half:], K[..., half:].transpose(-1, -2)) * s["scale"], valid)
    o = (torch.matmul(p1, V) - s["lam"].view(c["Hkv"], -1, 1) * torch.matmul(p2, V)).flatten(1, 2)
    if c["norm"]:
        o = o / torch.sqrt(o.square().mean(-1, keepdim=True) + EPS) * s["gain"]
    s["out"].copy_(o * 0.2)
    return [s["out"]]


# ---- the library's calls -------------------------------------------------------------------------

def _own(s):
    import int4_group_quantized_kvq_gb300 as kvq
    c = s["case"]
    if "cfg" not in s:  # kept by a serving program for as long as it runs
        s["cfg"] = kvq.config(c["Hkv"], c.get("d", 128), c.get("P", 16), c.get("Gk", 64), c.get("Gv", 128),
                              s.get("pages", 1))
        new = {"weights": kvq.new_int8_weights_workspace if c["codec"] == "int8" else kvq.new_weights_workspace,
               "diff": kvq.new_diff_workspace}.get(c["op"])
        s["workspace"] = new(s["cfg"], c["B"], c["Hq"], s["max_len"]) if new else None
    if c["op"] == "weights":
        call = kvq.kvq_int8_decode_attention_weights if c["codec"] == "int8" else kvq.kvq_decode_attention_weights
        call(s["cfg"], s["pool"], s["q"], s["table"], s["lens"], s["max_len"], s["scale"], c["decay"], s["weights"],
             s["out"], s["workspace"])
        return [s["out"], s["weights"]]
    if c["op"] == "select":
        kvq.kvq_evict_select(s["cfg"], s["weights"], s["lens"], s["max_len"], c["keep"], c["sinks"], c["recent"],
                             s["kept"], s["new_lens"])
        return [s["kept"], s["new_lens"]]
    if c["op"] == "compact":
        call = kvq.kvq_int8_evict_compact if c["codec"] == "int8" else kvq.kvq_evict_compact
        call(s["cfg"], s["pool"], s["table"], s["dst"], s["lens"], s["kept"], s["weights"])
        return [s["pool"], s["weights"]]
    kvq.kvq_diff_decode_attention(s["cfg"], s["pool"], s["q"], s["table"], s["lens"], s["max_len"], s["scale"],
                                  s["lam"], s["gain"], EPS, 0.2, s["out"], s["workspace"])
    return [s["out"]]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "select":
        c = state["case"]
        kept, new_lens = _plain_select(state["weights"], state["lens"], c["keep"], c["sinks"], c["recent"])
        return [state["kept"].copy_(kept), state["new_lens"].copy_(new_lens)]
    return {"weights": _plain_weights, "compact": _plain_compact, "diff": _plain_diff}[op](state)


# ---- exact values --------------------------------------------------------------------------------

def _exact_rows(s, b, n):
    """K and V of sequence b's first n positions in fp64, [Hkv, n, d], read byte by byte from the pool."""
    c = s["case"]
    d, P, H = c["d"], c["P"], c["Hkv"]
    sec, block = _sections(c)
    t = torch.arange(n, device=DEV)
    base = (s["table"][b, t // P].long() * H + torch.arange(H, device=DEV)[:, None]) * block  # [H, n]

    def read(part, count):
        off, row = sec[part]
        at = base + off + (t % P) * row
        return s["pool"][at[..., None] + torch.arange(count, device=DEV)].long()

    def values(codes, scales, group):
        dim = torch.arange(d, device=DEV)
        if c["codec"] == "int8":
            x = read(codes, d)
            f = read(scales, 4).to(torch.uint8).view(torch.float32).double()
            return torch.where(x > 127, x - 256, x).double() * f
        x = read(codes, d // 2)[..., dim // 2]
        x = torch.where(dim % 2 == 1, x // 16, x % 16) - 8
        f = read(scales, sec[scales][1]).to(torch.uint8).view(torch.float16).double()
        return x.double() * f[..., dim // group]

    return values(0, 2, c["Gk"]), values(1, 3, c["Gv"])


def exact(case, seed):
    c, s = case, prepare(case, seed)
    lens = _lens(c)
    if c["op"] == "select":
        return None  # whole numbers
    if c["op"] == "compact":
        w = s["weights"].double().cpu().numpy()
        kept = s["kept"].cpu().numpy()
        for b, n in enumerate(lens):
            for h in range(c["Hkv"]):
                new = np.zeros(n)
                m = min(n, c["keep"])
                new[:m] = w[b, h, kept[b, h, :m]]
                w[b, h, :n] = new
        return [None, torch.from_numpy(w)]
    out = torch.zeros((c["B"], c["Hq"], c["d"]), dtype=torch.float64, device=DEV)
    w = s["weights"].double() if c["op"] == "weights" else None
    r, half = c["Hq"] // c["Hkv"], c["d"] // 2
    for b, n in enumerate(lens):
        if n == 0:
            continue
        K, V = _exact_rows(s, b, n)
        for h in range(c["Hkv"]):
            q = s["q"][b, h * r:(h + 1) * r].double()
            if c["op"] == "weights":
                p = torch.softmax(q @ K[h].T * s["scale"], dim=-1)
                o = p @ V[h]
                w[b, h, :n] = c["decay"] * w[b, h, :n] + p.sum(0)
            else:
                p1 = torch.softmax(q[:, :half] @ K[h, :, :half].T * s["scale"], dim=-1)
                p2 = torch.softmax(q[:, half:] @ K[h, :, half:].T * s["scale"], dim=-1)
                o = (p1 - s["lam"][h * r:(h + 1) * r].double()[:, None] * p2) @ V[h]
                if c["norm"]:
                    o = o / torch.sqrt((o ** 2).mean(-1, keepdim=True) + EPS) * s["gain"].double()
                o = o * 0.2
            out[b, h * r:(h + 1) * r] = o
    return [out, w] if c["op"] == "weights" else [out]
