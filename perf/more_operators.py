"""Cases of the prompt and latent-cache operators: their inputs, plain forms and exact values.

Four operators that fill a quantized paged cache and attend to it with any number of new tokens per sequence:

  write         rotary positions (one to three axes) applied to q and to the new keys, keys and values quantized into
                their INT4 pages in the same pass; then the same rows read back as a prefix store does
  chunk         causal attention of the last rows of every sequence (a prompt, a part of one, a few drafted tokens) over
                its INT4 cache
  latent_write  new rows of a latent cache: the latent part normalised and quantized to 4 bits, the shared rotary key
                rotated, the queries' rotary part rotated; then the rows read back
  latent        attention whose keys and values are one shared latent vector per token (absorbed form), one token per
                sequence or several

With ``own`` false, ``run`` computes them in elementary torch operations; with ``own`` true it calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------------------------
# new_lo .. new_hi: new rows per sequence; old_lo .. old_hi: positions in the cache before them; pad: rows of the batch's
# arrays behind the last sequence.

def listed():
    return [
        # a decode step of a served batch: one new token each; latency
        dict(name="write step", op="write", B=64, Hq=32, Hkv=8, d=128, P=16, Gk=64, Gv=128, rot=128, inter=False, axes=1,
             new_lo=1, new_hi=1, old_lo=100, old_hi=4096, pad=0),
        # the prompts of four long documents at once, the rows of a fused q/k/v projection
        dict(name="write prompt", op="write", B=4, Hq=32, Hkv=8, d=128, P=16, Gk=64, Gv=128, rot=128, inter=False, axes=1,
             new_lo=8192, new_hi=8192, old_lo=0, old_hi=0, pad=0),
        # images and text, positions in time, height and width, heads turned in half, a padded batch
        dict(name="write axes ragged", op="write", B=13, Hq=15, Hkv=5, d=128, P=32, Gk=32, Gv=32, rot=64, inter=True,
             axes=3, new_lo=1, new_hi=2047, old_lo=0, old_hi=777, pad=97),
        # drafted tokens checked against long documents: few rows, the cache's bytes count
        dict(name="chunk draft", op="chunk", B=4, Hq=32, Hkv=8, d=128, P=16, Gk=64, Gv=128, new_lo=8, new_hi=8,
             old_lo=32761, old_hi=32761, pad=0),
        # one prompt from its first token
        dict(name="chunk prompt", op="chunk", B=1, Hq=32, Hkv=8, d=128, P=16, Gk=64, Gv=128, new_lo=8192, new_hi=8192,
             old_lo=0, old_hi=0, pad=0),
        # parts of long prompts behind what is cached already, one query head per kv head
        dict(name="chunk part mha", op="chunk", B=2, Hq=32, Hkv=32, d=128, P=64, Gk=128, Gv=128, new_lo=2048, new_hi=2048,
             old_lo=16384, old_hi=32768, pad=0),
        # a continuous batch: prompts, parts and single tokens together, three query heads per kv head
        dict(name="chunk ragged", op="chunk", B=24, Hq=12, Hkv=4, d=64, P=32, Gk=32, Gv=64, new_lo=1, new_hi=1023,
             old_lo=0, old_hi=4001, pad=33),
        # a decode step of a latent cache, 16 query heads
        dict(name="latent write step", op="latent_write", B=64, H=16, L=512, R=64, P=64, G=64, norm=True, inter=True,
             new_lo=1, new_hi=1, old_lo=100, old_hi=4096, pad=0),
        # prompts into the latent cache
        dict(name="latent write prompt", op="latent_write", B=5, H=32, L=512, R=64, P=64, G=64, norm=True, inter=True,
             new_lo=1000, new_hi=6143, old_lo=0, old_hi=513, pad=0),
        # single tokens of a served batch, all heads on this card
        dict(name="latent decode", op="latent", B=32, H=128, L=512, R=64, P=64, G=64, new_lo=1, new_hi=1,
             old_lo=1023, old_hi=8191, pad=0),
        # one long document, the heads shared over eight cards
        dict(name="latent decode long", op="latent", B=1, H=16, L=512, R=64, P=64, G=64, new_lo=1, new_hi=1,
             old_lo=131071, old_hi=131071, pad=0),
        # parts of prompts and drafted tokens over a smaller latent, an odd number of heads
        dict(name="latent chunk ragged", op="latent", B=9, H=20, L=256, R=64, P=16, G=32, new_lo=1, new_hi=255,
             old_lo=0, old_hi=3000, pad=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "chunk", "chunk", "latent_write", "latent", "latent"))
    B = _log(rng, 1, 64)
    c = dict(op=op, B=B, P=rng.choice((16, 32, 64)))
    if op in ("write", "chunk"):
        d = rng.choice((64, 128, 256) if op == "write" else (64, 128, 128))
        Hkv = rng.choice((1, 2, 3, 4, 5, 8, 16, 32))
        c.update(d=d, Hkv=Hkv, Hq=Hkv * rng.randint(1, 8 if Hkv <= 8 else 2),
                 Gk=rng.choice([g for g in (32, 64, 128) if g <= d]), Gv=rng.choice([g for g in (32, 64, 128) if g <= d]))
    if op == "write":
        rot = rng.choice([r for r in (32, 64, 128, 256) if r <= d])
        c.update(rot=rot, inter=rng.random() < 0.4, axes=rng.choice((1, 1, 2, 3)))
        # at most the rows of the largest listed write
        most = max(2, (32768 * 48 * 128) // (d * (c["Hq"] + 2 * Hkv) * B))
        hi = _log(rng, 1, min(8192, most))
        c.update(old_hi=_log(rng, 1, 4096))
    elif op == "chunk":
        hi = _log(rng, 1, 4096)
        old = _log(rng, 1, 32768)
        # at most the products and the cache rows of the largest listed chunk
        while B * c["Hq"] * d * hi * (old + hi) > 32 * 128 * 2 * 2048 * 26000 and hi > 1:
            hi = max(1, hi // 2)
        while B * Hkv * d * (old + hi) > 32 * 128 * 53000 and old > 1:
            old = max(1, old // 2)
            hi = max(1, hi // 2)
        c.update(old_hi=old)
    else:
        L = rng.choice((256, 512, 512))
        c.update(L=L, R=64, G=rng.choice((32, 64, 128)), H=rng.choice((1, 4, 7, 16, 20, 32, 64, 128)))
        if op == "latent_write":
            hi = _log(rng, 1, max(2, min(6143, 18000 * 32 // (c["H"] * B))))
            c.update(norm=rng.random() < 0.7, inter=rng.random() < 0.5, old_hi=_log(rng, 1, 4096))
        else:
            hi = rng.choice((1, 1, _log(rng, 1, 512)))
            old = _log(rng, 1, 65536)
            while B * c["H"] * hi * (old + hi) > 32 * 128 * 4608 and (hi > 1 or old > 1):
                old, hi = max(1, old // 2), max(1, hi // 2)
            while B * (old + hi) > 32 * 8192:
                old = max(1, old // 2)
            c.update(old_hi=old)
    c.update(new_hi=hi, new_lo=rng.choice((hi, 0, 1, hi // 2)), old_lo=rng.choice((c["old_hi"], 0, c["old_hi"] // 2)),
             pad=rng.choice((0, 0, rng.randint(1, 64))))
    c["new_lo"] = min(c["new_lo"], hi)
    return c


def _spread(lo, hi, n):
    """n numbers from lo to hi in even steps; the last one is hi."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _shape(c):
    """(new rows, positions in all) of every sequence: the longest histories with the fewest new rows."""
    new = _spread(c["new_lo"], c["new_hi"], c["B"])
    old = _spread(c["old_lo"], c["old_hi"], c["B"])[::-1]
    return new, [o + n for o, n in zip(old, new)]


def _row_bytes(c):
    """Bytes of one token's row in a block (all kv heads), section by section."""
    if c["op"].startswith("latent"):
        return (c["L"] // 2, 2 * (c["L"] // c["G"]), 2 * c["R"])
    return (c["d"] // 2, c["d"] // 2, 2 * (c["d"] // c["Gk"]), 2 * (c["d"] // c["Gv"]))


def _block_bytes(c):
    return (c["P"] * sum(_row_bytes(c)) + 15) // 16 * 16


def work(case):
    c = case
    new, total = _shape(c)
    rows, row = sum(new), sum(_row_bytes(c))
    pairs = sum(n * t - n * (n - 1) // 2 for n, t in zip(new, total))
    if c["op"] == "write":
        x = 2 * c["d"]
        return {"bytes": rows * (2 * c["Hq"] * x + 4 * c["Hkv"] * x + 2 * c["Hkv"] * row + 4 * c["rot"]),
                "flops": 3 * rows * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["op"] == "latent_write":
        x = 2 * (c["L"] + c["R"])
        return {"bytes": rows * (2 * x + 2 * row + 4 * c["H"] * c["R"] + 4 * c["R"]),
                "flops": rows * (4 * c["L"] + 3 * (c["H"] + 1) * c["R"])}
    seen = sum(t for n, t in zip(new, total) if n > 0)
    if c["op"] == "chunk":
        return {"bytes": seen * c["Hkv"] * row + 4 * rows * c["Hq"] * c["d"], "flops": 4 * pairs * c["Hq"] * c["d"]}
    return {"bytes": seen * row + 2 * rows * c["H"] * (2 * c["L"] + c["R"]),
            "flops": 2 * pairs * c["H"] * (2 * c["L"] + c["R"])}


# ---- inputs --------------------------------------------------------------------------------------

def _quantize(x, group):
    """fp32 x [.., n] as 4-bit codes (fp32 whole numbers) and fp16 scales [.., n / group]."""
    g = x.unflatten(-1, (-1, group))
    s = (g.abs().amax(-1, keepdim=True) / 7.0).half()
    s = torch.where(s == 0, torch.ones_like(s), s)
    return torch.round(g / s.float()).clamp(-7, 7).flatten(-2), s.squeeze(-1)


def _nibbles(codes):
    n = (codes + 8).to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _bytes_of(x):
    return x.contiguous().view(torch.uint8)


def _pool(c, gen, pages):
    """A pool of full pages: unit-normal rows; of the keys (the latents) four channels are larger."""
    P = c["P"]
    if c["op"].startswith("latent"):
        x = torch.randn((pages, P, c["L"]), generator=gen, device=DEV)
        x[..., :4] *= 4.0
        codes, s = _quantize(x.half().float(), c["G"])
        rope = torch.randn((pages, P, c["R"]), generator=gen, device=DEV).half()
        parts = [_nibbles(codes), _bytes_of(s), _bytes_of(rope)]
        block = torch.cat([t.flatten(1) for t in parts], dim=-1)
    else:
        H, d = c["Hkv"], c["d"]
        k = torch.randn((pages, H, P, d), generator=gen, device=DEV)
        big = torch.rand((H, d), generator=gen, device=DEV).topk(4, dim=-1).indices
        k = (k * torch.ones((H, d), device=DEV).scatter_(1, big, 20.0)[:, None, :]).half()
        kc, ks = _quantize(k.float(), c["Gk"])
        vc, vs = _quantize(torch.randn((pages, H, P, d), generator=gen, device=DEV).half().float(), c["Gv"])
        parts = [_nibbles(kc), _nibbles(vc), _bytes_of(ks), _bytes_of(vs)]
        block = torch.cat([t.flatten(2) for t in parts], dim=-1)
    return torch.nn.functional.pad(block, (0, _block_bytes(c) - block.shape[-1])).flatten()


def _angles(length, rot):
    """Cosines and sines of every position, [length, rot] fp32: rot / 2 cosines, then the sines."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    a = torch.arange(length, device=DEV, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], dim=-1).float()


def _sections(c):
    """How many of the rotary pairs each axis turns."""
    half, axes = c["rot"] // 2, c["axes"]
    if axes == 1:
        return [half]
    rest = half // (axes + 1)
    return [half - rest * (axes - 1)] + [rest] * (axes - 1)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    new, total = _shape(c)
    rows = sum(new) + c["pad"]
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    P = c["P"]
    max_len = max(1, max(total))
    blocks = (max_len + P - 1) // P
    need = [(t + P - 1) // P for t in total]
    pages = sum(need) + 1

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV).half()

    s = dict(case=c, new=new, total=total, cu_list=cu, cu=ints(cu), lens=ints(total), max_len=max_len, rows=rows,
             pages=pages, start=ints([t - n for n, t in zip(new, total)]))
    used = torch.arange(blocks, device=DEV) < ints(need)[:, None]
    s["table"] = torch.full((c["B"], blocks), -1, dtype=torch.int32, device=DEV)
    s["table"][used] = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)[:sum(need)]
    # which sequence and position each row belongs to (the plain forms' own use)
    s["row_seq"] = torch.repeat_interleave(torch.arange(c["B"], device=DEV), ints(new).long())
    at = torch.arange(sum(new), device=DEV) - s["cu"].long()[s["row_seq"]]
    s["row_pos"] = s["start"].long()[s["row_seq"]] + at
    if c["op"] == "write":
        H, Hq, d = c["Hkv"], c["Hq"], c["d"]
        s["pool"] = torch.zeros(pages * H * _block_bytes(c), dtype=torch.uint8, device=DEV)
        qkv = normal(rows, (Hq + 2 * H) * d)  # the rows of one projection: q, k and v of a token side by side
        s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, d)) for t in qkv.split([Hq * d, H * d, H * d], dim=1))
        big = torch.rand((H, d), generator=gen, device=DEV).topk(4, dim=-1).indices
        s["k"].mul_(torch.ones((H, d), device=DEV).scatter_(1, big, 20.0).half())
        s["table_cs"] = _angles(max_len + 64, c["rot"])
        s["positions"] = None
        if c["axes"] > 1:  # time as it goes, height and width within a picture of 32 x 24
            p = torch.nn.functional.pad(s["row_pos"], (0, c["pad"]))
            s["positions"] = torch.stack([p, p // 24 % 32, p % 24][:c["axes"]]).to(torch.int32).contiguous()
        s["q_out"] = torch.zeros((rows, Hq, d), dtype=torch.float16, device=DEV)
        s["k_out"], s["v_out"] = (torch.zeros((rows, H, d), dtype=torch.float16, device=DEV) for _ in range(2))
        return s
    if c["op"] == "latent_write":
        L, R = c["L"], c["R"]
        s["pool"] = torch.zeros(pages * _block_bytes(c), dtype=torch.uint8, device=DEV)
        s["rows_in"] = normal(rows, L + R)
        s["rows_in"][:, :4] *= 4.0
        s["gain"] = 1.0 + 0.1 * torch.randn(L, generator=gen, device=DEV) if c["norm"] else None
        s["q_pe"], s["q"] = normal(rows, c["H"], R), normal(rows, c["H"], L + R)
        s["table_cs"] = _angles(max_len + 64, R)
        s["out"] = torch.zeros((rows, L + R), dtype=torch.float16, device=DEV)
        return s
    s["pool"] = _pool(c, gen, pages)
    if c["op"] == "chunk":
        s["q"] = normal(rows, c["Hq"], c["d"])
        s["scale"] = c["d"] ** -0.5
        s["out"] = torch.zeros((rows, c["Hq"], c["d"]), dtype=torch.float16, device=DEV)
    else:
        s["q"] = normal(rows, c["H"], c["L"] + c["R"])
        s["scale"] = 0.5 * (c["L"] + c["R"]) ** -0.5
        s["out"] = torch.zeros((rows, c["H"], c["L"]), dtype=torch.float16, device=DEV)
    return s


# ---- plain forms ---------------------------------------------------------------------------------

def _rotate(x, cs, rot, inter):
    """The first rot elements of x [rows, heads, n] turned by cs [rows, rot], in fp32, each operation rounded once."""
    half = rot // 2
    c, n = cs[:, None, :half], cs[:, None, half:]
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :half], x[..., half:rot])
    u, w = a * c - b * n, b * c + a * n
    y = torch.stack([u, w], dim=-1).flatten(-2) if inter else torch.cat([u, w], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1).half()


def _row_angles(s):
    """Each row's cosines and sines, [rows of the sequences, rot]."""
    c = s["case"]
    if s.get("positions") is None:
        return s["table_cs"][s["row_pos"]]
    n, half = len(s["row_pos"]), c["rot"] // 2
    part, first = [], 0
    for axis, width in enumerate(_sections(c)):
        t = s["table_cs"][s["positions"][axis, :n].long()]
        part.append((t[:, first:first + width], t[:, half + first:half + first + width]))
        first += width
    return torch.cat([p[0] for p in part] + [p[1] for p in part], dim=-1)


def _behind(x, like):
    """x with zero rows behind it, as many rows as `like`."""
    return torch.nn.functional.pad(x, (0, 0) * (x.dim() - 1) + (0, like.shape[0] - x.shape[0]))


def _round_trip(x, group):
    codes, sc = _quantize(x.float(), group)
    return (codes.unflatten(-1, (-1, group)) * sc.float().unsqueeze(-1)).flatten(-2).half()


def _plain_write(s):
    c, n = s["case"], len(s["row_pos"])
    cs = _row_angles(s)
    q = _rotate(s["q"][:n], cs, c["rot"], c["inter"])
    k = _rotate(s["k"][:n], cs, c["rot"], c["inter"])
    return [_behind(q, s["q"]), _behind(_round_trip(k, c["Gk"]), s["k"]), _behind(_round_trip(s["v"][:n], c["Gv"]), s["v"])]


def _plain_latent_write(s):
    c, n = s["case"], len(s["row_pos"])
    L = c["L"]
    x = s["rows_in"][:n].float()
    y = x[:, :L]
    if s["gain"] is not None:  # the mean of squares in 64 bits: values next to a code's border follow it
        r = (1.0 / torch.sqrt(y.double().square().mean(-1, keepdim=True) + EPS)).float()
        y = y * r * s["gain"]
    cs = _row_angles(s)
    rope = _rotate(x[:, None, L:], cs, c["R"], c["inter"])[:, 0]
    q = s["q"].clone()
    q[:n, :, L:] = _rotate(s["q_pe"][:n], cs, c["R"], c["inter"])
    return [_behind(torch.cat([_round_trip(y, c["G"]), rope], dim=-1), s["out"]), q]


def _plain_rows(s, b):
    """Every cached row of sequence b in fp32: [K, V] each [Hkv, positions, d], or [[latent, rope]] [1, positions, L + R]."""
    c, P = s["case"], s["case"]["P"]
    n = s["total"][b]
    page = s["table"][b, :(n + P - 1) // P].long()
    heads = 1 if c["op"].startswith("latent") else c["Hkv"]
    x = s["pool"].view(-1, heads, _block_bytes(c))[page].transpose(0, 1)
    part, at = [], 0
    for r in _row_bytes(c):
        part.append(x[..., at:at + P * r].unflatten(-1, (P, r)).flatten(1, 2)[:, :n].contiguous())
        at += P * r

    def values(codes, scales, group):
        v = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float() - 8.0
        return (v.unflatten(-1, (-1, group)) * scales.view(torch.float16).float().unsqueeze(-1)).flatten(-2)

    if heads == 1 and "L" in c:
        return [torch.cat([values(part[0], part[1], c["G"]), part[2].view(torch.float16).float()], dim=-1)]
    return [values(part[0], part[2], c["Gk"]), values(part[1], part[3], c["Gv"])]


def _plain_attend(q, K, V, pos, scale):
    """q [rows, g, n], K [t, n], V [t, m], pos [rows]: softmax attention of every row to positions 0 .. pos, fp32."""
    z = torch.matmul(q.float(), K.T) * scale
    z = z.masked_fill(torch.arange(K.shape[0], device=DEV) > pos[:, None, None], -math.inf)
    e = torch.exp(z - z.amax(-1, keepdim=True))
    return torch.matmul(e / e.sum(-1, keepdim=True), V)


def _plain_attention(s):
    c = s["case"]
    out = torch.zeros_like(s["out"])
    for b in range(c["B"]):
        lo, hi = s["cu_list"][b], s["cu_list"][b + 1]
        if lo == hi:
            continue
        kv = _plain_rows(s, b)
        heads = kv[0].shape[0]
        g = s["q"].shape[1] // heads
        step = max(1, (1 << 30) // (g * s["total"][b]))  # scores of at most 4 GB at a time
        for h in range(heads):
            V = kv[1][h] if len(kv) == 2 else kv[0][h, :, :c["L"]]
            for r in range(lo, hi, step):
                to = min(hi, r + step)
                out[r:to, h * g:(h + 1) * g] = _plain_attend(s["q"][r:to, h * g:(h + 1) * g], kv[0][h], V,
                                                             s["row_pos"][r:to], s["scale"]).half()
    return [out]


# ---- the library's calls -------------------------------------------------------------------------

def _own(s):
    import int4_group_quantized_kvq_gb300 as kvq
    c = s["case"]
    if "cfg" not in s:  # kept by a serving program for as long as it runs
        if c["op"].startswith("latent"):
            s["cfg"] = kvq.latent_config(c["L"], c["R"], c["P"], c["G"], s["pages"])
        else:
            s["cfg"] = kvq.config(c["Hkv"], c["d"], c["P"], c["Gk"], c["Gv"], s["pages"])
        if c["op"] == "write":
            s["rope"] = kvq.rope(c["rot"], interleaved=c["inter"], sections=_sections(c) if c["axes"] > 1 else None)
        if c["op"] == "latent_write":
            s["rope"] = kvq.rope(c["R"], interleaved=c["inter"])
        if c["op"] == "chunk":
            s["workspace"] = kvq.new_chunk_workspace(s["cfg"], c["B"], c["Hq"], s["max_len"])
        if c["op"] == "latent":
            s["workspace"] = kvq.new_latent_workspace(s["cfg"], c["B"], c["H"], s["max_len"])
    if c["op"] == "write":
        kvq.kvq_rope_append(s["cfg"], s["rope"], s["pool"], s["q"], s["k"], s["v"], s["q_out"], s["table_cs"], s["table"],
                            s["start"], s["cu"], positions=s["positions"])
        kvq.kvq_dequantize_varlen(s["cfg"], s["pool"], s["table"], s["start"], s["cu"], s["k_out"], s["v_out"])
        return [s["q_out"], s["k_out"], s["v_out"]]
    if c["op"] == "latent_write":
        kvq.kvq_latent_append(s["cfg"], s["rope"], s["pool"], s["rows_in"], s["gain"], EPS, s["q_pe"], s["q"],
                              s["table_cs"], s["table"], s["start"], s["cu"])
        kvq.kvq_latent_dequantize(s["cfg"], s["pool"], s["table"], s["start"], s["cu"], s["out"])
        return [s["out"], s["q"]]
    call = kvq.kvq_chunk_attention if c["op"] == "chunk" else kvq.kvq_latent_attention
    call(s["cfg"], s["pool"], s["q"], s["table"], s["lens"], s["cu"], s["max_len"], s["scale"], s["out"], s["workspace"])
    return [s["out"]]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"write": _plain_write, "latent_write": _plain_latent_write}.get(op, _plain_attention)(state)


# ---- exact values --------------------------------------------------------------------------------

def _exact_turn(x, pos_of_pair, table, rot, inter):
    """x [rows, heads, n] in fp64, pair i of a row turned by the table's angle of position pos_of_pair[row, i]."""
    half = rot // 2
    pair = torch.arange(half, device=DEV)
    cos, sin = table.double()[pos_of_pair, pair], table.double()[pos_of_pair, half + pair]
    i, j = (2 * pair, 2 * pair + 1) if inter else (pair, pair + half)
    y = x.double().clone()
    y[..., i] = x[..., i].double() * cos[:, None] - x[..., j].double() * sin[:, None]
    y[..., j] = x[..., j].double() * cos[:, None] + x[..., i].double() * sin[:, None]
    return y


def _exact_codes(x, group):
    """What x [.., n] (fp64) stands for once it is held as codes and fp16 scales, in fp64."""
    shape = x.shape
    g = x.reshape(-1, group)
    s = (g.abs().max(dim=1).values.float() / 7).half().double()
    s[s == 0] = 1.0
    return (torch.clamp(torch.round(g / s[:, None]), -7, 7) * s[:, None]).reshape(shape)


def _exact_positions(s):
    """Position of every rotary pair of every row."""
    c, n = s["case"], len(s["row_pos"])
    half = c.get("rot", c.get("R")) // 2
    if s.get("positions") is None:
        return s["row_pos"][:, None].expand(n, half)
    axis = [a for a, w in enumerate(_sections(c)) for _ in range(w)]
    return s["positions"][torch.tensor(axis, device=DEV)][:, :n].T.long()


def _exact_cache(s, b, h, part, width, group, scales):
    """fp64 [positions, width] of one kv head's rows, read byte by byte; group 0: fp16 values."""
    c, P = s["case"], s["case"]["P"]
    heads = c.get("Hkv", 1)
    sizes = _row_bytes(c)
    off = [P * sum(sizes[:i]) for i in range(len(sizes))]
    t = torch.arange(s["total"][b], device=DEV)
    base = ((s["table"][b].long()[t // P] * heads + h) * _block_bytes(c))[:, None]
    dim = torch.arange(width, device=DEV)

    def half_at(p, index):
        at = base + off[p] + (t % P)[:, None] * sizes[p] + 2 * index
        return torch.stack([s["pool"][at], s["pool"][at + 1]], dim=-1).view(torch.float16)[..., 0].double()

    if group == 0:
        return half_at(part, dim)
    byte = s["pool"][base + off[part] + (t % P)[:, None] * sizes[part] + dim // 2].long()
    code = torch.where(dim % 2 == 1, byte // 16, byte % 16) - 8
    return code.double() * half_at(scales, dim // group)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    n = len(s["row_pos"])
    if c["op"] == "write":
        at = _exact_positions(s)
        q = _exact_turn(s["q"][:n], at, s["table_cs"], c["rot"], c["inter"])
        # the cache's definition rounds a turned key to fp16 before its codes are taken
        k = _exact_turn(s["k"][:n], at, s["table_cs"], c["rot"], c["inter"]).half().double()
        return [_behind(q, s["q"]), _behind(_exact_codes(k, c["Gk"]), s["k"]),
                _behind(_exact_codes(s["v"][:n].double(), c["Gv"]), s["v"])]
    if c["op"] == "latent_write":
        at, L = _exact_positions(s), c["L"]
        x = s["rows_in"][:n].double()
        y = x[:, :L]
        if c["norm"]:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / L + EPS) * s["gain"].double()
        rope = _exact_turn(s["rows_in"][:n, None, L:], at, s["table_cs"], c["R"], c["inter"])[:, 0]
        q = s["q"].double()
        q[:n, :, L:] = _exact_turn(s["q_pe"][:n], at, s["table_cs"], c["R"], c["inter"])
        return [_behind(torch.cat([_exact_codes(y, c["G"]), rope], dim=-1), s["out"]), q]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    heads = c.get("Hkv", 1)
    g = s["q"].shape[1] // heads
    for b in range(c["B"]):
        lo, hi = s["cu_list"][b], s["cu_list"][b + 1]
        if lo == hi:
            continue
        for h in range(heads):
            if c["op"] == "chunk":
                K = _exact_cache(s, b, h, 0, c["d"], c["Gk"], 2)
                V = _exact_cache(s, b, h, 1, c["d"], c["Gv"], 3)
            else:
                V = _exact_cache(s, b, h, 0, c["L"], c["G"], 1)
                K = torch.cat([V, _exact_cache(s, b, h, 2, c["R"], 0, 2)], dim=-1)
            step = max(1, (1 << 28) // (g * s["total"][b]))
            for r in range(lo, hi, step):
                to = min(hi, r + step)
                x = s["q"][r:to, h * g:(h + 1) * g].double()
                z = torch.einsum("rgn,tn->rgt", x, K) * s["scale"]
                hidden = torch.arange(s["total"][b], device=DEV)[None, :] > s["row_pos"][r:to, None]
                z.masked_fill_(hidden[:, None, :], -math.inf)
                out[r:to, h * g:(h + 1) * g] = torch.einsum("rgt,tm->rgm", torch.softmax(z, dim=-1), V)
    return [out]
