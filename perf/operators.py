"""The cache operators of a serving step, as cases to measure: the write of new
tokens with their rotary embedding (`write`), the dequantizing read-back of
cached tokens (`read`), and attention of ragged chunks of new tokens over the
paged cache (`attend`).

`run` computes them in a plain form (elementary torch operations in 32 bits,
`own` false) or through the package (`own` true). Both take the state that
`prepare` makes: the paged cache in the package's page layout, block tables,
lengths, and the new tokens.

Definitions
  write   k', q' = bf16(rotary(k)), bf16(rotary(q)) at each token's position,
          from a table of cosines and sines; k' and v quantized per (token, KV
          head) row and stored in the slots' pages; q' returned.
  read    the values that the codes of a run of tokens of each sequence stand
          for, as bf16, packed over the sequences.
  attend  row i of a sequence's n new tokens stands at position p = ctx - n + i
          and attends the tokens t <= p (with a window: p - window < t <= p) of
          the sequence's pages; softmax(scale q.K) V with grouped heads.
"""
import math
import random

import torch

own = False

BS = 16                                    # tokens per page
F8 = {"fp8": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
BITS = {"kivi2": 2, "kivi4": 4}
LLAMA = {"heads": 32, "kv": 8, "dim": 128}   # the 8B-shaped layer of the workloads
LARGE = {"heads": 64, "kv": 8, "dim": 128}   # the 70B-shaped layer
TINY = {"heads": 4, "kv": 2, "dim": 64}      # the tiny workload's layer


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of the 8B-shaped layer: a token for each of 64 sequences (call latency)
        {"name": "write-step-fp8", "kind": "write", "fmt": "fp8", **LLAMA, "batch": 64, "chunk_lo": 1, "chunk_hi": 1,
         "ctx_lo": 1024, "ctx_hi": 8192, "rotary": 128, "interleaved": False, "pad": 0, "lens": 1},
        # a prompt of 8,192 tokens written at once on the 70B-shaped layer
        {"name": "write-prompt-fp8", "kind": "write", "fmt": "fp8", **LARGE, "batch": 1, "chunk_lo": 8192, "chunk_hi": 8192,
         "ctx_lo": 8192, "ctx_hi": 8192, "rotary": 128, "interleaved": False, "pad": 0, "lens": 2},
        # ragged chunks that continue pages, a padded tail, part of each head rotated, pairs side by side,
        # then the new tokens read back as the cache holds them
        {"name": "write-ragged-int8", "kind": "write", "fmt": "int8", "heads": 32, "kv": 8, "dim": 64, "batch": 13, "chunk_lo": 1,
         "chunk_hi": 301, "ctx_lo": 301, "ctx_hi": 1000, "rotary": 32, "interleaved": True, "pad": 7, "lens": 3},
        # the unquantized cache, four prompts of about 1,000 tokens
        {"name": "write-prompts-bf16", "kind": "write", "fmt": "bf16", **LLAMA, "batch": 4, "chunk_lo": 900, "chunk_hi": 1100,
         "ctx_lo": 1100, "ctx_hi": 2048, "rotary": 128, "interleaved": False, "pad": 0, "lens": 4},
        # short prefixes taken out of the cache (call latency)
        {"name": "read-short-fp8", "kind": "read", "fmt": "fp8", **LLAMA, "batch": 16, "ctx_lo": 1, "ctx_hi": 255, "from_start": False, "lens": 5},
        # whole contexts of the 70B-shaped layer read back, to be moved or re-encoded
        {"name": "read-whole-int8", "kind": "read", "fmt": "int8", **LARGE, "batch": 32, "ctx_lo": 3900, "ctx_hi": 4300, "from_start": True, "lens": 6},
        # low-bit groups read back
        {"name": "read-groups-kivi4", "kind": "read", "fmt": "kivi4", **LARGE, "batch": 8, "ctx_lo": 4096, "ctx_hi": 8192, "from_start": False, "lens": 7},
        # continuous batching, decode only: one token for each of 64 sequences
        {"name": "attend-decode-fp8", "kind": "attend", "fmt": "fp8", **LLAMA, "batch": 64, "singles": 64, "chunk_lo": 1, "chunk_hi": 1,
         "ctx_lo": 1024, "ctx_hi": 8192, "window": 0, "out": "bf16", "lens": 8},
        # a prompt in chunks: 2,048 new tokens of two sequences behind a long prefix
        {"name": "attend-chunk-int8", "kind": "attend", "fmt": "int8", **LARGE, "batch": 2, "singles": 0, "chunk_lo": 2048, "chunk_hi": 2048,
         "ctx_lo": 8192, "ctx_hi": 8192, "window": 0, "out": "bf16", "lens": 9},
        # a mixed step: one sequence's prompt chunk beside single tokens of the others
        {"name": "attend-mixed-fp8", "kind": "attend", "fmt": "fp8", **LLAMA, "batch": 16, "singles": 15, "chunk_lo": 400, "chunk_hi": 512,
         "ctx_lo": 513, "ctx_hi": 4096, "window": 0, "out": "bf16", "lens": 10},
        # sliding-window layers over the unquantized cache
        {"name": "attend-window-bf16", "kind": "attend", "fmt": "bf16", **LLAMA, "batch": 4, "singles": 0, "chunk_lo": 777, "chunk_hi": 1024,
         "ctx_lo": 1024, "ctx_hi": 8192, "window": 1024, "out": "bf16", "lens": 11},
        # the tiny workload's layer: a few new tokens on short contexts (call latency), full-precision output
        {"name": "attend-tiny-int8c", "kind": "attend", "fmt": "int8c", **TINY, "batch": 2, "singles": 0, "chunk_lo": 1, "chunk_hi": 9,
         "ctx_lo": 37, "ctx_hi": 129, "window": 0, "out": "f32", "lens": 12},
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["write", "read", "attend"])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    c = {"kind": kind, "fmt": rng.choice(["fp8", "int8", "e5m2", "bf16", "int8c", "int8t"]), "heads": kv * group, "kv": kv, "dim": dim,
         "lens": rng.randrange(1 << 20)}
    if kind == "write":
        tokens = _spread(rng, 1, 8192)
        c["batch"] = _spread(rng, 1, min(tokens, 96))
        c["chunk_hi"] = max(1, tokens // c["batch"])
        c["chunk_lo"] = rng.randint(1, c["chunk_hi"])
        c["ctx_lo"] = c["chunk_hi"] + rng.randint(0, 500)
        c["ctx_hi"] = c["ctx_lo"] + rng.randint(0, 500)
        c["rotary"] = 16 * rng.randint(1, dim // 16)
        c["interleaved"] = rng.random() < 0.4
        c["pad"] = rng.choice([0, 0, 1, 5])
    elif kind == "read":
        if rng.random() < 0.3:
            c["fmt"] = rng.choice(["kivi2", "kivi4"])
        c["batch"] = _spread(rng, 1, 24)
        c["ctx_hi"] = _spread(rng, 1, 4300)
        c["ctx_lo"] = rng.randint(1, c["ctx_hi"])
        c["from_start"] = rng.random() < 0.5
    else:
        c["batch"] = _spread(rng, 1, 32)
        chunk = _spread(rng, 1, 1024)
        c["chunk_lo"] = rng.randint(1, chunk)
        c["chunk_hi"] = chunk
        c["singles"] = rng.randint(0, c["batch"])
        c["ctx_lo"] = chunk + rng.randint(0, 100)
        # the padded scores of the plain form stay below 2^30 values
        most = (1 << 30) // (c["batch"] * c["heads"] * chunk)
        c["ctx_hi"] = max(c["ctx_lo"], min(_spread(rng, 64, 8192), most))
        c["window"] = rng.choice([0, 0, 0, rng.randint(1, 2000)])
        c["out"] = rng.choice(["bf16", "bf16", "f32"])
    return c


def _lens(c):
    """(new tokens or tokens read, context) of each sequence, and where a read begins."""
    r = random.Random(c["lens"])
    rows = []
    for b in range(c["batch"]):
        ctx = r.randint(c["ctx_lo"], c["ctx_hi"])
        if c["kind"] == "read":
            start = 0 if c["from_start"] else r.randint(0, max(0, ctx - 1) // 2)
            if c["fmt"] in BITS:
                ctx = (ctx + 127) // 128 * 128
            rows.append((ctx - start, ctx, start))
        else:
            n = 1 if b < c.get("singles", 0) else r.randint(c["chunk_lo"], c["chunk_hi"])
            rows.append((n, ctx, ctx - n))
    return rows


def _cache_bytes_per_token(c):
    """Bytes of one token and KV head in the cache, K and V, scales included (per-channel
    scales of a group spread over its tokens)."""
    f, d = c["fmt"], c["dim"]
    if f in BITS:
        return 2 * d * BITS[f] / 8 + 4 + 4 * d / 128
    e = 2 if f == "bf16" else 1
    return 2 * d * e + {"fp8": 4, "e5m2": 4, "int8": 8}.get(f, 0)


def work(c):
    rows, hq, hk, d = _lens(c), c["heads"], c["kv"], c["dim"]
    new = sum(n for n, _, _ in rows)
    if c["kind"] == "write":
        total = new + c["pad"]
        # q, k, v read, q' written, the pages written, positions, slots, the angles of each token
        b = total * (2 * hq + 2 * hk) * d * 2 + new * hk * _cache_bytes_per_token(c) + total * (4 + 8 + 4 * c["rotary"])
        if c["fmt"].startswith("int8"):        # and the new tokens read back
            b += new * hk * (_cache_bytes_per_token(c) + 2 * d * 2)
        return {"bytes": b, "flops": 3 * total * (hq + hk) * c["rotary"] + 4 * new * hk * 2 * d}
    if c["kind"] == "read":
        return {"bytes": new * hk * (_cache_bytes_per_token(c) + 2 * d * 2), "flops": 2 * new * hk * 2 * d}
    seen = read = 0
    for n, ctx, start in rows:
        w = c["window"] or ctx
        seen += sum(min(p + 1, w) for p in range(start, ctx))
        read += min(ctx, n + w - 1)
    out = 2 if c["out"] == "bf16" else 4
    return {"bytes": read * hk * _cache_bytes_per_token(c) + new * hq * d * (2 + out), "flops": 4 * hq * d * seen}


# ------------------------------------------------------------------ page layout (plain)
def _k_pages(x, e):
    """[NB][Hk][16][D] -> the K page layout [NB][Hk][2][D e/16][8][16/e]."""
    nb, hk, _, d = x.shape
    return x.reshape(nb, hk, 2, 8, d * e // 16, 16 // e).permute(0, 1, 2, 4, 3, 5).contiguous()


def _v_pages(x, e):
    """[NB][Hk][16][D] -> the V page layout [NB][Hk][e][D][16/e]."""
    nb, hk, _, d = x.shape
    return x.reshape(nb, hk, e, 16 // e, d).permute(0, 1, 2, 4, 3).contiguous()


def _k_logical(p):
    return p.permute(0, 1, 2, 4, 3, 5).reshape(p.shape[0], p.shape[1], BS, -1)


def _v_logical(p):
    return p.permute(0, 1, 2, 4, 3).reshape(p.shape[0], p.shape[1], BS, -1)


def _pack(codes, bits):
    """Units of 16 codes (last axis) -> 2 bits bytes each."""
    m = codes.reshape(*codes.shape[:-1], 4, 4).to(torch.int32)      # [m][j], code 4m + j
    if bits == 2:
        w = m[..., 0, :] | m[..., 1, :] << 2 | m[..., 2, :] << 4 | m[..., 3, :] << 6
    else:
        w = torch.cat([m[..., 0, :] | m[..., 1, :] << 4, m[..., 2, :] | m[..., 3, :] << 4], -1)
    return w.to(torch.uint8)


def _unpack(w, bits):
    w = w.to(torch.int32)
    if bits == 2:
        return torch.cat([w & 3, w >> 2 & 3, w >> 4 & 3, w >> 6], -1)
    return torch.cat([w[..., :4] & 15, w[..., :4] >> 4, w[..., 4:] & 15, w[..., 4:] >> 4], -1)


# ------------------------------------------------------------------ quantization (plain)
def _encode(x, fmt, static):
    """Rows [..., Hk, D] in 32 bits -> (codes, scale): scale [..., Hk] or [..., Hk, 2]."""
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    if fmt in F8:
        t, top = F8[fmt]
        s = (x.abs().amax(-1) / top).to(torch.bfloat16)
        f = s.float()[..., None]
        q = torch.where(f > 0, x / f, torch.zeros_like(x)).clamp(-top, top)
        return q.to(t).view(torch.uint8), s
    if fmt == "int8":
        lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
        s = ((hi - lo) / 255.0).to(torch.bfloat16)
        f = s.float()
        zp = torch.where(f > 0, (-128 - torch.round(lo / f)).clamp(-128, 127), torch.zeros_like(f))
        q = torch.where(f[..., None] > 0, torch.round(x / f[..., None]) + zp[..., None], torch.zeros_like(x)).clamp(-128, 127)
        return q.to(torch.int8).view(torch.uint8), torch.stack([s, zp.to(torch.bfloat16)], -1)
    f = static.float().expand(x.shape[-2:]) if fmt == "int8c" else static.float()
    return torch.round(x / f).clamp(-127, 127).to(torch.int8).view(torch.uint8), None


def _decode(codes, scale, fmt, static):
    """The values that codes [..., Hk, 16, D] with scale [..., Hk, 16(, 2)] stand for, in 32 bits."""
    if fmt == "bf16":
        return codes.float()
    if fmt in F8:
        return codes.view(F8[fmt][0]).float() * scale.float()[..., None]
    x = codes.view(torch.int8).float()
    if fmt == "int8":
        return (x - scale[..., 1].float()[..., None]) * scale[..., 0].float()[..., None]
    return x * (static.float()[:, None, :] if fmt == "int8c" else static.float())


# ------------------------------------------------------------------ inputs
def _values(g, c, blocks, which):
    """[blocks][Hk][16][D] bf16 values as a projection gives them: unit spread, a few large K
    channels (the 8-bit floats' workload), a mean away from zero (the integers')."""
    x = torch.randn(blocks, c["kv"], BS, c["dim"], device="cuda", generator=g)
    if which == "k" and c["fmt"] in ("fp8", "e5m2", "bf16"):
        x[..., ::31] *= 6.0
    if c["fmt"].startswith("int8"):
        x += 0.3
    return x.to(torch.bfloat16)


def _fill(g, c, nb, which, static):
    """Pages of one cache array, and its scales, filled block range by block range."""
    fmt, hk, d = c["fmt"], c["kv"], c["dim"]
    pages = scales = None
    if fmt in BITS:
        return _fill_groups(g, c, nb, which)
    e = 2 if fmt == "bf16" else 1
    for a in range(0, nb, 8192):
        z = min(nb, a + 8192)
        codes, s = _encode(_values(g, c, z - a, which).transpose(1, 2).float(), fmt, static)
        codes = codes.transpose(1, 2)
        p = (_k_pages if which == "k" else _v_pages)(codes, e)
        if pages is None:
            pages = p.new_empty(nb, *p.shape[1:])
            scales = None if s is None else s.new_empty(nb, hk, BS, *s.shape[3:])
        pages[a:z] = p
        if s is not None:
            scales[a:z] = s.transpose(1, 2)
    return pages, scales


def _fill_groups(g, c, nb, which):
    """Low-bit pages: blocks 8i .. 8i+7 in storage order make up one group here, and the block
    tables keep them together; K has a (step, minimum) per channel of the group, V per token."""
    bits, hk, d = BITS[c["fmt"]], c["kv"], c["dim"]
    top = float(2 ** bits - 1)
    x = _values(g, c, nb, which).float()                                   # [NB][Hk][16][D]
    if which == "k":
        y = x.reshape(nb // 8, 8, hk, BS, d).permute(0, 2, 1, 3, 4).reshape(nb // 8, hk, 128, d)
        lo, hi = y.amin(2), y.amax(2)                                      # [groups][Hk][D]
        s, z = ((hi - lo) / top).to(torch.bfloat16), lo.to(torch.bfloat16)
        q = torch.round((y - z.float()[:, :, None]) / s.float()[:, :, None]).clamp(0, top)
        q = q.reshape(nb // 8, hk, 8, BS, d).permute(0, 2, 1, 3, 4).reshape(nb, hk, BS, d)
        meta = torch.zeros(nb // 8, 8, hk, BS, 2, dtype=torch.bfloat16, device="cuda")
        meta[:, :, :, : d // 8, 0] = s.reshape(nb // 8, hk, 8, d // 8).transpose(1, 2)
        meta[:, :, :, : d // 8, 1] = z.reshape(nb // 8, hk, 8, d // 8).transpose(1, 2)
        return _pack(_k_pages(q, 1), bits).reshape(nb, hk, -1), meta.reshape(nb, hk, BS, 2)
    lo, hi = x.amin(-1), x.amax(-1)
    s, z = ((hi - lo) / top).to(torch.bfloat16), lo.to(torch.bfloat16)
    q = torch.round((x - z.float()[..., None]) / s.float()[..., None]).clamp(0, top)
    return _pack(_v_pages(q, 1)[:, :, 0], bits).reshape(nb, hk, -1), torch.stack([s, z], -1)


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows, hk, hq, d, fmt = _lens(c), c["kv"], c["heads"], c["dim"], c["fmt"]
    batch = len(rows)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pages = [(ctx + BS - 1) // BS for _, ctx, _ in rows]
    unit = 8 if fmt in BITS else 1                                     # blocks that stay together
    groups = sum(-(-p // unit) for p in pages)
    nb = (groups + max(2, groups // 8)) * unit
    order = torch.randperm(nb // unit, device="cuda", generator=g)[:, None] * unit + torch.arange(unit, device="cuda")
    order = order.reshape(-1).to(torch.int32)
    width = max(pages)
    tables, at = torch.zeros(batch, width, dtype=torch.int32, device="cuda"), 0
    for b, p in enumerate(pages):
        tables[b, :p] = order[at:at + p]
        at += -(-p // unit) * unit
    s = {"case": c, "tables": tables, "nb": nb, "width": width, "ctx": i32([x for _, x, _ in rows]), "starts": i32([x for _, _, x in rows]),
         "max_ctx": max(x for _, x, _ in rows), "max_n": max(n for n, _, _ in rows)}
    cum = [0]
    for n, _, _ in rows:
        cum.append(cum[-1] + n)
    total = cum[-1]
    s["cu"], s["total"] = i32(cum), total
    n_of = torch.tensor([n for n, _, _ in rows], device="cuda")
    s["seq_of"] = torch.repeat_interleave(torch.arange(batch, device="cuda"), n_of)      # the plan of the plain form
    s["row_of"] = torch.arange(total, device="cuda") - s["cu"].long()[s["seq_of"]]
    s["pos"] = s["starts"].long()[s["seq_of"]] + s["row_of"]
    static = None
    if fmt == "int8c":
        static = [((torch.rand(hk, d, device="cuda", generator=g) + 0.5) * 4 / 127).to(torch.bfloat16) for _ in range(2)]
    elif fmt == "int8t":
        static = [((torch.rand(1, device="cuda", generator=g) + 0.5) * 4 / 127).to(torch.bfloat16) for _ in range(2)]
    s["static"] = static or [None, None]
    if c["kind"] == "write":
        e = 2 if fmt == "bf16" else 1
        dt = torch.bfloat16 if fmt == "bf16" else torch.uint8
        s["k"] = torch.zeros(nb, hk, 2, d * e // 16, 8, 16 // e, dtype=dt, device="cuda")
        s["v"] = torch.zeros(nb, hk, e, d, 16 // e, dtype=dt, device="cuda")
        shape = {"fp8": (nb, hk, BS), "e5m2": (nb, hk, BS), "int8": (nb, hk, BS, 2)}.get(fmt)
        s["ks"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda") if shape else s["static"][0]
        s["vs"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda") if shape else s["static"][1]
        t = total + c["pad"]
        x = torch.randn(t, hq + 2 * hk, d, device="cuda", generator=g)
        if fmt.startswith("int8"):
            x[:, hq:] += 0.3
        x = x.to(torch.bfloat16)                                       # one fused projection: q, k, v beside one another
        s["q"], s["kn"], s["vn"] = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        s["positions"] = torch.zeros(t, dtype=torch.int32, device="cuda")
        s["positions"][:total] = s["pos"]
        s["slots"] = torch.full((t,), -1, dtype=torch.int64, device="cuda")
        s["slots"][:total] = s["tables"][s["seq_of"], s["pos"] // BS].long() * BS + s["pos"] % BS
        half = c["rotary"] // 2
        angle = torch.arange(s["max_ctx"], dtype=torch.float64, device="cuda")[:, None] * 500000.0 ** (
            -torch.arange(half, dtype=torch.float64, device="cuda") / half)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        return s
    s["k"], s["ks"] = _fill(g, c, nb, "k", s["static"][0])
    s["v"], s["vs"] = _fill(g, c, nb, "v", s["static"][1])
    if fmt in ("int8c", "int8t"):
        s["ks"], s["vs"] = s["static"]
    if c["kind"] == "attend":
        s["q"] = torch.randn(total, hq, d, device="cuda", generator=g).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, cos, sin, rotary, interleaved):
    """bf16 rows [T][H][D]; cos, sin [T][rotary/2]; 32-bit products, rounded to bf16."""
    y = x.float()
    a, b = (y[..., 0:rotary:2], y[..., 1:rotary:2]) if interleaved else (y[..., : rotary // 2], y[..., rotary // 2:rotary])
    c, s = cos[:, None], sin[:, None]
    p, q = a * c - b * s, b * c + a * s
    r = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    return torch.cat([r, y[..., rotary:]], -1).to(torch.bfloat16)


def _write_plain(s):
    c, n = s["case"], s["total"]
    fmt, hk, d, half = c["fmt"], c["kv"], c["dim"], c["rotary"] // 2
    cs = s["cos_sin"][s["positions"].long()]
    q = _rotate(s["q"], cs[:, :half], cs[:, half:], c["rotary"], c["interleaved"])
    k = _rotate(s["kn"], cs[:, :half], cs[:, half:], c["rotary"], c["interleaved"])[:n]
    e = 2 if fmt == "bf16" else 1
    blk, t = s["slots"][:n] // BS, s["slots"][:n] % BS
    kc, ks = _encode(k.float(), fmt, s["static"][0])
    vc, vs = _encode(s["vn"][:n].float(), fmt, s["static"][1])
    s["k"][blk, :, t // 8, :, t % 8, :] = kc.reshape(n, hk, d * e // 16, 16 // e)
    s["v"][blk, :, t // (16 // e), :, t % (16 // e)] = vc
    if ks is not None:
        s["ks"][blk, :, t] = ks
        s["vs"][blk, :, t] = vs
    if fmt.startswith("int8"):
        return q, *_read_plain(s)
    return q


def _gathered(s, which, pages):
    """Values [.., Hk][16][D] in 32 bits of the blocks `pages` (an index of any shape)."""
    c = s["case"]
    fmt = c["fmt"]
    p, m = s[which][pages.reshape(-1)], s[which + "s"]
    if fmt in BITS:
        b = BITS[fmt]
        m = m[pages.reshape(-1)].float()
        n, hk, d = p.shape[0], c["kv"], c["dim"]
        if which == "k":
            x = _k_logical(_unpack(p.reshape(n, hk, 2, d // 16, 8, 2 * b), b)).float()
            return x, m
        x = _v_logical(_unpack(p.reshape(n, hk, 1, d, 2 * b), b)).float()
        return x * m[..., 0, None] + m[..., 1, None]
    codes = _k_logical(p) if which == "k" else _v_logical(p)
    static = s["static"][0 if which == "k" else 1]
    return _decode(codes.contiguous(), m[pages.reshape(-1)] if static is None and m is not None else None, fmt, static)


def _read_plain(s):
    c = s["case"]
    hk, d = c["kv"], c["dim"]
    page = s["pos"] // BS
    b, w = s["tables"].shape
    out = []
    for which in ("k", "v"):
        x = _gathered(s, which, s["tables"])
        if which == "k" and c["fmt"] in BITS:
            x, m = x
            wide = -(-w // 8) * 8                                       # whole groups of table entries
            m = torch.cat([m.reshape(b, w, hk, BS, 2), m.new_zeros(b, wide - w, hk, BS, 2)], 1)
            m = m.reshape(b, wide // 8, 8, hk, BS, 2)[..., : d // 8, :]
            m = m.permute(0, 1, 3, 2, 4, 5).reshape(b, wide // 8, 1, hk, 1, d, 2).expand(b, wide // 8, 8, hk, 1, d, 2)
            m = m.reshape(b, wide, hk, 1, d, 2)[:, :w]
            x = x.reshape(b, w, hk, BS, d) * m[..., 0] + m[..., 1]
        x = x.reshape(b, w, hk, BS, d)
        out.append(x[s["seq_of"], page, :, s["pos"] % BS].to(torch.bfloat16))
    return tuple(out)


def _attend_plain(s):
    c = s["case"]
    hk, d, hq = c["kv"], c["dim"], c["heads"]
    g, n, b, w = hq // hk, s["max_n"], s["tables"].shape[0], s["width"]
    kv = [_gathered(s, x, s["tables"]).reshape(b, w, hk, BS, d).transpose(1, 2).reshape(b, hk, w * BS, d) for x in ("k", "v")]
    rows = (s["cu"][:-1].long()[:, None] + torch.arange(n, device="cuda")).clamp(max=s["total"] - 1)
    q = s["q"][rows].float().reshape(b, n, hk, g, d).permute(0, 2, 3, 1, 4).reshape(b, hk, g * n, d)
    x = (q @ kv[0].transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(b, hk, g, n, w * BS)
    p = (s["starts"].long()[:, None] + torch.arange(n, device="cuda"))[:, None, None, :, None]
    t = torch.arange(w * BS, device="cuda")
    hidden = t > p
    if c["window"]:
        hidden = hidden | (t <= p - c["window"])
    hidden = hidden | (t >= s["ctx"].long()[:, None, None, None, None])
    x.masked_fill_(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    l = x.sum(-1, keepdim=True)
    o = (x.view(b, hk, g * n, w * BS) @ kv[1]).view(b, hk, g, n, d)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)[s["seq_of"], s["row_of"]]
    return o.to(torch.bfloat16) if c["out"] == "bf16" else o


# ------------------------------------------------------------------ the package's calls
def _own(s):
    from int8_quantized_paged_quantize_b200 import kvq
    c = s["case"]
    fmt = c["fmt"]
    if "cache" not in s:
        d = kvq.dims(s["nb"], c["kv"], c["heads"], c["dim"], s["width"])
        s["cache"] = (kvq.KiviCache(fmt, d, s["k"], s["v"], s["ks"], s["vs"], None) if fmt in BITS
                      else kvq.LayerCache(fmt, d, s["k"], s["v"], s["ks"], s["vs"]))
    cache = s["cache"]
    if c["kind"] == "write":
        q = cache.append_rope(s["q"], s["kn"], s["vn"], s["positions"], s["cos_sin"], s["slots"], interleaved=c["interleaved"])
        if fmt.startswith("int8"):
            return q, *cache.read(s["tables"], s["starts"], s["cu"], s["total"])
        return q
    if c["kind"] == "read":
        return cache.read(s["tables"], s["starts"], s["cu"], s["total"])
    if "ws" not in s:
        s["ws"] = cache.ragged_workspace(s["total"])
    return cache.ragged(s["q"], s["cu"], s["tables"], s["ctx"], s["max_ctx"], window=c["window"], workspace=s["ws"],
                        out_dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)


def run(s):
    c = s["case"]
    if own:
        got = _own(s)
    else:
        got = {"write": _write_plain, "read": _read_plain, "attend": _attend_plain}[c["kind"]](s)
    if c["kind"] == "write" and c["fmt"] == "bf16":
        return got, s["k"], s["v"]                 # the cache itself is what the write leaves behind
    if c["kind"] == "write" and c["fmt"] in F8:    # its codes as the numbers they are
        return got, s["k"].view(F8[c["fmt"]][0]), s["v"].view(F8[c["fmt"]][0]), s["ks"], s["vs"]
    return got


# ------------------------------------------------------------------ 64 bits
def _round_to(x, dtype):
    """64-bit values rounded once to `dtype` (by its spacing at each value, ties to even)."""
    f = torch.finfo(dtype)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=f.smallest_normal)))) * f.eps
    return torch.where(torch.isfinite(x), torch.round(x / step) * step, x).clamp(f.min, f.max)


def _exact_rows(x, fmt, static):
    """64-bit rows [T][Hk][D] -> (code values, scale, zero point, values)."""
    if fmt == "bf16":
        return x, None, None, x
    if fmt in F8:
        t, top = F8[fmt]
        s = _round_to(x.abs().amax(-1) / top, torch.bfloat16)
        code = _round_to((x / s[..., None]).nan_to_num(0.0).clamp(-top, top), t)
        return code, s, None, code * s[..., None]
    if fmt == "int8":
        lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
        s = _round_to((hi - lo) / 255, torch.bfloat16)
        z = (-128 - torch.round(lo / s)).clamp(-128, 127)
        code = (torch.round(x / s[..., None]) + z[..., None]).clamp(-128, 127)
        return code, s, z, (code - z[..., None]) * s[..., None]
    f = static.double()
    code = torch.round(x / f).clamp(-127, 127)
    return code, None, None, code * f


def _exact_write(s):
    c, n = s["case"], s["total"]
    fmt, rot = c["fmt"], c["rotary"]
    cs = s["cos_sin"].double()[s["positions"].long()]
    out = []
    for x in (s["q"], s["kn"]):
        y = x.double()
        z = y.clone()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
            co, si = cs[:, None, i], cs[:, None, rot // 2 + i]
            z[..., a] = y[..., a] * co - y[..., b] * si
            z[..., b] = y[..., b] * co + y[..., a] * si
        out.append(z)
    q, k, v = out[0], _round_to(out[1][:n], torch.bfloat16), s["vn"][:n].double()
    kq, vq = _exact_rows(k, fmt, s["static"][0]), _exact_rows(v, fmt, s["static"][1])
    if fmt.startswith("int8"):
        return q, kq[3], vq[3]
    e = 2 if fmt == "bf16" else 1
    got = [q]
    slot = s["slots"][:n]
    for which, x in (("k", kq[0]), ("v", vq[0])):
        flat = torch.zeros(s["nb"] * BS, c["kv"], c["dim"], dtype=torch.float64, device="cuda")
        flat[slot] = x
        pages = flat.view(s["nb"], BS, c["kv"], c["dim"]).transpose(1, 2)
        got.append((_k_pages if which == "k" else _v_pages)(pages, e))
    if fmt in F8:
        for x in (kq[1], vq[1]):
            flat = torch.zeros(s["nb"] * BS, c["kv"], dtype=torch.float64, device="cuda")
            flat[slot] = x
            got.append(flat.view(s["nb"], BS, c["kv"]).transpose(1, 2).contiguous())
    return tuple(got)


def _exact_values(s, b, which, a, z):
    """64-bit K or V [z - a][Hk][D] of tokens a .. z-1 of sequence b, token by token of the page layout."""
    c = s["case"]
    fmt, hk, d = c["fmt"], c["kv"], c["dim"]
    t = torch.arange(a, z, device="cuda")
    blk, o = s["tables"][b].long()[t // BS], t % BS
    if fmt in BITS:
        bits = BITS[fmt]
        p = s[which][blk].reshape(z - a, hk, -1, 2 * bits).to(torch.int64)            # units
        i, ch = torch.arange(z - a, device="cuda")[:, None], torch.arange(d, device="cuda")[None]
        if which == "k":
            unit, e = ((o[:, None] // 8) * (d // 16) + ch // 16) * 8 + o[:, None] % 8, ch % 16 + 0 * i
        else:
            unit, e = ch + 0 * i, o[:, None] + 0 * ch
        mm, j = e // 4, e % 4
        byte, shift = (j, 2 * mm) if bits == 2 else (4 * (mm // 2) + j, 4 * (mm % 2))
        code = (p[i, :, unit, byte] >> shift[..., None]) & (2 ** bits - 1)             # [T][D][Hk]
        code = code.transpose(1, 2).double()
        m = s[which + "s"].double()
        if which == "v":
            m = m[blk, :, o]                                                           # [T][Hk][2]
            return code * m[..., 0, None] + m[..., 1, None]
        home = s["tables"][b].long()[(t // 128)[:, None] * 8 + ch // (d // 8)]         # [T][D]
        m = m[home, :, ch % (d // 8) + 0 * home].transpose(1, 2)                       # [T][Hk][D][2]
        return code * m[..., 0] + m[..., 1]
    page = s[which][blk]
    if which == "k":
        x = page[torch.arange(z - a, device="cuda"), :, o // 8, :, o % 8].reshape(z - a, hk, d)
    else:
        per = page.shape[-1]
        x = page[torch.arange(z - a, device="cuda"), :, o // per, :, o % per]
    x = x.contiguous()
    if fmt == "bf16":
        return x.double()
    static = s["static"][0 if which == "k" else 1]
    if fmt in F8:
        return x.view(F8[fmt][0]).double() * s[which + "s"][blk, :, o].double()[..., None]
    x = x.view(torch.int8).double()
    if fmt == "int8":
        m = s[which + "s"][blk, :, o].double()
        return (x - m[..., 1, None]) * m[..., 0, None]
    return x * static.double()


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "write":
        return _exact_write(s)
    rows = _lens(c)
    if c["kind"] == "read":
        return tuple(torch.cat([_exact_values(s, b, w, start, ctx) for b, (_, ctx, start) in enumerate(rows)]) for w in ("k", "v"))
    g, out, at = c["heads"] // c["kv"], [], 0
    for b, (n, ctx, start) in enumerate(rows):
        a = max(0, start - c["window"] + 1) if c["window"] else 0
        k, v = _exact_values(s, b, "k", a, ctx), _exact_values(s, b, "v", a, ctx)
        p, t = torch.arange(start, ctx, device="cuda")[:, None], torch.arange(a, ctx, device="cuda")
        seen = (t <= p) & (t > p - c["window"]) if c["window"] else t <= p
        o = torch.empty(n, c["heads"], c["dim"], dtype=torch.float64, device="cuda")
        for h in range(c["heads"]):
            x = (s["q"][at:at + n, h].double() @ k[:, h // g].T) / math.sqrt(c["dim"])
            o[:, h] = torch.softmax(x.masked_fill(~seen, -math.inf), -1) @ v[:, h // g]
        out.append(o)
        at += n
    return torch.cat(out)
