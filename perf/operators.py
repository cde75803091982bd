"""Cases of the latent-cache and block-selection operators, with their plain forms.

Operators: the latent prologue (norm, rotary embedding, quantised append) with
the read-back of what it wrote; the read of a cache by range or by index;
sparse latent attention over a 4-bit cache; block keys; latent attention over
selected blocks.  Layouts are those of include/dsa.h:

  FP8 row  [dc e4m3 | dc/128 fp32 scales | dr bf16]
  Q4 row   [dc/2 code bytes | dr bf16 | dc/32 bf16 scales | zeros to 16 bytes]
           value 2i of a word's eight in nibble i, value 2i+1 in nibble i + 4,
           code 8 + rint(x / s), s = bf16(max(amax, 1e-4) / 7) per 32 values
"""
import math

import torch

if torch.cuda.is_available():
    DEV = "cuda"
else:
    DEV = "cpu"

own = False

BF16, FP8, Q4 = "bf16", "fp8", "q4"
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ row layouts
def row_bytes(fmt, dc, dr):
    if fmt == BF16:
        return 2 * (dc + dr)
    if fmt == FP8:
        return dc + dc // 32 + 2 * dr
    return (dc // 2 + 2 * dr + dc // 16 + 15) // 16 * 16


def bytes_of(x):
    """The bytes of a contiguous tensor, its last dimension spread out."""
    return x.contiguous().view(torch.uint8)


NIBBLE = (0, 4, 1, 5, 2, 6, 3, 7)      # value e of a word sits in nibble NIBBLE[e]


def pack_rows(x, fmt, dc):
    """x [..., dc + dr] (any float type) as cache rows of the format."""
    if fmt == BF16:
        return x.to(torch.bfloat16)
    dr = x.shape[-1] - dc
    lead = x.shape[:-1]
    pe = bytes_of(x[..., dc:].to(torch.bfloat16))
    c = x[..., :dc]
    if fmt == FP8:
        g = c.unflatten(-1, (dc // 128, 128))
        s = (g.abs().amax(-1).clamp_min(1e-4).float() / 448.0)
        codes = (g.float() / s[..., None]).clamp(-448, 448).to(E4M3).flatten(-2)
        return torch.cat((codes.view(torch.uint8), bytes_of(s), pe), -1)
    g = c.unflatten(-1, (dc // 32, 32))
    s = (g.abs().amax(-1).clamp_min(1e-4) / 7.0).to(torch.bfloat16)
    # the quotient in 64 bits: a value next to a border between two codes
    code = (torch.round(g.double() / s[..., None].double()).clamp(-7, 7) + 8).to(torch.int64)
    shift = 4 * torch.tensor(NIBBLE, device=x.device)
    word = (code.reshape(*lead, dc // 8, 8) << shift).sum(-1)
    # a word of 32 bits in int64, as four bytes
    octet = (word[..., None] >> torch.tensor((0, 8, 16, 24), device=x.device)) & 255
    octet = octet.flatten(-2).to(torch.uint8)
    pad = row_bytes(Q4, dc, dr) - (dc // 2 + 2 * dr + dc // 16)
    zeros = torch.zeros(*lead, pad, dtype=torch.uint8, device=x.device)
    return torch.cat((octet, pe, bytes_of(s), zeros), -1)


def unpack_rows(rows, fmt, dc, dr):
    """The values that cache rows stand for, each rounded to bf16 (as fp32)."""
    if fmt == BF16:
        return rows.float()
    if fmt == FP8:
        codes = rows[..., :dc].contiguous().view(E4M3).float()
        s = rows[..., dc:dc + dc // 32].contiguous().view(torch.float32)
        pe = rows[..., dc + dc // 32:].contiguous().view(torch.bfloat16)
        c = (codes.unflatten(-1, (dc // 128, 128)) * s[..., None]).flatten(-2)
    else:
        octet = rows[..., :dc // 2].unflatten(-1, (dc // 8, 4))
        nib = torch.stack((octet & 15, octet >> 4), -1).flatten(-2)     # nibbles 0..7 of a word
        code = nib[..., list(NIBBLE)].flatten(-2).float() - 8.0
        pe = rows[..., dc // 2:dc // 2 + 2 * dr].contiguous().view(torch.bfloat16)
        at = dc // 2 + 2 * dr
        s = rows[..., at:at + dc // 16].contiguous().view(torch.bfloat16).float()
        c = (code.unflatten(-1, (dc // 32, 32)) * s[..., None]).flatten(-2)
    return torch.cat((c.to(torch.bfloat16), pe), -1).float()


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 32 sequences: each writes its new row into the 4-bit
        # cache and takes back the values the cache now stands for
        dict(name="append-q4-B32", op="append", fmt=Q4, B=32, S=1, t_max=4096, start=4095,
             dc=512, dr=64, x="bf16", norm=True, rope=1),
        # an odd chunk from an fp32 projection into the FP8 cache, no norm, halves rotary
        dict(name="append-fp8-S1777", op="append", fmt=FP8, B=3, S=1777, t_max=2000, start=123,
             dc=512, dr=64, x="f32", norm=False, rope=2),
        # a batch of whole prompts into the 4-bit cache (prefill of 8192 tokens)
        dict(name="append-q4-S8192", op="append", fmt=Q4, B=8, S=8192, t_max=8192, start=0,
             dc=512, dr=64, x="bf16", norm=True, rope=1),
        # a prefill chunk takes back a whole 128K context to up-project it
        dict(name="read-q4-131072", op="read", fmt=Q4, B=1, t_max=131072, start=0, n=131072,
             gather=False, dc=512, dr=64, out="bf16"),
        # selected rows of FP8 caches as fp32, an unfilled slot here and there
        dict(name="read-fp8-rows", op="read", fmt=FP8, B=8, t_max=32768, start=0, n=2048,
             gather=True, dc=512, dr=64, out="f32"),
        # one sequence's decode step: the smallest attention
        dict(name="attn-q4-B1", op="attn", fmt=Q4, B=1, S=1, t_max=4096, start=4095, k=2048,
             Hq=128, dc=512, dr=64),
        # the long-context decode batch
        dict(name="attn-q4-B8", op="attn", fmt=Q4, B=8, S=1, t_max=131072, start=131071, k=2048,
             Hq=128, dc=512, dr=64),
        # a prefill chunk against a cached prompt, each query with its own selection
        dict(name="attn-q4-S1024", op="attn", fmt=Q4, B=1, S=1024, t_max=8192, start=7168, k=2048,
             Hq=128, dc=512, dr=64),
        # one new token per sequence finishes a block in each cache
        dict(name="keys-B32", op="keys", B=32, S=1, t_max=32768, start=32767, D=128, block=64),
        # the block keys of cached 128K contexts, built once
        dict(name="keys-131072", op="keys", B=8, S=131072, t_max=131072, start=0, D=128, block=64),
        # decode over 32 selected blocks of a 4-bit cache, the heads of one of eight ranks
        dict(name="blocks-q4-B32", op="blocks", fmt=Q4, B=32, S=1, t_max=32768, start=32740, kb=32,
             block=64, Hq=16, dc=512, dr=64),
        # a prefill chunk over selected blocks of a bf16 cache
        dict(name="blocks-bf16-S512", op="blocks", fmt=BF16, B=1, S=512, t_max=8192, start=7600,
             kb=16, block=128, Hq=128, dc=512, dr=64),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "read", "attn", "attn", "keys", "blocks", "blocks"))
    fmt = rng.choice((Q4, Q4, FP8, BF16))
    dc, dr = rng.choice(((512, 64), (512, 64), (512, 64), (256, 32), (128, 8), (384, 40)))
    if op == "append":
        B = spread(rng, 1, 64)
        S = spread(rng, 1, 65536 // B)
        start = rng.randrange(0, 500)
        return dict(op=op, fmt=fmt, B=B, S=S, t_max=start + S + rng.randrange(0, 300), start=start,
                    dc=dc, dr=dr, x=rng.choice(("bf16", "f32")), norm=rng.random() < 0.7,
                    rope=rng.randrange(0, 3))
    if op == "read":
        B = spread(rng, 1, 64)
        n = spread(rng, 1, 131072 // B)
        start = rng.randrange(0, 500)
        return dict(op=op, fmt=fmt, B=B, t_max=start + n + rng.randrange(0, 300), start=start, n=n,
                    gather=rng.random() < 0.5, dc=dc, dr=dr, out=rng.choice(("bf16", "f32")))
    if op == "keys":
        B = spread(rng, 1, 64)
        S = spread(rng, 1, 1048576 // B)
        block = rng.choice((4, 16, 32, 64, 128, 50))
        # the new tokens finish at least one block
        start = rng.randrange(0, 500) if S >= block else block * rng.randrange(8, 16) - S
        return dict(op=op, B=B, S=S, t_max=start + S + rng.randrange(0, 300), start=start,
                    D=rng.choice((128, 128, 64)), block=block)
    rows = spread(rng, 1, 512)                    # query rows: B of one token or one chunk
    B, S = (rows, 1) if rng.random() < 0.6 else (1, rows)
    ctx = spread(rng, 64, min(131072, 524288 // B))
    start = rng.randrange(0, ctx)
    t_max = start + S + rng.randrange(0, 100)
    Hq = rng.choice((1, 8, 16, 24, 32, 64, 80, 128, 128))
    if op == "attn":
        return dict(op=op, fmt=Q4, B=B, S=S, t_max=t_max, start=start, k=spread(rng, 1, 2048),
                    Hq=Hq, dc=dc, dr=dr)
    block = rng.choice((16, 32, 64, 128, 50))
    return dict(op=op, fmt=fmt, B=B, S=S, t_max=t_max, start=start,
                kb=spread(rng, 1, 2048 // block), block=block, Hq=Hq, dc=dc, dr=dr)


# --------------------------------------------------------------------- inputs
def picks(g, rows, n, avail):
    """rows x n distinct ids below avail[row], in ascending order and -1 behind
    them, as the top-k lists them."""
    most = int(avail.max())
    key = torch.rand(rows, max(most, 1), generator=g, device=DEV)
    at = torch.arange(max(most, 1), device=DEV)
    key = torch.where(at < avail[:, None], key, torch.full_like(key, 2.0))
    m = min(n, key.shape[1])
    val, ids = key.topk(m, dim=1, largest=False)
    ids = torch.where(val < 1.5, ids, torch.full_like(ids, most + 1)).sort(dim=1).values
    ids = torch.where(ids > most, torch.full_like(ids, -1), ids)
    out = torch.full((rows, n), -1, dtype=torch.int32, device=DEV)
    out[:, :m] = ids.int()
    return out


def make_cache(g, c):
    """A cache [B, t_max, row] of ~N(0, 1) latents, packed some rows at a time."""
    w = row_bytes(c["fmt"], c["dc"], c["dr"])
    B, t, d = c["B"], c["t_max"], c["dc"] + c["dr"]
    if c["fmt"] == BF16:
        cache = torch.empty(B * t, d, dtype=torch.bfloat16, device=DEV)
    else:
        cache = torch.empty(B * t, w, dtype=torch.uint8, device=DEV)
    for r in range(0, B * t, 65536):
        n = min(65536, B * t - r)
        cache[r:r + n] = pack_rows(torch.randn(n, d, generator=g, device=DEV), c["fmt"], c["dc"])
    return cache.view(B, t, -1)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = dict(case)
    op = c["op"]
    if op == "keys":
        keys = torch.randn(c["B"], c["t_max"], c["D"], generator=g, device=DEV)
        c["k_scale"] = keys.abs().amax(-1).clamp_min(1e-4) / 448.0
        c["k_cache"] = (keys / c["k_scale"][..., None]).to(E4M3).view(torch.uint8)
        n = (c["start"] + c["S"]) // c["block"]
        c["blk_cache"] = torch.zeros(c["B"], max(n, 1), c["D"], dtype=torch.uint8, device=DEV)
        c["blk_scale"] = torch.zeros(c["B"], max(n, 1), device=DEV)
        return c
    d = c["dc"] + c["dr"]
    if op == "append":
        xt = torch.bfloat16 if c["x"] == "bf16" else torch.float32
        c["kv"] = torch.randn(c["B"], c["S"], d, generator=g, device=DEV).to(xt)
        c["w"] = 1 + 0.1 * torch.randn(c["dc"], generator=g, device=DEV) if c["norm"] else None
        c["cs"] = None
        if c["rope"]:
            pos = torch.arange(c["start"], c["start"] + c["S"], device=DEV, dtype=torch.float64)
            j = torch.arange(c["dr"] // 2, device=DEV, dtype=torch.float64)
            a = pos[:, None] * 10000.0 ** (-2 * j / c["dr"])
            c["cs"] = torch.stack((a.cos(), a.sin()), -1).float().contiguous()
        shape = (c["B"], c["t_max"], row_bytes(c["fmt"], c["dc"], c["dr"]))
        c["cache"] = torch.zeros(shape, dtype=torch.uint8, device=DEV)
        if c["fmt"] == BF16:
            c["cache"] = c["cache"].view(torch.bfloat16)
        c["out"] = torch.empty(c["B"], c["S"], d, dtype=torch.bfloat16, device=DEV)
        return c
    c["cache"] = make_cache(g, c)
    if op == "read":
        c["idx"] = None
        if c["gather"]:
            n = c["B"] * c["n"]
            at = torch.randint(0, c["t_max"], (n,), generator=g, device=DEV)
            hole = torch.rand(n, generator=g, device=DEV) < 0.02
            c["idx"] = torch.where(hole, -1, at).int().view(c["B"], c["n"])
        ot = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        c["rows"] = torch.empty(c["B"], c["n"], d, dtype=ot, device=DEV)
        return c
    B, S = c["B"], c["S"]
    c["q"] = torch.randn(B, S, c["Hq"], d, generator=g, device=DEV).to(torch.bfloat16)
    seen = (c["start"] + 1 + torch.arange(S, device=DEV)).repeat(B)
    if op == "attn":
        c["idx"] = picks(g, B * S, c["k"], seen).view(B, S, c["k"])
    else:
        c["idx"] = picks(g, B * S, c["kb"], seen // c["block"]).view(B, S, c["kb"])
    c["scale"] = d ** -0.5
    c["out"] = torch.empty(B, S, c["Hq"], c["dc"], dtype=torch.bfloat16, device=DEV)
    c["lse"] = torch.empty(B, S, c["Hq"], device=DEV)
    # room for the split partials of either attention (a program keeps one workspace)
    c["ws"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    return c


# ---------------------------------------------------------------- plain forms
def rotate(x, cs, rope):
    """Rotary embedding of x [..., S, dr] by cs [S, dr/2, 2]: 1 = interleaved pairs."""
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if rope == 1 else (x[..., :half], x[..., half:])
    cos, sin = cs[..., 0], cs[..., 1]
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack((u, v), -1).flatten(-2) if rope == 1 else torch.cat((u, v), -1)


def plain_append(c):
    # in 64 bits: values next to a border between two codes
    dc, x = c["dc"], c["kv"].double()
    lat, pe = x[..., :dc], x[..., dc:]
    if c["norm"]:
        lat = lat * torch.rsqrt(lat.square().mean(-1, keepdim=True) + 1e-6) * c["w"].double()
    if c["rope"]:
        pe = rotate(pe, c["cs"].double(), c["rope"])
    rows = pack_rows(torch.cat((lat, pe), -1), c["fmt"], dc)
    at = slice(c["start"], c["start"] + c["S"])
    c["cache"][:, at] = rows
    return unpack_rows(c["cache"][:, at], c["fmt"], dc, c["dr"]).to(torch.bfloat16)


def plain_read(c):
    if c["idx"] is None:
        rows = c["cache"][:, c["start"]:c["start"] + c["n"]]
        got = unpack_rows(rows, c["fmt"], c["dc"], c["dr"])
    else:
        b = torch.arange(c["B"], device=DEV)[:, None]
        got = unpack_rows(c["cache"][b, c["idx"].long().clamp_min(0)], c["fmt"], c["dc"], c["dr"])
        got = torch.where((c["idx"] >= 0)[..., None], got, torch.zeros_like(got))
    return got.to(c["rows"].dtype)


def tokens(c):
    """The positions each query attends to [B, S, n] and which of them count."""
    limit = c["start"] + torch.arange(c["S"], device=DEV)[:, None]
    idx = c["idx"].long()
    if c["op"] == "attn":
        return idx.clamp_min(0), (idx >= 0) & (idx <= limit)
    m = c["block"]
    done = (limit + 1) // m                          # the query's finished blocks
    tail = done.expand(c["B"], c["S"], 1)            # and its unfinished one
    ok = torch.cat((torch.ones_like(tail, dtype=torch.bool), (idx >= 0) & (idx < done)), -1)
    blk = torch.cat((tail, idx), -1)
    pos = (blk[..., None] * m + torch.arange(m, device=DEV)).flatten(-2)
    ok = ok.repeat_interleave(m, -1) & (pos <= limit)
    return torch.where(ok, pos, torch.zeros_like(pos)), ok


def plain_attn(c):
    pos, ok = tokens(c)
    b = torch.arange(c["B"], device=DEV)[:, None, None]
    kv = unpack_rows(c["cache"][b, pos], c["fmt"], c["dc"], c["dr"])          # [B,S,n,d]
    z = torch.matmul(c["q"].float(), kv.transpose(-1, -2)) * c["scale"]
    z = z.masked_fill(~ok[:, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, kv[..., :c["dc"]]) / torch.where(total > 0, total, torch.ones_like(total))
    return out.to(torch.bfloat16), (top + torch.log(total)).squeeze(-1)


def plain_keys(c):
    m, first, last = c["block"], c["start"] // c["block"], (c["start"] + c["S"]) // c["block"]
    n = last - first
    k = c["k_cache"][:, first * m:last * m].view(E4M3).float()
    k = k * c["k_scale"][:, first * m:last * m, None]
    mean = k.view(c["B"], n, m, c["D"]).sum(2) / m
    s = mean.abs().amax(-1).clamp_min(1e-4) / 448.0
    c["blk_cache"][:, first:last] = (mean / s[..., None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
    c["blk_scale"][:, first:last] = s
    return c["blk_cache"].view(E4M3), c["blk_scale"]


def run(state):
    c = state
    op = c["op"]
    if not own:
        if op == "append":
            return plain_append(c)
        if op == "read":
            return plain_read(c)
        return plain_keys(c) if op == "keys" else plain_attn(c)
    import top_kv_selection_b200 as dsa
    if op == "keys":
        dsa.dsa_block_keys(c["k_cache"], c["k_scale"], c["start"], c["S"], c["block"],
                           c["blk_cache"], c["blk_scale"])
        return c["blk_cache"].view(E4M3), c["blk_scale"]
    fmt = {BF16: dsa.DSA_BF16, FP8: dsa.DSA_FP8_LATENT, Q4: dsa.DSA_Q4_LATENT}[c["fmt"]]
    if op == "append":
        dsa.dsa_latent_prologue(c["kv"], c["w"], 1e-6, c["cs"], c["rope"] == 1, c["start"],
                                c["cache"], fmt, c["dc"])
        dsa.dsa_latent_read(c["cache"], fmt, c["start"], c["out"], c["dc"])
        return c["out"]
    if op == "read":
        dsa.dsa_latent_read(c["cache"], fmt, c["start"], c["rows"], c["dc"], c["idx"])
        return c["rows"]
    if op == "attn":
        dsa.dsa_sparse_mla_attn_q4(c["q"], c["cache"], c["idx"], c["start"], c["scale"], c["dc"],
                                   c["out"], c["lse"], c["ws"])
    else:
        dsa.dsa_block_mla_attn(c["q"], c["cache"], fmt, c["idx"], c["block"], c["start"],
                               c["scale"], c["dc"], c["out"], c["lse"], c["ws"])
    return c["out"], c["lse"]


# ------------------------------------------------------------------------ work
def work(case):
    c, op = case, case["op"]
    if op == "keys":
        m, D = c["block"], c["D"]
        n = (c["start"] + c["S"]) // m - c["start"] // m
        return dict(bytes=c["B"] * max(n, 1) * (m + 1) * (D + 4), flops=c["B"] * n * m * D * 2)
    d, row = c["dc"] + c["dr"], row_bytes(c["fmt"], c["dc"], c["dr"])
    if op == "append":
        n = c["B"] * c["S"]
        return dict(bytes=n * (d * (2 if c["x"] == "bf16" else 4) + row + 2 * d), flops=n * 8 * d)
    if op == "read":
        n = c["B"] * c["n"]
        return dict(bytes=n * (row + d * (2 if c["out"] == "bf16" else 4) + 4 * c["gather"]),
                    flops=n * d)
    seen = [c["start"] + 1 + s for s in range(c["S"])]
    if op == "attn":
        each = [min(c["k"], n) for n in seen]
    else:
        m = c["block"]
        each = [min(c["kb"], n // m) * m + n % m for n in seen]
    pairs = sum(each) * c["B"]
    rows = min(sum(each), c["start"] + c["S"]) * c["B"]
    q = c["B"] * c["S"] * c["Hq"]
    slots = c["k"] if op == "attn" else c["kb"]
    return dict(bytes=rows * row + q * 2 * (d + c["dc"]) + 4 * q + 4 * c["B"] * c["S"] * slots,
                flops=2 * pairs * c["Hq"] * (d + c["dc"]))


# ----------------------------------------------------------- 64-bit definition
def values64(rows, fmt, dc, dr):
    """What cache rows [n, row] stand for, element by element from the layout."""
    if fmt == BF16:
        return rows.double()
    b = rows.long()
    v = torch.arange(dc, device=rows.device)
    if fmt == FP8:
        code, s = b[:, :dc], b[:, dc:dc + dc // 32].reshape(len(b), dc // 128, 4)
        e, f = (code >> 3) & 15, code & 7
        mag = torch.where(e == 0, f.double() / 512, (8 + f).double() * torch.exp2(e.double() - 10))
        val = torch.where(code >= 128, -mag, mag)
        bits = s[..., 0] | s[..., 1] << 8 | s[..., 2] << 16 | s[..., 3] << 24
        sc = bits.int().view(torch.float32).double()[:, v // 128]
        pe_at = dc + dc // 32
    else:
        nib = v % 8 // 2 + 4 * (v % 2)
        val = ((b[:, v // 8 * 4 + nib // 2] >> (4 * (nib % 2))) & 15).double() - 8
        pe_at = dc // 2
        sc = bf16_at(b, pe_at + 2 * dr + 2 * (v // 32))
    lat = (val * sc).to(torch.bfloat16).double()
    return torch.cat((lat, bf16_at(b, pe_at + 2 * torch.arange(dr, device=rows.device))), -1)


def bf16_at(b, at):
    """The bf16 numbers at byte offsets `at` of byte rows b."""
    return ((b[:, at] | b[:, at + 1] << 8) << 16).int().view(torch.float32).double()


def exact_append(c):
    dc, dr, S = c["dc"], c["dr"], c["S"]
    x = c["kv"].double().reshape(-1, dc + dr)
    lat, pe = x[:, :dc], x[:, dc:]
    if c["norm"]:
        lat = lat / (lat.pow(2).sum(-1, keepdim=True) / dc + 1e-6).sqrt() * c["w"].double()
    if c["rope"]:
        ang = c["cs"].double().repeat(c["B"], 1, 1)
        z = torch.view_as_complex(ang.contiguous())
        if c["rope"] == 1:
            y = torch.view_as_complex(pe.reshape(-1, dr // 2, 2).contiguous()) * z
            pe = torch.view_as_real(y).reshape(-1, dr)
        else:
            y = torch.complex(pe[:, :dr // 2], pe[:, dr // 2:]) * z
            pe = torch.cat((y.real, y.imag), -1)
    if c["fmt"] == FP8:
        g = lat.reshape(-1, dc // 128, 128)
        s = (g.abs().amax(-1, keepdim=True).clamp_min(1e-4).float() / 448).double()
        r = (g / s).clamp(-448, 448)
        step = torch.exp2(r.abs().clamp_min(2.0 ** -6).log2().floor() - 3)
        lat = (torch.round(r / step) * step * s).reshape(-1, dc)
    elif c["fmt"] == Q4:
        g = lat.reshape(-1, dc // 32, 32)
        s = (g.abs().amax(-1, keepdim=True).clamp_min(1e-4) / 7).to(torch.bfloat16).double()
        lat = (torch.round(g / s).clamp(-7, 7) * s).reshape(-1, dc)
    out = torch.cat((lat, pe), -1).to(torch.bfloat16).double()
    return out.reshape(c["B"], S, dc + dr)


def exact_keys(c):
    m, D, first = c["block"], c["D"], c["start"] // c["block"]
    codes, scales = torch.zeros_like(c["blk_cache"]).double(), torch.zeros_like(c["blk_scale"]).double()
    for e in range(first, (c["start"] + c["S"]) // m):
        at = slice(e * m, e * m + m)
        k = c["k_cache"][:, at].view(E4M3).double() * c["k_scale"][:, at, None].double()
        mean = k.mean(1)
        s = mean.abs().amax(-1).clamp_min(1e-4) / 448
        r = mean / s[:, None]
        step = torch.exp2(r.abs().clamp_min(2.0 ** -6).log2().floor() - 3)
        codes[:, e], scales[:, e] = torch.round(r / step) * step, s
    return codes, scales


def exact(case, seed):
    c = prepare(case, seed)
    dc, dr = c.get("dc"), c.get("dr")
    if c["op"] == "append":
        return exact_append(c)
    if c["op"] == "keys":
        return exact_keys(c)
    if c["op"] == "read":
        out = torch.zeros(c["B"], c["n"], dc + dr, dtype=torch.float64, device=DEV)
        for b in range(c["B"]):
            at = torch.arange(c["n"], device=DEV) + c["start"] if c["idx"] is None else c["idx"][b].long()
            for i in range(0, c["n"], 16384):
                a = at[i:i + 16384]
                v = values64(c["cache"][b, a.clamp_min(0)], c["fmt"], dc, dr)
                out[b, i:i + 16384] = v * (a >= 0)[:, None]
        return out
    out = torch.zeros(c["B"], c["S"], c["Hq"], dc, dtype=torch.float64, device=DEV)
    lse = torch.full((c["B"], c["S"], c["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        for s in range(c["S"]):
            i = c["start"] + s
            ids = c["idx"][b, s].long()
            if c["op"] == "attn":
                t = ids[(ids >= 0) & (ids <= i)]
            else:
                m = c["block"]
                ids = ids[(ids >= 0) & (ids < (i + 1) // m)]
                t = (ids[:, None] * m + torch.arange(m, device=DEV)).reshape(-1)
                t = torch.cat((t, torch.arange((i + 1) // m * m, i + 1, device=DEV)))
            if not len(t):
                continue
            v = values64(c["cache"][b, t], c["fmt"], dc, dr)
            z = c["q"][b, s].double() @ v.T * c["scale"]
            lse[b, s] = torch.logsumexp(z, -1)
            out[b, s] = torch.softmax(z, -1) @ v[:, :dc]
    return out, lse
