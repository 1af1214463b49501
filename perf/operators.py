"""Cases of the microscaled KV cache: quantising keys and values as they are
written, reading them back, attention of single tokens and of trees of drafted
tokens over the quantised pages, and keeping the accepted drafts.

The cache holds blocks of 32 channels of one token's key or value: an 8-bit
(e4m3) or 4-bit (e2m1) float per channel and one power-of-two scale.  With
``own`` false, ``run`` computes with elementary torch operations in fp32; with
``own`` true it calls the library.
"""
import math
import random

import torch

own = False

BLOCK = 32        # channels that share a scale
TILE = 32         # tokens of one tile of a pool
EXP_MIN, EXP_MAX = -64, 56   # range of the scale exponents
LARGE = 1 << 28   # channels of one step of a pool that are made at once
DEV = "cuda"

# The 16 values of an e2m1 code (sign in bit 3).
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------- cases

def _case(name, op, fmt, T=4, H=16, Hq=16, D=128, page=256, batch=1, ctx=(1024, 1024), new=(1, 1), **kw):
    c = {"name": name, "op": op, "fmt": fmt, "T": T, "H": H, "Hq": Hq, "D": D, "page": page, "batch": batch,
         "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0], "new_hi": new[1], "len_seed": 1,
         "x": "bf16", "q": "bf16", "out": "bf16", "tree": False, "cap": 0.0, "bias": False}
    c.update(kw)
    return c


def listed():
    return [
        # a serving step's new tokens, all four loop steps of 128 requests
        _case("append_b128_e4m3", "append", "e4m3", batch=128, ctx=(64, 320), new=(1, 1)),
        # a prompt of 8192 tokens of a 16-head layer enters the 4-bit cache
        _case("append_prompt8k_e2m1", "append", "e2m1", ctx=(8192, 8192), new=(8192, 8192)),
        # ragged prompts of a small fp32 model behind earlier tokens: odd lengths and starts
        _case("append_ragged_f32", "append", "e4m3", H=3, Hq=3, D=64, page=32, batch=7, ctx=(700, 2100),
              new=(1, 650), x="f32", out="f32"),
        # a short prefix read back, to be recomputed or moved to another cache
        _case("read_b4_e2m1", "read", "e2m1", batch=4, ctx=(320, 1000), new=(17, 300)),
        # a whole 16K context read back in bf16
        _case("read_16k_e4m3", "read", "e4m3", ctx=(16384, 16384), new=(16384, 16384)),
        # one token of one request against 32K tokens
        _case("attn_32k_e4m3", "attn", "e4m3", T=2, ctx=(32768, 32768)),
        # a tree of 64 drafted tokens against 32K tokens, two query heads per KV head
        _case("attn_32k_tree64_e2m1", "attn", "e2m1", T=1, Hq=32, ctx=(32832, 32832), new=(64, 64), tree=True),
        # a serving batch, single tokens, 4-bit cache, ragged contexts
        _case("attn_b32_e2m1", "attn", "e2m1", T=1, batch=32, ctx=(6144, 18432)),
        # a serving batch with small trees of drafts, some requests without any
        _case("attn_b32_tree_e4m3", "attn", "e4m3", T=1, batch=32, ctx=(6144, 18432), new=(0, 8), tree=True),
        # a small fp32 model: capped scores, a distance bias, an odd context
        _case("attn_small_cap_bias", "attn", "e4m3", H=2, Hq=4, D=64, page=32, batch=3, ctx=(129, 517), new=(3, 7),
              tree=True, q="f32", out="f32", cap=30.0, bias=True),
        # accepted drafts of a batch move to the end of their contexts, all loop steps
        _case("keep_b128_e4m3", "keep", "e4m3", batch=128, ctx=(500, 700), new=(33, 64)),
        _case("keep_b1_e2m1", "keep", "e2m1", ctx=(4097, 4097), new=(16, 16)),
    ]


def _loguniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attn", "attn", "keep"])
    fmt = rng.choice(["e4m3", "e2m1"])
    D = rng.choice([64, 128, 128])
    H = rng.choice([1, 2, 3, 8, 16, 16])
    group = rng.choice([1, 1, 2, 4])
    page = rng.choice([32, 64, 96, 256])
    T = rng.choice([1, 2, 4])
    batch = _loguniform(rng, 1, 128)
    c = dict(T=T, H=H, Hq=H * group, D=D, page=page, batch=batch)
    most = 600_000_000                   # channels that the case may hold in one pool
    room = max(64, most // (T * H * D * batch))
    if op in ("append", "read"):
        hi = _loguniform(rng, 33, min(room, 16384))
        new_hi = _loguniform(rng, 1, hi)
        ctx, new = (max(new_hi, hi // 2), hi), (max(1, new_hi // 3), new_hi)
        t = rng.choice(["bf16", "f32"])
        c.update(x=t, out=t)
    elif op == "keep":
        hi = _loguniform(rng, 80, min(max(room, 81), 8192))
        new_hi = rng.randint(4, 64)
        ctx, new = (max(new_hi, hi // 2), hi), (max(4, new_hi // 2), new_hi)
    else:
        hi = _loguniform(rng, 96, min(max(room, 97), 65536))
        new_hi = rng.choice([1, 1, rng.randint(2, 16), rng.randint(17, 64)])
        ctx, new = (max(new_hi, hi // 3), hi), (rng.randint(0, new_hi) if batch > 1 else new_hi, new_hi)
        c.update(tree=rng.random() < 0.7, cap=rng.choice([0.0, 0.0, 20.0, 50.0]), bias=rng.random() < 0.3,
                 q=rng.choice(["bf16", "bf16", "f32"]), out=rng.choice(["bf16", "bf16", "f32"]))
    c = _case("", op, fmt, ctx=ctx, new=new, len_seed=rng.randint(1, 1 << 20), **c)
    del c["name"]
    return c


def _lengths(case):
    """(context lengths, new tokens) of the requests; the new tokens are the
    last ones of each context."""
    r = random.Random(case["len_seed"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    new = [min(c, r.randint(case["new_lo"], case["new_hi"])) for c in ctx]
    if sum(new) == 0:
        new[0] = 1
    return ctx, new


def _n_keep(n):
    """Accepted tokens of n drafted ones: about a fifth of them."""
    return max(1, n // 5)


def work(case):
    ctx, new = _lengths(case)
    H, Hq, D, T = case["H"], case["Hq"], case["D"], case["T"]
    row = H * D * (8 if case["fmt"] == "e4m3" else 4) // 8 + H * D // BLOCK      # one token, K or V, one step
    rows = sum(new)
    ob = 2 if case["out"] == "bf16" else 4
    if case["op"] == "append":   # values in, codes out, the values they stand for out
        xb = 2 if case["x"] == "bf16" else 4
        return {"bytes": 2 * T * rows * (H * D * (xb + ob) + row), "flops": 2 * T * rows * H * D * 4}
    if case["op"] == "read":
        return {"bytes": 2 * T * rows * (H * D * ob + row), "flops": 2 * T * rows * H * D}
    if case["op"] == "keep":     # the moved tokens' codes in and out, their values out
        moved = sum(_n_keep(n) for n in new)
        return {"bytes": 2 * T * moved * (2 * row + H * D * ob), "flops": 2 * T * moved * H * D}
    qb = 2 if case["q"] == "bf16" else 4
    used = sum(c for c, n in zip(ctx, new) if n)
    pairs = sum(n * (c - n) + (n * n + n) // 2 for c, n in zip(ctx, new))
    return {"bytes": 2 * used * row + rows * Hq * (D * (qb + ob) + 4), "flops": 4 * pairs * Hq * D}


# ------------------------------------------------- the format, in plain torch

def _quantise(x, fmt):
    """x [..., D] -> (values of the codes [..., D] fp32, exponents [..., D/32]).
    The scale of a block is the smallest power of two that brings its largest
    magnitude within the codes' range; every step is exact in fp32."""
    top = 448.0 if fmt == "e4m3" else 6.0
    b = x.float().unflatten(-1, (-1, BLOCK))
    m, e = torch.frexp(b.abs().amax(-1))               # amax = m * 2^e, m in [0.5, 1)
    e = e - (9 if fmt == "e4m3" else 3)                # the codes' top is just below 2^9, 2^3
    e = e + (m > top / (512.0 if fmt == "e4m3" else 8.0))
    e = torch.where(m == 0, torch.full_like(e, EXP_MIN), e).clamp(EXP_MIN, EXP_MAX)
    y = torch.ldexp(b, -e.unsqueeze(-1)).clamp(-top, top)
    if fmt == "e4m3":
        y = y.to(torch.float8_e4m3fn).float()
    else:   # spacing 1/2 up to 2, then 1, then 2; ties to even multiples
        a = y.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        y = torch.copysign(torch.round(a / step) * step, y)
    return y.flatten(-2), e


def _values(y, e):
    return (y.unflatten(-1, (-1, BLOCK)) * torch.exp2(e.float()).unsqueeze(-1)).flatten(-2)


def _to_codes(y, fmt):
    """Code values -> one code per element (uint8)."""
    if fmt == "e4m3":
        return y.to(torch.float8_e4m3fn).view(torch.uint8)
    a = y.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4))
    return (code + torch.signbit(y) * 8).to(torch.uint8)


def _from_codes(code, fmt):
    if fmt == "e4m3":
        return code.view(torch.float8_e4m3fn).float()
    s = torch.tensor(E2M1 + [-v for v in E2M1], device=code.device)
    return s[code.long()]


def _pack(y, e, fmt, kind):
    """Code values [..., tokens, D] and exponents [..., tokens, D/32] -> pool
    bytes [..., tokens/32, tile bytes] in the layout that the header states."""
    code = _to_codes(y, fmt)
    D = y.shape[-1]
    nb = D // BLOCK
    lead = code.shape[:-2]
    t = code.shape[-2] // TILE
    if kind == "k":   # token (sub, g1, ab, g0), channel (b, c, i)
        z = code.reshape(*lead, t, 2, 4, 2, 2, nb, 4, 8)
        n = len(lead) + 1
        p = [n, n + 4, n + 1, n + 3, n + 5, n + 2, n + 6]          # sub b g1 g0 c ab i
    else:             # token (sub, c, t), channel (b, g, j)
        z = code.reshape(*lead, t, 2, 4, 4, nb, 8, 4)
        n = len(lead) + 1
        p = [n, n + 3, n + 4, n + 1, n + 5, n + 2]                 # sub b g c j t
    z = z.permute(*range(n), *p).reshape(*lead, t, 2, nb, 32, 16)  # [sub][b][lane][16 codes]
    if fmt == "e2m1":
        z = z[..., 0::2] | (z[..., 1::2] << 4)                     # low nibble first: 8 bytes
        z = z.unflatten(-3, (nb // 2, 2)).transpose(-3, -2)        # [sub][b/2][lane][b%2][8]
    z = z.reshape(*lead, t, -1)
    s = (e + 127).to(torch.uint8).reshape(*lead, t, 8, 4, nb).transpose(-2, -1)    # [quad of tokens][b][token]
    return torch.cat([z, s.reshape(*lead, t, TILE * nb)], -1).contiguous()


def _unpack(tiles, D, fmt, kind):
    """Inverse of _pack: [..., tiles, tile bytes] -> fp32 values [..., tokens, D]."""
    nb = D // BLOCK
    lead = tiles.shape[:-2]
    t = tiles.shape[-2]
    n = len(lead) + 1
    z, s = tiles.split([tiles.shape[-1] - TILE * nb, TILE * nb], -1)
    if fmt == "e2m1":
        z = z.reshape(*lead, t, 2, nb // 2, 32, 2, 8).transpose(-3, -2)
        z = torch.stack([z & 15, z >> 4], -1)
    if kind == "k":
        z = z.reshape(*lead, t, 2, nb, 4, 2, 4, 2, 8)              # sub b g1 g0 c ab i
        p = [n, n + 2, n + 5, n + 3, n + 1, n + 4, n + 6]
    else:
        z = z.reshape(*lead, t, 2, nb, 8, 4, 4, 4)                 # sub b g c j t
        p = [n, n + 3, n + 5, n + 1, n + 2, n + 4]
    code = z.permute(*range(n), *p).reshape(*lead, t * TILE, D)
    e = s.reshape(*lead, t, 8, nb, 4).transpose(-2, -1)
    e = e.reshape(*lead, t * TILE, nb).float() - 127
    return _values(_from_codes(code, fmt), e)


# ------------------------------------------------------------------- inputs

_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed, salt):
    return torch.Generator(device=DEV).manual_seed((seed * 7919 + salt) & 0x7FFFFFFF)


def _plan(case):
    """Lengths and page table: (ctx, new, new offsets, pages per request, table rows, pages of the pool)."""
    ctx, new = _lengths(case)
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    per = [-(-c // case["page"]) for c in ctx]
    total = sum(per)
    ids = list(range(total))
    random.Random(case["len_seed"] + 1).shuffle(ids)
    most = max(per)
    table, at = [], 0
    for p in per:
        table.append(ids[at:at + p] + [0] * (most - p))
        at += p
    return ctx, new, off, most, table, total


def _filled(case, seed, kind, t, pool):
    """The values that fill one loop step of a pool, some heads at a time:
    (first head, [heads][pool][D]), normal, a few key channels eight times as large."""
    H, D = case["H"], case["D"]
    few = H if H * pool * D < LARGE else 2
    for h0 in range(0, H, few):
        g = _gen(seed * 64 + h0, 100 + 2 * t + (kind == "v"))
        x = torch.randn((min(few, H - h0), pool, D), device=DEV, generator=g)
        if kind == "k":
            x[:, :, 3::37] *= 8.0
        yield h0, x


def _parents(case, seed, new):
    """Each request's tree: node i hangs from one of the nodes before it."""
    r = random.Random(seed * 31 + case["len_seed"])
    return [[-1] + [r.randint(max(0, i // 3 - 1), i - 1) for i in range(1, n)] if n else [] for n in new]


def _masks(parents):
    rows = []
    for p in parents:
        m = []
        for i, up in enumerate(p):
            m.append((m[up] if up >= 0 else 0) | 1 << i)
        rows += m
    return [x - (1 << 64) if x >> 63 else x for x in rows]


def _attn_inputs(case, seed, rows):
    q = torch.randn((rows, case["Hq"], case["D"]), device=DEV, generator=_gen(seed, 7)).to(_TORCH[case["q"]])
    slopes = torch.exp2(-8.0 * torch.arange(1, case["Hq"] + 1, device=DEV) / case["Hq"]) if case["bias"] else None
    return q, slopes


def _new_rows(case, seed, rows):
    """[T][rows][2][H][D]: keys and values as a fused projection leaves them."""
    x = torch.randn((case["T"], rows, 2, case["H"], case["D"]), device=DEV, generator=_gen(seed, 11))
    x[:, :, 0, :, 3::37] *= 8.0
    return x.to(_TORCH[case["x"]])


def _keep_lists(case, seed, new):
    """Accepted nodes: the root and then later ones, in order."""
    r = random.Random(seed * 17 + case["len_seed"])
    lists = []
    for n in new:
        k = _n_keep(n)
        lists.append([0] + sorted(r.sample(range(k, n), k - 1)) if n else [])
    return lists


def prepare(case, seed):
    ctx, new, off, most, table, total = _plan(case)
    rows = off[-1]
    pool = total * case["page"]
    dev = dict(device=DEV, dtype=torch.int32)
    s = {"case": case, "rows": rows, "pool": pool, "most": most, "max_ctx": max(ctx), "max_new": max(new),
         "ctx": torch.tensor(ctx, **dev), "off": torch.tensor(off, **dev), "pages": torch.tensor(table, **dev)}
    D, T, H, fmt = case["D"], case["T"], case["H"], case["fmt"]
    tile = 32 * D * (8 if fmt == "e4m3" else 4) // 8 + TILE * D // BLOCK
    for kind in ("k", "v"):
        p = torch.zeros((T, H, pool // TILE, tile), dtype=torch.uint8, device=DEV)
        if case["op"] != "append":
            for t in range(T):
                for h0, part in _filled(case, seed, kind, t, pool):
                    p[t, h0:h0 + len(part)] = _pack(*_quantise(part, fmt), fmt, kind)
        s["pool_" + kind] = p
    if case["op"] == "append":
        s["x"] = _new_rows(case, seed, rows)
    elif case["op"] == "attn":
        s["q"], s["slopes"] = _attn_inputs(case, seed, rows)
        s["mask"] = torch.tensor(_masks(_parents(case, seed, new)), dtype=torch.int64, device=DEV) \
            if case["tree"] else None
    elif case["op"] == "keep":
        keep = _keep_lists(case, seed, new)
        wide = max(len(k) for k in keep)
        s["keep"] = torch.tensor([k + [-1] * (wide - len(k)) for k in keep], **dev)
        s["n_keep"] = torch.tensor([len(k) for k in keep], **dev)
        # the same contexts once the accepted tokens have moved
        kept = [0]
        for k in keep:
            kept.append(kept[-1] + len(k))
        s["kept_ctx"] = torch.tensor([c - n + len(k) for c, n, k in zip(ctx, new, keep)], **dev)
        s["kept_off"] = torch.tensor(kept, **dev)
        s["kept_rows"], s["max_keep"] = kept[-1], wide
    return s


# ---------------------------------------------------------- plain operators

def _read_plain(s, kind, r, pos, start):
    """Values at position pos[i] >= start[r[i]] of request r[i], all steps: [T][rows][H][D] fp32."""
    c = s["case"]
    first = start.long() // TILE                        # the tiles that hold a request's tokens
    wide = -(-s["max_new"] // TILE) + 1
    n = (first[:, None] + torch.arange(wide, device=DEV)).clamp(max=s["most"] * c["page"] // TILE - 1)
    per = c["page"] // TILE
    at = s["pages"].long().gather(1, n // per) * per + n % per
    x = _unpack(s["pool_" + kind][:, :, at], c["D"], c["fmt"], kind)       # [T][H][B][tokens][D]
    return x[:, :, r, pos - first[r] * TILE].transpose(1, 2)


def _rows(off, rows):
    """Request, and number within it, of the rows off[r]..off[r+1]-1."""
    i = torch.arange(rows, device=DEV)
    r = torch.searchsorted(off[1:].long(), i, right=True)
    return r, i - off.long()[r]


def _attn_plain(s):
    c = s["case"]
    B, H, Hq, D = c["batch"], c["H"], c["Hq"], c["D"]
    t = c["T"] - 1
    k, v = (_unpack(s["pool_" + kind][t].unflatten(1, (-1, c["page"] // TILE))[:, s["pages"].long()].flatten(2, 3),
                    D, c["fmt"], kind) for kind in ("k", "v"))       # [H][B][N][D]
    N, M, G = k.shape[2], s["max_new"], Hq // H
    n_new = (s["off"][1:] - s["off"][:-1]).long()
    i = torch.arange(M, device=DEV)
    row = (s["off"][:-1].long()[:, None] + i).clamp(max=s["rows"] - 1)      # [B][M]
    there = i < n_new[:, None]
    q = s["q"].float()[row].view(B, M, H, G, D).permute(2, 0, 1, 3, 4).reshape(H, B, M * G, D)
    x = torch.matmul(q, k.transpose(2, 3)).view(H, B, M, G, N) * D ** -0.5
    # which of the new tokens each new token sees: [B][M][M]
    if c["tree"]:
        sees = (s["mask"][row][:, :, None] >> i) & 1 != 0
    else:
        sees = (i[None, :] <= i[:, None]).expand(B, M, M)
    sees = sees & there[:, None, :]
    depth = sees.sum(-1) - 1
    start = s["ctx"].long() - n_new
    n = torch.arange(N, device=DEV)
    node = (n - start[:, None]).clamp(0, M - 1)                     # [B][N]
    prefix = (n < start[:, None])
    inside = (n >= start[:, None]) & (n < s["ctx"].long()[:, None])
    seen = prefix[:, None] | (inside[:, None] & sees.gather(2, node[:, None].expand(B, M, N)))
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    if c["bias"]:
        at = torch.where(prefix, n.expand(B, N), start[:, None] + depth.gather(1, node))
        far = (start[:, None] + depth)[:, :, None] - at[:, None]    # [B][M][N]
        x = x - s["slopes"].view(H, 1, 1, G, 1) * far[None, :, :, None].float()
    x = torch.where(seen[None, :, :, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1)
    o = torch.matmul(p.view(H, B, M * G, N), v).view(H, B, M, G, D) / total.clamp(min=1e-37).unsqueeze(-1)
    lse = top.squeeze(-1) + torch.log(total)
    o = o.permute(1, 2, 0, 3, 4).reshape(B, M, Hq, D)[there]
    lse = lse.permute(1, 2, 0, 3).reshape(B, M, Hq)[there]
    return o.to(_TORCH[c["out"]]), lse


# --------------------------------------------------------------- the library

def _handle(s):
    """What a serving program keeps between calls: descriptors, output
    buffers, the workspace and the marshalled calls."""
    if "handle" in s:
        return s["handle"]
    from sub_bit_vector_b200 import loopvq as L
    c = s["case"]
    T, H, Hq, D = c["T"], c["H"], c["Hq"], c["D"]
    desc = L.make_mx_desc(T, H, D, L.LOOPVQ_MX_E4M3 if c["fmt"] == "e4m3" else L.LOOPVQ_MX_E2M1, n_heads_q=Hq)

    def layout(ctx, off, max_new, rows):
        return L.make_mx_layout(c["batch"], c["page"], s["most"], s["pool"], s["max_ctx"], max_new, rows, ctx, off,
                                s["pages"])

    lay = layout(s["ctx"], s["off"], s["max_new"], s["rows"])
    rows = s["kept_rows"] if c["op"] == "keep" else s["rows"]
    calls = []
    if c["op"] == "append":
        x = s["x"]
        calls.append(L.prepare_mx_write(desc, lay, 0, T, x[:, :, 0], x[:, :, 1], x.stride(0), x.stride(1), x.stride(3),
                                        s["pool_k"], s["pool_v"]))
    elif c["op"] == "keep":
        calls.append(L.prepare_mx_keep(desc, lay, s["keep"], s["n_keep"], s["max_keep"], s["pool_k"], s["pool_v"]))
        lay = layout(s["kept_ctx"], s["kept_off"], s["max_keep"], rows)
    if c["op"] == "attn":
        out = torch.empty((rows, Hq, D), dtype=_TORCH[c["out"]], device=DEV)
        outs = (out, torch.empty((rows, Hq), dtype=torch.float32, device=DEV))
        ws = torch.zeros(max(256, L.loopvq_mx_attn_workspace_bytes(desc, lay)), dtype=torch.uint8, device=DEV)
        calls.append(L.prepare_mx_attn(desc, lay, s["pool_k"], s["pool_v"], s["q"], Hq * D, D, s["mask"], T - 1,
                                       D ** -0.5, c["cap"], s["slopes"], outs[0], outs[1], ws))
    else:
        outs = tuple(torch.empty((T, rows, H, D), dtype=_TORCH[c["out"]], device=DEV) for _ in "kv")
        calls.append(L.prepare_mx_read(desc, lay, 0, T, s["pool_k"], s["pool_v"], outs[0], outs[1], rows * H * D,
                                       H * D, D))
    s["handle"] = (calls, outs)
    return s["handle"]


def run(s):
    if own:
        calls, outs = _handle(s)
        for call in calls:
            call()
        return outs
    c = s["case"]
    out = _TORCH[c["out"]]
    if c["op"] == "append":
        return tuple(_values(*_quantise(s["x"][:, :, i], c["fmt"])).to(out) for i in (0, 1))
    if c["op"] == "attn":
        return _attn_plain(s)
    start = (s["ctx"] - (s["off"][1:] - s["off"][:-1])).long()
    if c["op"] == "read":
        r, i = _rows(s["off"], s["rows"])
    else:       # the accepted tokens: what the first places hold once they have moved
        r, i = _rows(s["kept_off"], s["kept_rows"])
        i = s["keep"].long()[r, i]
    return tuple(_read_plain(s, kind, r, start[r] + i, start).to(out) for kind in ("k", "v"))


# ------------------------------------------------------------- in 64 bits

def _exact_values(x, fmt):
    """The definition: scale 2^e, e the least whole number in range with
    max|x| <= top * 2^e; then the nearest code value, ties to the even one."""
    top, lowest, digits = (448.0, -6, 3) if fmt == "e4m3" else (6.0, 0, 1)
    b = x.double().unflatten(-1, (-1, BLOCK))
    peak = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(peak / top)).clamp(EXP_MIN, EXP_MAX)
    e = torch.where(peak > top * torch.exp2(e), e + 1, e)          # log2 next to a whole number
    e = torch.where(peak <= top * torch.exp2(e - 1), e - 1, e).clamp(EXP_MIN, EXP_MAX)
    y = b / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=1e-300))).clamp(min=lowest) - digits)
    return ((torch.round(y / step) * step).clamp(-top, top) * torch.exp2(e)).flatten(-2)


def exact(case, seed):
    ctx, new, off, most, table, total = _plan(case)
    rows, pool, page = off[-1], total * case["page"], case["page"]
    H, Hq, D, fmt = case["H"], case["Hq"], case["D"], case["fmt"]
    if case["op"] == "append":
        x = _new_rows(case, seed, rows)
        return tuple(torch.cat([_exact_values(x[t:t + 1, :, i], fmt) for t in range(case["T"])]) for i in (0, 1))
    def at(r, pos):
        return [table[r][p // page] * page + p % page for p in pos]

    if case["op"] in ("read", "keep"):
        if case["op"] == "read":
            where = [a for r in range(case["batch"]) for a in at(r, range(ctx[r] - new[r], ctx[r]))]
        else:
            keep = _keep_lists(case, seed, new)
            where = [a for r in range(case["batch"]) for a in at(r, [ctx[r] - new[r] + k for k in keep[r]])]
        idx = torch.tensor(where, device=DEV)
        return tuple(torch.stack([torch.cat([_exact_values(x[:, idx], fmt) for _, x in _filled(case, seed, kind, t, pool)])
                                  .transpose(0, 1) for t in range(case["T"])]) for kind in ("k", "v"))
    t = case["T"] - 1
    q, slopes = _attn_inputs(case, seed, rows)
    trees = _parents(case, seed, new) if case["tree"] else [list(range(-1, n - 1)) for n in new]
    o = torch.zeros((rows, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((rows, Hq), -math.inf, dtype=torch.float64, device=DEV)
    G = Hq // H
    for (h0, K), (_, V) in zip(*(_filled(case, seed, kind, t, pool) for kind in ("k", "v"))):
        heads = slice(h0 * G, (h0 + len(K)) * G)
        for r in range(case["batch"]):
            if not new[r]:
                continue
            pre = ctx[r] - new[r]
            idx = torch.tensor(at(r, range(ctx[r])), device=DEV)
            k, v = (_exact_values(z[:, idx], fmt).repeat_interleave(G, 0) for z in (K, V))
            path, depth = [], []
            for i, up in enumerate(trees[r]):
                path.append((path[up] if up >= 0 else set()) | {i})
                depth.append(depth[up] + 1 if up >= 0 else 0)
            see = torch.tensor([[j in path[i] for j in range(new[r])] for i in range(new[r])])
            see = torch.cat([torch.ones((new[r], pre), dtype=torch.bool), see], 1).to(DEV)
            z = torch.einsum("nhd,hkd->hnk", q[off[r]:off[r + 1], heads].double(), k) / math.sqrt(D)
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if case["bias"]:
                place = torch.tensor(list(range(pre)) + [pre + d for d in depth], dtype=torch.float64, device=DEV)
                z = z - slopes[heads].double()[:, None, None] * (place[pre:, None] - place[None, :])
            z = z.masked_fill(~see, -math.inf)
            lse[off[r]:off[r + 1], heads] = torch.logsumexp(z, -1).T
            o[off[r]:off[r + 1], heads] = torch.einsum("hnk,hkd->nhd", torch.softmax(z, -1), v)
    return o, lse
