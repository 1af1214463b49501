"""Microscaled KV cache on the GPU against the fp64 oracle.

Writing, reading and moving are compared byte for byte.  Attention is compared
element by element within bounds that count its roundings.  With B the largest
scale * sum |q_d k_d| of a row, S the score's own rounding, A = sum p |v|:

* a score is a sum of D exact products in fp32: 3 roundings per block of 32
  channels and, inside a matrix instruction, at most 17 truncations of 2^-24 of
  a partial sum each: |ds| <= 32 * 2^-24 * B, and 2^-22 |s| for the factors;
* each weight carries 2 ds relatively (its own and the sum's), 2^-22 for the
  exponential, and its rounding to fp16: 2^-11 (fp32 in or out: 2^-21);
* a weight far below the largest: fp16 ends at 2^-24, so up to 2^-25 is lost of
  each, where the largest weight of the row and block stood at 2^8 or more:
  2^-33 of it.  A weight meets codes up to the format's top, and top * 2^e is
  at most twice the largest value of the block (the scale is the least that
  holds it, and rounding keeps it at half the top or more): N tokens lose
  N * 2^-32 * max p |v| of their block;
* the sums of up to 64 matrix instructions, partials and the division: 2^-17;
* a cap adds 2^-22 * cap to ds, a bias 2^-23 of itself;
* the output's rounding: 2^-8 |o| in bf16, 2^-24 |o| in fp32.
"""
import numpy as np
import pytest
import torch

import oracle as O
from sub_bit_vector_b200 import cache, loopvq as L

pytestmark = pytest.mark.gpu
FMT = {"e4m3": L.LOOPVQ_MX_E4M3, "e2m1": L.LOOPVQ_MX_E2M1}
TT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Setup:
    """A batch with shuffled pages: device arrays, layout and where tokens sit."""

    def __init__(self, ctx, new, *, D=128, fmt="e4m3", T=1, H=2, Hq=None, page=64, seed=0, spare=2, fill=0xFF):
        self.rng = np.random.default_rng(seed)
        self.ctx, self.new, self.D, self.fmt, self.T, self.H, self.page = ctx, new, D, fmt, T, H, page
        self.Hq = Hq or H
        self.off = np.concatenate([[0], np.cumsum(new)]).astype(int)
        self.rows = int(self.off[-1])
        per = [-(-c // page) for c in ctx]
        self.n_pages = sum(per) + spare
        ids = self.rng.permutation(self.n_pages)
        self.max_pages = max(1, max(per))
        self.table = np.full((len(ctx), self.max_pages), -1, dtype=np.int32)
        at = 0
        for r, p in enumerate(per):
            self.table[r, :p] = ids[at:at + p]
            at += p
        self.desc = L.make_mx_desc(T, H, D, FMT[fmt], n_heads_q=self.Hq)
        self.lay = self.layout(ctx, self.off)
        tb = O.mx_tile_bytes(D, fmt)
        self.shape = (T, H, self.n_pages * page // 32, tb)
        self.poolK = torch.full(self.shape, fill, dtype=torch.uint8, device="cuda")
        self.poolV = torch.full(self.shape, fill, dtype=torch.uint8, device="cuda")
        self.fault = torch.zeros(1, dtype=torch.int32, device="cuda")

    def layout(self, ctx, off, **kw):
        off = [int(o) for o in off]
        a = dict(max_ctx_len=max(1, max(ctx)), max_new=max(b - a for a, b in zip(off, off[1:])), total_new=off[-1])
        a.update(kw)
        return L.make_mx_layout(len(ctx), self.page, self.max_pages, self.n_pages * self.page, a["max_ctx_len"],
                                a["max_new"], a["total_new"], _i32(list(ctx)), _i32(off), _i32(self.table.tolist()))

    def pos(self, r, p):
        return int(self.table[r, p // self.page]) * self.page + p % self.page

    def write_all(self, K, V, dtype=torch.float32):
        """K, V: per request [T][ctx][H][D] arrays; every token is written as new."""
        off = np.concatenate([[0], np.cumsum(self.ctx)]).astype(int)
        lay = self.layout(self.ctx, off)
        k, v = (torch.from_numpy(np.concatenate(x, 1).astype(np.float32)).cuda().to(dtype) for x in (K, V))
        L.loopvq_mx_write(self.desc, lay, 0, self.T, k, v, k.stride(0), k.stride(1), k.stride(2), self.poolK, self.poolV,
                          self.fault)

    def faults(self):
        return int(self.fault.item())


def _values(rng, shape, kind, bf16=False):
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-3, 4, shape[:-1] + (1,)))
    if kind == "k":
        x[..., 3::37] *= 8
    x = x.astype(np.float32)
    return torch.from_numpy(x).to(torch.bfloat16).float().numpy() if bf16 else x


# ------------------------------------------------------------- write and read

@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("order", ["packed", "fused", "odd"])
@pytest.mark.parametrize("new", [[5, 0, 1, 100, 64], [5, 0, 1, 16, 3], [1, 1, 0, 1, 1]])
def test_write_and_read_bytes(fmt, D, dtype, order, new):
    """New tokens of ragged requests (none, one, a partial quad, a whole page and
    more) at odd starts: their bytes are the oracle's, all others keep theirs,
    and reading gives the codes' values.  Inputs packed, in a fused
    projection, or at an odd address (scalar loads)."""
    T, H = 2, 3
    s = Setup([37, 70, 5, 129, 64], new, D=D, fmt=fmt, T=T, H=H, page=32, seed=D + len(order), fill=0xA5)
    K = _values(s.rng, (T, s.rows, H, D), "k", dtype == "bf16")
    V = _values(s.rng, (T, s.rows, H, D), "v", dtype == "bf16")
    if order == "fused":
        x = torch.zeros((T, s.rows, H, 2, D), dtype=TT[dtype], device="cuda")
        k, v = x[:, :, :, 0], x[:, :, :, 1]
    elif order == "odd":
        base = [torch.zeros(T * s.rows * H * (D + 1) + 1, dtype=TT[dtype], device="cuda") for _ in "kv"]
        k, v = (b[1:].view(T, s.rows, H, D + 1)[..., :D] for b in base)
    else:
        k, v = (torch.zeros((T, s.rows, H, D), dtype=TT[dtype], device="cuda") for _ in "kv")
    k.copy_(torch.from_numpy(K))
    v.copy_(torch.from_numpy(V))
    L.loopvq_mx_write(s.desc, s.lay, 0, T, k, v, k.stride(0), k.stride(1), k.stride(2), s.poolK, s.poolV, s.fault)
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    if order == "odd":
        ko, vo = (torch.full((T, s.rows, H, D + 1), 7.0, dtype=TT[dtype], device="cuda")[..., :D] for _ in "kv")
    else:
        ko, vo = (torch.full((T, s.rows, H, D), 7.0, dtype=TT[dtype], device="cuda") for _ in "kv")
    L.loopvq_mx_read(s.desc, s.lay, 0, T, s.poolK, s.poolV, ko, vo, ko.stride(0), ko.stride(1), ko.stride(2), s.fault)
    assert s.faults() == 0
    for kind, X, pool, back in (("k", K, s.poolK, ko), ("v", V, s.poolV, vo)):
        want = np.full(s.shape, 0xA5, dtype=np.uint8)
        code, scale = O.mx_quantise(X, fmt)
        for r, n in enumerate(s.new):
            for i in range(n):
                for t in range(T):
                    for h in range(H):
                        row = s.off[r] + i
                        O.mx_store(want, t, h, s.pos(r, s.ctx[r] - n + i), code[t, row, h], scale[t, row, h], kind, fmt)
        np.testing.assert_array_equal(pool.cpu().numpy(), want)
        ref = torch.from_numpy(O.mx_values(code, scale, fmt)).to(TT[dtype])
        assert torch.equal(back.cpu(), ref)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_special_blocks(fmt):
    """Zeros of both signs, subnormals, values beyond the largest scale, ties, an
    infinity, a NaN; each in its own block, for K and V alike."""
    D = 128
    s = Setup([16], [16], D=D, fmt=fmt, H=1, page=32, fill=0)
    X = np.zeros((1, 16, 1, D), dtype=np.float32)
    X[0, 0, 0, :64] = -0.0
    X[0, 1, 0, 0:3] = [1e-45, -3e-39, 1e-38]
    X[0, 2, 0, 32:35] = [3.4e38, -2e38, 1e36]
    X[0, 3, 0, 5], X[0, 3, 0, 70] = np.inf, -np.inf
    X[0, 4, 0, 100] = np.nan
    X[0, 5, 0, :40] = np.linspace(-1, 1, 40)
    X[0, 6, 0, :16] = [448, 432, 17, 19, 6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -0.25, 2 ** -10, 3 * 2 ** -10]
    X[0, 7, 0, :9] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25]
    X[0, 8, 0, 0] = 2.0 ** -56 * 7
    x = torch.from_numpy(X).cuda()
    L.loopvq_mx_write(s.desc, s.lay, 0, 1, x, x, 0, D, D, s.poolK, s.poolV, s.fault)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    L.loopvq_mx_read(s.desc, s.lay, 0, 1, s.poolK, s.poolV, ko, vo, 0, D, D, s.fault)
    ref = torch.from_numpy(O.mx_values(*O.mx_quantise(X, fmt), fmt)).float()
    for o in (ko, vo):
        got = o.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(got.nan_to_num(0).view(torch.int32), ref.nan_to_num(0).view(torch.int32))


# ------------------------------------------------------------------ attention

def _tree(rng, n):
    m = []
    for i in range(n):
        up = int(rng.integers(-1, i)) if i else -1
        m.append((m[up] if up >= 0 else 0) | 1 << i)
    return m


def _masks(lists):
    return torch.tensor([x - (1 << 64) if x >> 63 else x for m in lists for x in m] or [0], dtype=torch.int64,
                        device="cuda")


def _check(s, q, K, V, masks, out, lse, *, cap=0.0, slopes=None, fine=False, scale=None, written=None):
    """out, lse (host fp64 arrays) against the oracle; K, V per request [ctx][H][D]
    values as read back."""
    scale = s.D ** -0.5 if scale is None else scale
    G = s.Hq // s.H
    worst = 0.0
    for r, (c, n) in enumerate(zip(s.ctx, s.new)):
        if n == 0:
            continue
        P = c - n
        m = masks[r] if masks is not None else [(2 << i) - 1 for i in range(n)]
        m = [x & ((1 << n) - 1) for x in m]
        sees = np.ones((n, c), dtype=bool)
        for i in range(n):
            sees[i, P:] = [m[i] >> j & 1 for j in range(n)]
        depth = np.array([bin(m[i] & ~(1 << i)).count("1") for i in range(n)])
        pos_q = P + depth
        pos_k = np.concatenate([np.arange(P), P + depth])
        if written is not None:
            sees &= written[r][None, :]
        for hq in range(s.Hq):
            k, v = K[r][:, hq // G], V[r][:, hq // G]
            qq = q[s.off[r]:s.off[r + 1], hq].astype(np.float64)
            sl = None if slopes is None else float(slopes[hq])
            o, l, a, big = O.mx_attention(qq, k, v, sees, pos_q, pos_k, scale, cap, sl)
            got = out[s.off[r]:s.off[r + 1], hq]
            gl = lse[s.off[r]:s.off[r + 1], hq]
            with np.errstate(invalid="ignore"):
                B = np.nanmax(np.where(sees, scale * (np.abs(qq) @ np.abs(k).T), 0), axis=1, initial=0)
            far = 0 if sl is None else abs(sl) * c
            ds = (32 * 2.0 ** -24 + 2.0 ** -22) * B + 2.0 ** -22 * cap + 2.0 ** -22 * far
            w = 2 * ds + 2.0 ** -22 + (2.0 ** -21 if fine else 2.0 ** -11) + 2.0 ** -17
            tol = a * w[:, None] + c * 2.0 ** -32 * big + np.abs(o) * (2.0 ** -24 if s.out == "f32" else 2.0 ** -8) + 1e-37
            assert np.array_equal(np.isnan(got), np.isnan(o)), (r, hq)
            fin = ~np.isnan(o)
            err = np.abs(got - o)
            assert (err[fin] <= tol[fin]).all(), (r, hq, float(np.max(err[fin] / tol[fin])))
            if fin.any():
                worst = max(worst, float(np.max(err[fin] / tol[fin])))
            inf = np.isneginf(l)
            assert np.array_equal(np.isneginf(gl), inf) and (got[inf] == 0).all()
            good = ~inf & ~np.isnan(l)
            assert (np.abs(gl[good] - l[good]) <= (ds + 2.0 ** -18 + 2.0 ** -22 * np.abs(l))[good]).all(), (r, hq)
    return worst


def _run(s, q, masks, *, q_t="bf16", out_t="bf16", cap=0.0, slopes=None, t=0, lay=None, ws=None, scale=None):
    s.out = out_t
    qd = q if isinstance(q, torch.Tensor) else torch.from_numpy(q).cuda().to(TT[q_t])
    lay = lay or s.lay
    out = torch.full((s.rows + 1, s.Hq, s.D), 7.0, dtype=TT[out_t], device="cuda")
    lse = torch.full((s.rows + 1, s.Hq), 7.0, device="cuda")
    if ws is None:
        ws = torch.full((L.loopvq_mx_attn_workspace_bytes(s.desc, lay),), 0xFF, dtype=torch.uint8, device="cuda")
    L.loopvq_mx_attn(s.desc, lay, s.poolK, s.poolV, qd, qd.stride(0), qd.stride(1),
                     None if masks is None else _masks(masks), t, s.D ** -0.5 if scale is None else scale, cap, slopes,
                     out, lse, ws, s.fault)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (o[s.rows] == 7).all() and (l[s.rows] == 7).all()      # the row behind the last one
    return o[:s.rows], l[:s.rows]


def _queries(s, q_t, gain=1.0):
    q = (s.rng.standard_normal((s.rows, s.Hq, s.D)) * gain).astype(np.float32)
    return torch.from_numpy(q).to(TT[q_t]).float().numpy()


def _filled(s, t=0):
    K = [_values(s.rng, (s.T, c, s.H, s.D), "k") for c in s.ctx]
    V = [_values(s.rng, (s.T, c, s.H, s.D), "v") for c in s.ctx]
    s.write_all(K, V)
    back = [[O.mx_values(*O.mx_quantise(x[t], s.fmt), s.fmt) for x in X] for X in (K, V)]
    return back


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("kind", ["single", "chain", "tree", "tree_cap_bias"])
def test_attention(fmt, D, types, kind):
    """Ragged contexts (a request whose only tokens are its new ones, one without
    new tokens, tile borders on both sides) and head groups of 1 and 3."""
    single = kind == "single"
    ctx = [1, 33, 300, 64, 1000, 31] if single else [3, 40, 300, 65, 1000, 31]
    new = [1, 1, 1, 0, 1, 1] if single else [3, 7, 0, 1, 19, 2]
    for Hq in (2, 6):
        s = Setup(ctx, new, D=D, fmt=fmt, Hq=Hq, seed=len(kind) + Hq)
        K, V = _filled(s)
        q = _queries(s, types[0])
        masks = [_tree(s.rng, n) for n in new] if "tree" in kind else None
        cap, slopes = 0.0, None
        if kind.endswith("bias"):
            cap, slopes = 5.0, torch.tensor([2.0 ** -(i + 1) for i in range(Hq)], device="cuda")
        o, l = _run(s, q, masks, q_t=types[0], out_t=types[1], cap=cap, slopes=slopes)
        _check(s, q, K, V, masks, o, l, cap=cap, slopes=slopes, fine="f32" in types)
        assert s.faults() == 0


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("n,Hq", [(64, 1), (64, 2), (63, 4), (9, 1), (8, 1), (17, 8)])
def test_attention_many_rows(types, n, Hq):
    """Up to 64 nodes and several query heads: more than one chunk of rows; bit 63 of a mask."""
    s = Setup([64 + 500, n, 700], [min(n, 64), n, 3], fmt="e2m1", H=1, Hq=Hq, seed=n + Hq, page=96)
    K, V = _filled(s)
    q = _queries(s, types[0])
    masks = [_tree(s.rng, k) for k in s.new]
    o, l = _run(s, q, masks, q_t=types[0], out_t=types[1])
    _check(s, q, K, V, masks, o, l, fine="f32" in types)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["tree", "chain", "cap_bias"])
def test_attention_on_the_tensor_cores(fmt, D, kind):
    """More rows than the warps' kernel takes: whole and partial chunks, requests
    with few rows or none beside them, contexts of the new tokens alone, tile
    borders, units that spread over several blocks."""
    new = [64, 0, 33, 1, 50, 64]
    s = Setup([64, 10, 33 + 31, 200, 3000, 97], new, D=D, fmt=fmt, H=2, Hq=8, seed=D + len(kind), page=96)
    K, V = _filled(s)
    q = _queries(s, "bf16")
    masks = None if kind == "chain" else [_tree(s.rng, n) for n in new]
    cap, slopes = 0.0, None
    if kind == "cap_bias":
        cap, slopes = 8.0, torch.tensor([2.0 ** -(i + 1) for i in range(8)], device="cuda")
    o, l = _run(s, q, masks, cap=cap, slopes=slopes)
    _check(s, q, K, V, masks, o, l, cap=cap, slopes=slopes)
    again = _run(s, q, masks, cap=cap, slopes=slopes)
    assert np.array_equal(o, again[0]) and np.array_equal(l, again[1]) and s.faults() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_tensor_core_rows_see_only_their_own(fmt):
    """NaN and infinite siblings, 0xFF bytes behind the contexts, rows that see
    nothing, a page outside the pool; then scores that rise by more than the
    slack from tile to tile, so that the sums are rescaled."""
    n, G = 60, 3
    s = Setup([200 + n, n + 5], [n, n], D=64, fmt=fmt, H=1, Hq=G, seed=30, page=32)
    K = [_values(s.rng, (1, c, 1, 64), "k") for c in s.ctx]
    V = [_values(s.rng, (1, c, 1, 64), "v") for c in s.ctx]
    K[0][0, 200 + 7, 0, 5] = np.nan
    V[0][0, 200 + 9, 0, 40] = np.inf
    V[1][0, 2, 0, 3] = np.nan            # in a prefix: every row sees it
    s.write_all(K, V)
    back = [[O.mx_values(*O.mx_quantise(x[0], fmt), fmt) for x in X] for X in (K, V)]
    masks = [_tree(s.rng, n) for _ in s.ctx]
    masks[0][11] = 0
    masks[0][13] |= 1 << 7
    masks[0][14] |= 1 << 9
    q = _queries(s, "bf16")
    o, l = _run(s, q, masks)
    _check(s, q, *back, masks, o, l)
    assert np.isnan(o[14]).any() and np.isfinite(o[0]).all() and np.isnan(o[n:, :, :32]).all()
    hole = s.table[0, 2]
    s.table[0, 2] = -1
    lay = s.layout(s.ctx, s.off)
    o, l = _run(s, q, masks, lay=lay)
    s.table[0, 2] = hole
    assert s.faults() == L.LOOPVQ_FAULT_POOL_RANGE
    written = [np.ones(c, dtype=bool) for c in s.ctx]
    written[0][64:96] = False
    _check(s, q, *back, masks, o, l, written=written)
    s.fault.zero_()
    o, l = _run(s, q, masks, lay=s.layout([260, 10 ** 6], s.off, max_ctx_len=260))
    assert s.faults() == L.LOOPVQ_FAULT_CTX_RANGE and (o[n:] == 7).all()
    # rising and falling scores
    s = Setup([1500], [n], D=64, fmt="e4m3", H=1, Hq=G, seed=31)
    K = [np.zeros((1, 1500, 1, 64), dtype=np.float32)]
    K[0][0, :, 0, 0] = np.concatenate([np.linspace(-300, 300, 1000), np.linspace(300, -300, 500)])
    V = [_values(s.rng, (1, 1500, 1, 64), "v") * np.exp2(s.rng.integers(-20, 20, (1, 1500, 1, 1)))]
    s.write_all(K, V)
    back = [[O.mx_values(*O.mx_quantise(x[0], "e4m3"), "e4m3") for x in X] for X in (K, V)]
    q = np.zeros((n, G, 64), dtype=np.float32)
    q[:, :, 0] = torch.from_numpy(s.rng.uniform(-1, 1, (n, G)).astype(np.float32)).to(torch.bfloat16).float().numpy()
    o, l = _run(s, q, None, scale=1.0)
    _check(s, q, *back, None, o, l, scale=1.0)


def test_tensor_core_blocks_far_apart():
    """Blocks of one token 2^30 apart: on the tensor cores the small one is rounded
    to 2^-24 of the token's largest scale, 2^-25 of 2^E at most, and 2^E is at most
    twice the token's largest value over the top of the format."""
    n, G = 64, 2
    s = Setup([300], [n], D=128, fmt="e4m3", H=1, Hq=G, seed=32)
    K = [_values(s.rng, (1, 300, 1, 128), "k")]
    V = [_values(s.rng, (1, 300, 1, 128), "v")]
    V[0][..., 32:64] *= 2.0 ** -30
    V[0][..., 64:96] *= 2.0 ** -12
    s.write_all(K, V)
    k, v = (O.mx_values(*O.mx_quantise(x[0][0], "e4m3"), "e4m3") for x in (K, V))
    q = _queries(s, "bf16")
    o, l = _run(s, q, None)
    big = np.abs(v[:, 0]).max(-1)
    sees = np.tril(np.ones((n, 300), dtype=bool), 300 - n)
    for hq in range(G):
        qq = q[:, hq].astype(np.float64)
        ref, _, a, top = O.mx_attention(qq, k[:, 0], v[:, 0], sees, None, None, 128 ** -0.5)
        x = np.where(sees, 128 ** -0.5 * (qq @ k[:, 0].T), -np.inf)
        p = np.exp(x - x.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        B = 128 ** -0.5 * (np.abs(qq) @ np.abs(k[:, 0]).T).max(-1, keepdims=True)
        w = 2 * (32 * 2.0 ** -24 + 2.0 ** -22) * B + 2.0 ** -22 + 2.0 ** -11 + 2.0 ** -17
        # a weight holds the token's factor here: its end is 2^-33 of the largest weight of the row, times codes up to the top
        floor = 300 * 2.0 ** -32 * (p * big).max(-1, keepdims=True) + 2.0 ** -25 * 2 / 448 * (p @ big)[:, None]
        assert (np.abs(o[:, hq] - ref) <= a * w + floor + 2.0 ** -8 * np.abs(ref)).all()
        assert (np.abs(o[:, hq, 64:96] - ref[:, 64:96]) <= (a * w + floor + 2.0 ** -8 * np.abs(ref))[:, 64:96]).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_masks_of_every_kind(fmt):
    """Rows that see nothing, bits beyond the new tokens, a row that does not see
    itself, one that sees a later token."""
    s = Setup([4, 36, 3], [4, 4, 3], fmt=fmt, seed=3)
    K, V = _filled(s)
    q = _queries(s, "f32")
    masks = [[0, 0b10, 0xFFFFFFF0, 0b1111], [0, 0b1000, 0b1001, (1 << 64) - 1], [0, 0, 0]]
    o, l = _run(s, q, masks, q_t="f32", out_t="f32")
    _check(s, q, K, V, masks, o, l, fine=True)
    assert np.isneginf(l[0]).all() and np.isneginf(l[2]).all() and np.isfinite(l[4]).all()
    slopes = torch.tensor([0.5, 0.25], device="cuda")
    o, l = _run(s, q, masks, q_t="f32", out_t="f32", slopes=slopes)
    _check(s, q, K, V, masks, o, l, fine=True, slopes=slopes)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32")])
def test_what_is_not_seen_never_arrives(fmt, types):
    """A sibling with NaN and infinite keys and values, and 0xFF bytes behind the
    contexts, reach only the rows that see them."""
    s = Setup([70, 5], [6, 5], fmt=fmt, seed=4)
    K = [_values(s.rng, (1, c, 2, s.D), "k") for c in s.ctx]
    V = [_values(s.rng, (1, c, 2, s.D), "v") for c in s.ctx]
    K[0][0, 64 + 2, 0, 5] = np.nan
    V[0][0, 64 + 3, 1, 7] = np.inf
    V[1][0, 1, 0, 40] = np.nan
    s.write_all(K, V)
    back = [[O.mx_values(*O.mx_quantise(x[0], fmt), fmt) for x in X] for X in (K, V)]
    masks = [[1, 3, 4, 8, 0b10001, 0b101100], [1, 2, 4, 8, 0b11000]]
    q = _queries(s, types[0])
    o, l = _run(s, q, masks, q_t=types[0], out_t=types[1])
    _check(s, q, *back, masks, o, l, fine="f32" in types)
    assert np.isnan(o).any() and np.isfinite(o[0]).all()


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32")])
def test_scales_far_apart(types):
    """Values whose scales differ by 2^60 within a block of channels, the large
    ones behind weights just as small: both parts count.  Keys with blocks
    2^30 apart."""
    s = Setup([200], [1], fmt="e4m3", H=1, D=64, seed=5)
    K = [_values(s.rng, (1, 200, 1, 64), "k")]
    V = [_values(s.rng, (1, 200, 1, 64), "v")]
    q = np.zeros((1, 1, 64), dtype=np.float32)
    q[0, 0, 0] = 1.0
    K[0][0, :, 0, :] = 0
    K[0][0, ::2, 0, 0] = 41.5         # weight 2^-41.5 ln .. of the even tokens against the odd ones' 1
    K[0][0, ::2, 0, 0] *= -1
    V[0][0, ::2] *= 2.0 ** 40
    V[0][0, 1::2] *= 2.0 ** -20
    s.write_all(K, V)
    back = [[O.mx_values(*O.mx_quantise(x[0], "e4m3"), "e4m3") for x in X] for X in (K, V)]
    o, l = _run(s, q, None, q_t=types[0], out_t=types[1], scale=1.0)
    _check(s, q, *back, None, o, l, fine="f32" in types, scale=1.0)


def test_rising_scores():
    """Scores that grow along the context (each tile above the last by more than
    the slack) and fall again: the references are raised many times."""
    for types in (("bf16", "bf16"), ("f32", "f32")):
        s = Setup([900], [2], fmt="e4m3", H=1, D=64, seed=6)
        K = [np.zeros((1, 900, 1, 64), dtype=np.float32)]
        K[0][0, :, 0, 0] = np.concatenate([np.linspace(-300, 300, 600), np.linspace(300, -300, 300)])
        V = [_values(s.rng, (1, 900, 1, 64), "v")]
        s.write_all(K, V)
        back = [[O.mx_values(*O.mx_quantise(x[0], "e4m3"), "e4m3") for x in X] for X in (K, V)]
        q = np.zeros((2, 1, 64), dtype=np.float32)
        q[:, 0, 0] = [1.0, -0.5]
        o, l = _run(s, q, None, q_t=types[0], out_t=types[1], scale=1.0)
        _check(s, q, *back, None, o, l, fine="f32" in types, scale=1.0)


def test_queries_of_any_size_and_order():
    """Queries of 2^-100 and 2^100 (scores near 0, and one-hot weights), infinite
    and NaN ones; strided, and at an odd address."""
    s = Setup([100, 40], [3, 2], fmt="e4m3", D=64, seed=7)
    K, V = _filled(s)
    q = _queries(s, "bf16")
    q[1] *= 2.0 ** -100
    q[2] *= 2.0 ** 18
    buf = torch.zeros(s.rows * 400 + 8, dtype=torch.bfloat16, device="cuda")
    for shift in (0, 1):
        view = torch.as_strided(buf, (s.rows, 2, 64), (400, 136, 1), shift)
        view.copy_(torch.from_numpy(q))
        o, l = _run(s, view, None)
        _check(s, q, K, V, None, o, l)
    bad = q.copy()
    bad[0, 0, 3], bad[3, 1, 9] = np.nan, np.inf
    o, l = _run(s, bad, None)
    assert np.isnan(o[0, 0]).all() and np.isnan(o[3, 1]).all()
    keep = np.ones((5, 2), dtype=bool)
    keep[0, 0] = keep[3, 1] = False
    o2, _ = _run(s, q, None)
    assert np.array_equal(o[keep], o2[keep])


@pytest.mark.parametrize("ctx,new", [(20000, 1), (40001, 1), (20000, 6), (20011, 64)])
def test_attention_long(ctx, new):
    s = Setup([ctx, 77], [new, 1], fmt="e2m1", H=1, Hq=2, seed=8, page=256)
    K, V = _filled(s)
    q = _queries(s, "bf16")
    o, l = _run(s, q, None)
    _check(s, q, K, V, None, o, l)


def test_a_loop_step_of_several():
    s = Setup([90], [4], fmt="e2m1", T=3, seed=9)
    for t in (2, 0):
        s.rng = np.random.default_rng(9)
        K, V = _filled(s, t)
        q = _queries(s, "bf16")
        o, l = _run(s, q, None, t=t)
        _check(s, q, K, V, None, o, l)


def test_same_call_same_bits():
    s = Setup([3000, 500, 9000], [5, 1, 9], seed=10, Hq=4)
    _filled(s)
    q = _queries(s, "bf16")
    masks = [_tree(s.rng, n) for n in s.new]
    first = _run(s, q, masks)
    for _ in range(3):
        again = _run(s, q, masks)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_wide_batch():
    """More requests than a warp has lanes, most of them short, some idle."""
    rng = np.random.default_rng(11)
    ctx = [int(x) for x in rng.integers(1, 90, 150)]
    new = [int(min(c, x)) for c, x in zip(ctx, rng.integers(0, 3, 150))]
    s = Setup(ctx, new, D=64, H=1, fmt="e2m1", seed=11, page=32)
    K, V = _filled(s)
    q = _queries(s, "f32")
    o, l = _run(s, q, None, q_t="f32", out_t="f32")
    _check(s, q, K, V, None, o, l, fine=True)


# ----------------------------------------------------------------------- keep

@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("D", [64, 128])
def test_keep_bytes(fmt, D):
    """Any order, the same source twice, nothing kept, everything reversed; all
    other bytes stay."""
    T, H = 2, 5
    s = Setup([50, 33, 64, 95, 7], [20, 33, 64, 64, 0], D=D, fmt=fmt, T=T, H=H, page=32, seed=D)
    K = [_values(s.rng, (T, c, H, D), "k") for c in s.ctx]
    V = [_values(s.rng, (T, c, H, D), "v") for c in s.ctx]
    s.write_all(K, V)
    lists = [[0, 3, 4, 19], [], list(range(63, -1, -1)), [5, 5, 1, 63, 0, 33, 40, 2], []]
    before = [p.cpu().numpy().copy() for p in (s.poolK, s.poolV)]
    keep = np.full((5, 64), -1)
    for r, a in enumerate(lists):
        keep[r, :len(a)] = a
    L.loopvq_mx_keep(s.desc, s.lay, _i32(keep.tolist()), _i32([len(a) for a in lists]), 64, s.poolK, s.poolV, s.fault)
    assert s.faults() == 0
    for kind, X, pool, want in (("k", K, s.poolK, before[0]), ("v", V, s.poolV, before[1])):
        for r, a in enumerate(lists):
            P = s.ctx[r] - s.new[r]
            code, scale = O.mx_quantise(X[r], fmt)
            for i, f in enumerate(a):
                for t in range(T):
                    for h in range(H):
                        O.mx_store(want, t, h, s.pos(r, P + i), code[t, P + f, h], scale[t, P + f, h], kind, fmt)
        np.testing.assert_array_equal(pool.cpu().numpy(), want)


# --------------------------------------------------------------------- faults

def test_lengths_and_pages_out_of_range_are_left_out():
    """Bad lengths and page ids set their fault bits; the rows and tokens that
    they concern stay as they were, all others are right."""
    D, H = 64, 2
    s = Setup([40, 50, 100], [2, 3, 4], D=D, H=H, page=32, seed=12)
    K, V = _filled(s)
    q = _queries(s, "f32")
    good_o, good_l = _run(s, q, None, q_t="f32", out_t="f32")
    x = torch.ones((1, s.rows, H, D), device="cuda")
    for ctx, off in (([40, 51 + 200, 100], s.off), ([40, -1, 100], s.off), ([40, 2, 100], s.off),
                     ([40, 50, 100], [0, 2, 1, 9]), ([40, 50, 100], [0, 2, 30, 9])):
        s.fault.zero_()
        lay = s.layout(ctx, off, max_ctx_len=100, max_new=4, total_new=9)
        before = s.poolK.clone()
        o, l = _run(s, q, None, q_t="f32", out_t="f32", lay=lay)
        assert s.faults() == L.LOOPVQ_FAULT_CTX_RANGE
        assert np.array_equal(o[:2], good_o[:2]) and (o[2:5] == 7).all() and (l[2:5] == 7).all() or off is not s.off
        s.fault.zero_()
        n = _i32([1, 1, 1])
        L.loopvq_mx_keep(s.desc, lay, _i32([[0], [0], [0]]), n, 1, s.poolK, s.poolV, s.fault)
        assert s.faults() == L.LOOPVQ_FAULT_CTX_RANGE and torch.equal(s.poolK, before)
        out = torch.full((1, s.rows, H, D), 7.0, device="cuda")
        s.fault.zero_()
        L.loopvq_mx_read(s.desc, lay, 0, 1, s.poolK, s.poolV, out, out.clone(), 0, H * D, D, s.fault)
        assert s.faults() == L.LOOPVQ_FAULT_CTX_RANGE and (off is not s.off or bool((out[:, 2:5] == 7).all()))
    # a page outside the pool: its 32 tokens are not there
    for bad in (-1, s.n_pages, 2 ** 31 - 1):
        keep_id = s.table[2, 1]
        s.table[2, 1] = bad
        lay = s.layout(s.ctx, s.off)
        s.fault.zero_()
        o, l = _run(s, q, None, q_t="f32", out_t="f32", lay=lay)
        assert s.faults() == L.LOOPVQ_FAULT_POOL_RANGE
        written = [np.ones(c, dtype=bool) for c in s.ctx]
        written[2][32:64] = False
        _check(s, q, K, V, None, o, l, fine=True, written=written)
        before = s.poolK.clone(), s.poolV.clone()
        off = [0, 0, 0, 70]
        wide = torch.ones((1, 70, H, D), device="cuda")
        s.fault.zero_()
        L.loopvq_mx_write(s.desc, s.layout([40, 50, 100], off), 0, 1, wide, wide, 0, H * D, D, s.poolK, s.poolV, s.fault)
        assert s.faults() == L.LOOPVQ_FAULT_POOL_RANGE
        s.table[2, 1] = keep_id
        same = (s.poolK == before[0])[:, :, keep_id].all()
        assert bool(same)
        s.poolK.copy_(before[0])
        s.poolV.copy_(before[1])
    # an index that keep cannot move
    for lists, n in (([[4], [0], [0]], [1, 0, 0]), ([[-1], [0], [0]], [1, 0, 0]), ([[0], [0], [0]], [5, 0, 0]),
                     ([[0], [0], [0]], [-1, 0, 0])):
        before = s.poolK.clone()
        s.fault.zero_()
        L.loopvq_mx_keep(s.desc, s.lay, _i32(lists), _i32(n), 1, s.poolK, s.poolV, s.fault)
        assert s.faults() == L.LOOPVQ_FAULT_CTX_RANGE and torch.equal(s.poolK, before)


def test_no_fault_word():
    s = Setup([40], [2], seed=13)
    _filled(s)
    q = torch.zeros((2, 2, 128), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q), None
    lay = s.layout([41], [0, 2], max_ctx_len=40)
    ws = torch.zeros(L.loopvq_mx_attn_workspace_bytes(s.desc, lay), dtype=torch.uint8, device="cuda")
    L.loopvq_mx_attn(s.desc, lay, s.poolK, s.poolV, q, 256, 128, None, 0, 0.1, 0.0, None, out, lse, ws)
    torch.cuda.synchronize()


# ------------------------------------------------------- together, and its use

@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_cache_in_use(fmt):
    """Prompts, a step of drafted trees, keeping what was accepted, single
    tokens, one request ending and its pages going to another; every attention
    against the oracle on the values that the history left."""
    T, H, Hq, D, B = 2, 2, 4, 64, 3
    rng = np.random.default_rng(14)
    c = cache.MXCache(n_loop=T, n_heads_kv=H, n_heads_q=Hq, head_dim=D, batch=B, max_ctx_len=160, page_tokens=32, n_pages=11,
                      format=fmt, out_dtype=torch.float32)
    hist = [[np.zeros((T, 0, H, D))] * 2 for _ in range(B)]     # values as read back

    def step(n_new, masks=None, accept=None, cap=0.0):
        c.extend(n_new)
        K, V = (_values(rng, (T, c.rows, H, D), kind, True) for kind in "kv")
        off = np.concatenate([[0], np.cumsum(n_new)])
        for r in range(B):
            for i, X in enumerate((K, V)):
                back = O.mx_values(*O.mx_quantise(X[:, off[r]:off[r + 1]], fmt), fmt)
                hist[r][i] = np.concatenate([hist[r][i], back], 1)
        k, v = (torch.from_numpy(x).cuda().to(torch.bfloat16) for x in (K, V))
        if cap:
            c.write(k, v)
        for t in range(T):
            if not cap:
                c.write(k[t], v[t], t)
            q = torch.from_numpy(rng.standard_normal((c.rows, Hq, D)).astype(np.float32)).cuda().to(torch.bfloat16)
            if max(n_new) > 64:          # a long prompt is written, not attended to
                with pytest.raises(L.LoopVQError):
                    c.attend(t, q)
                continue
            out, lse = c.attend(t, q, None if masks is None else _masks(masks), softcap=cap)
            s = Setup.__new__(Setup)
            s.ctx, s.new, s.off, s.H, s.Hq, s.D, s.out = c.ctx, c.new, off, H, Hq, D, "f32"
            _check(s, q.float().cpu().numpy(), [x[0][t] for x in hist], [x[1][t] for x in hist], masks,
                   out.double().cpu().numpy(), lse.double().cpu().numpy(), cap=cap, fine=True)
        if accept is not None:
            P = [c.ctx[r] - n_new[r] for r in range(B)]
            c.keep(accept)
            for r in range(B):
                a = list(range(n_new[r])) if accept[r] is None else accept[r]
                hist[r] = [np.concatenate([x[:, :P[r]], x[:, P[r]:][:, a]], 1) for x in hist[r]]
                assert c.ctx[r] == hist[r][0].shape[1]

    step([45, 97, 3], cap=20.0)
    step([12, 0, 5], [_tree(rng, 12), [], _tree(rng, 5)], [[0, 4, 7, 11], None, [0, 1]])
    step([1, 1, 1])
    step([30, 20, 40], [_tree(rng, 30), _tree(rng, 20), _tree(rng, 40)], [[29, 3], [], None])
    c.truncate(1, 0)
    hist[1] = [np.zeros((T, 0, H, D))] * 2
    step([60, 1, 60])
    k, v = c.read(0, 40, 51, first_step=1)
    assert np.array_equal(k.double().cpu().numpy(), hist[0][0][1:, 40:51])
    assert np.array_equal(v.double().cpu().numpy(), hist[0][1][1:, 40:51])
    assert c.device_faults() == 0


def test_captured_step_replays_on_new_inputs():
    """Write, attend, keep and read captured into a graph; two graphs with a
    workspace each replayed on two streams at once; eager calls in between."""
    def make(seed):
        s = Setup([200, 90], [6, 3], seed=seed, D=64, Hq=4)
        _filled(s)
        s.masks = _masks([_tree(s.rng, n) for n in s.new])
        s.k = torch.zeros((1, s.rows, 2, 64), dtype=torch.bfloat16, device="cuda")
        s.v, s.q = torch.zeros_like(s.k), torch.zeros((s.rows, 4, 64), dtype=torch.bfloat16, device="cuda")
        s.keep, s.n = _i32([[0, 4, 5], [2, 0, 0]]), _i32([3, 1])
        ws = torch.zeros(L.loopvq_mx_attn_workspace_bytes(s.desc, s.lay), dtype=torch.uint8, device="cuda")
        s.res = [torch.zeros((s.rows, 4, 64), device="cuda"), torch.zeros((s.rows, 4), device="cuda"),
                 torch.zeros((1, s.rows, 2, 64), device="cuda"), torch.zeros((1, s.rows, 2, 64), device="cuda")]
        s.calls = [L.prepare_mx_write(s.desc, s.lay, 0, 1, s.k, s.v, 0, 128, 64, s.poolK, s.poolV, s.fault),
                   L.prepare_mx_attn(s.desc, s.lay, s.poolK, s.poolV, s.q, 256, 64, s.masks, 0, 0.125, 0.0, None,
                                     s.res[0], s.res[1], ws, s.fault),
                   L.prepare_mx_keep(s.desc, s.lay, s.keep, s.n, 3, s.poolK, s.poolV, s.fault),
                   L.prepare_mx_read(s.desc, s.lay, 0, 1, s.poolK, s.poolV, s.res[2], s.res[3], 0, 128, 64, s.fault)]
        return s

    two = [make(20), make(21)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    torch.cuda.synchronize()
    for s, st in zip(two, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for call in s.calls:
                call()
        graphs.append(g)
    for rep in range(3):
        for s in two:
            for x in (s.k, s.v, s.q):
                x.copy_(torch.randn(x.shape, device="cuda"))
        pools = [(s.poolK.clone(), s.poolV.clone()) for s in two]
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        got = [[x.clone() for x in s.res] for s in two]
        for s, p, res in zip(two, pools, got):
            s.poolK.copy_(p[0])
            s.poolV.copy_(p[1])
            for x in s.res:
                x.zero_()
            for call in s.calls:
                call()
            assert all(torch.equal(a, b) for a, b in zip(res, s.res)) and s.faults() == 0
            assert bool(res[0].abs().sum() > 0)


def test_offsets_past_32_bits():
    """A pool whose last pages lie beyond 2^31 bytes and 2^31 codes."""
    D, H, page = 128, 16, 256
    n_pages = (1 << 31) // (H * page * 132) + 40
    s = Setup([300], [300], D=D, H=1, page=page)
    desc = L.make_mx_desc(1, H, D, FMT["e4m3"])
    pools = [torch.zeros((1, H, n_pages * page // 32, O.mx_tile_bytes(D, "e4m3")), dtype=torch.uint8, device="cuda")
             for _ in "kv"]
    assert pools[0].numel() > 1 << 31
    table = _i32([[n_pages - 1, n_pages - 7]])
    lay = L.make_mx_layout(1, page, 2, n_pages * page, 300, 300, 300, _i32([300]), _i32([0, 300]), table)
    x = torch.randn((1, 300, H, D), device="cuda")
    L.loopvq_mx_write(desc, lay, 0, 1, x, x, 0, H * D, D, *pools)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    L.loopvq_mx_read(desc, lay, 0, 1, *pools, ko, vo, 0, H * D, D)
    ref = O.mx_values(*O.mx_quantise(x.cpu().numpy(), "e4m3"), "e4m3")
    assert np.array_equal(ko.double().cpu().numpy(), ref) and np.array_equal(vo.double().cpu().numpy(), ref)
    s.desc, s.H, s.Hq, s.new, s.off, s.rows = desc, H, H, [1], [0, 1], 1
    s.poolK, s.poolV = pools
    lay = L.make_mx_layout(1, page, 2, n_pages * page, 300, 1, 1, _i32([300]), _i32([0, 1]), table)
    q = _queries(s, "bf16")
    o, l = _run(s, q, None, lay=lay)
    _check(s, q, [ref[0]], [ref[0]], None, o, l)


@pytest.mark.parametrize("Hq,new", [(2, [[2, 3], [3, 1], [0, 2]]), (4, [[64, 3], [40, 20], [1, 60]])])
def test_captured_attention_replays_on_new_lengths(Hq, new):
    """One graph, lengths and rows changed in place between its replays, within
    the bounds that the layout gave: both kernels of rows."""
    s = Setup([700, 900], new[0], D=64, H=1, Hq=Hq, seed=40, fmt="e2m1")
    K, V = _filled(s)
    rows = max(sum(n) for n in new)
    ctx, off = _i32([700, 900]), _i32([0, 0, 0])
    lay = L.make_mx_layout(2, s.page, s.max_pages, s.n_pages * s.page, 900, 64, rows, ctx, off, _i32(s.table.tolist()))
    q = torch.from_numpy(s.rng.standard_normal((rows, Hq, 64)).astype(np.float32)).cuda().to(torch.bfloat16)
    out, lse = torch.zeros((rows, Hq, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((rows, Hq), device="cuda")
    ws = torch.full((L.loopvq_mx_attn_workspace_bytes(s.desc, lay),), 0xFF, dtype=torch.uint8, device="cuda")
    call = L.prepare_mx_attn(s.desc, lay, s.poolK, s.poolV, q, Hq * 64, 64, None, 0, 0.125, 0.0, None, out, lse, ws, s.fault)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    s.out = "bf16"
    for lengths, n in zip(([700, 900], [45, 333], [64, 900]), new):
        s.ctx, s.new, s.off = lengths, n, np.concatenate([[0], np.cumsum(n)]).astype(int)
        ctx.copy_(_i32(lengths))
        off.copy_(_i32(s.off.tolist()))
        out.fill_(7)
        lse.fill_(7)
        g.replay()
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        _check(s, q.double().cpu().numpy(), [k[:c] for k, c in zip(K, lengths)], [v[:c] for v, c in zip(V, lengths)], None, o, l)
        assert (o[s.off[-1]:] == 7).all() and (l[s.off[-1]:] == 7).all() and s.faults() == 0
