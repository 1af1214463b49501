"""Microscaled KV cache on the GPU where its contract ends.

Bounds as in test_gpu_mx.py, whose batch and oracle helpers are used; what is
added to the error ds of a score is derived at each test.
"""
import numpy as np
import pytest
import torch

import oracle as O
from sub_bit_vector_b200 import cache, loopvq as L
from test_gpu_mx import Setup, _filled, _i32, _queries, _run, _values

pytestmark = pytest.mark.gpu


def _close(s, q, K, V, out, lse, *, cap=0.0, fine=False, scale=None, more=None):
    """Chains of new tokens against the oracle.  ds = (32 * 2^-24 + 2^-22) B +
    more(qq, k, B) per row."""
    scale = s.D ** -0.5 if scale is None else scale
    cap = float(np.float32(cap))
    G = s.Hq // s.H
    for r, (c, n) in enumerate(zip(s.ctx, s.new)):
        sees = np.tril(np.ones((n, c), dtype=bool), c - n)
        for hq in range(s.Hq if n else 0):
            k, v = K[r][:, hq // G], V[r][:, hq // G]
            rows = slice(s.off[r], s.off[r + 1])
            qq = q[rows, hq].astype(np.float64)
            o, l, a, big = O.mx_attention(qq, k, v, sees, None, None, scale, cap)
            B = np.where(sees, scale * (np.abs(qq) @ np.abs(k).T), 0).max(1)
            ds = (32 * 2.0 ** -24 + 2.0 ** -22) * B + (0 if more is None else more(qq, k, B))
            # two weights' scores are off by ds each: e^(2 ds) - 1, which is 2 ds where that is small
            w = np.expm1(np.minimum(2 * ds, 50.0)) + 2.0 ** -22 + (2.0 ** -21 if fine else 2.0 ** -11) + 2.0 ** -17
            tol = a * w[:, None] + c * 2.0 ** -32 * big + np.abs(o) * (2.0 ** -24 if s.out == "f32" else 2.0 ** -8) + 1e-37
            err = np.abs(out[rows, hq] - o)
            assert (err <= tol).all(), (r, hq, float(np.max(err / tol)))
            assert (np.abs(lse[rows, hq] - l) <= ds + 2.0 ** -18 + 2.0 ** -22 * np.abs(l)).all(), (r, hq)


# Rows (new tokens x query heads of a KV head) that reach every form of the
# attention: halves and blocks in columns, rows in columns, the tensor cores.
ROWS = [(1, 1), (2, 1), (3, 1), (7, 1), (20, 1), (33, 4)]


@pytest.mark.parametrize("cap", [1e-30, 1.0, 64.0, 65.0, 1e3, 1e4, 1e6, 1e8])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("D", [64, 128])
def test_caps_of_any_size(D, types, cap):
    """s = cap * tanh(s / cap) for caps far below and far above the scores.  With
    fp32 in or out, or a cap above 64, the error is relative to the score: 2^-22 of
    tanhf and four roundings are below 2^-20 B, whatever the cap.  With bf16 in and out and a cap up to 64: 2^-22 of the cap."""
    fine = "f32" in types
    for n, G in ROWS:
        s = Setup([190 + n, n + 3], [n, n], D=D, fmt="e4m3", H=1, Hq=G, seed=n + D, page=64)
        K, V = _filled(s)
        for gain in (1.0, 60.0):
            q = _queries(s, types[0], gain)
            o, l = _run(s, q, None, q_t=types[0], out_t=types[1], cap=cap)
            _close(s, q, K, V, o, l, cap=cap, fine=fine,
                   more=lambda qq, k, B: 2.0 ** -20 * B if fine or cap > 64 else 2.0 ** -22 * cap)
        assert s.faults() == 0


@pytest.mark.parametrize("cap", [1e-45, 3e-39, 2.0 ** 126, 3e38])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("D", [64, 128])
def test_caps_at_the_ends_of_fp32(D, types, cap):
    """Caps whose reciprocal or whose product with log2 e is no fp32 number, and
    queries of zeros among the others (0 times that reciprocal is 0).  A
    reciprocal of 2^-128 in steps of 2^-149 is right to 2^-22: 2^-20 B as above.
    s / cap itself is rounded to half a step of 2^-149: 2^-150 of the cap."""
    fine = "f32" in types
    for n, G in ROWS:
        s = Setup([190 + n, n + 3], [n, n], D=D, fmt="e4m3", H=1, Hq=G, seed=n + D, page=64)
        K, V = _filled(s)
        q = _queries(s, types[0], 60.0)
        q[::2] = 0
        o, l = _run(s, q, None, q_t=types[0], out_t=types[1], cap=cap)
        _close(s, q, K, V, o, l, cap=cap, fine=fine,
               more=lambda qq, k, B: 2.0 ** -20 * B + 2.0 ** -150 * cap if fine or cap > 64 else 2.0 ** -22 * cap)
        assert s.faults() == 0


@pytest.mark.parametrize("scale,gain", [(3.0e38, 2.0 ** -127), (2.0 ** -100, 2.0 ** 97)])
def test_softmax_scales_at_the_ends_of_fp32(scale, gain):
    """The largest scale that is taken, and a small one, on queries that make the
    scores ordinary again."""
    for n, G in ROWS:
        s = Setup([190 + n], [n], D=64, fmt="e4m3", H=1, Hq=G, seed=n, page=64)
        K, V = _filled(s)
        q = (_queries(s, "bf16").astype(np.float64) * gain).astype(np.float32)
        q = torch.from_numpy(q).to(torch.bfloat16).float().numpy()
        for cap in (0.0, 30.0, 1e6):
            o, l = _run(s, q, None, cap=cap, scale=scale)
            _close(s, q, K, V, o, l, cap=cap, scale=float(np.float32(scale)),
                   more=lambda qq, k, B: 2.0 ** -20 * B + 2.0 ** -22 * min(cap, 64))


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_kernels_that_follow_closely_see_the_last_ones_bytes(fmt, new):
    """Write, keep, read and attend again and again in one stream with no host wait
    between them, each input made by the operation before it: every result is
    what the calls give one at a time."""
    s = Setup([300, 190 + new, new], [new, new, new], D=128, fmt=fmt, H=4, Hq=8, page=64, seed=new)
    _filled(s)
    first = s.poolK.clone(), s.poolV.clone()
    x = torch.from_numpy(s.rng.standard_normal((2, s.rows, s.H, s.D)).astype(np.float32)).cuda().to(torch.bfloat16)
    keep, n_keep = _i32([[new - 1], [0], [new // 2]]), _i32([1, 1, 1])
    ws = torch.zeros(L.loopvq_mx_attn_workspace_bytes(s.desc, s.lay), dtype=torch.uint8, device="cuda")

    def go(wait):
        s.poolK.copy_(first[0])
        s.poolV.copy_(first[1])
        a, res = x.clone(), []
        for i in range(40):
            a = a * -1.25 if i % 3 else a * 0.5 + 1        # a torch kernel writes the rows
            wait()
            L.loopvq_mx_write(s.desc, s.lay, 0, 1, a[0], a[1], 0, s.H * s.D, s.D, s.poolK, s.poolV, s.fault)
            wait()
            k, v = torch.empty_like(a[0:1]), torch.empty_like(a[0:1])
            L.loopvq_mx_read(s.desc, s.lay, 0, 1, s.poolK, s.poolV, k, v, 0, s.H * s.D, s.D, s.fault)
            wait()
            L.loopvq_mx_keep(s.desc, s.lay, keep, n_keep, 1, s.poolK, s.poolV, s.fault)
            wait()
            out = torch.empty((s.rows, s.Hq, s.D), dtype=torch.bfloat16, device="cuda")
            L.loopvq_mx_attn(s.desc, s.lay, s.poolK, s.poolV, torch.cat([k[0], v[0]], 1), 8 * s.D, s.D, None, 0, 0.02, 0.0,
                             None, out, None, ws, s.fault)
            wait()
            a = torch.stack([out[:, :s.H], out[:, s.H:]])  # the next rows come from this output
            res += [k, v, out]
        torch.cuda.synchronize()
        return res

    for a, b in zip(go(torch.cuda.synchronize), go(lambda: None)):
        assert torch.equal(a, b)
    assert s.faults() == 0


def test_prompts_beside_trees_are_kept():
    """A step with a prompt of more than 64 tokens, a tree and a single token: the
    accepted nodes move, the rest stays."""
    rng = np.random.default_rng(50)
    c = cache.MXCache(n_loop=2, n_heads_kv=2, head_dim=64, batch=3, max_ctx_len=200, page_tokens=32, format="e2m1",
                      out_dtype=torch.float32)
    hist = [[np.zeros((2, 0, 2, 64))] * 2 for _ in range(3)]
    for n_new, accept in (([40, 33, 0], None), ([100, 9, 1], [None, [0, 3, 8, 5], None]), ([1, 70, 6], [[], range(65), [5, 1]])):
        c.extend(n_new)
        X = [_values(rng, (2, c.rows, 2, 64), kind) for kind in "kv"]
        c.write(*(torch.from_numpy(x).cuda() for x in X))
        off = np.concatenate([[0], np.cumsum(n_new)])
        if accept is not None:
            c.keep(accept)
        for r, n in enumerate(n_new):
            a = list(range(n)) if accept is None or accept[r] is None else list(accept[r])
            for i, x in enumerate(X):
                back = O.mx_values(*O.mx_quantise(x[:, off[r]:off[r + 1]][:, a], "e2m1"), "e2m1")
                hist[r][i] = np.concatenate([hist[r][i], back], 1)
    for r in range(3):
        for got, want in zip(c.read(r), hist[r]):
            assert np.array_equal(got.double().cpu().numpy(), want)
    assert c.device_faults() == 0


def test_steps_on_another_stream_and_in_a_graph():
    """A step's calls wait on a stream of their own while the host begins the next
    steps, which make arrays of the same sizes; a graph of a step is replayed
    after them."""
    def steps(stream, wait):
        rng = np.random.default_rng(60)
        c = cache.MXCache(n_loop=1, n_heads_kv=2, n_heads_q=4, head_dim=64, batch=3, max_ctx_len=320, page_tokens=32)
        res, graphs = [], []
        torch.cuda.synchronize()
        for i in range(6):
            new = [int(x) for x in rng.integers(1, 9, 3)] if i else [100, 40, 64]
            c.extend(new)
            k, v = (torch.from_numpy(_values(rng, (c.rows, 2, 64), kind)).cuda().to(torch.bfloat16) for kind in "kv")
            q = torch.from_numpy(rng.standard_normal((c.rows, 4, 64)).astype(np.float32)).cuda().to(torch.bfloat16)
            torch.cuda.current_stream().synchronize()
            with torch.cuda.stream(stream):
                if wait:
                    torch.cuda._sleep(20_000_000)       # about 10 ms: the calls below have not begun when extend returns
                c.write(k, v, 0)
                if max(new) <= 64:
                    res.append(c.attend(0, q))
            if i == 3:
                torch.cuda.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    res.append(c.attend(0, q))
                graphs.append((g, q))
            for x in (k, v, q):
                x.record_stream(stream)
        torch.cuda.synchronize()
        for x in res[3]:                               # the graph's outputs: of its step, whatever came after
            x.zero_()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert c.device_faults() == 0
        return [x.clone() for pair in res for x in pair]

    plain = steps(torch.cuda.current_stream(), False)
    for a, b in zip(plain, steps(torch.cuda.Stream(), True)):
        assert torch.equal(a, b)
    assert torch.equal(plain[6], plain[4]) and torch.equal(plain[7], plain[5])


@pytest.mark.parametrize("apart", [12, 20, 30])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("D", [64, 128])
def test_key_blocks_far_apart(D, types, apart):
    """The first block of channels of every key 2^apart times as large as the
    others, met by queries that are as much smaller there, or zero.

    q is taken to half of 2^-38 of its row's largest element (fp32 too, whose
    second term ends there): 2^-39 max|q| |k_d| per channel.  On the tensor cores
    a key's element is taken to half of 2^-24 of 2^E, exactly if its block is
    less than 2^15 below E's; 2^E <= 2 max|k| / 448: 2^-24 max|k| / 448 |q_d|."""
    scale = D ** -0.5
    for n, G in ROWS:
        s = Setup([200 + n], [n], D=D, fmt="e4m3", H=1, Hq=G, seed=apart + n, page=64)
        K = [_values(s.rng, (1, c, 1, D), "k") for c in s.ctx]
        V = [_values(s.rng, (1, c, 1, D), "v") for c in s.ctx]
        K[0][..., :32] *= 2.0 ** apart
        s.write_all(K, V)
        back = [[O.mx_values(*O.mx_quantise(x[0], "e4m3"), "e4m3") for x in X] for X in (K, V)]
        for factor in (0.0, 2.0 ** -apart):
            q = _queries(s, types[0])
            q[..., :32] *= factor
            o, l = _run(s, q, None, q_t=types[0], out_t=types[1])
            on_tensor_cores = types[0] == "bf16" and n * G > 64

            def more(qq, k, B):
                d = scale * 2.0 ** -39 * np.abs(qq).max(-1) * np.abs(k).sum(-1).max()
                if on_tensor_cores and apart > 12:
                    d = d + scale * 2.0 ** -24 / 448 * np.abs(k).max() * np.abs(qq[:, 32:]).sum(-1)
                return d
            _close(s, q, *back, o, l, fine="f32" in types, more=more)
        assert s.faults() == 0


# ------------------------------------------------- lengths out of range

BAD_LENGTHS = [([40, 251, 100], None), ([40, -1, 100], None), ([40, 2, 100], None), ([40, 50, 100], [0, 2, 1, 0]),
               ([40, 50, 100], [0, 2, 30, 9])]


def _batch():
    s = Setup([40, 50, 100], [2, 3, 4], D=64, H=2, page=32, seed=12)
    K, V = _filled(s)
    return s, K, V


def _valid(s, off):
    """Requests that the bad lengths leave: all but the second, and if the
    offsets are bad, the third too (its rows begin at a wrong place)."""
    return (0, 2) if off is None else (0,)


@pytest.mark.parametrize("ctx,off", BAD_LENGTHS)
@pytest.mark.parametrize("many", [False, True])
def test_writes_of_bad_lengths_touch_nothing(ctx, off, many):
    """Both kernels of the write (few tokens, whole tiles): the pools' bytes are
    the oracle's for the requests that are in range, and the old ones elsewhere."""
    s, _, _ = _batch()
    want = [p.cpu().numpy().copy() for p in (s.poolK, s.poolV)]
    X = [_values(s.rng, (s.rows, s.H, s.D), kind) for kind in "kv"]
    k, v = (torch.from_numpy(x).cuda() for x in X)
    lay = s.layout(ctx, s.off if off is None else off, max_ctx_len=100, max_new=20 if many else 4, total_new=9)
    L.loopvq_mx_write(s.desc, lay, 0, 1, k, v, 0, s.H * s.D, s.D, s.poolK, s.poolV, s.fault)
    assert s.faults() == L.LOOPVQ_FAULT_CTX_RANGE
    ok = _valid(s, off)
    for kind, x, w, pool in (("k", X[0], want[0], s.poolK), ("v", X[1], want[1], s.poolV)):
        code, scale = O.mx_quantise(x, s.fmt)
        for r in ok:
            for i in range(s.new[r]):
                for h in range(s.H):
                    O.mx_store(w, 0, h, s.pos(r, s.ctx[r] - s.new[r] + i), code[s.off[r] + i, h], scale[s.off[r] + i, h],
                               kind, s.fmt)
        np.testing.assert_array_equal(pool.cpu().numpy(), w)


@pytest.mark.parametrize("ctx,off", BAD_LENGTHS)
def test_keeps_of_bad_lengths_touch_nothing(ctx, off):
    """Index 1 to place 0 moves bytes: of the requests in range, and no others."""
    s, _, _ = _batch()
    before = [p.cpu().numpy().copy() for p in (s.poolK, s.poolV)]
    lay = s.layout(ctx, s.off if off is None else off, max_ctx_len=100, max_new=4, total_new=9)
    L.loopvq_mx_keep(s.desc, lay, _i32([[1], [1], [1]]), _i32([1, 1, 1]), 1, s.poolK, s.poolV, s.fault)
    assert s.faults() == L.LOOPVQ_FAULT_CTX_RANGE
    for kind, w, pool in (("k", before[0], s.poolK), ("v", before[1], s.poolV)):
        old = w.copy()
        for r in _valid(s, off):
            P = s.ctx[r] - s.new[r]
            src, dst = s.pos(r, P + 1), s.pos(r, P)
            for h in range(s.H):
                code = np.array([old[0, h, src // 32][O.mx_place(src % 32, d, kind, s.D, s.fmt)[0]] for d in range(s.D)])
                scale = np.array([old[0, h, src // 32][O.mx_scale_place(src % 32, b, s.D, s.fmt)] for b in range(s.D // 32)])
                O.mx_store(w, 0, h, dst, code, scale, kind, s.fmt)
        assert not np.array_equal(w, old)
        np.testing.assert_array_equal(pool.cpu().numpy(), w)


@pytest.mark.parametrize("ctx,off", BAD_LENGTHS)
@pytest.mark.parametrize("many", [False, True])
def test_reads_and_attention_of_bad_lengths_leave_rows(ctx, off, many):
    """Rows of the requests in range are right, all others stay as they were; few
    tokens and whole tiles, the warps' attention and the tensor cores'."""
    s, K, V = _batch()
    Hq = 64 if many else 2
    s.desc, s.Hq = L.make_mx_desc(1, s.H, s.D, L.LOOPVQ_MX_E4M3, n_heads_q=Hq), Hq
    q = _queries(s, "bf16")
    lay = s.layout(ctx, s.off if off is None else off, max_ctx_len=100, max_new=20 if many else 4, total_new=9)
    o, l = _run(s, q, None, lay=lay)
    assert s.faults() == L.LOOPVQ_FAULT_CTX_RANGE
    s.fault.zero_()
    ko, vo = (torch.full((1, s.rows, s.H, s.D), 7.0, device="cuda") for _ in "kv")
    L.loopvq_mx_read(s.desc, lay, 0, 1, s.poolK, s.poolV, ko, vo, 0, s.H * s.D, s.D, s.fault)
    assert s.faults() == L.LOOPVQ_FAULT_CTX_RANGE
    ko, vo = ko.double().cpu().numpy()[0], vo.double().cpu().numpy()[0]
    rows = np.zeros(s.rows, dtype=bool)
    new = [0] * 3
    for r in _valid(s, off):
        rows[s.off[r]:s.off[r + 1]] = True
        new[r] = s.new[r]
        P = s.ctx[r] - s.new[r]
        assert np.array_equal(ko[s.off[r]:s.off[r + 1]], K[r][P:]) and np.array_equal(vo[s.off[r]:s.off[r + 1]], V[r][P:])
    for x in (o, l, ko, vo):
        assert (x[~rows] == 7).all()
    s.new = new
    _close(s, q, K, V, o, l)


# ------------------------------------------------- calls that stand elsewhere

def test_captured_after_other_nodes():
    """A graph in which these kernels follow nothing, a copy, a fill, a kernel of
    torch and a join of two streams: replays give what eager calls give."""
    s = Setup([200, 90], [6, 3], seed=70, D=64, Hq=4)
    _filled(s)
    src = torch.from_numpy(s.rng.standard_normal((2, s.rows, 2, 64)).astype(np.float32)).cuda().to(torch.bfloat16)
    x, q = torch.zeros_like(src), torch.zeros((2, s.rows, 4, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((3, s.rows, 4, 64), dtype=torch.bfloat16, device="cuda")
    back = torch.zeros((2, 1, s.rows, 2, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros((2, L.loopvq_mx_attn_workspace_bytes(s.desc, s.lay)), dtype=torch.uint8, device="cuda")

    def write():
        L.loopvq_mx_write(s.desc, s.lay, 0, 1, x[0], x[1], 0, 128, 64, s.poolK, s.poolV, s.fault)

    def read():
        L.loopvq_mx_read(s.desc, s.lay, 0, 1, s.poolK, s.poolV, back[0], back[1], 0, 128, 64, s.fault)

    def attn(i, w=0):
        L.loopvq_mx_attn(s.desc, s.lay, s.poolK, s.poolV, q[i // 2], 256, 64, None, 0, 0.125, 0.0, None, out[i], None, ws[w],
                         s.fault)

    side = torch.cuda.Stream()

    def go():
        main = torch.cuda.current_stream()
        attn(0)                              # follows nothing
        x.copy_(src)                         # a copy
        write()
        side.wait_stream(main)
        q[0].copy_(src[0].repeat(1, 2, 1))   # kernels of torch, beside the read
        with torch.cuda.stream(side):
            read()
        main.wait_stream(side)
        attn(1)                              # a join
        side.wait_stream(main)
        with torch.cuda.stream(side):
            attn(0, 1)                       # beside the next call, with a workspace of its own
        q[1].fill_(0.25)                     # a fill
        attn(2)
        main.wait_stream(side)
        read()

    pools = s.poolK.clone(), s.poolV.clone()

    def again(run):
        s.poolK.copy_(pools[0])
        s.poolV.copy_(pools[1])
        for t in (x, q, out, back):
            t.zero_()
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        return [t.clone() for t in (out, back, s.poolK, s.poolV)]

    def one_at_a_time():
        for step in (lambda: attn(0), lambda: x.copy_(src), write, read, lambda: q[0].copy_(src[0].repeat(1, 2, 1)),
                     lambda: attn(1), lambda: attn(0, 1), lambda: q[1].fill_(0.25), lambda: attn(2)):
            step()
            torch.cuda.synchronize()

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    want = again(one_at_a_time)
    for _ in range(3):
        for a, b in zip(want, again(g.replay)):
            assert torch.equal(a, b)
    assert s.faults() == 0


@pytest.mark.parametrize("Hq", [1, 4])
def test_requests_that_share_the_pages_of_a_prefix(Hq):
    """40 requests (more than a warp has lanes) whose tables begin with the same
    pages, 17 to 30 tokens each behind them; a query of NaN and one of
    infinities among the rows; the warps' kernel and the tensor cores."""
    n, D, page = 17, 64, 32
    rng = np.random.default_rng(80)
    new = [n + int(x) for x in rng.integers(0, 14, 40)]
    s = Setup([96 + x for x in new], new, D=D, fmt="e4m3", H=1, Hq=Hq, seed=81, page=page)
    s.table[:, :3] = s.table[0, :3]
    s.lay = s.layout(s.ctx, s.off)
    pre = [_values(rng, (1, 96, 1, D), kind) for kind in "kv"]
    own = [[_values(rng, (1, x, 1, D), kind) for x in new] for kind in "kv"]
    k, v = (torch.from_numpy(x).cuda() for x in pre)
    L.loopvq_mx_write(s.desc, s.layout([96] + [0] * 39, [0] + [96] * 40), 0, 1, k, v, 0, D, D, s.poolK, s.poolV, s.fault)
    k, v = (torch.from_numpy(np.concatenate(x, 1)).cuda() for x in own)
    L.loopvq_mx_write(s.desc, s.lay, 0, 1, k, v, 0, D, D, s.poolK, s.poolV, s.fault)
    back = [[O.mx_values(*O.mx_quantise(np.concatenate([p, x], 1)[0], "e4m3"), "e4m3") for x in o] for p, o in zip(pre, own)]
    q = _queries(s, "bf16")
    o, l = _run(s, q, None)
    _close(s, q, *back, o, l)
    bad = q.copy()
    bad[3, 0, 5], bad[100, Hq - 1, 9] = np.nan, np.inf
    o2, _ = _run(s, bad, None)
    same = np.ones((s.rows, Hq), dtype=bool)
    same[3, 0] = same[100, Hq - 1] = False
    assert np.array_equal(o2[same], o[same]) and np.isnan(o2[~same]).all()
    assert s.faults() == 0
