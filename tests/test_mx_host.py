"""Microscaled KV cache, on the CPU: the oracle's format against values written
out by hand, every refusal of the entry points (all return before a launch),
the binding's checks and MXCache's bookkeeping."""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O
from sub_bit_vector_b200 import cache, loopvq as L

FAKE = 1 << 20
BAD, UNSUP, SMALL = L.LOOPVQ_ERR_INVALID_ARG, L.LOOPVQ_ERR_UNSUPPORTED, L.LOOPVQ_ERR_WORKSPACE_TOO_SMALL


# ------------------------------------------------------------------ the format

def test_tables():
    assert list(O.mx_table("e2m1")[:8]) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    t = O.mx_table("e4m3")
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(t, want)


@pytest.mark.parametrize("fmt,top", [("e4m3", 448.0), ("e2m1", 6.0)])
def test_scales_and_ties(fmt, top):
    x = np.zeros((5, 32))
    x[0, 0] = top                    # fits with e = 0
    x[1, 0] = top * (1 + 2.0 ** -20)  # needs e = 1
    x[2, 0] = 2.0 ** 100             # e = 56 saturates
    x[3, 0] = 2.0 ** -140
    x[4, 3] = np.inf
    code, scale = O.mx_quantise(x, fmt)
    assert list(scale[:, 0]) == [127, 128, 127 + 56, 127 - 64, 255]
    v = O.mx_values(code, scale, fmt)
    assert v[0, 0] == top and v[2, 0] == top * 2.0 ** 56 and v[3, 0] == 0 and np.isnan(v[4]).all()
    # ties to the even code, per sign
    y = np.zeros((1, 32))
    if fmt == "e2m1":
        y[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
        want = [6, 0, 1, 1, 2, 2, 4, 4]
    else:
        y[0, :6] = [448, 2.0 ** -10, 3 * 2.0 ** -10, 17, 19, 432]
        want = [448, 0, 2.0 ** -8, 16, 20, 448]   # 432: between 416 (odd) and 448 (even)
    for s in (1, -1):
        y2 = y * s
        v = O.mx_values(*O.mx_quantise(y2, fmt), fmt)[0]
        assert list(v[:len(want)]) == [s * w for w in want]


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["k", "v"])
def test_tile_places_are_a_permutation(fmt, D, kind):
    seen = {O.mx_place(n, d, kind, D, fmt) for n in range(32) for d in range(D)}
    sc = {O.mx_scale_place(n, b, D, fmt) for n in range(32) for b in range(D // 32)}
    size = O.mx_tile_bytes(D, fmt)
    assert len(seen) == 32 * D and len(sc) == D
    assert {p for p, _ in seen} | sc == set(range(size)) and not {p for p, _ in seen} & sc


# ------------------------------------------------------------------- refusals

def _desc(**kw):
    a = dict(n_loop=2, n_heads_kv=2, head_dim=128, format=L.LOOPVQ_MX_E4M3, n_heads_q=4)
    a.update(kw)
    return L.make_mx_desc(**a)


def _lay(**kw):
    a = dict(batch=2, page_tokens=64, max_pages=4, pool_tokens=512, max_ctx_len=256, max_new=4, total_new=8,
             ctx_len=FAKE, new_off=FAKE, pages=FAKE)
    a.update(kw)
    return L.make_mx_layout(**a)


def _write(d, l, **kw):
    a = dict(first=0, n=2, k=FAKE, v=FAKE, xd=L.LOOPVQ_BF16, st=0, sn=256, sh=128, pk=FAKE, pv=FAKE, fb=None)
    a.update(kw)
    return L._lib.loopvq_mx_write(ctypes.byref(d), ctypes.byref(l), a["first"], a["n"], a["k"], a["v"], a["xd"], a["st"],
                                  a["sn"], a["sh"], a["pk"], a["pv"], a["fb"], None)


def _read(d, l, **kw):
    a = dict(first=0, n=2, k=FAKE, v=FAKE, xd=L.LOOPVQ_BF16, st=4096, sn=256, sh=128, pk=FAKE, pv=FAKE, fb=None)
    a.update(kw)
    return L._lib.loopvq_mx_read(ctypes.byref(d), ctypes.byref(l), a["first"], a["n"], a["pk"], a["pv"], a["k"], a["v"],
                                 a["xd"], a["st"], a["sn"], a["sh"], a["fb"], None)


def _attn(d, l, **kw):
    a = dict(pk=FAKE, pv=FAKE, q=FAKE, qd=L.LOOPVQ_BF16, qn=512, qh=128, mask=None, t=0, scale=0.1, cap=0.0, slopes=None,
             out=FAKE, od=L.LOOPVQ_BF16, lse=None, ws=FAKE, wsb=1 << 40, fb=None)
    a.update(kw)
    return L._lib.loopvq_mx_attn(ctypes.byref(d), ctypes.byref(l), a["pk"], a["pv"], a["q"], a["qd"], a["qn"], a["qh"],
                                 a["mask"], a["t"], a["scale"], a["cap"], a["slopes"], a["out"], a["od"], a["lse"],
                                 a["ws"], a["wsb"], a["fb"], None)


def _keep(d, l, **kw):
    a = dict(keep=FAKE, n=FAKE, mx=4, pk=FAKE, pv=FAKE, fb=None)
    a.update(kw)
    return L._lib.loopvq_mx_keep(ctypes.byref(d), ctypes.byref(l), a["keep"], a["n"], a["mx"], a["pk"], a["pv"],
                                 a["fb"], None)


CALLS = [_write, _read, _attn, _keep]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,status", [
    (dict(n_loop=0), BAD), (dict(n_heads_kv=0), BAD), (dict(n_heads_q=3), BAD), (dict(format=2), BAD),
    (dict(head_dim=0), BAD), (dict(head_dim=96), UNSUP), (dict(head_dim=256), UNSUP),
    (dict(n_heads_kv=70000, n_heads_q=70000), UNSUP)])
def test_descriptors_refused(call, kw, status):
    assert call(_desc(**kw), _lay()) == status


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=65536), dict(page_tokens=0), dict(page_tokens=48), dict(max_pages=0),
    dict(pool_tokens=0), dict(pool_tokens=100), dict(max_ctx_len=-1), dict(max_ctx_len=257), dict(max_new=-1),
    dict(total_new=-1), dict(ctx_len=None), dict(new_off=None), dict(pages=None), dict(pages=FAKE + 2)])
def test_layouts_refused(call, kw):
    assert call(_desc(), _lay(**kw)) == BAD


@pytest.mark.parametrize("call,kw,status", [
    (_write, dict(first=-1), BAD), (_write, dict(first=1), BAD), (_write, dict(n=0), BAD), (_write, dict(xd=5), BAD),
    (_write, dict(st=-1), BAD), (_write, dict(k=None), BAD), (_write, dict(v=FAKE + 1), BAD),
    (_write, dict(pk=FAKE + 8), BAD), (_write, dict(pv=None), BAD), (_write, dict(fb=FAKE + 1), BAD),
    (_read, dict(n=3), BAD), (_read, dict(sn=0), BAD), (_read, dict(st=0), BAD), (_read, dict(sh=0), BAD),
    (_read, dict(k=FAKE + 1), BAD), (_read, dict(sh=-128), BAD),
    (_attn, dict(t=2), BAD), (_attn, dict(t=-1), BAD), (_attn, dict(qd=3), BAD), (_attn, dict(od=3), BAD),
    (_attn, dict(cap=-1.0), BAD), (_attn, dict(cap=float("nan")), BAD), (_attn, dict(cap=float("inf")), BAD),
    (_attn, dict(scale=float("nan")), BAD), (_attn, dict(mask=FAKE + 4), BAD), (_attn, dict(q=None), BAD),
    (_attn, dict(out=FAKE + 8), BAD), (_attn, dict(ws=FAKE + 128), BAD), (_attn, dict(ws=None), BAD),
    (_attn, dict(wsb=255), SMALL), (_attn, dict(slopes=FAKE + 2), BAD), (_attn, dict(lse=FAKE + 2), BAD),
    (_attn, dict(qn=-1), BAD), (_attn, dict(pk=None), BAD),
    (_keep, dict(keep=None), BAD), (_keep, dict(n=FAKE + 1), BAD), (_keep, dict(mx=0), BAD), (_keep, dict(pv=FAKE + 4), BAD)])
def test_arguments_refused(call, kw, status):
    assert call(_desc(), _lay(), **kw) == status


def test_more_than_64_new_tokens_refused_by_attention_and_keep():
    lay = _lay(max_new=65, total_new=130)
    assert _attn(_desc(), lay) == UNSUP and _keep(_desc(), lay) == UNSUP
    assert L.loopvq_mx_attn_workspace_bytes(_desc(), lay) == 0


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw", [dict(total_new=0), dict(max_new=0), dict(max_ctx_len=0)])
def test_calls_without_rows_do_nothing(call, kw):
    assert call(_desc(), _lay(**kw)) == L.LOOPVQ_OK


def test_sizes():
    assert L.loopvq_mx_pool_bytes(_desc(), 64) == 2 * 2 * 64 * (128 + 4)
    assert L.loopvq_mx_pool_bytes(_desc(format=L.LOOPVQ_MX_E2M1), 64) == 2 * 2 * 64 * (64 + 4)
    assert L.loopvq_mx_pool_bytes(_desc(), 33) == 0 and L.loopvq_mx_pool_bytes(_desc(head_dim=96), 64) == 0
    assert L.loopvq_mx_attn_workspace_bytes(_desc(), _lay()) >= 256
    assert L.loopvq_mx_attn_workspace_bytes(_desc(), _lay(batch=0)) == 0
    # the largest layout: sizes stay finite and positive
    big = _lay(batch=65535, max_pages=1 << 20, max_ctx_len=1 << 25, max_new=64, total_new=65535 * 64,
               pool_tokens=1 << 40)
    assert 0 < L.loopvq_mx_attn_workspace_bytes(_desc(n_heads_kv=65535, n_heads_q=65535), big) < 1 << 30


def test_binding_checks_what_the_kernels_read():
    d, lay = _desc(), _lay()
    with pytest.raises(TypeError):
        L.make_mx_layout(1, 64, 4, 512, 256, 1, 1, torch.zeros(1, dtype=torch.int64), FAKE, FAKE)
    with pytest.raises(ValueError):
        L.make_mx_layout(2, 64, 4, 512, 256, 1, 1, FAKE, torch.zeros(2, dtype=torch.int32), FAKE)
    with pytest.raises(ValueError):
        L.make_mx_layout(2, 64, 4, 512, 256, 1, 1, FAKE, FAKE, torch.zeros((4, 2), dtype=torch.int32).T)
    x = torch.zeros((8, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):      # host memory
        L.loopvq_mx_write(d, lay, 0, 1, x, x, 0, 256, 128, FAKE, FAKE)
    with pytest.raises(ValueError):      # 9 rows of 8
        L._mx_rows(d, _lay(total_new=9), 0, 1, x, x, 0, 256, 128)
    L._mx_rows(d, lay, 0, 1, x, x, 0, 256, 128)
    with pytest.raises(TypeError):
        L._mx_rows(d, lay, 0, 1, x, x.float(), 0, 256, 128)
    with pytest.raises(ValueError):
        L._mx_pools(d, lay, torch.zeros(100, dtype=torch.uint8), FAKE)
    with pytest.raises(TypeError):
        L._want("tree_mask", torch.zeros(8, dtype=torch.int32), ("int64", "uint64"), 8)


# ---------------------------------------------------------------- MXCache

def _cache(**kw):
    a = dict(n_loop=1, n_heads_kv=1, head_dim=64, batch=3, max_ctx_len=200, page_tokens=32, n_pages=12, device="cpu")
    a.update(kw)
    return cache.MXCache(**a)


def test_cache_pages_and_lengths(monkeypatch):
    moved = []
    monkeypatch.setattr(L, "loopvq_mx_keep", lambda d, lay, keep, n, mx, *a: moved.append((keep.tolist(), n.tolist(), mx)))
    c = _cache()
    c.extend([33, 0, 64])
    assert c.rows == 97 and [len(p) for p in c.pages] == [2, 0, 2] and len(c.free) == 8
    assert c.layout.max_new == 64 and c.layout.total_new == 97
    c.extend([5, 1, 0])
    c.keep([[0, 3], None, None])
    assert c.ctx == [35, 1, 64] and moved == [([[0, 3], [0, -1], [-1, -1]], [2, 1, 0], 2)]
    with pytest.raises(RuntimeError):
        c.attend(0, torch.zeros(1))
    c.extend([31, 0, 0])                 # into a third page, and back out of it
    assert len(c.pages[0]) == 3
    c.keep([[0, 1], [], []])             # a prefix of the new tokens: nothing moves
    assert c.ctx[0] == 37 and len(c.pages[0]) == 2 and len(moved) == 1
    c.truncate(2, 0)
    assert c.pages[2] == [] and len(c.free) == 9
    used = sum(c.pages, [])
    assert sorted(used + c.free) == list(range(12))


def test_cache_refusals():
    c = _cache()
    with pytest.raises(ValueError):
        _cache(format="e5m2")
    with pytest.raises(ValueError):
        _cache(page_tokens=40)
    with pytest.raises(ValueError):
        _cache(head_dim=96)
    with pytest.raises(ValueError):
        c.extend([1, 2])
    with pytest.raises(ValueError):
        c.extend([201, 0, 0])
    with pytest.raises(RuntimeError):
        c.extend([200, 200, 200])        # 21 pages of 12
    assert c.ctx == [0, 0, 0] and len(c.free) == 12
    c.extend([4, 0, 0])
    with pytest.raises(ValueError):
        c.keep([[4], [], []])
    with pytest.raises(ValueError):
        c.keep([[0, 1, 2, 3, 0], [], []])
    with pytest.raises(ValueError):
        c.write(torch.zeros(3, 1, 64), torch.zeros(3, 1, 64), 0)
    with pytest.raises(ValueError):
        c.truncate(0, 5)
    with pytest.raises(ValueError):
        c.read(0, 2, 9)
