"""Microscaled KV cache, on the CPU: what its sources, binding and MXCache's
bookkeeping promise at the ends of their contracts."""
import glob
import os
import re

import pytest
import torch

from sub_bit_vector_b200 import loopvq as L
from test_mx_host import FAKE, UNSUP, _attn, _cache, _desc, _keep, _lay, _read, _write

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sub_bit_vector_b200", "csrc")


def test_no_read_only_loads_in_kernels_that_start_early():
    """The read-only path (__ldg, ld.global.nc, __restrict__ pointers that the
    compiler may turn into it) is for data that nothing writes while the kernel
    lives.  These kernels may be resident before the one that writes their
    inputs has ended."""
    files = sorted(glob.glob(os.path.join(CSRC, "mx*.cu*")))
    assert len(files) == 5
    for f in files:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(f).read(), flags=re.S)
        assert "griddepcontrol.wait" in code or "mx_begin()" in code or f.endswith("mx_attn.cuh")
        for word in ("__ldg(", ".nc", "__restrict__", "ldg("):
            assert word not in code, (os.path.basename(f), word)


# ------------------------------------------------------------------ the binding

X = torch.zeros((8, 4, 128), dtype=torch.bfloat16)      # host memory: no call here reaches a launch


def _prepare(name, **kw):
    """prepare_mx_* with valid arguments but for kw."""
    d, lay = kw.pop("desc", _desc()), kw.pop("lay", _lay())
    a = dict(fault_bits=None, workspace=torch.zeros(1 << 20, dtype=torch.uint8), loop_step=0)
    a.update(kw)
    f = a["fault_bits"]
    if name == "write":
        return L.prepare_mx_write(d, lay, a["loop_step"], 1, X, X, 0, 512, 128, FAKE, FAKE, f)
    if name == "read":
        return L.prepare_mx_read(d, lay, a["loop_step"], 1, FAKE, FAKE, X, X, 0, 512, 128, f)
    if name == "attn":
        return L.prepare_mx_attn(d, lay, FAKE, FAKE, X, 512, 128, None, a["loop_step"], 0.1, 0.0, None, X, None,
                                 a["workspace"], f)
    return L.prepare_mx_keep(d, lay, FAKE, FAKE, 4, FAKE, FAKE, f)


CALLS = ["write", "read", "attn", "keep"]


@pytest.mark.parametrize("name", CALLS)
def test_fault_words_are_checked(name, monkeypatch):
    """The kernels write the fault word by its address: one on the host, of
    another type or of no elements is refused before any launch."""
    seen = []
    here = L._here
    with monkeypatch.context() as m:     # the other arguments of this test are in host memory too
        m.setattr(L, "_here", lambda *t: seen.extend(t))
        word = torch.zeros(1, dtype=torch.int32)
        try:
            _prepare(name, fault_bits=word)
        except RuntimeError:             # without a GPU, at the current device: all checks have passed
            pass
        assert any(t is word for t in seen)
        for bad, error in ((torch.zeros(1, dtype=torch.int64), TypeError), (torch.zeros(0, dtype=torch.int32), ValueError)):
            with pytest.raises(error, match="fault_bits"):
                _prepare(name, fault_bits=bad)
    with pytest.raises(ValueError, match="not on a CUDA device"):
        here(torch.zeros(1, dtype=torch.int32))


def test_workspaces_are_consecutive(monkeypatch):
    """A workspace's size is taken from its number of elements."""
    monkeypatch.setattr(L, "_here", lambda *t: None)
    with pytest.raises(ValueError, match="workspace"):
        _prepare("attn", workspace=torch.zeros((1 << 10, 1 << 10), dtype=torch.uint8)[:, ::2])


@pytest.mark.parametrize("name", CALLS)
def test_layouts_made_by_hand_are_taken(name, monkeypatch):
    """The exported structure, filled with raw addresses, without make_mx_layout."""
    monkeypatch.setattr(L, "_here", lambda *t: None)
    monkeypatch.setattr(L, "_prepared", lambda name, args, keep, stream: "prepared")
    lay = L.loopvq_mx_layout(2, 64, 4, 256, 4, 8, 512, FAKE, FAKE, FAKE)
    assert _prepare(name, lay=lay) == "prepared"


@pytest.mark.parametrize("name", CALLS)
def test_prepared_calls_keep_what_was_checked(name, monkeypatch):
    """A descriptor or layout that its owner changes, or uses again for another
    call, does not change the calls that were prepared from it."""
    monkeypatch.setattr(L, "_here", lambda *t: None)
    monkeypatch.setattr(L, "_prepared", lambda name, args, keep, stream: args)
    desc, lay = _desc(), _lay()
    args = _prepare(name, desc=desc, lay=lay)
    lay.total_new, lay.pool_tokens, desc.n_heads_kv = 1 << 20, 1 << 30, 1 << 10
    assert args[0]._obj.n_heads_kv == 2 and args[1]._obj.total_new == 8 and args[1]._obj.pool_tokens == 512


# ------------------------------------------------------- the ends of integers

@pytest.mark.parametrize("call", [_write, _read, _attn, _keep])
def test_contexts_whose_positions_pass_31_bits_refused(call):
    """The kernels look up to three tiles past a context's last token, in ints."""
    lay = dict(page_tokens=1 << 20, max_pages=1 << 11, pool_tokens=1 << 31)
    for length in (2 ** 31 - 1, 2 ** 31 - 128):
        assert call(_desc(), _lay(max_ctx_len=length, **lay)) == UNSUP
    assert call(_desc(), _lay(max_ctx_len=2 ** 31 - 129, total_new=0, **lay)) == L.LOOPVQ_OK


@pytest.mark.parametrize("call", [_write, _read, _attn, _keep])
def test_pools_whose_bytes_pass_63_bits_refused(call):
    """2 steps x 2 heads x 132 bytes a token: a size that wraps to a few bytes
    would let a small pool pass for a large one."""
    for tokens in (1 << 56, (1 << 59) + 32, (1 << 62)):
        assert L.loopvq_mx_pool_bytes(_desc(), tokens) == 0
        assert call(_desc(), _lay(pool_tokens=tokens)) == UNSUP
    assert L.loopvq_mx_pool_bytes(_desc(), 1 << 53) == (1 << 55) * 132
    assert call(_desc(), _lay(pool_tokens=1 << 53, total_new=0)) == L.LOOPVQ_OK


@pytest.mark.parametrize("name", ["batch", "page_tokens", "max_pages", "max_ctx_len", "max_new", "total_new"])
def test_layout_numbers_that_do_not_fit_refused(name):
    """2^32 tokens would have become 0, and the call one that does nothing."""
    with pytest.raises(OverflowError, match=name):
        _lay(**{name: 1 << 32})


def test_numbers_that_do_not_fit_refused(monkeypatch):
    with pytest.raises(OverflowError, match="n_loop"):
        _desc(n_loop=(1 << 32) + 1)
    with pytest.raises(OverflowError, match="pool_tokens"):
        _lay(pool_tokens=1 << 64)
    monkeypatch.setattr(L, "_here", lambda *t: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    for name in ("write", "read", "attn"):
        with pytest.raises(OverflowError):
            _prepare(name, loop_step=1 << 32)


# ---------------------------------------------------------------- MXCache

def test_requests_counted_from_the_end(monkeypatch):
    """read(-1) names the last request as truncate(-1) does; it used to read no
    request and return memory that nothing had written."""
    c = _cache()
    c.extend([5, 0, 70])
    lays = []
    monkeypatch.setattr(L, "loopvq_mx_read", lambda d, lay, *a: lays.append(lay))
    for r in (2, -1):
        c.read(r, 10, 64)
        lay = lays.pop()
        assert lay.total_new == lay.max_new == 54
        assert [t.tolist() for t in lay._keep[:2]] == [[0, 0, 64], [0, 0, 0, 54]]
    for call in (lambda r: c.read(r), lambda r: c.truncate(r, 0)):
        for r in (3, -4):
            with pytest.raises(IndexError):
                call(r)
    c.truncate(-1, 0)
    assert c.ctx == [5, 0, 0]


def test_a_prompt_beside_a_tree_is_kept(monkeypatch):
    """The kernel takes up to 64 new tokens of a request; a prompt that stays as it
    is, or loses its end, is not sent to it."""
    sent = []
    monkeypatch.setattr(L, "loopvq_mx_keep", lambda d, lay, keep, n, mx, *a: sent.append(
        (keep.tolist(), n.tolist(), mx, lay.max_new, [t.tolist() for t in lay._keep[:2]])))
    c = _cache()
    c.extend([0, 30, 0])
    c.extend([100, 5, 1])
    with pytest.raises(ValueError, match="64"):
        c.keep([[0, 2], [0], [0]])
    assert c.ctx == [100, 35, 1] and not sent
    c.keep([None, [0, 2], None])
    assert sent == [([[-1, -1], [0, 2], [-1, -1]], [0, 2, 0], 2, 5, [[100, 35, 1], [0, 0, 5, 5]])]
    assert c.ctx == [100, 32, 1]
    c.extend([70, 5, 1])
    c.keep([list(range(66)), [4], []])
    assert sent[1:] == [([[-1], [4], [-1]], [0, 1, 0], 1, 5, [[170, 37, 2], [0, 0, 5, 5]])]
    assert c.ctx == [166, 33, 1]


def test_a_steps_arrays_outlive_calls_on_other_streams_and_graphs(monkeypatch):
    """The arrays that extend makes go back to the allocator with the next step.
    Calls on another stream, which may still read them then, are made known to it;
    a graph, which may read them at any time, keeps them."""
    class Stream:
        def __init__(self, number):
            self.cuda_stream = number

    class Array:
        def __init__(self):
            self.on = []

        def record_stream(self, stream):
            self.on.append(stream.cuda_stream)

    now = {"stream": Stream(1), "capturing": False}
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now["stream"])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now["capturing"])
    c = _cache()
    c.extend([3, 0, 0])
    c.device, c.made_on = torch.device("cuda"), 1
    c.layout._keep = [Array() for _ in range(3)]
    assert c._step() is c.layout and all(a.on == [] for a in c.layout._keep)
    now["stream"] = Stream(2)
    c._step()
    assert all(a.on == [2] for a in c.layout._keep) and c.captured == []
    now["capturing"] = True
    c._step()
    c._step()
    assert c.captured == [c.layout] and all(a.on == [2] for a in c.layout._keep)


def test_an_extend_that_fails_changes_nothing(monkeypatch):
    """No memory for the arrays of a step, or a stream that is being captured: the
    cache is as it was, and the same extend may be tried again."""
    c = _cache()
    c.extend([40, 3, 0])
    before = [list(c.ctx), list(c.new), c.rows, [list(p) for p in c.pages], list(c.free), c.layout]

    def fail(*a):
        raise RuntimeError("out of memory")

    with monkeypatch.context() as m:
        m.setattr(L, "make_mx_layout", fail)
        with pytest.raises(RuntimeError, match="out of memory"):
            c.extend([30, 1, 65])
    assert before == [c.ctx, c.new, c.rows, c.pages, c.free, c.layout]
    c.extend([30, 1, 65])
    assert c.ctx == [70, 4, 65] and [len(p) for p in c.pages] == [3, 1, 3] and len(c.free) == 5
    assert sorted(sum(c.pages, []) + c.free) == list(range(12))


def test_idle_steps_take_empty_rows_of_any_strides(monkeypatch):
    """No request has a new token: rows without elements, whose strides mean
    nothing, are no error."""
    calls = []
    monkeypatch.setattr(L, "loopvq_mx_write", lambda d, lay, *a: calls.append(lay.total_new))
    c = _cache()
    c.extend([0, 0, 0])
    empty = torch.zeros(0).as_strided((0, 1, 64), (64, 64, 3))
    c.write(empty, empty, 0)
    assert calls == [0]
    c.extend([1, 0, 0])
    with pytest.raises(ValueError, match="consecutive channels"):
        c.write(torch.zeros((1, 1, 128))[..., ::2], torch.zeros((1, 1, 64)), 0)
