"""Host side of the 8-bit cache's binding on CPU tensors, with a library that records its calls and launches nothing."""

import contextlib
import threading
import time
from types import SimpleNamespace

import pytest
import torch

from block_sparse_long_dual_b200 import sfa

CPU = torch.device("cpu")


class Library:
    """Stands for libsfa.so: keeps (name, arguments) of every call; sizes are 256 bytes."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 256 if name.endswith("_workspace") else 0
        return call


class Graph:
    """Stands for a CUDA graph: replaying repeats the library calls recorded while it was captured."""

    def replay(self):
        self.lib.calls += self.held


@pytest.fixture
def lib(monkeypatch):
    lib = Library()

    @contextlib.contextmanager
    def capture(graph):
        n = len(lib.calls)
        yield
        graph.lib, graph.held = lib, lib.calls[n:]
        del lib.calls[n:]

    stream = SimpleNamespace(device=CPU, cuda_stream=0, wait_stream=lambda other: None)
    monkeypatch.setattr(sfa, "load", lambda: lib)
    monkeypatch.setattr(sfa, "_cuda", lambda t, name: None)
    monkeypatch.setattr(sfa, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "Stream", lambda device=None: stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "CUDAGraph", Graph)
    monkeypatch.setattr(torch.cuda, "graph", capture)
    return lib


def cache(block=128, **share):
    c = sfa.KvCache8.empty(batch=1, heads_kv=2, capacity=256, head_dim=64, block=block, weight=False, device="cpu")
    if not share:
        return c
    held = dict(k=c.k, v=c.v, k_scale=c.k_scale, v_scale=c.v_scale, lens=c.lens)
    return sfa.KvCache8(**{**held, **share}, block=block)


def decoder():
    return sfa.FasaDecode(batch=1, heads_q=4, heads_kv=2, seq_len=256, head_dim=64, fc=[[0, 1, 2, 3]] * 2, k=8,
                          device="cpu")


def q():
    return torch.zeros((1, 4, 64), dtype=torch.bfloat16)


# ---------------------------------------------------------------------------
# the graph step of the selecting decoder
# ---------------------------------------------------------------------------
def read_by(lib, since):
    """What the calls from `since` on read of a cache: {call: its sfa_cache8 fields}."""
    out = {}
    for name, args in lib.calls[since:]:
        if name in ("sfa_cache8_fc_gather", "sfa_cache8_attn_list"):
            c = args[1]._obj
            out[name] = (c.k, c.v, c.k_scale, c.v_scale, c.lens, c.block)
    return out


@pytest.mark.parametrize("other", ["k_scale", "v_scale", "lens", "k", "v", "block"])
def test_a_step_never_replays_the_graph_of_another_cache(lib, other):
    """Two handles that share every tensor but one (or, with another block, all but the scales)."""
    m, a, x = decoder(), cache(), q()
    share = {n: getattr(a, n) for n in ("k", "v", "k_scale", "v_scale", "lens") if n != other}
    if other == "block":
        for n in ("k_scale", "v_scale"):  # the larger array's start: the same address for both handles
            big = torch.ones((1, 2, 4))
            share[n] = big
            setattr(a, n, torch.as_strided(big, (1, 2, 2), (4, 2, 1)))
        a = sfa.KvCache8(k=a.k, v=a.v, k_scale=a.k_scale, v_scale=a.v_scale, lens=a.lens)
    b = cache(block=64 if other == "block" else 128, **share)
    for c in (a, b, a, b):
        n = len(lib.calls)
        m.step(x, c, pos=3)
        want = (c.k.data_ptr(), c.v.data_ptr(), c.k_scale.data_ptr(), c.v_scale.data_ptr(), c.lens.data_ptr(), c.block)
        assert read_by(lib, n) == {"sfa_cache8_fc_gather": want, "sfa_cache8_attn_list": want}


def test_a_step_with_the_same_buffers_replays_one_graph(lib, monkeypatch):
    made = []
    monkeypatch.setattr(torch.cuda, "CUDAGraph", lambda: made.append(Graph()) or made[-1])
    m, a, x = decoder(), cache(), q()
    for _ in range(3):
        m.step(x, a, pos=3)
    again = sfa.KvCache8(k=a.k, v=a.v, k_scale=a.k_scale, v_scale=a.v_scale, lens=a.lens)
    m.step(x, again, pos=3)
    assert len(made) == 1
    m.step(x, a, pos=4)
    assert len(made) == 2


def test_a_step_checks_queries_of_another_shape_at_the_same_address(lib):
    m, a = decoder(), cache()
    big = torch.zeros(512, dtype=torch.bfloat16)
    m.step(big[:256].view(1, 4, 64), a, pos=3)
    with pytest.raises(ValueError, match="q must be"):
        m.step(big.view(1, 4, 128), a, pos=3)


# ---------------------------------------------------------------------------
# what the selecting decoder refuses
# ---------------------------------------------------------------------------
def test_a_missing_value_cache_or_position_is_named(lib):
    m, x, K = decoder(), q(), torch.zeros((1, 2, 256, 64), dtype=torch.bfloat16)
    for call in (lambda: m(x, K), lambda: m.attend(x, K), lambda: m.step(x, K, pos=3)):
        with pytest.raises(TypeError, match="V_cache"):
            call()
    for call in (lambda: m.step(x, K, K), lambda: m.step(x, cache())):
        with pytest.raises(TypeError, match="pos"):
            call()
    assert not lib.calls or {n for n, _ in lib.calls} == {"sfa_decode_workspace"}


def test_a_position_before_the_cache_is_the_librarys_to_refuse(lib, monkeypatch):
    """As for every other caller of the compact-key copy: SFA_ERR_INVALID_ARG, whichever cache is given."""
    m, x, K = decoder(), q(), torch.zeros((1, 2, 256, 64), dtype=torch.bfloat16)
    for name in ("sfa_decode_fc_gather", "sfa_cache8_fc_gather"):
        monkeypatch.setattr(lib, name, lambda s, c, fc, nfc, pos0, *rest: 1 if pos0 < 0 else 0, raising=False)
    for call in (lambda: m.step(x, K, K, -1), lambda: m.step(x, cache(), pos=-1)):
        with pytest.raises(sfa.SfaError, match="SFA_ERR_INVALID_ARG"):
            call()


# ---------------------------------------------------------------------------
# host threads
# ---------------------------------------------------------------------------
def together(lib, name, word, calls):
    """Runs the calls in a thread each; every library call `name` lasts a while.  The largest number of them that
    were under way at once with the same `word` (an argument)."""
    inside, most, guard = {}, [0], threading.Lock()

    def slow(*args):
        at = word(args)
        with guard:
            inside[at] = inside.get(at, 0) + 1
            most[0] = max(most[0], inside[at])
        time.sleep(0.02)
        with guard:
            inside[at] -= 1
        return 0

    setattr(lib, name, slow)
    start = threading.Barrier(len(calls))
    threads = [threading.Thread(target=lambda f=f: (start.wait(), f())) for f in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return most[0]


def test_threads_never_share_the_handles_workspace(lib):
    """An attention is two launches with the partial results of one in the workspace: a second thread's call on the
    same stream must not get between them."""
    c = cache()
    assert together(lib, "sfa_cache8_attn", lambda args: args[10], [lambda: c.attend(q())] * 6) == 1


def test_threads_append_one_after_the_other(lib):
    """An append at the lengths is two launches, which read and then advance them."""
    c, rows = cache(), torch.zeros((1, 2, 1, 64), dtype=torch.bfloat16)
    assert together(lib, "sfa_cache8_append", lambda args: 0, [lambda: c.append(rows, rows)] * 6) == 1


# ---------------------------------------------------------------------------
# the eviction's list
# ---------------------------------------------------------------------------
def evicting(keep=5, **kw):
    src = sfa.KvCache8.empty(batch=1, heads_kv=2, capacity=256, head_dim=64, device="cpu")
    dst = sfa.KvCache8.empty(batch=1, heads_kv=2, capacity=64, head_dim=64, device="cpu")
    return sfa.cache8_evict(src, dst, keep=keep, **kw)


def test_an_eviction_without_a_list_works_in_the_workspace_it_is_given(lib):
    ws = torch.zeros(255, dtype=torch.uint8)
    got = evicting(workspace=ws)
    name, args = lib.calls[-1]
    assert name == "sfa_cache8_evict" and args[6] is None and args[7] == ws.data_ptr() and args[8] == 255
    assert got.shape == (1, 2, 5) and got.dtype == torch.int32 and got.data_ptr() == ws.data_ptr()
    idx = torch.zeros((1, 2, 5), dtype=torch.int32)
    assert evicting(idx=idx, workspace=ws) is idx and lib.calls[-1][1][6] == idx.data_ptr()
    own = evicting()
    assert lib.calls[-1][1][6] == own.data_ptr() and own.shape == (1, 2, 5)
