"""The 8-bit cache's calls refuse bad arguments on the host, before any launch (no GPU needed)."""

import ctypes

import pytest
import torch

from block_sparse_long_dual_b200 import build as sfa_build
from block_sparse_long_dual_b200 import sfa

P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    sfa_build.build()
    return sfa.load()


def S(B=2, Hq=8, Hkv=2, L=1000, d=128, dt=sfa.BF16):
    return sfa.Shape(B, Hq, Hkv, L, d, dt)


def C(block=128, **kw):
    a = dict(k=1 << 30, v=2 << 30, k_scale=3 << 30, v_scale=(3 << 30) + (1 << 20), lens=(3 << 30) + (2 << 20),
             weight=(3 << 30) + (4 << 20))
    a.update(kw)
    return sfa.Cache8(a["k"], a["v"], a["k_scale"], a["v_scale"], a["lens"], a["weight"], block)


def append(lib, s=None, c=None, K=P, V=P, n=4, at=None, counts=None):
    return lib.sfa_cache8_append(ctypes.byref(s or S()), ctypes.byref(c or C()), K, V, n, at, counts, None, None)


def attn(lib, s=None, c=None, q=P, nq=1, back=0, scale=0.0, o=P, w_in=None, w_out=None, ws=P, nbytes=1 << 40):
    return lib.sfa_cache8_attn(ctypes.byref(s or S()), ctypes.byref(c or C()), q, nq, back, scale, o, None, w_in,
                               w_out, ws, nbytes, None, None)


def lst(lib, s=None, c=None, q=P, idx=P, k=4, scale=0.0, o=P):
    return lib.sfa_cache8_attn_list(ctypes.byref(s or S()), ctypes.byref(c or C()), q, idx, k, scale, o, None, None,
                                    None)


def dst(**kw):
    a = dict(k=5 << 30, v=6 << 30, k_scale=7 << 30, v_scale=(7 << 30) + (1 << 20), lens=(7 << 30) + (2 << 20),
             weight=(7 << 30) + (4 << 20))
    a.update(kw)
    return C(**a)


def evict(lib, s=None, a=None, b=None, dl=200, keep=100, recent=10, idx=P, ws=None, n=0):
    return lib.sfa_cache8_evict(ctypes.byref(s or S()), ctypes.byref(a or C()), ctypes.byref(b or dst()), dl, keep,
                                recent, idx, ws, n, None, None)


@pytest.mark.parametrize("s,code", [
    (S(dt=sfa.F32), 3), (S(d=96), 2), (S(B=0), 2), (S(L=0), 2), (S(Hq=6, Hkv=4), 2), (S(Hq=6, Hkv=2), 4),
    (S(B=1 << 12, Hkv=8, L=1 << 16), 4),
])
def test_shapes(lib, s, code):
    assert attn(lib, s=s) == code and lst(lib, s=s) == code
    assert lib.sfa_cache8_attn_workspace(ctypes.byref(s), 1, 0) == 0
    if s.heads_q % s.heads_kv == 0 and s.heads_q // s.heads_kv != 3:  # the calls without q ignore heads_q
        assert append(lib, s=s) == code and evict(lib, s=s) == code


def test_blocks_and_arrays(lib):
    for call in (append, attn, lst):
        assert call(lib, c=C(block=96)) == 2
        for name in ("k", "v", "k_scale", "v_scale", "lens"):
            assert call(lib, c=C(**{name: None})) == 1
        assert call(lib, c=C(k=(1 << 30) + 8)) == 1


def test_append(lib):
    assert append(lib, K=None) == 1 and append(lib, V=None) == 1 and append(lib, n=0) == 1
    assert append(lib, K=P + 2) == 1
    assert append(lib, at=(3 << 30) + (2 << 20) + 4) == 1   # positions inside the lengths
    assert append(lib, counts=(3 << 30) + (2 << 20)) == 1


def test_attn(lib):
    assert attn(lib, q=None) == 1 and attn(lib, o=None) == 1 and attn(lib, q=P + 4) == 1
    assert attn(lib, nq=0) == 1 and attn(lib, back=-1) == 1 and attn(lib, scale=float("nan")) == 1
    assert attn(lib, nq=5) == 4                       # 4 heads x 5 queries > 16 rows
    assert attn(lib, w_in=P) == 1                     # nowhere to add to
    need = lib.sfa_cache8_attn_workspace(ctypes.byref(S()), 1, 0)
    more = lib.sfa_cache8_attn_workspace(ctypes.byref(S()), 1, 1)
    assert more >= need + 2 * 2 * 4 * 1000 * 4        # the scores of every query row
    assert attn(lib, ws=None) == 5 and attn(lib, nbytes=need - 1) == 5 and attn(lib, ws=P + 16) == 5
    assert attn(lib, w_out=P, nbytes=need) == 5
    assert lib.sfa_cache8_attn_workspace(ctypes.byref(S()), 0, 0) == 0
    assert lib.sfa_cache8_attn_workspace(ctypes.byref(S()), 5, 0) == 0


def test_list(lib):
    assert lst(lib, q=None) == 1 and lst(lib, idx=None) == 1 and lst(lib, o=None) == 1
    assert lst(lib, k=0) == 1 and lst(lib, scale=float("inf")) == 1


def test_evict(lib):
    assert evict(lib, keep=0) == 1 and evict(lib, recent=-1) == 1 and evict(lib, recent=101) == 1
    assert evict(lib, dl=99) == 1
    assert evict(lib, a=C(weight=None)) == 1
    assert evict(lib, b=dst(block=64)) == 2
    assert evict(lib, b=dst(k=(1 << 30) + 64)) == 1      # into the source's keys
    assert evict(lib, b=dst(lens=(3 << 30) + (2 << 20))) == 1
    assert evict(lib, idx=(1 << 30) + 1024) == 1 and evict(lib, idx=(7 << 30) - 16) == 1  # the list in a cache
    need = lib.sfa_cache8_evict_workspace(ctypes.byref(S()), 100)
    assert evict(lib, idx=None, ws=6 << 30, n=need) == 1
    assert need >= 2 * 2 * 100 * 4
    assert evict(lib, idx=None) == 5 and evict(lib, idx=None, ws=P, n=need - 1) == 5
    assert lib.sfa_cache8_evict_workspace(ctypes.byref(S()), 0) == 0


def test_gather(lib):
    f = lib.sfa_cache8_fc_gather
    fc = (ctypes.c_int * 8)(0, 5, 9, 63, 1, 2, 3, 4)
    s, c = ctypes.byref(S()), ctypes.byref(C())
    assert f(s, c, None, 4, 0, 10, P, None) == 1 and f(s, c, fc, 4, 0, 10, None, None) == 1
    assert f(s, c, fc, 3, 0, 10, P, None) == 1 and f(s, c, fc, 4, 995, 6, P, None) == 1
    assert f(s, c, fc, 4, -1, 6, P, None) == 1
    assert f(s, c, (ctypes.c_int * 8)(0, 5, 5, 6, 1, 2, 3, 4), 4, 0, 10, P, None) == 1


def test_binding_checks_the_cache_tensors():
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        sfa.KvCache8(k=z((1, 1, 64, 64)).to(torch.float8_e4m3fn), v=None, k_scale=None, v_scale=None, lens=None)
    with pytest.raises(ValueError, match=r"\[B, Hkv, capacity, d\]"):
        sfa.KvCache8(k=z((64, 64)), v=None, k_scale=None, v_scale=None, lens=None)
