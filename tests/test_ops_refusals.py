"""Refusals of the shared-prefix, weights and eviction entry points, without a GPU: every invalid call returns its
error code before any device work, and the sizes of the workspaces cover every smaller call."""
import ctypes
import itertools
import math
import random

import pytest
import torch

import tree_indexed_sparse_03_b200 as z
from tree_indexed_sparse_03_b200 import zha as zb

P = 1 << 20  # a stand-in address (aligned, never used: every call below is refused first)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from tree_indexed_sparse_03_b200 import build_lib
    build_lib.build()
    return z.lib()


def cfg(**kw):
    base = dict(d=128, n_q_heads=32, n_kv_heads=4, block=4, levels=1, n_refs=1, p=1.0, dtype="bf16", capacity=4096)
    base.update(kw)
    return z.make_config(**base)


def prefix(L, c=None, **kw):
    a = dict(K=P, V=P, ld=1000, n=900, K_own=P, V_own=P, ld_own=64, own_len=P, Q=P, O=P, lse=P, B=2, m=1, scratch=P,
             nbytes=BIG)
    a.update(kw)
    c = c or cfg()
    return L.zha_prefix_decode(ctypes.byref(c), a["K"], a["V"], a["ld"], a["n"], a["K_own"], a["V_own"], a["ld_own"],
                               a["own_len"], a["Q"], a["O"], a["lse"], a["B"], a["m"], a["scratch"], a["nbytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(K=None), zb.ZHA_ERR_INVALID), (dict(V=None), zb.ZHA_ERR_INVALID), (dict(Q=None), zb.ZHA_ERR_INVALID),
    (dict(O=None), zb.ZHA_ERR_INVALID), (dict(scratch=None), zb.ZHA_ERR_INVALID),
    (dict(K_own=None), zb.ZHA_ERR_INVALID), (dict(V_own=None), zb.ZHA_ERR_INVALID),
    (dict(own_len=None), zb.ZHA_ERR_INVALID), (dict(n=-1), zb.ZHA_ERR_INVALID), (dict(n=1001), zb.ZHA_ERR_INVALID),
    (dict(ld=1 << 31), zb.ZHA_ERR_INVALID), (dict(ld_own=-1), zb.ZHA_ERR_INVALID),
    (dict(ld_own=1 << 31), zb.ZHA_ERR_INVALID), (dict(B=0), zb.ZHA_ERR_INVALID), (dict(m=0), zb.ZHA_ERR_INVALID),
    (dict(B=1 << 20), zb.ZHA_ERR_UNSUPPORTED), (dict(B=1 << 30, m=1 << 30), zb.ZHA_ERR_UNSUPPORTED),
    (dict(K=P + 8), zb.ZHA_ERR_INVALID), (dict(V=P + 2), zb.ZHA_ERR_INVALID), (dict(K_own=P + 8), zb.ZHA_ERR_INVALID),
    (dict(Q=P + 4), zb.ZHA_ERR_INVALID), (dict(O=P + 4), zb.ZHA_ERR_INVALID), (dict(lse=P + 2), zb.ZHA_ERR_INVALID),
    (dict(own_len=P + 1), zb.ZHA_ERR_INVALID), (dict(scratch=P + 128), zb.ZHA_ERR_INVALID),
    (dict(nbytes=256), zb.ZHA_ERR_CAPACITY),
])
def test_prefix_refusals(L, kw, code):
    before = L.zha_launch_count()
    assert prefix(L, **kw) == code
    assert L.zha_last_error() and L.zha_launch_count() == before


def test_prefix_refuses_bad_configs(L):
    assert prefix(L, cfg(d=96)) == zb.ZHA_ERR_UNSUPPORTED
    assert prefix(L, cfg(n_q_heads=30)) == zb.ZHA_ERR_UNSUPPORTED
    assert L.zha_prefix_scratch_bytes(ctypes.byref(cfg(d=96)), 1, 1, 10, 0) == 0
    assert L.zha_prefix_scratch_bytes(ctypes.byref(cfg()), 0, 1, 10, 0) == 0
    assert L.zha_weights_scratch_bytes(ctypes.byref(cfg()), 1, 0) == 0
    assert L.zha_prefix_decode(None, P, P, 1, 1, P, P, 1, P, P, P, P, 1, 1, P, BIG, None) == zb.ZHA_ERR_INVALID


def weights(L, c=None, **kw):
    a = dict(K=P, V=P, ld=1000, n=900, Q=P, O=P, m=4, causal=1, acc_in=P, ld_in=900, acc_out=P, ld_out=900, scratch=P,
             nbytes=BIG)
    a.update(kw)
    c = c or cfg()
    return L.zha_dense_weights(ctypes.byref(c), a["K"], a["V"], a["ld"], a["n"], a["Q"], a["O"], a["m"], a["causal"],
                               a["acc_in"], a["ld_in"], a["acc_out"], a["ld_out"], a["scratch"], a["nbytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(K=None), zb.ZHA_ERR_INVALID), (dict(V=None), zb.ZHA_ERR_INVALID), (dict(O=None), zb.ZHA_ERR_INVALID),
    (dict(Q=None), zb.ZHA_ERR_INVALID), (dict(acc_out=None), zb.ZHA_ERR_INVALID),
    (dict(scratch=None), zb.ZHA_ERR_INVALID), (dict(n=0), zb.ZHA_ERR_INVALID), (dict(n=1001), zb.ZHA_ERR_INVALID),
    (dict(m=0), zb.ZHA_ERR_INVALID), (dict(m=901), zb.ZHA_ERR_INVALID), (dict(causal=2), zb.ZHA_ERR_INVALID),
    (dict(ld_in=899), zb.ZHA_ERR_INVALID), (dict(ld_out=899), zb.ZHA_ERR_INVALID),
    (dict(acc_in=P + 4), zb.ZHA_ERR_INVALID),               # overlaps acc_out without being it
    (dict(ld_in=950), zb.ZHA_ERR_INVALID),                  # the same buffer with another stride
    (dict(K=P + 8), zb.ZHA_ERR_INVALID), (dict(acc_out=P + 2), zb.ZHA_ERR_INVALID),
    (dict(m=1 << 20, causal=0), zb.ZHA_ERR_UNSUPPORTED), (dict(scratch=P + 16), zb.ZHA_ERR_INVALID),
    (dict(nbytes=512), zb.ZHA_ERR_CAPACITY),
])
def test_weights_refusals(L, kw, code):
    before = L.zha_launch_count()
    assert weights(L, **kw) == code
    assert L.zha_last_error() and L.zha_launch_count() == before


def evict(L, c=None, **kw):
    MB = 1 << 20
    a = dict(K=P, V=P + 16 * MB, ld=1000, n=900, acc=P + 32 * MB, ld_acc=900, keep=100, first=4, last=8,
             K_out=P + 48 * MB, V_out=P + 64 * MB, ld_out=100, acc_out=P + 80 * MB, ld_acc_out=100, idx=P + 96 * MB, scratch=P + 112 * MB, nbytes=BIG)
    a.update(kw)
    c = c or cfg()
    return L.zha_cache_evict(ctypes.byref(c), a["K"], a["V"], a["ld"], a["n"], a["acc"], a["ld_acc"], a["keep"],
                             a["first"], a["last"], a["K_out"], a["V_out"], a["ld_out"], a["acc_out"],
                             a["ld_acc_out"], a["idx"], a["scratch"], a["nbytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(K=None), zb.ZHA_ERR_INVALID), (dict(V_out=None), zb.ZHA_ERR_INVALID), (dict(acc=None), zb.ZHA_ERR_INVALID),
    (dict(idx=None), zb.ZHA_ERR_INVALID), (dict(n=1001), zb.ZHA_ERR_INVALID), (dict(n=0, keep=0), zb.ZHA_ERR_INVALID),
    (dict(keep=0), zb.ZHA_ERR_INVALID), (dict(keep=901), zb.ZHA_ERR_INVALID), (dict(first=-1), zb.ZHA_ERR_INVALID),
    (dict(last=-1), zb.ZHA_ERR_INVALID), (dict(first=50, last=51), zb.ZHA_ERR_INVALID),
    (dict(first=2 ** 62, last=2 ** 62), zb.ZHA_ERR_INVALID), (dict(ld_acc=899), zb.ZHA_ERR_INVALID),
    (dict(ld_out=99), zb.ZHA_ERR_INVALID), (dict(ld_acc_out=99), zb.ZHA_ERR_INVALID),
    (dict(K_out=P, ld_out=500), zb.ZHA_ERR_INVALID),        # in place with another row stride
    (dict(K_out=P + 256), zb.ZHA_ERR_INVALID),              # shifted by one row
    (dict(V_out=P), zb.ZHA_ERR_INVALID),                    # V over K
    (dict(V_out=P + (48 << 20)), zb.ZHA_ERR_INVALID),       # two outputs in one place
    (dict(idx=P + (32 << 20)), zb.ZHA_ERR_INVALID),         # the list over the sums
    (dict(K=P + 8), zb.ZHA_ERR_INVALID), (dict(acc_out=P + (80 << 20) + 2), zb.ZHA_ERR_INVALID),
    (dict(n=50000, ld=50000, ld_acc=50000, scratch=None, acc=P + (1 << 30), K_out=P + (2 << 30), V=P + (3 << 30),
          V_out=P + (4 << 30)), zb.ZHA_ERR_INVALID),        # a long cache needs its workspace
    (dict(n=50000, ld=50000, ld_acc=50000, nbytes=1024, acc=P + (1 << 30), K_out=P + (2 << 30), V=P + (3 << 30),
          V_out=P + (4 << 30)), zb.ZHA_ERR_CAPACITY),
])
def test_evict_refusals(L, kw, code):
    before = L.zha_launch_count()
    assert evict(L, **kw) == code
    assert L.zha_last_error() and L.zha_launch_count() == before


def test_evict_workspace_grows_with_the_cache(L):
    ref = ctypes.byref(cfg())
    sizes = [L.zha_evict_scratch_bytes(ref, n) for n in (1, 16384, 16385, 40961, 300000, 1 << 20, (1 << 31) - 1)]
    assert sizes[0] == sizes[1] == 0 and sizes[2] > 4 * 3 * 2048 * 4 and sizes == sorted(sizes)
    assert L.zha_evict_scratch_bytes(ref, 0) == 0 and L.zha_evict_scratch_bytes(ref, 1 << 31) == 0


def test_tree_evict_and_status_refuse_null(L):
    assert L.zha_tree_evict(None, P, 10, 5, 0, 0, P, None, 0, None) == zb.ZHA_ERR_INVALID
    assert L.zha_scratch_status(None, None) == zb.ZHA_ERR_INVALID


def test_bindings_refuse_host_tensors_and_wrong_shapes(L):
    c = cfg(d=64, n_q_heads=4, n_kv_heads=2)
    bf = torch.bfloat16
    K = torch.zeros(2, 16, 64, dtype=bf)
    Q = torch.zeros(3, 4, 64, dtype=bf)
    dec = zb.PrefixDecoder.__new__(zb.PrefixDecoder)
    dec.cfg = c
    with pytest.raises(ValueError):
        dec(K, K, 16, Q)
    w = zb.DenseWeights.__new__(zb.DenseWeights)
    w.cfg = c
    with pytest.raises(ValueError):
        w(K, K, 16, Q)
    with pytest.raises(ValueError):
        z.cache_evict(c, K, K.clone(), 16, torch.zeros(2, 16), 4)


@pytest.mark.parametrize("d,hq,hkv,dtype", [(128, 32, 4, "bf16"), (64, 6, 2, "bf16"), (128, 5, 5, "f32"), (64, 8, 1, "f32")])
def test_workspaces_cover_smaller_calls(L, d, hq, hkv, dtype):
    """A workspace sized for (B, m, n, own) serves every call with no more of each (the sizes themselves are what a
    call of that size is checked against, so covering is: never smaller than a smaller call's)."""
    c = cfg(d=d, n_q_heads=hq, n_kv_heads=hkv, dtype=dtype)
    ref = ctypes.byref(c)
    Bs, ms, ns, owns = (1, 2, 3, 9, 40, 64), (1, 2, 5, 8), (0, 1, 65, 777, 20000, 262144), (0, 1, 64, 129, 1024)
    size = {k: L.zha_prefix_scratch_bytes(ref, *k) for k in itertools.product(Bs, ms, ns, owns)}
    for (B, m, n, o), s in size.items():
        assert s > 256
        for k in ((Bs[max(0, Bs.index(B) - 1)], m, n, o), (B, ms[max(0, ms.index(m) - 1)], n, o),
                  (B, m, ns[max(0, ns.index(n) - 1)], o), (B, m, n, owns[max(0, owns.index(o) - 1)])):
            assert size[k] <= s, (k, (B, m, n, o))
    ms, ns = (1, 2, 7, 33, 64, 1000, 4099), (1, 63, 65, 777, 4099, 65536, 300000)
    size = {k: L.zha_weights_scratch_bytes(ref, *k) for k in itertools.product(ms, ns)}
    for (m, n), s in size.items():
        assert s > 256
        for k in ((ms[max(0, ms.index(m) - 1)], n), (m, ns[max(0, ns.index(n) - 1)])):
            assert size[k] <= s, (k, (m, n))


def test_workspace_requests_that_are_refused_keep_their_code(L):
    """The size functions answer 0 for a request that no call would take; the classes raise what the call would return."""
    with pytest.raises(z.ZhaError) as e:
        z.PrefixDecoder(cfg(), 1 << 20, 100)
    assert e.value.code == zb.ZHA_ERR_UNSUPPORTED and "2^24" in str(e.value)
    with pytest.raises(z.ZhaError) as e:
        z.DenseWeights(cfg(d=96), 1, 100)
    assert e.value.code == zb.ZHA_ERR_UNSUPPORTED and "head dim" in str(e.value)
    with pytest.raises(z.ZhaError) as e:
        z.PrefixDecoder(cfg(), 0, 100)
    assert e.value.code == zb.ZHA_ERR_INVALID
    with pytest.raises(z.ZhaError) as e:
        z.DenseWeights(cfg(), 1, 0)
    assert e.value.code == zb.ZHA_ERR_INVALID
    assert L.zha_last_error_code() == zb.ZHA_ERR_INVALID
    assert evict(L, nbytes=0, n=50000, ld=50000, ld_acc=50000, acc=P + (1 << 30), K_out=P + (2 << 30), V=P + (3 << 30),
                 V_out=P + (4 << 30)) == L.zha_last_error_code() == zb.ZHA_ERR_CAPACITY


@pytest.mark.parametrize("d,hq,hkv,dtype", [(128, 32, 4, "bf16"), (64, 6, 2, "bf16"), (64, 300, 2, "bf16"),
                                            (128, 5, 5, "f32"), (64, 8, 1, "f32"), (64, 96, 3, "f32")])
def test_workspaces_hold_what_calls_need(L, d, hq, hkv, dtype):
    """A workspace of the size that one shape asks for passes the check of every call with no more of anything: the
    call's own need, not the size function, decides.  A misaligned result, looked at after the workspace, keeps every
    call from reaching the device."""
    c = cfg(d=d, n_q_heads=hq, n_kv_heads=hkv, dtype=dtype)
    ref = ctypes.byref(c)
    rng = random.Random(5)

    def log(lo, hi):
        return min(hi, int(lo + math.exp(rng.uniform(0, math.log(hi - lo + 1))) - 1))

    for _ in range(4000):
        big = (log(1, 130), log(1, 40), log(0, 400000), rng.choice([0, log(1, 3000)]))
        if rng.random() < 0.3:
            small = big
        else:
            small = tuple(log(min(lo, b), b) if rng.random() < 0.7 else b for lo, b in zip((1, 1, 0, 0), big))
        size = L.zha_prefix_scratch_bytes(ref, *big)
        assert size > 0
        B, m, n, own = small
        args = dict(B=B, m=m, n=n, ld=n, ld_own=own, lse=P + 2)
        assert prefix(L, c, nbytes=size, **args) == zb.ZHA_ERR_INVALID, (small, big, L.zha_last_error())
        assert b"aligned" in L.zha_last_error()
        assert prefix(L, c, nbytes=300, **args) == zb.ZHA_ERR_CAPACITY
    for _ in range(4000):
        big = (log(1, 5000), log(1, 400000))
        small = big if rng.random() < 0.3 else (log(1, big[0]), log(1, big[1]))
        size = L.zha_weights_scratch_bytes(ref, *big)
        assert size > 0
        m, n = small
        args = dict(m=m, n=n, ld=n, ld_in=n, ld_out=n, causal=0, acc_out=P + 2)
        assert weights(L, c, nbytes=size, **args) == zb.ZHA_ERR_INVALID, (small, big, L.zha_last_error())
        assert b"aligned" in L.zha_last_error()
