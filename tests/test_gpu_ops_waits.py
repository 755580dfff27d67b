"""Waits of the tensor-core kernels that run out: ZHA_ERR_TIMEOUT through the workspace's status word, and the workspace
and the context as good as before.

ZHA_WAIT_CYCLES (read by every call) bounds the waits on copies and matrix products: 0 makes a wait that is not over at
its first look give up, larger bounds let the roles of a CTA get further before they leave.  Every role then waits, with
a bound of its own, for the copies and products it has in flight.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import tree_indexed_sparse_03_b200 as z
    from tree_indexed_sparse_03_b200 import zha as zb

BOUNDS = [0, 300, 1000, 3000, 10000, 30000]


def cfg_of(d, hkv, group, capacity=1 << 20):
    return z.make_config(d=d, n_q_heads=hkv * group, n_kv_heads=hkv, block=4, levels=1, n_refs=1, p=1.0, dtype="bf16",
                         capacity=capacity)


def rnd(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def run_out(dec, call, monkeypatch, bound):
    """One call under the bound; its status is TIMEOUT for a bound of 0, TIMEOUT or fine for the others."""
    monkeypatch.setenv("ZHA_WAIT_CYCLES", str(bound))
    call()
    monkeypatch.delenv("ZHA_WAIT_CYCLES")
    torch.cuda.synchronize()
    try:
        dec.status()
        assert bound > 0
    except z.ZhaError as e:
        assert e.code == zb.ZHA_ERR_TIMEOUT
    dec.status()  # looking cleared it


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,group,B,m,n,own", [(2, 4, 3, 1, 900, 300), (1, 8, 40, 1, 5000, 200), (1, 8, 40, 8, 400001, 70)])
def test_prefix_waits_that_run_out(monkeypatch, d, hkv, group, B, m, n, own):
    """Own caches that end inside a tile, shared and separate rows of the two streams, shares long enough for the
    accumulator to leave tensor memory."""
    K, V, Q = rnd(1, hkv, n, d), rnd(2, hkv, n, d), rnd(3, B, m, hkv * group, d, scale=2.0)
    Ko, Vo = rnd(4, B, hkv, own, d), rnd(5, B, hkv, own, d)
    ln = torch.tensor([own - (b * 37) % own for b in range(B)], dtype=torch.int32, device="cuda")
    dec = z.PrefixDecoder(cfg_of(d, hkv, group), B, n, own, m)
    want, lse = dec(K, V, n, Q, Ko, Vo, ln, want_lse=True)
    torch.cuda.synchronize()
    dec.status()
    for bound in BOUNDS:
        run_out(dec, lambda: dec(K, V, n, Q, Ko, Vo, ln, want_lse=True), monkeypatch, bound)
        o, l = dec(K, V, n, Q, Ko, Vo, ln, want_lse=True)
        torch.cuda.synchronize()
        dec.status()
        assert torch.equal(o, want) and torch.equal(l, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("outputs", [True, False])
@pytest.mark.parametrize("hkv,group,m,n", [(2, 4, 1, 900), (2, 4, 33, 900), (1, 8, 300, 3000), (2, 150, 5, 700)])
def test_weights_waits_that_run_out(monkeypatch, d, outputs, hkv, group, m, n):
    K, V, Q = rnd(1, hkv, n, d), rnd(2, hkv, n, d), rnd(3, m, hkv * group, d, scale=2.0)
    dec = z.DenseWeights(cfg_of(d, hkv, group), m, n)

    def call():
        return dec(K, V if outputs else None, n, Q, causal=True)

    want = call()
    torch.cuda.synchronize()
    dec.status()
    for bound in BOUNDS:
        run_out(dec, call, monkeypatch, bound)
        got = call()
        torch.cuda.synchronize()
        dec.status()
        assert torch.equal(got[1], want[1]) and (not outputs or torch.equal(got[0], want[0]))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("outputs", [True, False])
@pytest.mark.parametrize("hkv,group,m,n", [(2, 4, 1, 900), (2, 4, 33, 901), (1, 8, 300, 3000), (2, 150, 5, 700)])
def test_sums_in_place_survive_a_wait_that_runs_out(monkeypatch, d, outputs, hkv, group, m, n):
    """Running sums that a call adds to in place are all as they were when one of its waits ran out, and stay so until
    the status has been looked at; all complete otherwise."""
    K, V, Q = rnd(1, hkv, n, d), rnd(2, hkv, n, d), rnd(3, m, hkv * group, d, scale=2.0)
    before = torch.rand(hkv, n + 3, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    dec = z.DenseWeights(cfg_of(d, hkv, group), m, n)
    after = before.clone()
    after[:, :n] = dec(K, V if outputs else None, n, Q, before, causal=True)[1]
    for bound in BOUNDS:
        acc = before.clone()

        def call():
            dec(K, V if outputs else None, n, Q, acc, causal=True, acc_out=acc)

        monkeypatch.setenv("ZHA_WAIT_CYCLES", str(bound))
        call()
        monkeypatch.delenv("ZHA_WAIT_CYCLES")
        if bound == 0:
            call()  # nobody has looked
        torch.cuda.synchronize()
        try:
            dec.status()
            assert bound > 0 and torch.equal(acc, after)
        except z.ZhaError as e:
            assert e.code == zb.ZHA_ERR_TIMEOUT and torch.equal(acc, before)
            call()
            torch.cuda.synchronize()
            dec.status()
            assert torch.equal(acc, after)
