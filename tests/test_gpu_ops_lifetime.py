"""What a call on another stream uses may be dropped as soon as the call returns: its memory is handed out again only once
that stream is done."""
import pytest
import torch

from synth.workloads import random_tree_case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import tree_indexed_sparse_03_b200 as z

D, HKV, G, N, B, OWN = 64, 2, 4, 3000, 3, 200


def cfg_of(dtype="bf16"):
    return z.make_config(d=D, n_q_heads=HKV * G, n_kv_heads=HKV, block=4, levels=1, n_refs=1, p=1.0, dtype=dtype,
                         capacity=N)


def rnd(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def busy():
    """A stream that is busy for about half a second."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(1_000_000_000)
    return s


def overwrite(sizes, places):
    """New tensors of the sizes, filled with NaN bits: none lies where the dropped ones were."""
    new = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    for t in new:
        t.fill_(0xFF)
    spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in new]
    assert not any(lo < p + n and p < hi for lo, hi in spans for p, n in places)
    return new


def places_of(*tensors):
    return [(t.data_ptr(), t.numel() * t.element_size()) for t in tensors]


@pytest.mark.parametrize("how", ["argument", "current"])
def test_decoder_dropped_while_its_stream_runs(how):
    K, V, Q = rnd(1, HKV, N, D), rnd(2, HKV, N, D), rnd(3, B, 1, HKV * G, D, scale=2.0)
    want = z.PrefixDecoder(cfg_of(), B, N)(K, V, N, Q)
    torch.cuda.synchronize()
    dec = z.PrefixDecoder(cfg_of(), B, N)
    s = busy()
    if how == "argument":
        o = dec(K, V, N, Q, stream=s)
    else:
        with torch.cuda.stream(s):
            o = dec(K, V, N, Q)
    places = places_of(dec.scratch)
    del dec
    keep = overwrite([n for _, n in places], places)
    assert not s.query()
    s.synchronize()
    assert torch.equal(o, want) and keep


def test_prefix_inputs_dropped_while_the_stream_runs():
    def inputs():
        return (rnd(1, HKV, N, D), rnd(2, HKV, N, D), N, rnd(3, B, 1, HKV * G, D, scale=2.0), rnd(4, B, HKV, OWN, D),
                rnd(5, B, HKV, OWN, D), torch.tensor([OWN, 3, 90], dtype=torch.int32, device="cuda"))
    dec = z.PrefixDecoder(cfg_of(), B, N, OWN)
    want = dec(*inputs())
    args = inputs()
    torch.cuda.synchronize()
    s = busy()
    o = dec(*args, stream=s)
    places = places_of(*(t for t in args if isinstance(t, torch.Tensor)))
    del args
    keep = overwrite([n for _, n in places], places)
    assert not s.query()
    s.synchronize()
    assert torch.equal(o, want) and keep


def test_weights_temporary_and_inputs():
    def inputs():
        return rnd(1, HKV, N, D), rnd(2, HKV, N, D), N, rnd(3, 30, HKV * G, D, scale=2.0), torch.ones(HKV, N, device="cuda")
    want = z.DenseWeights(cfg_of(), 30, N)(*inputs(), causal=True)
    args = inputs()
    dec = z.DenseWeights(cfg_of(), 30, N)
    torch.cuda.synchronize()
    s = busy()
    o, a = dec(*args, causal=True, stream=s)
    places = places_of(dec.scratch, *(t for t in args if isinstance(t, torch.Tensor)))
    del dec, args
    keep = overwrite([n for _, n in places], places)
    assert not s.query()
    s.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(a, want[1]) and keep


def test_evict_inputs_dropped_while_the_stream_runs():
    n, keep_n = 20000, 700  # long enough for a workspace

    def inputs():
        g = torch.Generator(device="cuda").manual_seed(6)
        return rnd(1, HKV, n, D), rnd(2, HKV, n, D), n, torch.rand(HKV, n, generator=g, device="cuda"), keep_n
    outs = [torch.zeros(HKV, keep_n, D, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    want = z.cache_evict(cfg_of(), *inputs(), K_out=outs[0], V_out=outs[1])
    args = inputs()
    torch.cuda.synchronize()
    s = busy()
    idx, acc = z.cache_evict(cfg_of(), *args, K_out=outs[2], V_out=outs[3], stream=s)
    places = places_of(*(t for t in args if isinstance(t, torch.Tensor)))
    del args
    keep = overwrite([m for _, m in places], places)
    assert not s.query()
    s.synchronize()
    assert torch.equal(idx, want[0]) and torch.equal(acc, want[1]) and keep
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])


def test_tree_dropped_while_its_eviction_runs():
    n, keep_n = 3000, 800
    K, V, refs, _ = random_tree_case(21, n_tokens=n, d=128, n_q_heads=8, n_kv_heads=1, n_refs=4, batch=1, dtype="bf16")
    cfg = z.make_config(d=128, n_q_heads=8, n_kv_heads=1, block=4, levels=3, n_refs=4, p=0.9, dtype="bf16", capacity=n)
    sums = torch.rand(1, n, generator=torch.Generator().manual_seed(2))

    def tree():
        t = z.ZhaTree(cfg, K.cuda(), V.cuda(), refs.cuda())
        t.build(n)
        return t
    want = tree().evict(sums.cuda(), keep_n, first=1, last=10)
    t, acc = tree(), sums.cuda()
    torch.cuda.synchronize()
    s = busy()
    idx = t.evict(acc, keep_n, first=1, last=10, stream=s)
    places = places_of(acc, t.K, t.V, t.refs, t.nodes, t.scratch)
    del t, acc
    keep = overwrite([m for _, m in places], places)
    assert not s.query()
    s.synchronize()
    assert torch.equal(idx, want) and keep


def test_workspaces_are_not_made_inside_a_capture():
    """Refused before anything reaches the stream: the capture goes on and its graph replays."""
    K, V, Q = rnd(1, HKV, N, D), rnd(2, HKV, N, D), rnd(3, B, 1, HKV * G, D, scale=2.0)
    dec = z.PrefixDecoder(cfg_of(), B, N)
    want = dec(K, V, N, Q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(ValueError):
            z.prefix_decode(cfg_of(), K, V, N, Q)
        with pytest.raises(ValueError):
            z.DenseWeights(cfg_of(), 30, N)
        o = dec(K, V, N, Q)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)
