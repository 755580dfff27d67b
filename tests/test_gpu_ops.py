"""Shared-prefix attention, attention-weight sums and eviction on the GPU against plain fp64 implementations.

Tolerances.  The stored inputs are the same on both sides.  A logit is an fp32 sum of d exact (bf16) or once-rounded
(fp32) products, |logit| stays below 16 here: rounding of the logit and of the exponent's argument 16 * 2^-23, of the
exponential 2^-22, so a weight is off by about 3e-6 of itself; where weights enter a bf16 product they do so as two bf16 parts, which
leave half a step of the second part, 2^-9 * 2^-8 = 2^-17 = 7.6e-6 at most.  Together 1.1e-5 relative per weight, and the
fp32 sums of up to 4,000 terms per accumulator add errors of random sign, below 64 * 2^-24 = 4e-6.  So an output, a weighted mean of rows
of V, is off by at most 2e-5 * max|V|, a token's sum of weights by at most 2e-5 of itself, and a log-sum-exp by 2e-5 (+ 2^-22 of itself).
Positions are whole numbers and moved rows are copies: equal.
"""
import math

import pytest
import torch

import oracle.zha_oracle as zo
from synth.workloads import generate, small_topics

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import tree_indexed_sparse_03_b200 as z
    from tree_indexed_sparse_03_b200 import zha as zb

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
REL = 2e-5


def cfg_of(dtype, d, hkv, group, capacity=1 << 20):
    return z.make_config(d=d, n_q_heads=hkv * group, n_kv_heads=hkv, block=4, levels=1, n_refs=1, p=1.0, dtype=dtype,
                         capacity=capacity)


def rnd(seed, *shape, dtype="bf16", scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(DT[dtype])


def prefix_ref(K, V, n, Q, K_own, V_own, lens):
    """fp64, one query head at a time: (O, lse)."""
    B, m, hq, d = Q.shape
    hkv = K.shape[0]
    G = hq // hkv
    O = torch.zeros(B, m, hq, d, dtype=torch.float64)
    lse = torch.full((B, m, hq), -math.inf, dtype=torch.float64)
    for b in range(B):
        L = lens[b] if lens is not None else 0
        for h in range(hkv):
            for i in range(m):
                seen = max(0, L - m + i + 1)
                k, v = K[h, :n].double(), V[h, :n].double()
                if seen:
                    k = torch.cat([k, K_own[b, h, :seen].double()])
                    v = torch.cat([v, V_own[b, h, :seen].double()])
                if k.shape[0] == 0:
                    continue
                x = Q[b, i, h * G:(h + 1) * G].double() @ k.T / math.sqrt(d)
                lse[b, i, h * G:(h + 1) * G] = torch.logsumexp(x, 1)
                O[b, i, h * G:(h + 1) * G] = torch.softmax(x, 1) @ v
    return O, lse


def close(got, want, tol, what):
    assert got.shape == want.shape
    g = got.cpu().double()
    assert torch.isfinite(g).equal(torch.isfinite(want)), what
    fin = torch.isfinite(want)
    err = (g[fin] - want[fin]).abs()
    tol = tol[fin] if isinstance(tol, torch.Tensor) else tol
    assert bool((err <= tol).all()), f"{what}: {float(err.max())}"


def check_prefix(dtype, d, hkv, group, B, m, n, own, lens, seed=1, ld=None):
    """Rows past n and past a sequence's length hold NaN and infinities: they are never used."""
    ld = ld or n
    K, V = rnd(seed, hkv, ld, d, dtype=dtype), rnd(seed + 1, hkv, ld, d, dtype=dtype)
    K[:, n:], V[:, n:] = math.nan, math.inf
    Q = rnd(seed + 2, B, m, hkv * group, d, dtype=dtype, scale=2.0)
    Ko = Vo = ln = None
    if own:
        Ko, Vo = rnd(seed + 3, B, hkv, own, d, dtype=dtype), rnd(seed + 4, B, hkv, own, d, dtype=dtype)
        for b in range(B):
            Ko[b, :, lens[b]:], Vo[b, :, lens[b]:] = math.inf, math.nan
        ln = torch.tensor(lens, dtype=torch.int32).cuda()
    want_o, want_l = prefix_ref(K, V, n, Q, Ko, Vo, lens if own else None)
    dec = z.PrefixDecoder(cfg_of(dtype, d, hkv, group), B, n, own, m)
    args = (K.cuda(), V.cuda(), n, Q.cuda(), Ko.cuda() if own else None, Vo.cuda() if own else None, ln)
    o, lse = dec(*args, want_lse=True)
    o2 = dec(*args)
    torch.cuda.synchronize()
    dec.status()
    close(o, want_o, REL * float(V[:, :n].abs().max() if n else 6.0) + 1e-6, "O")
    close(lse, want_l, REL + 2.0 ** -22 * 16, "lse")
    assert torch.equal(o, o2)  # the same bits on every call


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
@pytest.mark.parametrize("hkv,group,B,m,n,own,lens", [
    (1, 1, 1, 1, 1, 0, None),                       # one key, one row
    (2, 4, 1, 1, 64, 0, None),
    (1, 8, 1, 1, 127, 1, [1]),
    (2, 2, 2, 1, 777, 37, [37, 1]),
    (1, 3, 5, 1, 129, 64, [0, 64, 63, 1, 33]),      # a sequence with nothing of its own
    (3, 7, 2, 5, 300, 140, [140, 5]),               # drafted tokens, odd groups
    (1, 5, 3, 8, 0, 70, [70, 8, 3]),                # no prefix; query tokens that see no key
    (2, 8, 19, 1, 1025, 129, [(b * 37) % 130 for b in range(19)]),
    (1, 8, 70, 4, 515, 20, [(b * 7) % 21 for b in range(70)]),
    (4, 8, 3, 1, 5003, 260, [260, 0, 131]),
    (4, 3, 120, 1, 100, 300, [(b * 61) % 301 for b in range(120)]),  # several short segments per CTA
])
def test_prefix(dtype, d, hkv, group, B, m, n, own, lens):
    check_prefix(dtype, d, hkv, group, B, m, n, own, lens, ld=n + 5 if n % 2 else n)


@pytest.mark.parametrize("dtype,group,B,m", [("bf16", 8, 40, 8), ("f32", 4, 6, 6), ("bf16", 17, 1, 16)])
def test_prefix_many_rows(dtype, group, B, m):
    """Several row blocks per head and more rows of one sequence than one row block holds."""
    check_prefix(dtype, 64, 1, group, B, m, 2050, 150, [(b * 53 + m) % 151 for b in range(B)], seed=5)


def test_prefix_without_own_is_dense():
    K, V = rnd(1, 4, 20000, 128).cuda(), rnd(2, 4, 20000, 128).cuda()
    Q = rnd(3, 3, 32, 128, scale=2.0).cuda()
    cfg = z.make_config(d=128, n_q_heads=32, n_kv_heads=4, block=4, levels=1, n_refs=1, p=1.0, dtype="bf16",
                        capacity=20000, max_batch=3)
    a = z.prefix_decode(cfg, K, V, 20000, Q)
    b = z.dense_decode(cfg, K, V, 20000, Q)
    torch.cuda.synchronize()
    assert (a - b).abs().max().item() <= 2 * REL * float(V.abs().max())


def test_prefix_lengths_outside_the_cache_are_clamped():
    K, V = rnd(1, 1, 100, 64).cuda(), rnd(2, 1, 100, 64).cuda()
    Q = rnd(3, 2, 1, 2, 64).cuda()
    Ko, Vo = rnd(4, 2, 1, 16, 64).cuda(), rnd(5, 2, 1, 16, 64).cuda()
    cfg = cfg_of("bf16", 64, 1, 2)
    dec = z.PrefixDecoder(cfg, 2, 100, 16)
    a = dec(K, V, 100, Q, Ko, Vo, torch.tensor([1 << 30, -5], dtype=torch.int32, device="cuda"))
    b = dec(K, V, 100, Q, Ko, Vo, torch.tensor([16, 0], dtype=torch.int32, device="cuda"))
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefix_workspace_reused_by_smaller_calls(dtype):
    """Long own caches first, then short ones (fewer tiles than the plan has CTAs for) in the same workspace: nothing
    that the first call left there is taken up."""
    hkv, B, d, own = 2, 3, 64, 1024
    cfg = cfg_of(dtype, d, hkv, 2)
    Q = rnd(1, B, 1, 4, d, dtype=dtype, scale=2.0)
    K, V = rnd(2, hkv, 300, d, dtype=dtype), rnd(3, hkv, 300, d, dtype=dtype)
    Ko, Vo = rnd(4, B, hkv, own, d, dtype=dtype), rnd(5, B, hkv, own, d, dtype=dtype)
    dec = z.PrefixDecoder(cfg, B, 300, own)
    for n, lens in ((300, [1024, 900, 1000]), (0, [130, 300, 1]), (5, [1, 0, 257]), (300, [0, 0, 0]), (0, [0, 700, 0])):
        want, lse = prefix_ref(K, V, n, Q, Ko, Vo, lens)
        o, l = dec(K.cuda(), V.cuda(), n, Q.cuda(), Ko.cuda(), Vo.cuda(),
                   torch.tensor(lens, dtype=torch.int32, device="cuda"), want_lse=True)
        close(o, want, REL * float(V.abs().max()) + 1e-6, f"{n} {lens}")
        close(l, lse, 3e-5, f"{n} {lens}")


def test_prefix_large_logits_and_shifted_rows():
    """Logits of several hundred, one key far above the rest late in the prefix: the running maximum moves."""
    d, n = 128, 3000
    K, V = rnd(1, 1, n, d), rnd(2, 1, n, d)
    Q = rnd(3, 1, 1, 8, d, scale=2.0)
    K[0, 2990] = 8 * Q[0, 0, 3]
    K[0, 5] = 4 * Q[0, 0, 3]
    K[0, 1500] = 3 * Q[0, 0, 6]
    want, lse = prefix_ref(K, V, n, Q, None, None, None)
    o, l = z.prefix_decode(cfg_of("bf16", d, 1, 8), K.cuda(), V.cuda(), n, Q.cuda(), want_lse=True)
    # logits reach 400: the exponent's argument is rounded to 400 * 2^-23 = 5e-5
    close(o, want, 7e-5 * float(V.abs().max()), "O")
    close(l, lse, 2e-4, "lse")


def test_prefix_slices_streams_and_graphs():
    """Heads that are slices of a longer cache, another stream than the current one, a captured call replayed on
    changed inputs, and two decoders whose graphs replay at once."""
    d, n, B = 128, 1500, 4
    cfg = cfg_of("bf16", d, 2, 4)
    big_k, big_v = rnd(1, 2, 4000, d).cuda(), rnd(2, 2, 4000, d).cuda()
    Q = rnd(3, B, 1, 8, d, scale=2.0).cuda()
    Ko, Vo = rnd(4, B, 2, 40, d).cuda(), rnd(5, B, 2, 40, d).cuda()
    ln = torch.tensor([40, 3, 0, 17], dtype=torch.int32, device="cuda")
    want, _ = prefix_ref(big_k[:, :n].cpu(), big_v[:, :n].cpu(), n, Q.cpu(), Ko.cpu(), Vo.cpu(), ln.tolist())
    dec = z.PrefixDecoder(cfg, B, n, 40)
    tol = REL * float(big_v.abs().max())
    close(dec(big_k[:, :n], big_v[:, :n], n, Q, Ko, Vo, ln), want, tol, "slice")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = dec(big_k, big_v, n, Q, Ko, Vo, ln, stream=s)
    s.synchronize()
    close(o, want, tol, "other stream")
    torch.cuda.synchronize()
    dec2 = z.PrefixDecoder(cfg, B, n, 40)
    out1, out2 = torch.zeros(B, 1, 8, d, device="cuda"), torch.zeros(B, 1, 8, d, device="cuda")
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        dec(big_k, big_v, n, Q, Ko, Vo, ln, out=out1)
    with torch.cuda.graph(g2):
        dec2(big_k, big_v, n, Q, Ko, Vo, ln, out=out2)
    for step in range(2):
        Q.copy_(rnd(30 + step, B, 1, 8, d, scale=2.0))
        ln.copy_(torch.tensor([1 + step, 40, 20, 0], dtype=torch.int32))
        want, _ = prefix_ref(big_k[:, :n].cpu(), big_v[:, :n].cpu(), n, Q.cpu(), Ko.cpu(), Vo.cpu(), ln.tolist())
        torch.cuda.synchronize()
        g1.replay()
        with torch.cuda.stream(s):
            g2.replay()
        torch.cuda.synchronize()
        close(out1, want, tol, "replay")
        close(out2, want, tol, "replay beside another")
    dec.status()
    dec2.status()


@pytest.mark.parametrize("B,m,own,rising", [(1, 1, 0, False), (1, 1, 0, True), (40, 8, 60, False), (40, 8, 60, True),
                                              (2, 1, 600001, True)])
def test_prefix_long(B, m, own, rising):
    """Shares of many tiles: the accumulator is added up outside tensor memory several times, also while the running maximum
    moves (rising: keys grow along the cache by a factor of 16, each longer key ahead of all before it)."""
    n, hkv, d = 700003, 1, 64
    K, V = rnd(1, hkv, n, d).cuda(), rnd(2, hkv, n, d).cuda()
    Q = rnd(3, B, m, 4, d, scale=2.0).cuda()
    if rising:
        K = (K * (0.25 + 3.75 * torch.arange(n, device="cuda")[:, None] / n)).to(torch.bfloat16)
    Ko, Vo = (rnd(4, B, hkv, own, d).cuda(), rnd(5, B, hkv, own, d).cuda()) if own else (None, None)
    ln = torch.tensor([own - (b * 7) % (own + 1) for b in range(B)], dtype=torch.int32, device="cuda") if own else None
    dec = z.PrefixDecoder(cfg_of("bf16", d, hkv, 4, capacity=n), B, n, own, m)
    o, lse = dec(K, V, n, Q, Ko, Vo, ln, want_lse=True)
    torch.cuda.synchronize()
    dec.status()
    k, v = K[0].double(), V[0].double()
    worst = norm = 0.0
    for b in range(0, B, 13):
        for i in range(m):
            seen = max(0, int(ln[b]) - m + i + 1) if own else 0
            kk = torch.cat([k, Ko[b, 0, :seen].double()]) if seen else k
            vv = torch.cat([v, Vo[b, 0, :seen].double()]) if seen else v
            x = Q[b, i].double() @ kk.T / math.sqrt(d)
            want = torch.softmax(x, 1) @ vv
            worst += float((o[b, i].double() - want).square().sum())
            norm += float(want.square().sum())
            # logits up to 64: the exponent's argument is rounded to 64 * 2^-23 = 8e-6, weights to 1.9e-5 in all; the same
            # for the sum
            assert float((o[b, i].double() - want).abs().max()) <= 4e-5 * float(v.abs().max())
            assert float((lse[b, i].double() - torch.logsumexp(x, 1)).abs().max()) <= 4e-5
    # by the 2-norm: 16 tiles of 16 products add at most 256 * 2^-24 = 1.5e-5 of an output (all of the same sign), beside the 1.9e-5
    assert math.sqrt(worst / norm) <= 3.4e-5


def test_prefix_without_any_key():
    """No prefix and no own caches: every query sees nothing."""
    cfg = cfg_of("bf16", 128, 2, 3)
    o, lse = z.prefix_decode(cfg, None, None, 0, rnd(1, 2, 1, 6, 128).cuda(), want_lse=True)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    assert z.prefix_decode(cfg, None, None, 0, rnd(1, 0, 1, 6, 128).cuda()).shape == (0, 1, 6, 128)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_back_to_back(dtype):
    """Forty calls of two operators in one workspace each, nothing waiting between them (each starts under the end of the one
    before): the bits of the same calls made one at a time."""
    d, n, B = 64, 900, 3
    cfg = cfg_of(dtype, d, 2, 4)
    K, V = rnd(1, 2, n, d, dtype=dtype).cuda(), rnd(2, 2, n, d, dtype=dtype).cuda()
    Ko, Vo = rnd(3, B, 2, 300, d, dtype=dtype).cuda(), rnd(4, B, 2, 300, d, dtype=dtype).cuda()
    ln = [torch.tensor([(i * 97) % 301, (i * 31) % 301, 300], dtype=torch.int32, device="cuda") for i in range(20)]
    Qs = [rnd(10 + i, B, 1, 8, d, dtype=dtype, scale=2.0).cuda() for i in range(20)]
    dec, w = z.PrefixDecoder(cfg, B, n, 300), z.DenseWeights(cfg, 40, n)
    Qw = [rnd(50 + i, 40, 8, d, dtype=dtype, scale=2.0).cuda() for i in range(20)]

    def one(i):
        o = dec(K, V, n - i, Qs[i], Ko, Vo, ln[i], want_lse=True)
        return [*o, *w(K, V, n - 2 * i, Qw[i], causal=bool(i & 1))]

    alone = []
    for i in range(20):
        alone.append([t.clone() for t in one(i)])
        torch.cuda.synchronize()
    together = [one(i) for i in range(20)]
    torch.cuda.synchronize()
    dec.status()
    w.status()
    for x, y in zip(alone, together):
        assert all(torch.equal(p, q) for p, q in zip(x, y))


# ---------------------------------------------------------------- weights
def weights_ref(K, V, n, Q, acc, causal):
    m, hq, d = Q.shape
    hkv = K.shape[0]
    G = hq // hkv
    O = torch.zeros(m, hq, d, dtype=torch.float64)
    out = acc[:, :n].double().clone() if acc is not None else torch.zeros(hkv, n, dtype=torch.float64)
    for h in range(hkv):
        x = torch.einsum("igd,nd->ign", Q[:, h * G:(h + 1) * G].double(), K[h, :n].double()) / math.sqrt(d)
        if causal:
            seen = n - m + 1 + torch.arange(m)
            x = x.masked_fill(torch.arange(n)[None, None, :] >= seen[:, None, None], -math.inf)
        w = torch.softmax(x, 2)
        out[h] += w.sum((0, 1))
        O[:, h * G:(h + 1) * G] = torch.einsum("ign,nd->igd", w, V[h, :n].double())
    return O, out


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
@pytest.mark.parametrize("hkv,group,m,n,causal", [
    (1, 1, 1, 1, True), (2, 4, 1, 64, False), (1, 8, 1, 4099, False), (2, 2, 3, 129, True), (1, 3, 65, 65, True),
    (3, 5, 33, 1000, False), (1, 8, 130, 2051, True), (1, 7, 515, 515, True), (2, 8, 16, 700, True),
])
def test_weights(dtype, d, hkv, group, m, n, causal):
    ld = n + 3
    K, V = rnd(1, hkv, ld, d, dtype=dtype), rnd(2, hkv, ld, d, dtype=dtype)
    K[:, n:], V[:, n:] = math.nan, math.nan
    Q = rnd(3, m, hkv * group, d, dtype=dtype, scale=2.0)
    acc = torch.rand(hkv, n + 2, generator=torch.Generator().manual_seed(4)) * 3
    want_o, want_a = weights_ref(K, V, n, Q, acc, causal)
    dec = z.DenseWeights(cfg_of(dtype, d, hkv, group), m, n)
    Kc, Vc, Qc, ac = K.cuda(), V.cuda(), Q.cuda(), acc.cuda()
    o, a = dec(Kc, Vc, n, Qc, ac, causal=causal)
    tol_a = REL * want_a + 1e-6
    close(o, want_o, REL * float(V[:, :n].abs().max()) + 1e-6, "O")
    close(a, want_a, tol_a, "acc")
    none, alone = dec(Kc, None, n, Qc, None, causal=causal)
    assert none is None
    base = weights_ref(K, V, n, Q, None, causal)[1]
    close(alone, base, REL * base + 1e-6, "sums alone")
    # in place, and what lies past n stays
    inplace = ac.clone()
    _, same = dec(Kc, Vc, n, Qc, inplace, causal=causal, acc_out=inplace)
    assert same is inplace and torch.equal(inplace[:, n:], ac[:, n:]) and torch.equal(inplace[:, :n], a)
    dec.status()
    # the weights of one query head sum to one
    assert abs(float(alone.double().sum()) - m * hkv * group) <= REL * m * hkv * group


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_workspace_reused_and_wide_groups(dtype):
    """One workspace for calls of many shapes, and more query heads per KV head than a tile has rows."""
    d, n, group = 64, 1300, 150
    dec = z.DenseWeights(cfg_of(dtype, d, 1, group), 40, n)
    K, V = rnd(1, 1, n, d, dtype=dtype), rnd(2, 1, n, d, dtype=dtype)
    Q = rnd(3, 40, group, d, dtype=dtype, scale=2.0)
    for m, nn, causal in ((40, 1300, False), (40, 40, True), (1, 1, False), (7, 700, True), (40, 300, True), (2, 257, False)):
        want_o, want_a = weights_ref(K, V, nn, Q[:m], None, causal)
        o, a = dec(K.cuda(), V.cuda(), nn, Q[:m].cuda(), causal=causal)
        close(o, want_o, REL * float(V.abs().max()) + 1e-6, f"{m} {nn}")
        close(a, want_a, REL * want_a + 1e-6, f"{m} {nn}")


@pytest.mark.parametrize("dtype,d,hkv,group,m,n", [("bf16", 64, 5, 3, 95, 300), ("bf16", 128, 40, 1, 2, 130),
                                                   ("bf16", 64, 200, 1, 1, 90), ("f32", 64, 200, 2, 1, 70)])
def test_weights_many_short_segments(dtype, d, hkv, group, m, n):
    """Several segments per CTA: whole ones between two that its neighbours share, blocks of a few rows among them."""
    K, V, Q = rnd(1, hkv, n, d, dtype=dtype), rnd(2, hkv, n, d, dtype=dtype), rnd(3, m, hkv * group, d, dtype=dtype, scale=2.0)
    dec = z.DenseWeights(cfg_of(dtype, d, hkv, group), m, n)
    for causal in (True, False):
        want_o, want_a = weights_ref(K, V, n, Q, None, causal)
        o, a = dec(K.cuda(), V.cuda(), n, Q.cuda(), causal=causal)
        close(o, want_o, REL * float(V.abs().max()) + 1e-6, "O")
        close(a, want_a, REL * want_a + 1e-6, "acc")
    dec.status()


@pytest.mark.parametrize("m", [1, 70])
def test_weights_long(m):
    """One step (kept logits) and a window over a long context, against fp64 on the GPU."""
    n, d, G = 500001, 64, 4
    K, V = rnd(1, 1, n, d).cuda(), rnd(2, 1, n, d).cuda()
    Q = rnd(3, m, G, d, scale=2.0).cuda()
    dec = z.DenseWeights(cfg_of("bf16", d, 1, G, capacity=n), m, n)
    o, a = dec(K, V, n, Q, causal=True)
    torch.cuda.synchronize()
    dec.status()
    acc = torch.zeros(n, dtype=torch.float64, device="cuda")
    worst = norm = 0.0
    for i in range(m):
        seen = n - m + 1 + i
        w = torch.softmax(Q[i].double() @ K[0, :seen].double().T / math.sqrt(d), 1)
        acc[:seen] += w.sum(0)
        want = w @ V[0, :seen].double()
        worst += float((o[i].double() - want).square().sum())
        norm += float(want.square().sum())
    assert bool(((a[0].double() - acc).abs() <= REL * acc + 1e-6).all())
    # weights to 1.1e-5 (above), beside them at most 256 cut-off additions of 2^-24 = 1.5e-5
    assert math.sqrt(worst / norm) <= 2.6e-5


def test_weights_graph_and_stream():
    n, m, d = 700, 9, 64
    K, V, Q = rnd(1, 2, n, d).cuda(), rnd(2, 2, n, d).cuda(), rnd(3, m, 6, d, scale=2.0).cuda()
    acc = torch.zeros(2, n, device="cuda")
    dec = z.DenseWeights(cfg_of("bf16", d, 2, 3), m, n)
    out = torch.zeros(m, 6, d, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, a = dec(K, V, n, Q, acc, causal=True, stream=s)
    s.synchronize()
    want_o, want_a = weights_ref(K.cpu(), V.cpu(), n, Q.cpu(), None, True)
    close(o, want_o, REL * 6, "stream")
    close(a, want_a, REL * want_a + 1e-6, "stream")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec(K, V, n, Q, acc, causal=True, acc_out=acc, out=out)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    close(acc, 3 * want_a, 3 * (REL * want_a + 1e-6), "three replays add up")
    dec.status()


# ---------------------------------------------------------------- eviction
def evict_ref(acc, n, keep, first, last):
    key = torch.where(acc[:, :n].isnan(), torch.full_like(acc[:, :n], -math.inf), acc[:, :n]).double()
    # NaN below everything, minus infinity included
    low = acc[:, :n].isnan()
    order = torch.argsort(low[:, first:n - last].to(torch.int8), dim=1, stable=True)
    by = torch.gather(key[:, first:n - last], 1, order)
    order = torch.gather(order, 1, torch.argsort(by, dim=1, descending=True, stable=True))
    ends = torch.cat([torch.arange(first), torch.arange(n - last, n)]).expand(acc.shape[0], -1)
    return torch.sort(torch.cat([order[:, :keep - first - last] + first, ends], 1), 1).values


def sums_case(kind, hkv, n, seed):
    g = torch.Generator().manual_seed(seed)
    a = torch.rand(hkv, n, generator=g) ** 8
    if kind == "ties":
        a = torch.floor(a * 4) / 4
    elif kind == "equal":
        a = torch.full((hkv, n), 0.25)
    elif kind == "special":
        a = torch.randn(hkv, n, generator=g)
        a[:, ::7] = 0.0
        a[:, 3::7] = -0.0
        a[:, 5::11] = math.nan
        a[:, 6::13] = math.inf
        a[:, 2::17] = -math.inf
    elif kind == "small":
        a = a * 1e-42  # subnormal
    return a


@pytest.mark.parametrize("dtype,d,hkv", [("bf16", 128, 2), ("f32", 64, 3), ("bf16", 64, 1), ("f32", 128, 1)])
@pytest.mark.parametrize("kind,n,keep,first,last", [
    ("plain", 1, 1, 0, 0), ("plain", 5, 5, 2, 3), ("plain", 4097, 1, 0, 0), ("plain", 4097, 1000, 4, 64),
    ("ties", 3001, 1500, 1, 0), ("ties", 9000, 123, 0, 100), ("equal", 2500, 700, 3, 9), ("special", 5003, 2600, 0, 1),
    ("special", 5003, 4990, 7, 0), ("small", 2049, 600, 0, 0), ("plain", 300001, 70007, 4, 1024),
    ("plain", 3000, 100, 60, 40), ("plain", 66000, 65999, 1, 1), ("ties", 16384, 9000, 0, 0), ("special", 16385, 9001, 0, 0),
    ("equal", 70001, 30000, 5, 7), ("special", 50007, 49000, 3, 40000), ("plain", 40000, 300, 200, 100),
])
def test_evict(dtype, d, hkv, kind, n, keep, first, last):
    if n > 100000 and (dtype, d) != ("bf16", 128):
        pytest.skip("the long cache once is enough")
    acc = sums_case(kind, hkv, n + 2, 3)
    K, V = rnd(1, hkv, n + 4, d, dtype=dtype), rnd(2, hkv, n + 4, d, dtype=dtype)
    want = evict_ref(acc, n, keep, first, last)
    pick = torch.arange(hkv)[:, None]
    wk, wv, wa = K[pick, want], V[pick, want], acc[pick, want]
    cfg = cfg_of(dtype, d, hkv, 1)
    Kc, Vc, ac = K.cuda(), V.cuda(), acc.cuda()
    ko, vo = torch.full_like(Kc[:, :keep + 3], 7.0), torch.full_like(Vc[:, :keep + 3], 7.0)
    idx, ao = z.cache_evict(cfg, Kc, Vc, n, ac, keep, first=first, last=last, K_out=ko, V_out=vo)
    assert torch.equal(idx.cpu().long(), want)
    assert torch.equal(ko[:, :keep].cpu(), wk) and torch.equal(vo[:, :keep].cpu(), wv)
    assert bool((ko[:, keep:] == 7).all()) and bool((vo[:, keep:] == 7).all())
    assert torch.equal(ao.cpu().nan_to_num(nan=-9.0), wa.nan_to_num(nan=-9.0))
    assert torch.equal(Kc.cpu(), K) and torch.equal(Vc.cpu(), V)
    # in place: the same rows, the ones behind left as they were, the sums behind cleared
    idx2, same = z.cache_evict(cfg, Kc, Vc, n, ac, keep, first=first, last=last)
    assert same is ac and torch.equal(idx2, idx)
    assert torch.equal(Kc[:, :keep].cpu(), wk) and torch.equal(Vc[:, :keep].cpu(), wv)
    assert torch.equal(Kc[:, keep:].cpu(), K[:, keep:]) and torch.equal(Vc[:, keep:].cpu(), V[:, keep:])
    assert torch.equal(ac[:, :keep].cpu().nan_to_num(nan=-9.0), wa.nan_to_num(nan=-9.0))
    assert bool((ac[:, keep:n] == 0).all())
    assert torch.equal(ac[:, n:].cpu().nan_to_num(nan=-9.0), acc[:, n:].nan_to_num(nan=-9.0))


def test_evict_slices_stream_and_graph():
    """Outputs with another row stride, sums that are a slice, another stream, a captured call replayed."""
    hkv, n, keep, d = 2, 2000, 600, 128
    K, V = rnd(1, hkv, 3000, d).cuda(), rnd(2, hkv, 3000, d).cuda()
    acc = torch.rand(hkv, 2500, generator=torch.Generator().manual_seed(1)).cuda()
    cfg = cfg_of("bf16", d, hkv, 1)
    ko, vo = torch.zeros(hkv, 900, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(hkv, 900, d, dtype=torch.bfloat16,
                                                                                     device="cuda")
    want = evict_ref(acc.cpu(), n, keep, 2, 5)
    pick = torch.arange(hkv)[:, None]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    idx, ao = z.cache_evict(cfg, K[:, :n], V[:, :n], n, acc[:, :n], keep, first=2, last=5, K_out=ko[:, :keep],
                            V_out=vo[:, :keep], stream=s)
    s.synchronize()
    assert torch.equal(idx.cpu().long(), want)
    assert torch.equal(ko[:, :keep].cpu(), K.cpu()[pick, want]) and bool((ko[:, keep:] == 0).all())
    assert torch.equal(ao.cpu(), acc.cpu()[pick, want])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx2, ao2 = z.cache_evict(cfg, K, V, n, acc, keep, first=2, last=5, K_out=ko, V_out=vo)
    acc.copy_(torch.rand(hkv, 2500, generator=torch.Generator().manual_seed(2)))
    g.replay()
    torch.cuda.synchronize()
    want = evict_ref(acc.cpu(), n, keep, 2, 5)
    assert torch.equal(idx2.cpu().long(), want) and torch.equal(vo[:, :keep].cpu(), V.cpu()[pick, want])


# ---------------------------------------------------------------- together
def test_prompt_weights_eviction_tree_and_prefix():
    """A prompt's last queries weigh the cache, the cache is cut, the tree over the rest decodes, tokens are
    appended, and a batch attends behind the shortened cache: each against fp64 on the kept tokens."""
    n, keep, first, last, m = 6000, 2500, 4, 100, 16
    w = small_topics(n, d=128, n_q_heads=8, n_kv_heads=2, block=4, levels=3, n_refs=4, p=1.0, batch=2)
    inp = generate(w, n_total=n + 8)
    cfg = z.make_config(d=128, n_q_heads=8, n_kv_heads=2, block=4, levels=3, n_refs=4, p=1.0, dtype="bf16",
                        capacity=n + 8, max_batch=2)
    K, V = inp.K[:, :n + 8].cuda().contiguous(), inp.V[:, :n + 8].cuda().contiguous()
    tree = z.ZhaTree(cfg, K, V, inp.refs.cuda().contiguous())
    tree.build(n)
    window = rnd(9, m, 8, 128, scale=2.0)
    acc = torch.zeros(2, n + 8, device="cuda")
    dw = z.DenseWeights(cfg, m, n)
    dw(tree.K, None, n, window.cuda(), acc, causal=True, acc_out=acc)
    want_acc = weights_ref(inp.K, inp.V, n, window, None, True)[1]
    close(acc[:, :n], want_acc, REL * want_acc + 1e-6, "sums")
    sums = acc.cpu()
    idx = tree.evict(acc, keep, first=first, last=last)
    torch.cuda.synchronize()
    tree.status()
    want = evict_ref(sums, n, keep, first, last)
    assert torch.equal(idx.cpu().long(), want) and tree.size == keep
    assert bool((acc[:, keep:n] == 0).all())
    tree.append(inp.K[:, n:n + 8].cuda(), inp.V[:, n:n + 8].cuda())
    pick = torch.arange(2)[:, None]
    Kk = torch.cat([inp.K[pick, want], inp.K[:, n:n + 8]], 1)
    Vk = torch.cat([inp.V[pick, want], inp.V[:, n:n + 8]], 1)
    Q = inp.Q[0]
    O = tree.decode(Q.cuda())  # p = 1: every kept token
    torch.cuda.synchronize()
    tree.status()
    for b in range(2):
        for h in range(8):
            ref = zo.dense(Kk[h // 4].double().numpy(), Vk[h // 4].double().numpy(), Q[b, h].double().numpy(), keep + 8)
            assert abs(O[b, h].cpu().double().numpy() - ref).max() <= REL * float(Vk.abs().max()) + 1e-6
    # a batch behind the shortened cache, each sequence with its own tokens
    B, own = 3, 20
    Qb = rnd(11, B, 1, 8, 128, scale=2.0)
    Ko, Vo = rnd(12, B, 2, own, 128), rnd(13, B, 2, own, 128)
    ln = [20, 7, 1]
    want_o, _ = prefix_ref(Kk, Vk, keep, Qb, Ko, Vo, ln)
    o = z.prefix_decode(cfg, tree.K, tree.V, keep, Qb.cuda(), Ko.cuda(), Vo.cuda(),
                        torch.tensor(ln, dtype=torch.int32, device="cuda"))
    close(o, want_o, REL * float(Vk.abs().max()) + 1e-6, "behind the shortened cache")


def test_refusals_on_device():
    cfg = cfg_of("bf16", 64, 2, 2)
    K = torch.zeros(2, 64, 64, dtype=torch.bfloat16, device="cuda")
    Q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    acc = torch.zeros(2, 64, device="cuda")
    dec = z.PrefixDecoder(cfg, 1, 32)
    with pytest.raises(ValueError):
        dec(K, K, 64, Q)                                  # more tokens than it was made for
    with pytest.raises(ValueError):
        dec(K, K, 32, Q.expand(2, 1, 4, 64).contiguous())  # more sequences
    with pytest.raises(ValueError):
        dec(K.transpose(0, 1).contiguous().transpose(0, 1), K, 32, Q)  # token-major cache
    with pytest.raises(ValueError):
        dec(K[:, ::2], K[:, ::2], 16, Q)                  # rows not one after another
    with pytest.raises(ValueError):
        dec(K, K, 32, Q, K_own=K[None])
    with pytest.raises(ValueError):
        dec(K, K, 32, Q.float())
    w = z.DenseWeights(cfg, 2, 64)
    with pytest.raises(zb.ZhaError):
        w(K, K, 1, torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"), acc, causal=True)  # m > n
    with pytest.raises(ValueError):
        w(K, K, 64, Q[0], acc.double())
    with pytest.raises(ValueError):
        w(K, None, 64, Q[0], acc, out=torch.zeros(1, 4, 64, device="cuda"))
    with pytest.raises(zb.ZhaError):
        w(K, K, 60, Q[0], acc[:, :60], acc_out=acc[:, 1:61])  # sums that overlap
    with pytest.raises(zb.ZhaError):
        z.cache_evict(cfg, K, K, 64, acc, 10)             # K and V in one buffer, both shortened in place
    with pytest.raises(ValueError):
        z.cache_evict(cfg, K, K.clone(), 64, acc, 65)
    with pytest.raises(zb.ZhaError):
        z.cache_evict(cfg, K, K.clone(), 64, acc, 10, first=8, last=8)
    if torch.cuda.device_count() > 1:
        with torch.cuda.device(1), pytest.raises(ValueError):
            dec(K, K, 32, Q)


def test_gpu_launch_counts():
    """The operators run in the library's kernels."""
    before = z.launch_count()
    cfg = cfg_of("bf16", 64, 1, 1)
    K = torch.zeros(1, 10, 64, dtype=torch.bfloat16, device="cuda")
    z.prefix_decode(cfg, K, K, 10, torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda"))
    assert z.launch_count() > before
