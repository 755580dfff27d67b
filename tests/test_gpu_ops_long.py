"""Shared-prefix attention and attention-weight sums over long caches, against fp64 on the GPU, by relative errors.

Tolerances.  |logit| stays below 16 (64 where keys rise).  A logit's error in natural units is a weight's relative
error.
* bf16: the tensor pipe adds d/16 products of exact terms and cuts off, d/16 * 2^-23 of a partial sum below 16 at most:
  7.7e-6 (d = 64) and 1.5e-5 (d = 128) if all fell the same way; the scale, the exponent's argument (below 40 in powers
  of two), the log-sum-exp and its conversion round once each, 2^-24 of a value below 40: 4 * 40 * ln 2 * 2^-24 = 6.6e-6 at
  most; ex2 2^-22.  A sum of weights is off by at most 1.5e-5 (d = 64) and 2.2e-5 (d = 128) of itself.
* fp32: d roundings of partial sums of |q k| / sqrt d, which add up to about 0.64 * 2 * sqrt d: 64 * 2^-24 * 10 = 3.9e-5
  (d = 64), 128 * 2^-24 * 14.5 = 1.1e-4 (d = 128) if all fell the same way, and 6.9e-6 as above.
* Outputs: the weights' error; for bf16 half a step of the second bf16 part, 2^-17 = 7.6e-6, and the accumulator, which
  takes 16 tiles of 16 products: 256 * 2^-24 = 1.5e-5 on average for additions that cut off.  Errors of different keys are as
  unrelated as the keys' shares of the output, so by the 2-norm an output is off by the same fraction of itself.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import tree_indexed_sparse_03_b200 as z

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
WEIGHT = {("bf16", 64): 1.5e-5, ("bf16", 128): 2.2e-5, ("f32", 64): 4.6e-5, ("f32", 128): 1.2e-4}
OUT = {k: w + (2.3e-5 if k[0] == "bf16" else 0.0) for k, w in WEIGHT.items()}


def cfg_of(dtype, d, hkv, group, capacity):
    return z.make_config(d=d, n_q_heads=hkv * group, n_kv_heads=hkv, block=4, levels=1, n_refs=1, p=1.0, dtype=dtype,
                         capacity=capacity)


def rnd(seed, *shape, dtype="bf16", scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(DT[dtype])


@pytest.mark.parametrize("B,m,own,rising", [(1, 1, 0, False), (1, 1, 0, True), (40, 8, 60, False), (40, 8, 60, True),
                                            (2, 1, 600001, True)])
def test_prefix_long_wide_heads(B, m, own, rising):
    """Heads of 128: an accumulator of two 64-column halves leaves tensor memory several times, also while the running
    maximum moves (keys grow along the cache by a factor of 16, logits up to 64)."""
    n, d, G = 700003, 128, 4
    K, V, Q = rnd(1, 1, n, d), rnd(2, 1, n, d), rnd(3, B, m, G, d, scale=2.0)
    if rising:
        K = (K * (0.25 + 3.75 * torch.arange(n, device="cuda")[:, None] / n)).to(torch.bfloat16)
    Ko, Vo = (rnd(4, B, 1, own, d), rnd(5, B, 1, own, d)) if own else (None, None)
    lens = [own - (b * 7) % (own + 1) for b in range(B)]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda") if own else None
    dec = z.PrefixDecoder(cfg_of("bf16", d, 1, G, n), B, n, own, m)
    o, lse = dec(K, V, n, Q, Ko, Vo, ln, want_lse=True)
    torch.cuda.synchronize()
    dec.status()
    k, v = K[0].double(), V[0].double()
    worst = norm = 0.0
    for b in range(0, B, 13):
        for i in range(m):
            seen = max(0, lens[b] - m + i + 1) if own else 0
            kk = torch.cat([k, Ko[b, 0, :seen].double()]) if seen else k
            vv = torch.cat([v, Vo[b, 0, :seen].double()]) if seen else v
            x = Q[b, i].double() @ kk.T / math.sqrt(d)
            want = torch.softmax(x, 1) @ vv
            worst += float((o[b, i].double() - want).square().sum())
            norm += float(want.square().sum())
            # rising: logits up to 64, four times the bound of a weight
            assert float((lse[b, i].double() - torch.logsumexp(x, 1)).abs().max()) <= (4 if rising else 1) * WEIGHT["bf16", d]
    assert math.sqrt(worst / norm) <= OUT["bf16", d] + (3 * WEIGHT["bf16", d] if rising else 0.0)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("B,m,n,own", [(1, 1, 60001, 0), (3, 1, 20000, 700), (9, 5, 20003, 130)])
def test_prefix_by_the_norm(dtype, d, B, m, n, own):
    hkv, G = 2, 4
    K, V = rnd(1, hkv, n, d, dtype=dtype), rnd(2, hkv, n, d, dtype=dtype)
    Q = rnd(3, B, m, hkv * G, d, dtype=dtype, scale=2.0)
    Ko, Vo = (rnd(4, B, hkv, own, d, dtype=dtype), rnd(5, B, hkv, own, d, dtype=dtype)) if own else (None, None)
    lens = [own - (b * 53) % (own + 1) for b in range(B)]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda") if own else None
    o, lse = z.prefix_decode(cfg_of(dtype, d, hkv, G, n), K, V, n, Q, Ko, Vo, ln, want_lse=True)
    for b in range(B):
        for h in range(hkv):
            for i in range(m):
                seen = max(0, lens[b] - m + i + 1) if own else 0
                k, v = K[h].double(), V[h].double()
                if seen:
                    k, v = torch.cat([k, Ko[b, h, :seen].double()]), torch.cat([v, Vo[b, h, :seen].double()])
                heads = slice(h * G, (h + 1) * G)
                x = Q[b, i, heads].double() @ k.T / math.sqrt(d)
                want = torch.softmax(x, 1) @ v
                err = (o[b, i, heads].double() - want).norm(dim=1) / want.norm(dim=1)
                assert float(err.max()) <= OUT[dtype, d], (b, h, i)
                assert float((lse[b, i, heads].double() - torch.logsumexp(x, 1)).abs().max()) <= WEIGHT[dtype, d]


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("m,n", [(1, 500001), (4, 130001), (5, 130001), (70, 130001)])
@pytest.mark.parametrize("outputs", [True, False])
def test_weights_by_their_own_size(dtype, d, m, n, outputs):
    """Every token's sum to a fraction of itself, however small (kept logits for m <= 4), their total, their norm."""
    G = 4
    K, V, Q = rnd(1, 1, n, d, dtype=dtype), rnd(2, 1, n, d, dtype=dtype), rnd(3, m, G, d, dtype=dtype, scale=2.0)
    dec = z.DenseWeights(cfg_of(dtype, d, 1, G, n), m, n)
    o, a = dec(K, V if outputs else None, n, Q, causal=True)
    torch.cuda.synchronize()
    dec.status()
    k, v = K[0].double(), V[0].double()
    want = torch.zeros(n, dtype=torch.float64, device="cuda")
    worst = norm = 0.0
    for i in range(m):
        seen = n - m + 1 + i
        w = torch.softmax(Q[i].double() @ k[:seen].T / math.sqrt(d), 1)
        want[:seen] += w.sum(0)
        if outputs:
            x = w @ v[:seen]
            worst += float((o[i].double() - x).square().sum())
            norm += float(x.square().sum())
    tol = WEIGHT[dtype, d]
    got = a[0].double()
    assert float(((got - want).abs() / want).max()) <= tol
    assert float((got - want).norm() / want.norm()) <= tol and abs(float(got.sum()) - m * G) <= tol * m * G
    if outputs:
        assert math.sqrt(worst / norm) <= OUT[dtype, d]


@pytest.mark.parametrize("dtype,d,hkv,n", [("bf16", 128, 3, 6000011), ("f32", 64, 2, 9000005)])
def test_offsets_past_32_bits(dtype, d, hkv, n):
    """Caches of more than 2^32 bytes (bf16: of more than 2^31 elements) per tensor: every head of each operator against
    fp64, eviction's rows against the positions it returns, into other buffers and in place."""
    G, keep, first, last = 2, 40000, 3, 500
    K, V = (torch.empty(hkv, n, d, dtype=DT[dtype], device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (K, V):
        for h in range(hkv):
            for i in range(0, n, 1 << 20):
                part = t[h, i:i + (1 << 20)]
                part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    assert K.numel() * K.element_size() > 2 ** 32
    cfg = cfg_of(dtype, d, hkv, G, n)
    Q = rnd(3, 1, hkv * G, d, dtype=dtype, scale=2.0)
    o, lse = z.prefix_decode(cfg, K, V, n, Q, want_lse=True)
    ow, acc = z.DenseWeights(cfg, 1, n)(K, V, n, Q)
    x = torch.empty(hkv, G, n, dtype=torch.float64, device="cuda")
    for h in range(hkv):
        for i in range(0, n, 1 << 20):
            x[h, :, i:i + (1 << 20)] = Q[0, h * G:(h + 1) * G].double() @ K[h, i:i + (1 << 20)].double().T / math.sqrt(d)
    w = torch.softmax(x, 2)
    want = torch.zeros(hkv, G, d, dtype=torch.float64, device="cuda")
    for h in range(hkv):
        for i in range(0, n, 1 << 20):
            want[h] += w[h, :, i:i + (1 << 20)] @ V[h, i:i + (1 << 20)].double()
    tol = OUT[dtype, d]
    for got in (o, ow):
        err = (got[0].double().view(hkv, G, d) - want).norm(dim=2) / want.norm(dim=2)
        assert float(err.max()) <= tol
    assert float((lse[0].double().view(hkv, G) - torch.logsumexp(x, 2)).abs().max()) <= WEIGHT[dtype, d]
    sums = w.sum(1)
    assert float(((acc.double() - sums).abs() / sums).max()) <= WEIGHT[dtype, d]
    del x, w, sums
    ko, vo = (torch.empty(hkv, keep, d, dtype=DT[dtype], device="cuda") for _ in range(2))
    idx, ao = z.cache_evict(cfg, K, V, n, acc, keep, first=first, last=last, K_out=ko, V_out=vo)
    mid = torch.sort(acc[:, first:n - last], dim=1, descending=True, stable=True).indices[:, :keep - first - last] + first
    ends = torch.cat([torch.arange(first, device="cuda"), torch.arange(n - last, n, device="cuda")]).expand(hkv, -1)
    assert torch.equal(idx.long(), torch.sort(torch.cat([mid, ends], 1), 1).values)
    for h in range(hkv):
        at = idx[h].long()
        assert torch.equal(ko[h], K[h][at]) and torch.equal(vo[h], V[h][at]) and torch.equal(ao[h], acc[h][at])
    idx2, _ = z.cache_evict(cfg, K, V, n, acc, keep, first=first, last=last)
    assert torch.equal(idx2, idx) and torch.equal(K[:, :keep], ko) and torch.equal(V[:, :keep], vo)
    assert torch.equal(acc[:, :keep], ao) and not bool(acc[:, keep:].any())
