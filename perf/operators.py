"""Cases of the cache operators around dense and routed decode, their plain forms and the library's calls.

Three operators over one KV cache ``[Hkv, tokens, d]``:

* ``prefix``: attention of a batch whose sequences share a long prefix and have own caches of their own lengths;
* ``weights``: dense attention that also adds every token's softmax weight to the token's running sum;
* ``evict``: the cache shortened to the tokens with the largest sums, in token order.

``own`` False computes the plain form with elementary torch operations in fp32; True makes the library's calls.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # two short chats over a small shared instruction, fp32: launch latency
        dict(name="prefix_small_f32", op="prefix", dtype="f32", d=64, hkv=2, group=2, n=777, own=37, batch=2, m=1),
        # one token for each of sixteen requests behind one 32K document
        dict(name="prefix_batch16", op="prefix", dtype="bf16", d=128, hkv=4, group=8, n=32768, own=512, batch=16, m=1),
        # seven requests that each check five drafted tokens, ragged lengths, narrow heads
        dict(name="prefix_draft_odd", op="prefix", dtype="bf16", d=64, hkv=1, group=8, n=5003, own=301, batch=7, m=5),
        # one token for each of 64 requests behind a 256K context: the largest
        dict(name="prefix_batch64_256k", op="prefix", dtype="bf16", d=128, hkv=4, group=8, n=262144, own=1024, batch=64,
             m=1),
        # one decode step of a short fp32 context: launch latency
        dict(name="weights_small_f32", op="weights", dtype="f32", d=64, hkv=2, group=2, n=777, m=1, causal=False,
             out=True),
        # one decode step over 256K tokens that keeps the running sums up to date
        dict(name="weights_step_256k", op="weights", dtype="bf16", d=128, hkv=4, group=8, n=262144, m=1, causal=False,
             out=True),
        # the last 64 queries of a 64K prompt as the observation window, sums alone
        dict(name="weights_window", op="weights", dtype="bf16", d=128, hkv=4, group=8, n=65536, m=64, causal=True,
             out=False),
        # a whole prompt of odd length, attention outputs and sums
        dict(name="weights_prompt_odd", op="weights", dtype="bf16", d=64, hkv=1, group=8, n=4099, m=4099, causal=True,
             out=True),
        # a short fp32 cache cut to a quarter: launch latency
        dict(name="evict_small_f32", op="evict", dtype="f32", d=64, hkv=1, n=4096, keep=1024, first=4, last=64),
        # a 256K cache cut to a quarter
        dict(name="evict_256k", op="evict", dtype="bf16", d=128, hkv=4, n=262144, keep=65536, first=4, last=1024),
        # a 1M cache cut to a half: the largest cache
        dict(name="evict_1m", op="evict", dtype="bf16", d=128, hkv=4, n=1048576, keep=524288, first=16, last=4096),
        # a few tokens dropped from an odd cache of narrow heads
        dict(name="evict_odd", op="evict", dtype="bf16", d=64, hkv=3, n=30011, keep=29989, first=1, last=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefix", "weights", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "evict":
        n = _log(rng, 1024, 1048576 if dtype == "bf16" else 524288) // (2 if hkv == 8 else 1)
        keep = rng.randint(1, n)
        keep = min(keep, 524288 * 4 * 128 // (hkv * d * (1 if dtype == "bf16" else 2)))
        first = rng.randint(0, min(16, keep))
        last = rng.randint(0, min(4096, keep - first))
        return dict(op=op, dtype=dtype, d=d, hkv=hkv, n=n, keep=keep, first=first, last=last)
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    heads = hkv * group
    if op == "prefix":
        most = 2 ** 38 if dtype == "bf16" else 2 ** 33  # multiply-adds of the two products
        batch, m = _log(rng, 1, 64), rng.choice([1, 1, 2, 5, 8])
        own_max = max(m, _log(rng, 8, 2048))
        n = _log(rng, 512, 262144)
        n = max(64, min(n, most // (4 * d * heads * batch * m) - own_max))
        return dict(op=op, dtype=dtype, d=d, hkv=hkv, group=group, n=n, own=own_max, batch=batch, m=m)
    most = 2 ** 36 if dtype == "bf16" else 2 ** 32
    n = _log(rng, 512, 262144)
    causal = rng.random() < 0.6
    m = _log(rng, 1, 4099)
    m = max(1, min(m, most // (4 * d * heads * n)))
    if causal:
        m = min(m, n)
    return dict(op=op, dtype=dtype, d=d, hkv=hkv, group=group, n=n, m=m, causal=causal, out=rng.random() < 0.5)


def own_lens(case):
    """Own tokens of each sequence: spread over [m, own]."""
    lo, hi = min(case["m"], case["own"]), case["own"]
    return [lo + (hi - lo) * ((b * 7919 + 61) % 101) // 100 for b in range(case["batch"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    dt, d, hkv, n = DT[case["dtype"]], case["d"], case["hkv"], case["n"]
    st = dict(case=dict(case), K=rnd(hkv, n, d).to(dt), V=rnd(hkv, n, d).to(dt))
    if case["op"] == "prefix":
        B, m, hq = case["batch"], case["m"], hkv * case["group"]
        # queries twice as long as the keys: logits of standard deviation 2, a few hundred tokens carry most weight
        st["Q"] = (2 * rnd(B, m, hq, d)).to(dt)
        st["K_own"], st["V_own"] = rnd(B, hkv, case["own"], d).to(dt), rnd(B, hkv, case["own"], d).to(dt)
        st["own_len"] = torch.tensor(own_lens(case), dtype=torch.int32, device="cuda")
    elif case["op"] == "weights":
        st["Q"] = (2 * rnd(case["m"], hkv * case["group"], d)).to(dt)
        # sums of earlier steps: most tokens have little, a few have much
        st["acc"] = torch.rand(hkv, n, generator=g, device="cuda") ** 8 * 4
    else:
        acc = torch.rand(hkv, n, generator=g, device="cuda") ** 8 * 64
        # tokens that nothing has attended to yet tie at zero
        st["acc"] = torch.where(torch.rand(hkv, n, generator=g, device="cuda") < 0.1, torch.zeros_like(acc), acc)
        st["K_out"], st["V_out"] = torch.empty_like(st["K"][:, :case["keep"]]), torch.empty_like(st["V"][:, :case["keep"]])
    return st


def _plain_prefix(st):
    c = st["case"]
    B, m, hkv, G, d, w = c["batch"], c["m"], c["hkv"], c["group"], c["d"], c["own"]
    scale = 1.0 / math.sqrt(d)
    q = st["Q"].float().view(B, m, hkv, G, d).permute(2, 0, 1, 3, 4).reshape(hkv, B * m * G, d)
    qb = q.view(hkv, B, m * G, d).transpose(0, 1)
    sp = (q @ st["K"].float().transpose(1, 2)) * scale
    so = (qb @ st["K_own"].float().transpose(2, 3)) * scale
    seen = st["own_len"].long()[:, None] - m + 1 + torch.arange(m, device="cuda")  # own tokens query i sees
    ok = torch.arange(w, device="cuda") < seen.repeat_interleave(G, dim=1)[:, :, None]
    so = so.masked_fill(~ok[:, None], -math.inf)
    top = torch.maximum(sp.amax(-1).view(hkv, B, m * G), so.amax(-1).transpose(0, 1))
    ep = torch.exp(sp.sub_(top.view(hkv, B * m * G, 1)))
    eo = torch.exp(so - top.transpose(0, 1)[..., None])
    total = ep.sum(-1).view(hkv, B, m * G) + eo.sum(-1).transpose(0, 1)
    o = (ep @ st["V"].float()).view(hkv, B, m * G, d) + (eo @ st["V_own"].float()).transpose(0, 1)
    o = (o / total[..., None]).view(hkv, B, m, G, d).permute(1, 2, 0, 3, 4).reshape(B, m, hkv * G, d)
    lse = (torch.log(total) + top).view(hkv, B, m, G).permute(1, 2, 0, 3).reshape(B, m, hkv * G)
    return {"o": o.contiguous(), "lse": lse.contiguous()}


def _plain_weights(st):
    c = st["case"]
    m, hkv, G, d, n = c["m"], c["hkv"], c["group"], c["d"], c["n"]
    q = st["Q"].float().view(m, hkv, G, d).permute(1, 0, 2, 3).reshape(hkv, m * G, d)
    s = (q @ st["K"].float().transpose(1, 2)) * (1.0 / math.sqrt(d))
    if c["causal"]:
        last = (n - m + torch.arange(m, device="cuda")).repeat_interleave(G)
        s = s.masked_fill_(torch.arange(n, device="cuda") > last[:, None], -math.inf)
    e = torch.exp(s.sub_(s.amax(-1, keepdim=True)))
    w = e.div_(e.sum(-1, keepdim=True))
    got = {"acc": st["acc"] + w.sum(1)}
    if c["out"]:
        o = (w @ st["V"].float()).view(hkv, m, G, d).permute(1, 0, 2, 3).reshape(m, hkv * G, d)
        got["o"] = o.contiguous()
    return got


def _plain_evict(st):
    c = st["case"]
    n, keep, first, last, d = c["n"], c["keep"], c["first"], c["last"], c["d"]
    a = st["acc"]
    order = torch.sort(a[:, first:n - last], dim=1, descending=True, stable=True).indices[:, :keep - first - last] + first
    ends = torch.cat([torch.arange(first, device="cuda"), torch.arange(n - last, n, device="cuda")])
    idx = torch.sort(torch.cat([order, ends.expand(a.shape[0], -1)], dim=1), dim=1).values
    rows = idx[..., None].expand(-1, -1, d)
    return {"idx": idx.int(), "acc": torch.gather(a, 1, idx), "K": torch.gather(st["K"], 1, rows),
            "V": torch.gather(st["V"], 1, rows)}


def run(st):
    c = st["case"]
    if own:
        import tree_indexed_sparse_03_b200 as z
        if "handle" not in st:  # a program keeps its configuration and workspaces
            group = c.get("group", 1)
            cfg = z.make_config(d=c["d"], n_q_heads=c["hkv"] * group, n_kv_heads=c["hkv"], block=4, levels=1, n_refs=1,
                                p=1.0, dtype=c["dtype"], capacity=c["n"])
            if c["op"] == "prefix":
                st["handle"] = z.PrefixDecoder(cfg, c["batch"], c["n"], own_max=c["own"], m=c["m"])
            elif c["op"] == "weights":
                st["handle"] = z.DenseWeights(cfg, c["m"], c["n"])
            else:
                st["handle"] = cfg
        h = st["handle"]
        if c["op"] == "prefix":
            o, lse = h(st["K"], st["V"], c["n"], st["Q"], st["K_own"], st["V_own"], st["own_len"], want_lse=True)
            return {"o": o, "lse": lse}
        if c["op"] == "weights":
            o, acc = h(st["K"], st["V"] if c["out"] else None, c["n"], st["Q"], st["acc"], causal=c["causal"])
            return {"acc": acc, "o": o} if c["out"] else {"acc": acc}
        idx, acc = z.cache_evict(h, st["K"], st["V"], c["n"], st["acc"], c["keep"], first=c["first"], last=c["last"],
                                 K_out=st["K_out"], V_out=st["V_out"])
        return {"idx": idx, "acc": acc, "K": st["K_out"], "V": st["V_out"]}
    if c["op"] == "prefix":
        return _plain_prefix(st)
    return _plain_weights(st) if c["op"] == "weights" else _plain_evict(st)


def _pairs(case):
    """(query row, key) pairs of one query head that a mask leaves."""
    n, m = case["n"], case["m"]
    if case["op"] == "prefix":
        seen = sum(max(0, L - m + 1 + i) for L in own_lens(case) for i in range(m))
        return case["batch"] * m * n + seen
    return m * n - (m * (m - 1) // 2 if case["causal"] else 0)


def work(case):
    es, d, hkv, n = (4 if case["dtype"] == "f32" else 2), case["d"], case["hkv"], case["n"]
    if case["op"] == "evict":
        keep = case["keep"]
        # the sums of all tokens, the kept rows of K and V read and written, the kept sums and indices written
        return {"bytes": hkv * (4 * n + keep * (4 * d * es + 8)), "flops": 0}
    hq = hkv * case["group"]
    if case["op"] == "prefix":
        rows = case["batch"] * case["m"] * hq
        cache = hkv * (n + sum(own_lens(case))) * 2 * d * es
        return {"bytes": cache + rows * (d * es + 4 * d + 4) + 4 * case["batch"], "flops": 4 * d * hq * _pairs(case)}
    rows = case["m"] * hq
    if case["out"]:
        return {"bytes": hkv * n * (2 * d * es + 8) + rows * d * (es + 4), "flops": 4 * d * hq * _pairs(case)}
    return {"bytes": hkv * n * (d * es + 8) + rows * d * es, "flops": 2 * d * hq * _pairs(case)}


def exact(case, seed):
    """From the definitions in fp64, one KV head and one block of query tokens at a time."""
    st = prepare(case, seed)
    d, hkv, n = case["d"], case["hkv"], case["n"]
    if case["op"] == "evict":
        keep, first, last = case["keep"], case["first"], case["last"]
        idx = []
        for h in range(hkv):
            rank = st["acc"][h].double().clone()
            rank[:first] = math.inf
            rank[n - last:] = math.inf
            border = torch.sort(rank, descending=True).values[keep - 1]
            above = rank > border
            tied = torch.nonzero(rank == border).flatten()[: keep - int(above.sum())]
            above[tied] = True
            idx.append(torch.nonzero(above).flatten())
        idx = torch.stack(idx)
        pick = torch.arange(hkv, device="cuda")[:, None]
        return {"idx": idx.int(), "acc": st["acc"][pick, idx].double(), "K": st["K"][pick, idx].double(),
                "V": st["V"][pick, idx].double()}
    G = case["group"]
    if case["op"] == "prefix":
        B, m = case["batch"], case["m"]
        o = torch.empty(B, m, hkv * G, d, dtype=torch.float64, device="cuda")
        lse = torch.empty(B, m, hkv * G, dtype=torch.float64, device="cuda")
        for h in range(hkv):
            K, V = st["K"][h].double(), st["V"][h].double()
            for b in range(B):
                L = own_lens(case)[b]
                keys = torch.cat([K, st["K_own"][b, h, :L].double()])
                vals = torch.cat([V, st["V_own"][b, h, :L].double()])
                for i in range(m):
                    seen = n + max(0, L - m + 1 + i)
                    x = st["Q"][b, i, h * G:(h + 1) * G].double() @ keys[:seen].T / math.sqrt(d)
                    lse[b, i, h * G:(h + 1) * G] = torch.logsumexp(x, dim=1)
                    o[b, i, h * G:(h + 1) * G] = torch.softmax(x, dim=1) @ vals[:seen]
        return {"o": o, "lse": lse}
    m = case["m"]
    acc = st["acc"].double()
    o = torch.empty(m, hkv * G, d, dtype=torch.float64, device="cuda")
    step = max(1, min(m, (1 << 27) // (G * n)))
    at = torch.arange(n, device="cuda")
    for h in range(hkv):
        K, V = st["K"][h].double(), st["V"][h].double()
        for i0 in range(0, m, step):
            i1 = min(m, i0 + step)
            x = torch.einsum("igd,nd->ign", st["Q"][i0:i1, h * G:(h + 1) * G].double(), K) / math.sqrt(d)
            if case["causal"]:
                seen = n - m + 1 + torch.arange(i0, i1, device="cuda")
                x = torch.where(at[None, None, :] < seen[:, None, None], x, torch.full_like(x, -math.inf))
            w = torch.softmax(x, dim=2)
            acc[h] += w.sum((0, 1))
            o[i0:i1, h * G:(h + 1) * G] = torch.einsum("ign,nd->igd", w, V)
    return {"acc": acc, "o": o} if case["out"] else {"acc": acc}
