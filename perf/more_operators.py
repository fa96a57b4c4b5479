"""The operators of a bounded key/value cache, as cases to be timed.

A program that serves long conversations from a cache of bounded size runs them in this order:
a prompt goes through an attention with a sliding window whose first few tokens stay visible; each
step, new tokens (one, or a tree of drafted ones) attend over the window of their sequence's pages;
in layers that attend to everything, each step adds the weights that the cached positions received
to a running sum; and from time to time every sequence is cut back to its first positions, its last
ones and those between them that received the most weight.

With ``own`` false, ``run`` computes an operator with elementary torch operations in 32 bits
and rounds once; with ``own`` true it makes the library's calls.  Head counts, head dimensions
and types are those of the library's workloads (Hq/Hkv 2/1, 16/8, 32/8; D 64 and 128; fp16, bf16).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one short prompt through a tiny model: launch latency
        {"name": "window_prompt_one", "op": "prompt", "lens": "200", "window": 64, "sinks": 4, "Hq": 2, "Hkv": 1, "D": 64,
         "dtype": "f16", "fused": False},
        # a prefill batch of mixed prompts, q/k/v cut from one projection
        {"name": "window_prompts_mixed", "op": "prompt", "lens": "4096,33,2000,1,777,1024,128,3001,513,256,90,1500",
         "window": 512, "sinks": 4, "Hq": 16, "Hkv": 8, "D": 128, "dtype": "f16", "fused": True},
        # two long documents
        {"name": "window_prompts_long", "op": "prompt", "lens": "16384,9001", "window": 2048, "sinks": 64, "Hq": 32, "Hkv": 8,
         "D": 128, "dtype": "bf16", "fused": False},
        # one decoding step of a batch (a tree of one token each)
        {"name": "window_one_token", "op": "step", "ctx": "8191,4000,8000,1,6500,7777,513,8191,3000,8100,5000,64,7000,8191,2222,6000",
         "tree": "1", "window": 1024, "sinks": 4, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "layers": 1},
        # verifying draft trees of different sizes
        {"name": "window_trees", "op": "step", "ctx": "12000,700,5000,2049,9000,130,7000,3333", "tree": "26,32,7,1,48,33,60,16",
         "window": 4096, "sinks": 128, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 32, "layers": 1},
        # one decoding step: the weights that every cached position receives are added to its sum
        {"name": "weigh_step", "op": "weigh", "lens": "8192,4001,8001,2,6501,7778,514,8192,3001,8101,5001,65,7001,8192,2223,6001",
         "new": "1", "fresh": False, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64},
        # behind a long prompt: the weights of its last 32 tokens alone decide
        {"name": "weigh_prompt_end", "op": "weigh", "lens": "32000", "new": "32", "fresh": True, "Hq": 32, "Hkv": 8, "D": 128,
         "dtype": "bf16", "page": 128},
        # whole prompts: the weights of every token
        {"name": "weigh_prompts", "op": "weigh", "lens": "4096,33,2000,1,777,1024,128,3001,513,256,90,1500",
         "new": "4096,33,2000,1,777,1024,128,3001,513,256,90,1500", "fresh": True, "Hq": 16, "Hkv": 8, "D": 128, "dtype": "f16",
         "page": 32},
        # a short chat is cut back in a one-layer model: latency
        {"name": "evict_one", "op": "evict", "lens": "300", "sinks": 4, "heavy": 60, "recent": 64, "Hkv": 8, "D": 64, "dtype": "f16",
         "page": 16, "layers": 1},
        # a batch of conversations goes back to 1024 positions each
        {"name": "evict_batch", "op": "evict", "lens": "8192,4001,8001,900,6501,7778,1025,8192,3001,8101,5001,65,7001,8192,2223,6001",
         "sinks": 4, "heavy": 508, "recent": 512, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "layers": 4},
        # the oldest positions go, the window and its first tokens stay (no weights)
        {"name": "evict_oldest", "op": "evict", "lens": "2500,2304,2222,4000,2600,2100,2048,2301,2304,3000,3200,2049,2900,2400,2304,2222",
         "sinks": 4, "heavy": 0, "recent": 2044, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 32, "layers": 4},
        # one very long document keeps a quarter
        {"name": "evict_long", "op": "evict", "lens": "65000", "sinks": 16, "heavy": 12000, "recent": 4000, "Hkv": 8, "D": 128,
         "dtype": "bf16", "page": 128, "layers": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "step", "weigh", "evict"])
    Hq, Hkv = rng.choice([(2, 1), (16, 8), (32, 8), (8, 8), (12, 4)])
    c = {"op": op, "Hkv": Hkv, "D": rng.choice([64, 128]), "dtype": rng.choice(["f16", "bf16"])}
    if op != "evict":
        c |= {"Hq": Hq}
    if op != "prompt":
        c |= {"page": rng.choice([16, 32, 64, 128, 256])}
    if op in ("prompt", "step"):
        c |= {"window": _log(rng, 1, 3000), "sinks": rng.choice([0, 1, 4, _log(rng, 1, 500)])}
    if op in ("prompt", "weigh"):
        longest = _log(rng, 16, 6000)
        lens = [longest] + [_log(rng, 1, longest) for _ in range(rng.randint(0, 11))]
        rng.shuffle(lens)
        c |= {"lens": ",".join(map(str, lens))}
    if op == "prompt":
        c |= {"fused": rng.random() < 0.5}
    if op == "weigh":
        kind = rng.choice(["one", "some", "all"])
        new = {"one": [1] * len(lens), "some": [_log(rng, 1, n) for n in lens], "all": lens}[kind]
        c |= {"new": ",".join(map(str, new)), "fresh": rng.random() < 0.5}
    if op == "step":
        n = rng.randint(1, 12)
        c |= {"ctx": ",".join(str(_log(rng, 1, 20000)) for _ in range(n)), "layers": 1,
              "tree": rng.choice(["1", ",".join(str(_log(rng, 1, 64)) for _ in range(n))])}
    if op == "evict":
        n, longest = rng.randint(1, 16), _log(rng, 40, 8000)
        c |= {"lens": ",".join(str(_log(rng, 20, longest)) for _ in range(n)), "layers": rng.randint(1, 4),
              "sinks": rng.choice([0, 4, rng.randint(1, 100)]), "heavy": rng.choice([0, _log(rng, 1, longest)]),
              "recent": _log(rng, 1, longest)}
    return c


def _ints(text):
    return [int(x) for x in str(text).split(",")]


def _each(text, n):
    t = _ints(text)
    return t if len(t) == n else t * n


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)
    h = torch.Generator()
    h.manual_seed(7919 * seed + 11)
    return g, h


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(lens):
    return _i32([0] + torch.tensor(lens).cumsum(0).tolist())


def _cache(case, lens, layers, g, h):
    """Pools, and page tables of sequences of these lengths over shuffled pages (-1 behind the last one)."""
    page, need = case["page"], [-(-n // case["page"]) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=h).tolist()
    # table, lengths and references lie in one tensor, so that a pass that starts over copies them at once
    width = max(need) + 1
    state = torch.zeros(len(lens) * (width + 1) + n_pages, dtype=torch.int32)
    table = state[:len(lens) * width].view(len(lens), width)
    table.fill_(-1)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    state[len(lens) * width:len(lens) * (width + 1)] = torch.tensor(lens, dtype=torch.int32)
    used = table[table >= 0].long()
    state[len(lens) * (width + 1):] = torch.bincount(used, minlength=n_pages).to(torch.int32)
    state = state.cuda()
    shape = (layers, n_pages, case["Hkv"], page, case["D"])
    k, v = (torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[case["dtype"]]) for _ in range(2))
    a, b = len(lens) * width, len(lens) * (width + 1)
    return {"k": k, "v": v, "state": state, "table": state[:a].view(len(lens), width), "lens": state[a:b], "refs": state[b:],
            "host_lens": list(lens)}


def _handle(s):
    """What a program keeps of a cache: the library's description of it, where there is one."""
    if own:
        from gqa_attention_forward_gb300 import binding
        s["cache"] = binding.KVPages(s["k"], s["v"], s["table"], s["lens"], s["refs"])
    return s


def _gather(pool, row, at, page):
    """Positions ``at`` of a sequence with this table row: [Hkv, len(at), D]."""
    return pool[row[at // page].long(), :, at % page].transpose(0, 1)


def prepare(case, seed):
    g, h = _gen(seed)
    op, D, Hkv, dt = case["op"], case["D"], case["Hkv"], DTYPES[case["dtype"]]
    s = {"op": op, "scale": 1.0 / math.sqrt(D)}

    def rows(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    if op == "prompt":
        lens, Hq = _ints(case["lens"]), case["Hq"]
        total = sum(lens)
        if case["fused"]:  # one projection's output, cut along the heads
            x = rows(total, Hq + 2 * Hkv, D)
            q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            q, k, v = rows(total, Hq, D), rows(total, Hkv, D), rows(total, Hkv, D)
        return s | {"q": q, "k": k, "v": v, "cu": _cu(lens), "host_lens": lens, "window": case["window"], "sinks": case["sinks"]}
    if op == "step":
        ctx = _ints(case["ctx"])
        T = _each(case["tree"], len(ctx))
        s |= _cache(case, [c + t for c, t in zip(ctx, T)], case["layers"], g, h)
        parents = []
        for t in T:  # a random tree: each token follows an earlier one, or the last committed token (-1)
            parents += [-1] + [int(torch.randint(-1, i, (1,), generator=h)) for i in range(1, t)]
        s |= {"q": rows(sum(T), case["Hq"], D), "cu": _cu(T), "parents": _i32(parents), "T": max(T),
              "window": case["window"], "sinks": case["sinks"]}
        return _handle(s)
    lens = _ints(case["lens"])
    s |= _cache(case, lens, case.get("layers", 1), g, h)
    positions = s["table"].shape[1] * case["page"]
    if op == "weigh":
        new = _each(case["new"], len(lens))
        q = rows(sum(new), case["Hq"], D)
        s |= {"q": q, "cu": _cu(new), "host_new": new, "fresh": case["fresh"]}
        # what the attention of the same step has left: the log-sum-exp of each query row
        s["lse"] = torch.empty((case["Hq"], sum(new)), dtype=torch.float32, device="cuda")
        at = 0
        for i, (n, t) in enumerate(zip(lens, new)):
            k = _gather(s["k"][0], s["table"][i], torch.arange(n, device="cuda"), case["page"]).float()
            for r in range(0, t, 1024):
                x = q[at + r:at + min(r + 1024, t)].float().view(-1, Hkv, case["Hq"] // Hkv, D)
                x = torch.einsum("thgd,hld->hgtl", x, k).mul_(s["scale"])
                pos = torch.arange(n - t + r, n - t + r + x.shape[2], device="cuda")
                x.masked_fill_(torch.arange(n, device="cuda") > pos[:, None], -math.inf)
                s["lse"][:, at + r:at + r + x.shape[2]] = torch.logsumexp(x, -1).reshape(case["Hq"], -1)
            at += t
        # sums of the steps before, and what another sequence may have left behind the end
        s["weights"] = torch.rand((1, len(lens), Hkv, positions), generator=g, device="cuda")
        s["weights0"] = s["weights"].clone()
        return _handle(s)
    # evict: sums over many steps, most of them small, a few large, some never looked at
    w = torch.randn((case.get("layers", 1), len(lens), Hkv, positions), generator=g, device="cuda").mul_(2.0).exp_()
    w[w < 0.02] = 0.0
    if case["heavy"] == 0:
        w = None
    s |= {"weights": w, "sinks": case["sinks"], "heavy": case["heavy"], "recent": case["recent"],
          "seqs": torch.randperm(len(lens), generator=h).to(torch.int32).cuda()}
    # cut again and again on one state: tables, lengths, references and weights as they were before
    s |= {"state0": s["state"].clone(), "weights0": None if w is None else w.clone()}
    return _handle(s)


# ---------------------------------------------------------------- one pass
def run(s):
    return {"prompt": _prompt, "step": _step, "weigh": _weigh, "evict": _evict}[s["op"]](s)


def _softmax_product(scores, mask, v):
    """softmax over the allowed columns times v, and the log-sum-exp; scores are overwritten."""
    scores.masked_fill_(~mask, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = scores.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / total, (m + total.log()).squeeze(-1)


def _prompt(s):
    q, k, v, window, sinks = s["q"], s["k"], s["v"], s["window"], s["sinks"]
    if own:
        from gqa_attention_forward_gb300 import binding
        return binding.attention_varlen(q, k, v, s["cu"], scale=s["scale"], window=window, sinks=sinks)
    total, Hq, D = q.shape
    Hkv = k.shape[1]
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty((Hq, total), dtype=torch.float32, device=q.device)
    at = 0
    for n in s["host_lens"]:
        for r in range(0, n, 1024):  # a block of rows and the band of keys that some of them see
            e = min(r + 1024, n)
            lo = max(0, r - window + 1)
            key = torch.cat([torch.arange(min(sinks, lo), device=q.device), torch.arange(lo, e, device=q.device)])
            kf, vf = (x[at + key].float().transpose(0, 1) for x in (k, v))
            qf = q[at + r:at + e].float().view(e - r, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3)
            scores = torch.matmul(qf.reshape(Hkv, -1, D), kf.transpose(1, 2)).mul_(s["scale"]).view(Hkv, Hq // Hkv, e - r, -1)
            pos = torch.arange(r, e, device=q.device)[:, None]
            x, l = _softmax_product(scores, (key <= pos) & ((key > pos - window) | (key < sinks)), vf[:, None])
            o[at + r:at + e] = x.permute(2, 0, 1, 3).reshape(e - r, Hq, D).to(q.dtype)
            lse[:, at + r:at + e] = l.reshape(Hq, e - r)
        at += n
    return o, lse


def _step(s):
    q, cu, window, sinks = s["q"], s["cu"], s["window"], s["sinks"]
    if own:
        from gqa_attention_forward_gb300 import binding
        return binding.attention_tree(q, s["cache"], cu, parents=s["parents"], scale=s["scale"], window=window, sinks=sinks)
    k, v, lens = s["k"][0], s["v"][0], s["lens"].long()
    total, Hq, D = q.shape
    n, T, page, Hkv = lens.numel(), s["T"], k.shape[2], k.shape[1]
    t = cu.diff().long()
    base = lens - t
    pos = torch.arange(T, device=q.device)
    valid = pos < t[:, None]
    at = torch.where(valid, cu[:-1, None].long() + pos, 0)
    # ancestors: (1 + parent matrix) to the power T counts the ways down, zero where there is none
    par = torch.where(valid, s["parents"].long()[at], -1)
    step = (par[:, :, None] == pos).double() + torch.eye(T, dtype=torch.float64, device=q.device)
    anc = torch.linalg.matrix_power(step, T) > 0  # [n, token, ancestor or itself]
    depth = anc.sum(-1) - 1
    near = (depth[:, None, :] > depth[:, :, None] - window) | ((base[:, None] + depth)[:, None, :] < sinks)
    # the positions that some token of the sequence sees: the first ones, the window, the tree
    longest = max(s["host_lens"])
    m = min(longest, min(sinks, longest) + window - 1 + T)
    lo = (lens - (m - min(sinks, longest))).clamp(min=0)
    key = torch.arange(m, device=q.device)
    first = torch.minimum(lo, torch.full_like(lo, sinks))[:, None]
    key = torch.where(key < first, key, lo[:, None] + key - first)  # [n, m], past the end where a sequence is short
    inside = key < lens[:, None]
    key = torch.where(inside, key, 0)
    pages = torch.gather(s["table"].long(), 1, key // page)
    kf = k[pages, :, key % page].float().transpose(1, 2)
    vf = v[pages, :, key % page].float().transpose(1, 2)
    node = key - base[:, None]
    tree = torch.gather(anc & near, 2, node.clamp(0, T - 1)[:, None].expand(n, T, m)) & (node >= 0)[:, None]
    at_pos = (base[:, None] + depth)[:, :, None]
    old = (node < 0)[:, None] & ((key[:, None] > at_pos - window) | (key < sinks)[:, None])
    mask = (tree | old) & inside[:, None] | ~valid[:, :, None]
    qf = q[at].float().view(n, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    scores = torch.matmul(qf.reshape(n, Hkv, -1, D), kf.transpose(2, 3)).mul_(s["scale"])
    o, lse = _softmax_product(scores.view(n, Hkv, Hq // Hkv, T, m), mask[:, None, None], vf[:, :, None])
    o = o.permute(0, 3, 1, 2, 4).reshape(n, T, Hq, D)[valid]
    lse = lse.permute(0, 3, 1, 2).reshape(n, T, Hq)[valid]
    return o.to(q.dtype), lse.t().contiguous()


def _weigh(s):
    q, lse, weights = s["q"], s["lse"], s["weights"]
    if not s["fresh"]:  # taken again and again on one state, each time from the same sums
        weights.copy_(s["weights0"])
    if own:
        from gqa_attention_forward_gb300 import binding
        binding.kv_weigh(s["cache"], weights, q, lse, s["cu"], scale=s["scale"], accumulate=not s["fresh"])
        return weights
    k, page = s["k"][0], s["k"].shape[3]
    total, Hq, D = q.shape
    Hkv = k.shape[1]
    at = 0
    for i, (n, t) in enumerate(zip(s["host_lens"], s["host_new"])):
        key = torch.arange(n, device=q.device)
        kf = _gather(k, s["table"][i], key, page).float()
        x = weights[0, i]
        x[:, n - t:n] = 0.0  # the new tokens' own positions begin here
        if s["fresh"]:
            x[:, :n - t] = 0.0
        for r in range(0, t, 1024):
            e = min(r + 1024, t)
            qf = q[at + r:at + e].float().view(e - r, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
            p = torch.matmul(qf, kf.transpose(1, 2)).mul_(s["scale"]).view(Hkv, Hq // Hkv, e - r, n)
            p = p.sub_(lse[:, at + r:at + e].view(Hkv, Hq // Hkv, e - r, 1)).exp_()
            pos = torch.arange(n - t + r, n - t + e, device=q.device)
            x[:, :n] += p.masked_fill_(key > pos[:, None], 0.0).sum((1, 2))
        at += t
    return weights


def _pools(s):
    x = {n: s[n] for n in ("k", "v", "table", "lens", "refs")}
    return x if s["weights"] is None else x | {"weights": s["weights"]}


def _evict(s):
    k, v, table, lens, refs, weights = (s[x] for x in ("k", "v", "table", "lens", "refs", "weights"))
    sinks, heavy, recent = s["sinks"], s["heavy"], s["recent"]
    s["state"].copy_(s["state0"])
    if weights is not None:
        weights.copy_(s["weights0"])
    if own:
        from gqa_attention_forward_gb300 import binding
        binding.kv_evict(s["cache"], s["seqs"], weights, sinks=sinks, heavy=heavy, recent=recent)
        return _pools(s)
    layers, N, Hkv, page, D = k.shape
    keep, dev = sinks + heavy + recent, k.device
    L = torch.arange(layers, device=dev)[:, None, None]
    H = torch.arange(Hkv, device=dev)[None, :, None]
    for i, n in enumerate(s["host_lens"]):
        if n <= keep:
            continue
        at = torch.arange(n, device=dev).expand(layers, Hkv, n)
        best = at[:, :, :0]
        if heavy > 0:  # ties go to the lowest position
            best = torch.sort(weights[:, i, :, sinks:n - recent], dim=-1, descending=True, stable=True).indices[:, :, :heavy] + sinks
        src = torch.cat([at[:, :, :sinks], torch.sort(best, dim=-1).values, at[:, :, n - recent:]], -1)
        dst = at[:, :, :keep]
        row = table[i].long()
        for x in (k, v):
            x[L, row[dst // page], H, dst % page] = x[L, row[src // page], H, src % page]
        if weights is not None:
            weights[:, i, :, :keep] = torch.gather(weights[:, i], 2, src)
            weights[:, i, :, keep:n] = 0.0
        used = -(-keep // page)
        refs -= torch.bincount(row[used:][row[used:] >= 0], minlength=N).to(torch.int32)
        table[i, used:] = -1
    lens.clamp_(max=keep)
    return _pools(s)


# ---------------------------------------------------------------- floors
def _seen(p, window, sinks):
    """Keys that position p sees."""
    return min(p + 1, window) + max(0, min(sinks, p - window + 1))


def work(case):
    op, D, Hkv = case["op"], case["D"], case["Hkv"]
    row = D * 2
    if op == "prompt":
        lens = _ints(case["lens"])
        n = sum(lens)
        return {"bytes": n * (2 * case["Hq"] + 2 * Hkv) * row + n * case["Hq"] * 4,
                "flops": 4 * case["Hq"] * D * sum(_seen(p, case["window"], case["sinks"]) for x in lens for p in range(x))}
    if op == "step":
        ctx = _ints(case["ctx"])
        T = _each(case["tree"], len(ctx))
        n, seen = sum(T), [_seen(c, case["window"], case["sinks"]) for c in ctx]
        return {"bytes": sum(x + t - 1 for x, t in zip(seen, T)) * 2 * Hkv * row + n * case["Hq"] * (2 * row + 4),
                "flops": 4 * case["Hq"] * D * sum(x * t for x, t in zip(seen, T))}
    lens = _ints(case["lens"])
    if op == "weigh":
        new = _each(case["new"], len(lens))
        return {"bytes": sum(lens) * Hkv * (row + (4 if case["fresh"] else 8)) + sum(new) * case["Hq"] * (row + 4),
                "flops": 2 * case["Hq"] * D * sum(t * (n - t) + t * (t + 1) // 2 for n, t in zip(lens, new))}
    keep, bytes_ = case["sinks"] + case["heavy"] + case["recent"], 0
    for n in lens:
        if n > keep:
            moved = case["heavy"] + case["recent"]
            bytes_ += case["layers"] * Hkv * (moved * 2 * 2 * row + (0 if case["heavy"] == 0 else (n - case["sinks"]) * 8))
    return {"bytes": bytes_ + len(lens) * 8, "flops": 0}


# ---------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, dev, Hkv = case["op"], "cuda", case["Hkv"]
    f64 = {"dtype": torch.float64, "device": dev}
    if op in ("prompt", "step"):
        q, window, sinks = s["q"].double(), case["window"], case["sinks"]
        total, Hq, D = q.shape
        G = Hq // Hkv
        o, lse, cu = torch.empty(q.shape, **f64), torch.empty((Hq, total), **f64), s["cu"].tolist()
        for i, (a, b) in enumerate(zip(cu, cu[1:])):
            for r in range(a, b, 512):
                e = min(r + 512, b)
                if op == "prompt":
                    # rows r .. e of the sequence: the union of the keys they see
                    keys = sorted(set(range(min(sinks, e - a))) | set(range(max(0, r - a - window + 1), e - a)))
                    at = torch.tensor(keys, device=dev)
                    kk, vv = s["k"][a + at].double(), s["v"][a + at].double()
                    p = torch.arange(r - a, e - a, device=dev)[:, None]
                    see = (at <= p) & ((p - at < window) | (at < sinks))
                else:
                    n = s["host_lens"][i]
                    base, par = n - (b - a), s["parents"][a:b].tolist()
                    seen_by = []
                    for t in range(r - a, e - a):  # positions along the token's path, the token itself last
                        path, u = [], t
                        while u >= 0:
                            path.append(u)
                            u = par[u]
                        path = list(range(base)) + [base + u for u in reversed(path)]
                        seen_by.append(set(path[:sinks]) | set(path[-window:]))
                    keys = sorted(set().union(*seen_by))
                    at = torch.tensor(keys, device=dev)
                    kk, vv = (_gather(x[0], s["table"][i], at, case["page"]).transpose(0, 1).double() for x in (s["k"], s["v"]))
                    place = {key: j for j, key in enumerate(keys)}
                    see = np.zeros((e - r, len(keys)), dtype=bool)
                    for t, mine in enumerate(seen_by):
                        see[t, [place[key] for key in mine]] = True
                    see = torch.from_numpy(see).to(dev)
                for h in range(Hkv):
                    x = torch.einsum("tgd,ld->gtl", q[r:e, h * G:(h + 1) * G], kk[:, h]) * s["scale"]
                    x = x.masked_fill(~see, -math.inf)
                    l = torch.logsumexp(x, -1)
                    o[r:e, h * G:(h + 1) * G] = torch.einsum("gtl,ld->tgd", torch.exp(x - l[:, :, None]), vv[:, h])
                    lse[h * G:(h + 1) * G, r:e] = l
        return o, lse
    page = case["page"]
    if op == "weigh":
        out, q, lse = s["weights"].double(), s["q"].double(), s["lse"].double()
        G, at = case["Hq"] // Hkv, 0
        for i, n in enumerate(s["host_lens"]):
            t = s["host_new"][i]
            old = n - t
            out[0, i, :, 0 if case["fresh"] else old:n] = 0.0
            key = torch.arange(n, device=dev)
            for h in range(Hkv):
                kk = _gather(s["k"][0], s["table"][i], key, page)[h].double()
                for g in range(G):
                    for r in range(0, t, 2048):
                        x = q[at + r:at + min(t, r + 2048), h * G + g] @ kk.T * s["scale"]
                        x = torch.exp(x - lse[h * G + g, at + r:at + min(t, r + 2048), None])
                        out[0, i, h, :n] += torch.tril(x, old + r).sum(0)
            at += t
        return out
    # what eviction keeps is written out sequence by sequence, layer by layer and head by head
    sinks, heavy, recent = case["sinks"], case["heavy"], case["recent"]
    keep = sinks + heavy + recent
    k, v = s["k"].double(), s["v"].double()
    w = None if s["weights"] is None else s["weights"].cpu().numpy().astype(np.float64)
    table, refs, lens = s["table"].cpu().numpy().copy(), s["refs"].cpu().numpy().copy(), list(s["host_lens"])
    for i, n in enumerate(s["host_lens"]):
        if n <= keep:
            continue
        for layer in range(case["layers"]):
            for h in range(Hkv):
                middle = np.arange(sinks, n - recent)
                if heavy:
                    order = np.lexsort((middle, -w[layer, i, h, middle]))  # heaviest first, then lowest
                    middle = np.sort(middle[order[:heavy]])
                else:
                    middle = middle[:0]
                src = np.concatenate([np.arange(sinks), middle, np.arange(n - recent, n)])
                a, ao, b, bo = (torch.from_numpy(x).to(dev).long() for x in (
                    table[i, src // page], src % page, table[i, np.arange(keep) // page], np.arange(keep) % page))
                for x in (k, v):
                    x[layer, b, h, bo] = x[layer, a, h, ao]
                if w is not None:
                    w[layer, i, h, :keep] = w[layer, i, h, src]
                    w[layer, i, h, keep:n] = 0.0
        for j in range(-(-keep // page), table.shape[1]):
            if table[i, j] >= 0:
                refs[table[i, j]] -= 1
                table[i, j] = -1
        lens[i] = keep
    out = {"k": k, "v": v, "table": _i32(table.tolist()), "lens": _i32(lens), "refs": _i32(refs.tolist())}
    return out if w is None else out | {"weights": torch.from_numpy(w).to(dev)}
