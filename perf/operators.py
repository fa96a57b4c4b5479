"""The operators of packed prompts and of the paged key/value cache, as cases to be timed.

A serving program runs them in this order: prompts of different lengths go through one
packed causal attention; their keys and values are appended to the pages of a cache; each
step, a tree of drafted tokens (one token in plain decoding) attends over the pages, and the
accepted path of the tree stays in the cache; sequences fork and are freed as a search or a
sampler goes on, and from time to time the live pages are moved to the front of the pool.

With ``own`` false, ``run`` computes an operator with elementary torch operations in 32 bits
and rounds once; with ``own`` true it makes the library's calls.  Head counts, head dimensions
and types are those of the library's workloads (Hq/Hkv 2/1, 16/8, 32/8; D 64 and 128; fp16, bf16).
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one short prompt through a tiny model: launch latency
        {"name": "prompt_one", "op": "varlen", "lens": "37", "Hq": 2, "Hkv": 1, "D": 64, "dtype": "f16", "fused": False},
        # a batch of chat turns, from one token to a page of text, q/k/v cut from one projection
        {"name": "prompts_short", "op": "varlen", "lens": "1,17,64,100,128,129,200,255,256,300,333,400,411,480,500,512",
         "Hq": 16, "Hkv": 8, "D": 128, "dtype": "f16", "fused": True},
        # a prefill batch of mixed prompts
        {"name": "prompts_mixed", "op": "varlen", "lens": "4096,33,2000,1,777,1024,128,3001,513,256,90,1500",
         "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "fused": False},
        # two long documents
        {"name": "prompts_long", "op": "varlen", "lens": "16384,9001", "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16",
         "fused": False},
        # a small draft tree over a short chat: latency
        {"name": "tree_small", "op": "tree", "ctx": "300", "tree": "8", "Hq": 16, "Hkv": 8, "D": 64, "dtype": "f16",
         "page": 16, "layers": 1},
        # one decoding step of a batch (a tree of one token each)
        {"name": "tree_one_token", "op": "tree", "ctx": "8191,4000,8000,1,6500,7777,513,8191,3000,8100,5000,64,7000,8191,2222,6000",
         "tree": "1", "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "layers": 1},
        # verifying draft trees of different sizes
        {"name": "tree_batch", "op": "tree", "ctx": "12000,700,5000,2049,9000,130,7000,3333", "tree": "26,64,7,1,48,33,60,16",
         "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 32, "layers": 1},
        # one draft tree over a very long context
        {"name": "tree_long", "op": "tree", "ctx": "131000", "tree": "25", "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16",
         "page": 64, "layers": 1},
        # a step of a beam search: the losing beams are freed and the winners forked into their place
        {"name": "pages_beam", "op": "beam", "parents": 24, "children": 96, "ctx": 900, "Hkv": 8, "D": 128, "dtype": "bf16",
         "page": 16, "layers": 8, "pages": 3000},
        # a fragmented pool made dense
        {"name": "pages_compact", "op": "compact", "seqs": 48, "ctx": 1500, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64,
         "layers": 4, "pages": 2400},
        # the keys and values of prefilled prompts go into their pages
        {"name": "pages_append", "op": "append", "lens": "4096,33,2000,1,777,1024,128,3001,513,256,90,1500", "ctx": 100,
         "Hkv": 8, "D": 128, "dtype": "bf16", "page": 32, "fused": True},
        # after verification: the accepted path of each tree stays, in every layer
        {"name": "pages_accept", "op": "accept", "seqs": 32, "ctx": 1000, "tree": 48, "accepted": 5, "Hkv": 8, "D": 128,
         "dtype": "bf16", "page": 32, "layers": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["varlen", "varlen", "tree", "tree", "beam", "compact", "append", "accept"])
    Hq, Hkv = rng.choice([(2, 1), (16, 8), (32, 8), (8, 8), (12, 4)])
    c = {"op": op, "Hkv": Hkv, "D": rng.choice([64, 128]), "dtype": rng.choice(["f16", "bf16"])}
    if op in ("varlen", "append"):
        longest = _log(rng, 16, 6000)
        lens = [longest] + [_log(rng, 1, longest) for _ in range(rng.randint(0, 11))]
        rng.shuffle(lens)
        c |= {"lens": ",".join(map(str, lens)), "fused": rng.random() < 0.5}
    if op in ("varlen", "tree"):
        c |= {"Hq": Hq}
    if op != "varlen":
        c |= {"page": rng.choice([16, 32, 64, 128])}
    if op == "append":
        c |= {"ctx": _log(rng, 1, 2000)}
    if op == "tree":
        n = rng.randint(1, 12)
        c |= {"ctx": ",".join(str(_log(rng, 1, 20000)) for _ in range(n)), "layers": 1,
              "tree": rng.choice(["1", ",".join(str(_log(rng, 1, 64)) for _ in range(n))])}
    if op == "beam":
        n = rng.randint(1, 16)
        c |= {"parents": n, "children": n * rng.randint(1, 4), "ctx": _log(rng, 30, 900), "layers": rng.randint(1, 8)}
        c["pages"] = (n * (1 + c["children"] // n)) * (c["ctx"] * 2 // c["page"] + 2) + 5
    if op == "compact":
        c |= {"seqs": rng.randint(2, 32), "ctx": _log(rng, 30, 1500), "layers": rng.randint(1, 4)}
        c["pages"] = 2 * c["seqs"] * (c["ctx"] * 3 // 2 // c["page"] + 2)
    if op == "accept":
        c |= {"seqs": rng.randint(1, 32), "ctx": _log(rng, 10, 2000), "tree": rng.randint(8, 64),
              "accepted": rng.randint(1, 6), "layers": rng.randint(1, 8)}
    return c


def _ints(text):
    return [int(x) for x in str(text).split(",")]


def _tree_sizes(case):
    n, t = len(_ints(case["ctx"])), _ints(case["tree"])
    return t if len(t) == n else t * n


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    h = torch.Generator()
    h.manual_seed(7919 * seed + 3)
    return g, h


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(lens):
    return _i32([0] + torch.tensor(lens).cumsum(0).tolist())


def _pool(case, n_pages, layers, g):
    shape = (layers, n_pages, case["Hkv"], case["page"], case["D"])
    return [torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[case["dtype"]]) for _ in range(2)]


def _tables(lens, page, pool_pages, h, longest=0):
    """Page tables of sequences of these lengths over shuffled pages (-1 behind the last one)."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(pool_pages, generator=h).tolist()
    table = torch.full((len(lens), -(-max(longest, *lens, 1) // page) + 2), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return table


def _refs(table, n_pages):
    used = table[table >= 0].long()
    return torch.bincount(used, minlength=n_pages).to(torch.int32)


def _handle(s):
    """What a program keeps of a cache: the library's description of it, where there is one."""
    if own:
        from gqa_attention_forward_gb300 import binding
        s["cache"] = binding.KVPages(s["k"], s["v"], s["table"], s["lens"], s["refs"])
    return s


def prepare(case, seed):
    g, h = _gen(seed)
    op, D, Hkv, dt = case["op"], case["D"], case["Hkv"], DTYPES[case["dtype"]]
    s = {"op": op, "scale": 1.0 / math.sqrt(D)}

    def rows(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    if op == "varlen":
        lens, Hq = _ints(case["lens"]), case["Hq"]
        total = sum(lens)
        if case["fused"]:  # one projection's output, cut along the heads
            x = rows(total, Hq + 2 * Hkv, D)
            q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            q, k, v = rows(total, Hq, D), rows(total, Hkv, D), rows(total, Hkv, D)
        return s | {"q": q, "k": k, "v": v, "cu": _cu(lens), "longest": max(lens)}
    if op == "tree":
        ctx, T, Hq, page = _ints(case["ctx"]), _tree_sizes(case), case["Hq"], case["page"]
        lens = [c + t for c, t in zip(ctx, T)]
        n_pages = sum(-(-n // page) for n in lens) + 3
        k, v = _pool(case, n_pages, case["layers"], g)
        table = _tables(lens, page, n_pages, h)
        parents = []
        for t in T:  # a random tree: each token follows an earlier one, or the last committed token (-1)
            parents += [-1] + [int(torch.randint(-1, i, (1,), generator=h)) for i in range(1, t)]
        total = sum(T)
        s |= {"q": rows(total, Hq, D), "k": k, "v": v, "table": table.cuda(), "lens": _i32(lens),
              "refs": _refs(table, n_pages).cuda(), "cu": _cu(T), "parents": _i32(parents), "T": max(T),
              "longest": max(lens)}
        return _handle(s)
    page, layers = case["page"], case.get("layers", 1)
    if op == "beam":
        # rows [0, n) of the table are the winners, rows [n, n + m) the losing beams that the step replaces
        n, m, N = case["parents"], case["children"], case["pages"]
        lens = [int(x) for x in torch.randint(max(1, case["ctx"] // 2), case["ctx"] * 2, (n,), generator=h)]
        table = _tables(lens, page, N, h, case["ctx"] * 2)
        table = torch.cat([table, torch.full((m, table.shape[1]), -1, dtype=torch.int32)])
        full = (torch.tensor(lens) // page).tolist()
        free = sorted(set(range(N)) - set(table[table >= 0].tolist()))
        src = [i % n for i in range(m)]
        for i, p in enumerate(src):
            table[n + i, :full[p]] = table[p, :full[p]]
            if lens[p] % page:
                table[n + i, full[p]] = free.pop(0)
        k, v = _pool(case, N, layers, g)
        pick = torch.randint(0, n, (m,), generator=h).tolist()
        s |= {"k": k, "v": v, "table": table.cuda(), "lens": _i32(lens + [lens[p] for p in src]),
              "refs": _refs(table, N).cuda(), "losers": _i32(list(range(n, n + m))), "winners": _i32(pick)}
        # the step is taken again and again on one state, each time from the same beams
        s |= {"table0": s["table"].clone(), "lens0": s["lens"].clone(), "refs0": s["refs"].clone()}
        return _handle(s)
    if op == "compact":
        n, N = case["seqs"], case["pages"]
        lens = [int(x) for x in torch.randint(max(1, case["ctx"] // 2), case["ctx"] * 3 // 2, (n,), generator=h)]
        table = _tables(lens, page, N, h, case["ctx"] * 3 // 2)
        if n > 2:  # the last sequence shares the full pages of the first
            full = min(lens[0], lens[-1]) // page
            table[-1, :full] = table[0, :full]
        k, v = _pool(case, N, layers, g)
        s |= {"k": k, "v": v, "table": table.cuda(), "lens": _i32(lens), "refs": _refs(table, N).cuda()}
        # compacting is timed again and again on one state: the tables as they were before
        s |= {"table0": s["table"].clone(), "refs0": s["refs"].clone()}
        return _handle(s)
    if op == "append":
        new = _ints(case["lens"])
        lens = [case["ctx"] + i % 7 + n for i, n in enumerate(new)]
        N = sum(-(-n // page) for n in lens) + 3
        k, v = _pool(case, N, 1, g)
        table = _tables(lens, page, N, h)
        total = sum(new)
        if case["fused"]:
            x = rows(total, 2 * Hkv, D)
            k_new, v_new = x[:, :Hkv], x[:, Hkv:]
        else:
            k_new, v_new = rows(total, Hkv, D), rows(total, Hkv, D)
        s |= {"k": k, "v": v, "table": table.cuda(), "lens": _i32(lens), "refs": _refs(table, N).cuda(),
              "k_new": k_new, "v_new": v_new, "cu": _cu(new)}
        return _handle(s)
    # accept: the path's first token stays where it is and the others come from behind the path, as in a tree whose
    # levels are wide, so that the step can be taken again on one state
    n, T, a = case["seqs"], case["tree"], case["accepted"]
    lens = [case["ctx"] + 13 * i + T for i in range(n)]
    N = sum(-(-x // page) for x in lens) + 3
    k, v = _pool(case, N, layers, g)
    table = _tables(lens, page, N, h)
    path = torch.full((n, a), -1, dtype=torch.int32)
    taken = torch.randint(1, a + 1, (n,), generator=h)
    for i in range(n):
        m = min(int(taken[i]), T - a + 1)
        taken[i] = m
        path[i, 0] = 0
        if m > 1:
            path[i, 1:m] = torch.sort(torch.randperm(T - a, generator=h)[:m - 1] + a).values.to(torch.int32)
    s |= {"k": k, "v": v, "table": table.cuda(), "lens": _i32(lens), "refs": _refs(table, N).cuda(),
          "cu": _cu([T] * n), "path": path.cuda(), "taken": taken.to(torch.int32).cuda()}
    s |= {"lens0": s["lens"].clone()}
    return _handle(s)


# ---------------------------------------------------------------- one pass
def run(s):
    return {"varlen": _varlen, "tree": _tree, "beam": _beam, "compact": _compact, "append": _append, "accept": _accept}[s["op"]](s)


def _softmax_product(scores, mask, v):
    """softmax over the allowed columns times v, and the log-sum-exp; scores are overwritten."""
    scores.masked_fill_(~mask, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = scores.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / total, (m + total.log()).squeeze(-1)


def _varlen(s):
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu"]
    if own:
        from gqa_attention_forward_gb300 import binding
        return binding.attention_varlen(q, k, v, cu, causal=True, scale=s["scale"])
    total, Hq, D = q.shape
    Hkv, m = k.shape[1], s["longest"]
    start, lens = cu[:-1].long(), cu.diff().long()
    pos = torch.arange(m, device=q.device)
    valid = pos < lens[:, None]
    at = torch.where(valid, start[:, None] + pos, 0)  # [n, m]: sequences padded to the longest
    n = lens.numel()
    kf = k[at].float().permute(0, 2, 1, 3)
    vf = v[at].float().permute(0, 2, 1, 3)
    qf = q[at].float().view(n, m, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    scores = torch.matmul(qf.reshape(n, Hkv, -1, D), kf.transpose(2, 3)).mul_(s["scale"])
    scores = scores.view(n, Hkv, Hq // Hkv, m, m)
    mask = (pos[:, None] >= pos)[None, None, None]  # a padded row sees keys too; it is dropped below
    o, lse = _softmax_product(scores, mask, vf[:, :, None])
    o = o.permute(0, 3, 1, 2, 4).reshape(n, m, Hq, D)[valid]
    lse = lse.permute(0, 3, 1, 2).reshape(n, m, Hq)[valid]
    return o.to(q.dtype), lse.t().contiguous()


def _tree(s):
    q, cu = s["q"], s["cu"]
    if own:
        from gqa_attention_forward_gb300 import binding
        return binding.attention_tree(q, s["cache"], cu, parents=s["parents"], scale=s["scale"])
    k, v, lens = s["k"][0], s["v"][0], s["lens"].long()
    total, Hq, D = q.shape
    n, T, L, page = lens.numel(), s["T"], s["longest"], k.shape[2]
    Hkv = k.shape[1]
    t = cu.diff().long()
    pos = torch.arange(T, device=q.device)
    valid = pos < t[:, None]
    at = torch.where(valid, cu[:-1, None].long() + pos, 0)
    # ancestors: (1 + parent matrix) to the power T counts the ways down, zero where there is none
    par = torch.where(valid, s["parents"].long()[at], -1)
    step = (par[:, :, None] == pos).double() + torch.eye(T, dtype=torch.float64, device=q.device)
    anc = torch.linalg.matrix_power(step, T) > 0  # [n, token, ancestor or itself]
    key = torch.arange(L, device=q.device)
    pages = s["table"][:, : -(-L // page)].long().clamp(min=0)
    kf = k[pages].float().permute(0, 2, 1, 3, 4).reshape(n, Hkv, -1, D)[:, :, :L]
    vf = v[pages].float().permute(0, 2, 1, 3, 4).reshape(n, Hkv, -1, D)[:, :, :L]
    base = lens - t
    node = key - base[:, None]  # [n, L]: which token of the tree a position holds
    inside = (node >= 0) & (key < lens[:, None])
    seen = torch.gather(anc, 2, node.clamp(0, T - 1)[:, None].expand(n, T, L)) & inside[:, None]
    mask = seen | (node < 0)[:, None]
    qf = q[at].float().view(n, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    scores = torch.matmul(qf.reshape(n, Hkv, -1, D), kf.transpose(2, 3)).mul_(s["scale"])
    scores = scores.view(n, Hkv, Hq // Hkv, T, L)
    o, lse = _softmax_product(scores, mask[:, None, None], vf[:, :, None])
    o = o.permute(0, 3, 1, 2, 4).reshape(n, T, Hq, D)[valid]
    lse = lse.permute(0, 3, 1, 2).reshape(n, T, Hq)[valid]
    return o.to(q.dtype), lse.t().contiguous()


def _state(s):
    return {x: s[x] for x in ("k", "v", "table", "lens", "refs")}


def _beam(s):
    k, v, table, lens, refs = (s[x] for x in ("k", "v", "table", "lens", "refs"))
    table.copy_(s["table0"])
    lens.copy_(s["lens0"])
    refs.copy_(s["refs0"])
    if own:
        from gqa_attention_forward_gb300 import binding
        binding.kv_free(s["cache"], s["losers"])
        binding.kv_fork(s["cache"], s["winners"], s["losers"])
        return _state(s)
    a, b, page = s["winners"].long(), s["losers"].long(), k.shape[3]
    N = refs.numel()
    # free: one reference less for each page of a loser
    old = table[b]
    refs -= torch.bincount(old[old >= 0].long(), minlength=N).to(torch.int32)
    # fork: full pages are shared; a page that is not full is copied to the lowest free page
    n = lens[a].long()
    full, rest = n // page, n % page
    col = torch.arange(table.shape[1], device=k.device)
    row = torch.where(col < full[:, None], table[a], -1)
    free = torch.nonzero(refs == 0).squeeze(1)
    part = torch.nonzero(rest > 0).squeeze(1)
    dst = free[: part.numel()]
    src = table[a[part], full[part]].long()
    row[part, full[part]] = dst.to(torch.int32)
    keep = (torch.arange(page, device=k.device) < rest[part, None])[None, :, None, :, None]
    k[:, dst] = torch.where(keep, k[:, src], k[:, dst])
    v[:, dst] = torch.where(keep, v[:, src], v[:, dst])
    table[b] = row
    lens[b] = lens[a]
    refs += torch.bincount(row[row >= 0].long(), minlength=N).to(torch.int32)
    return _state(s)


def _compact(s):
    k, v, table, refs = (s[x] for x in ("k", "v", "table", "refs"))
    table.copy_(s["table0"])
    refs.copy_(s["refs0"])
    if own:
        from gqa_attention_forward_gb300 import binding
        live = binding.kv_compact(s["cache"])
        return _state(s) | {"live": live}
    used = refs > 0
    live = used.sum()
    index = torch.arange(refs.numel(), device=k.device)
    holes = index[~used & (index < live)]
    movers = index[used & (index >= live)]
    k[:, holes] = k[:, movers]
    v[:, holes] = v[:, movers]
    refs[holes] = refs[movers]
    refs[movers] = 0
    to = index.clone()
    to[movers] = holes
    table.copy_(torch.where(table >= 0, to[table.long().clamp(min=0)].to(torch.int32), table))
    return _state(s) | {"live": live.to(torch.int32).view(1)}


def _append(s):
    if own:
        from gqa_attention_forward_gb300 import binding
        binding.kv_append(s["cache"], s["k_new"], s["v_new"], s["cu"])
        return s["k"], s["v"]
    cu, lens, page = s["cu"].long(), s["lens"].long(), s["k"].shape[3]
    total = s["k_new"].shape[0]
    t = torch.arange(total, device=cu.device)
    seq = (t[:, None] >= cu[1:]).sum(1)
    pos = lens[seq] - (cu[seq + 1] - t)
    at, row = s["table"][seq, pos // page].long(), pos % page
    s["k"][0, at, :, row] = s["k_new"]
    s["v"][0, at, :, row] = s["v_new"]
    return s["k"], s["v"]


def _accept(s):
    s["lens"].copy_(s["lens0"])
    if own:
        from gqa_attention_forward_gb300 import binding
        binding.kv_accept(s["cache"], s["cu"], s["path"], s["taken"])
        return s["k"], s["v"], s["lens"]
    k, v, lens, page = s["k"], s["v"], s["lens"], s["k"].shape[3]
    base = lens.long() - s["cu"].diff().long()
    path, taken = s["path"].long(), s["taken"].long()
    j = torch.arange(path.shape[1], device=k.device)
    i, j = torch.nonzero(j < taken[:, None], as_tuple=True)
    src, dst = base[i] + path[i, j], base[i] + j
    ps, pd = s["table"][i, src // page].long(), s["table"][i, dst // page].long()
    k[:, pd, :, dst % page] = k[:, ps, :, src % page]
    v[:, pd, :, dst % page] = v[:, ps, :, src % page]
    lens.copy_(base + taken)
    return k, v, lens


# ---------------------------------------------------------------- floors
def work(case):
    op, D, Hkv = case["op"], case["D"], case["Hkv"]
    row = D * 2
    if op == "varlen":
        lens = _ints(case["lens"])
        n = sum(lens)
        return {"bytes": n * (2 * case["Hq"] + 2 * Hkv) * row + n * case["Hq"] * 4,
                "flops": 4 * case["Hq"] * D * sum(x * (x + 1) // 2 for x in lens)}
    if op == "tree":
        ctx, T = _ints(case["ctx"]), _tree_sizes(case)
        n = sum(T)
        return {"bytes": sum(c + t for c, t in zip(ctx, T)) * 2 * Hkv * row + n * case["Hq"] * (2 * row + 4),
                "flops": 4 * case["Hq"] * D * sum(t * c + t for c, t in zip(ctx, T))}
    page, layers = case["page"], case.get("layers", 1)
    if op == "beam":  # half a page of each child, and the tables of the children
        cols = case["ctx"] * 5 // 4 // page + 1
        return {"bytes": case["children"] * (layers * 2 * Hkv * row * page + 5 * 4 * cols) + case["pages"] * 4, "flops": 0}
    if op == "compact":  # live pages behind the live count are read and written
        live = min(1.0, case["seqs"] * (case["ctx"] + page / 2) / page / case["pages"])
        return {"bytes": live * (1 - live) * case["pages"] * layers * 2 * Hkv * page * row * 2 + case["pages"] * 4, "flops": 0}
    if op == "append":
        return {"bytes": sum(_ints(case["lens"])) * Hkv * row * 4, "flops": 0}
    return {"bytes": max(1, case["accepted"] - 1) / 2 * case["seqs"] * layers * Hkv * row * 4 + case["seqs"] * 64, "flops": 0}


# ---------------------------------------------------------------- the definitions, in 64 bits
def _exact_rows(q, k, v, scale, allowed):
    """One sequence and one kv head: q [G, T, D], k, v [L, D], allowed [T, L]; a block of rows at a time."""
    o = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    for r in range(0, q.shape[1], 2048):
        x = torch.einsum("gtd,ld->gtl", q[:, r:r + 2048], k) * scale
        x = x.masked_fill(~allowed(r, min(r + 2048, q.shape[1])), -math.inf)
        lse[:, r:r + 2048] = torch.logsumexp(x, -1)
        o[:, r:r + 2048] = torch.einsum("gtl,ld->gtd", torch.exp(x - lse[:, r:r + 2048, None]), v)
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    op, dev = case["op"], "cuda"
    if op in ("varlen", "tree"):
        q = s["q"].double()
        total, Hq, D = q.shape
        G = Hq // case["Hkv"]
        o = torch.empty(q.shape, dtype=torch.float64, device=dev)
        lse = torch.empty((Hq, total), dtype=torch.float64, device=dev)
        cu = s["cu"].tolist()
        for i, (a, b) in enumerate(zip(cu, cu[1:])):
            if op == "varlen":
                ks, vs = s["k"][a:b].double().transpose(0, 1), s["v"][a:b].double().transpose(0, 1)

                def allowed(r0, r1, n=b - a):
                    return torch.ones(r1 - r0, n, dtype=torch.bool, device=dev).tril(r0)
            else:
                n = int(s["lens"][i])
                at = s["table"][i, [p // case["page"] for p in range(n)]].long()
                off = torch.arange(n, device=dev) % case["page"]
                ks, vs = (x[0][at, :, off].double().transpose(0, 1) for x in (s["k"], s["v"]))
                see = torch.ones(b - a, n, dtype=torch.bool)
                see[:, n - (b - a):] = False
                par = s["parents"][a:b].tolist()
                for t in range(b - a):
                    u = t
                    while u >= 0:
                        see[t, n - (b - a) + u] = True
                        u = par[u]
                see = see.to(dev)

                def allowed(r0, r1, see=see):
                    return see[r0:r1]
            for h in range(case["Hkv"]):
                x, l = _exact_rows(q[a:b, h * G:(h + 1) * G].transpose(0, 1), ks[h], vs[h], s["scale"], allowed)
                o[a:b, h * G:(h + 1) * G] = x.transpose(0, 1)
                lse[h * G:(h + 1) * G, a:b] = l
        return o, lse
    # the cache's operators move values and count pages: written out page by page and row by row
    k, v, page = s["k"].double(), s["v"].double(), case["page"]
    table, lens, refs = s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()

    def whole(x, like):
        return torch.tensor(x, dtype=torch.int32, device=dev).view(like.shape)

    if op == "beam":
        for c in s["losers"].tolist():
            for p in table[c]:
                if p >= 0:
                    refs[p] -= 1
            table[c] = [-1] * len(table[c])
        for a, c in zip(s["winners"].tolist(), s["losers"].tolist()):
            lens[c] = lens[a]
            for j in range(-(-lens[a] // page)):
                rest = lens[a] - j * page
                p = table[a][j]
                if rest < page:
                    p = refs.index(0)
                    k[:, p, :, :rest] = k[:, table[a][j], :, :rest]
                    v[:, p, :, :rest] = v[:, table[a][j], :, :rest]
                table[c][j] = p
                refs[p] += 1
        return {"k": k, "v": v, "table": whole(table, s["table"]), "lens": whole(lens, s["lens"]), "refs": whole(refs, s["refs"])}
    if op == "compact":
        live = sum(r > 0 for r in refs)
        for p in range(live, len(refs)):
            if refs[p] > 0:
                d = refs.index(0)
                k[:, d], v[:, d] = k[:, p], v[:, p]
                refs[d], refs[p] = refs[p], 0
                table = [[d if x == p else x for x in r] for r in table]
        return {"k": k, "v": v, "table": whole(table, s["table"]), "lens": whole(lens, s["lens"]), "refs": whole(refs, s["refs"]),
                "live": torch.tensor([live], dtype=torch.int32, device=dev)}
    cu = s["cu"].tolist()
    if op == "append":
        for i, (a, b) in enumerate(zip(cu, cu[1:])):
            done = a
            while done < b:  # a page at a time
                p = lens[i] - (b - done)
                m = min(b - done, page - p % page)
                k[0, table[i][p // page], :, p % page:p % page + m] = s["k_new"][done:done + m].double().transpose(0, 1)
                v[0, table[i][p // page], :, p % page:p % page + m] = s["v_new"][done:done + m].double().transpose(0, 1)
                done += m
        return k, v
    for i, (path, m) in enumerate(zip(s["path"].tolist(), s["taken"].tolist())):
        base = lens[i] - (cu[i + 1] - cu[i])
        for j in range(m):
            a, b = base + path[j], base + j
            k[:, table[i][b // page], :, b % page] = k[:, table[i][a // page], :, a % page]
            v[:, table[i][b // page], :, b % page] = v[:, table[i][a // page], :, a % page]
        lens[i] = base + m
    return k, v, whole(lens, s["lens"])
