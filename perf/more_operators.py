"""Cases of the speculative decoding operators: their inputs, their plain forms and their definition in 64 bits.

Three operators that a decode step with drafted tokens runs one after the other:

  attend   attention of a tree of drafted tokens over a paged bf16 cache: a node sees the cached keys, itself and
           its ancestors (16 query / 8 KV heads of 128)
  verify   the path of drafted tokens that the target's probabilities accept, from given random numbers, and the
           token that follows it
  commit   the accepted path's keys and values appended to the cache of every layer

`run` computes the plain forms with elementary torch operations where `own` is false, and makes the calls of
codec_token_tts_gb300 where it is true. All sizes not in a case are the backbone's: 16 query and 8 KV heads of
128, 64-token cache blocks. Node 0 of a tree is the pending token; a parent's index is below its children's.
"""
import math
import random

import torch

own = False

NQ, NKV, HD, BLK = 16, 8, 128, 64
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one stream a few seconds into an utterance, five tokens drafted in a row: the smallest call, all latency
        {"name": "attend_1x333_chain6", "op": "attend", "seqs": 1, "nodes": 6, "shape": "chain", "ctx": 333, "ragged": False, "io": "bf16"},
        # a batched step over ragged caches with trees of an odd size, fp32 queries
        {"name": "attend_16x2000_tree25_f32", "op": "attend", "seqs": 16, "nodes": 25, "shape": "tree", "ctx": 2000, "ragged": True, "io": "f32"},
        # a full batch with the largest trees
        {"name": "attend_64x2000_tree64", "op": "attend", "seqs": 64, "nodes": 64, "shape": "tree", "ctx": 2000, "ragged": True, "io": "bf16"},
        # a few streams with very long caches
        {"name": "attend_8x65537_tree31", "op": "attend", "seqs": 8, "nodes": 31, "shape": "tree", "ctx": 65537, "ragged": False, "io": "bf16"},
        # one stream's codebook tokens, drafted in a row
        {"name": "verify_1x2048_chain6", "op": "verify", "seqs": 1, "nodes": 6, "shape": "chain", "vocab": 2048, "pad": 0, "mode": "drawn"},
        # a batch of codebook trees whose drafts are the draft model's most probable tokens
        {"name": "verify_64x2048_tree25_ranked", "op": "verify", "seqs": 64, "nodes": 25, "shape": "tree", "vocab": 2048, "pad": 0, "mode": "ranked"},
        # the text vocabulary, a batched step with trees drawn from the draft's distribution
        {"name": "verify_64x151676_tree12", "op": "verify", "seqs": 64, "nodes": 12, "shape": "tree", "vocab": 151676, "pad": 4, "mode": "drawn"},
        # a batch decoded greedily: the argmax of each node's logits against the drafts
        {"name": "verify_64_tree64_greedy", "op": "verify", "seqs": 64, "nodes": 64, "shape": "tree", "vocab": 2048, "pad": 0, "mode": "greedy"},
        # one stream's accepted tokens into the 28 layers' caches
        {"name": "commit_28x1_chain6", "op": "commit", "layers": 28, "seqs": 1, "nodes": 6, "ctx": 333},
        # a batch's accepted tokens
        {"name": "commit_28x64_tree25", "op": "commit", "layers": 28, "seqs": 64, "nodes": 25, "ctx": 190},
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("attend", "attend", "verify", "commit"))
    nodes, shape = _log(rng, 1, 64), rng.choice(("chain", "tree"))
    if op == "attend":
        ctx = 0 if rng.random() < 0.05 else _log(rng, 1, 65537)
        io = rng.choice(("f32", "bf16"))
        seqs = max(1, min(64, _log(rng, 1, 64), (8 if io == "bf16" else 4) * 65537 // (ctx + 64)))
        if ctx * seqs > 131072:
            nodes = min(nodes, 31)
        return {"op": op, "seqs": seqs, "nodes": nodes, "shape": shape, "ctx": ctx, "ragged": rng.random() < 0.6, "io": io}
    if op == "verify":
        vocab = _log(rng, 2, 200000)
        seqs = _log(rng, 1, 64)
        if seqs * nodes * vocab > 64 * 12 * 151676:
            nodes = max(1, 64 * 12 * 151676 // (seqs * vocab))
        return {"op": op, "seqs": seqs, "nodes": nodes, "shape": shape, "vocab": vocab, "pad": rng.choice((0, 0, 1, 3, 8)),
                "mode": rng.choice(("drawn", "drawn", "ranked", "greedy"))}
    layers = rng.choice((1, 5, 28))
    seqs = _log(rng, 1, 64)
    return {"op": op, "layers": layers, "seqs": seqs, "nodes": min(nodes, 25), "ctx": _log(rng, 25, 192 * 64 // seqs if seqs > 12 else 1000)}


def _lens(case):
    """Cached keys of each sequence, by the case alone."""
    B, C = case["seqs"], case["ctx"]
    lo = C // 10
    return [C - (b * 7919) % (C - lo + 1) for b in range(B)] if case.get("ragged") else [C] * B


def _nodes(case):
    """Nodes of each sequence's tree: most are full, some are smaller."""
    N = case["nodes"]
    return [N if b % 3 < 2 else N - (b * 5) % (N // 2 + 1) for b in range(case["seqs"])]


def work(case):
    """The bytes read and written once, and the operations of the products."""
    B, N = case["seqs"], case["nodes"]
    if case["op"] == "attend":
        e, nodes, lens = 4 if case["io"] == "f32" else 2, _nodes(case), _lens(case)
        row = 2 * NKV * HD * 2
        pairs = sum(n * k + n * (n + 1) // 2 if case["shape"] == "chain" else n * k + 4 * n for n, k in zip(nodes, lens))
        return {"bytes": (sum(lens) + sum(nodes)) * row + 2 * sum(nodes) * NQ * HD * e, "flops": 4.0 * NQ * HD * pairs}
    if case["op"] == "verify":
        # the row at which a sequence's path ends, and the draft's
        rows = {"drawn": 2, "ranked": 1, "greedy": 0}[case["mode"]]
        return {"bytes": B * (rows * case["vocab"] * 4 + N * 16 + 8), "flops": 2.0 * B * rows * case["vocab"]}
    tokens = sum(_accepted(case))
    return {"bytes": 2 * case["layers"] * tokens * 2 * NKV * HD * 2, "flops": 0.0}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _accepted(case):
    """Nodes of each sequence's accepted path (commit), by the case alone: a few, the pending token among them."""
    return [1 + (b * 3 + 2) % min(8, case["nodes"]) for b in range(case["seqs"])]


def _trees(case, seed):
    """Parents [B][N], at most four children a node; and each node's rank among its siblings."""
    rng = random.Random(seed)
    N, parents, ranks = case["nodes"], [], []
    for _ in range(case["seqs"]):
        kids, par, rank = [0] * N, [-1], [0]
        for i in range(1, N):
            p = i - 1
            if case["shape"] == "tree":
                p = rng.choice([j for j in range(max(0, i - 12), i) if kids[j] < 4])
            par.append(p)
            rank.append(kids[p])
            kids[p] += 1
        parents.append(par)
        ranks.append(rank)
    return _ints(parents), _ints(ranks)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    B, N = case["seqs"], case["nodes"]
    if case["op"] == "attend":
        C = case["ctx"]
        io, nb = IO[case["io"]], max(1, -(-C // BLK))
        # keys of unit RMS times a gain near 1, values with a size of their own for each channel
        s["pool"] = torch.empty(B * nb, 2, NKV, BLK, HD, dtype=torch.bfloat16, device="cuda")
        size = torch.exp(0.5 * _randn(g, NKV, 1, HD))
        for at in range(0, B * nb, 1024):
            part = _randn(g, min(1024, B * nb - at), 2, NKV, BLK, HD)
            part[:, 1] *= size
            s["pool"][at : at + 1024] = part
        s["table"] = torch.randperm(B * nb, generator=g, device="cuda").int().reshape(B, nb)
        s["lens"], s["n"] = _ints(_lens(case)), _ints(_nodes(case))
        s["parents"], _ = _trees(case, seed)
        s["q"] = (1.5 * _randn(g, B * N, NQ * HD)).to(io)
        s["k"] = _randn(g, B * N, NKV * HD).bfloat16()
        s["v"] = (_randn(g, B * N, NKV, HD) * size[:, 0]).reshape(B * N, NKV * HD).bfloat16()
        s["out"] = torch.zeros(B * N, NQ * HD, dtype=io, device="cuda")
        if own:
            import codec_token_tts_gb300 as tts
            s["tts"], s["cache"] = tts, tts.KvCache(s["pool"], s["table"])
            s["ws"] = torch.empty(max(1, tts.tts_bb_tree_attention_workspace(B, N, C)), dtype=torch.uint8, device="cuda")
    elif case["op"] == "verify":
        V = case["vocab"]
        s["n"] = _ints(_nodes(case))
        s["parents"], rank = _trees(case, seed)
        rows = torch.arange(B, device="cuda")[:, None] * N + s["parents"].long().clamp(min=0)
        if case["mode"] == "greedy":
            # an argmax a node; most drafts are the argmax of their parent, the others any id
            s["best"] = torch.randint(0, V, (B, N), generator=g, device="cuda").int()
            hit = (rank == 0) & (torch.rand(B, N, generator=g, device="cuda") < 0.8)
            any_id = torch.randint(0, V, (B, N), generator=g, device="cuda").int()
            s["tokens"] = torch.where(hit, s["best"].reshape(-1)[rows], any_id)
        else:
            # peaked distributions, the draft's near the target's
            z = 2.5 * _randn(g, B * N, V)
            s["target"] = torch.zeros(B * N, V + case["pad"], device="cuda")
            s["target"][:, :V] = torch.softmax(z, -1)
            z += 0.5 * _randn(g, B * N, V)
            draft = torch.zeros(B * N, V + case["pad"], device="cuda")
            draft[:, :V] = torch.softmax(z, -1)
            k = min(4, V)
            if case["mode"] == "drawn":
                picks = torch.multinomial(draft[:, :V], 4, replacement=True, generator=g)
            else:
                picks = draft[:, :V].topk(k, -1).indices
            s["tokens"] = picks[rows, rank.long() % picks.shape[1]].int()
            s["draft"] = draft if case["mode"] == "drawn" else None
            s["u"], s["u_next"] = torch.rand(B, N, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
        s["count"], s["next"] = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
        s["path"] = torch.zeros(B, N, dtype=torch.int32, device="cuda")
        if own:
            import codec_token_tts_gb300 as tts
            s["tts"] = tts
    else:
        L, C = case["layers"], case["ctx"]
        nb = -(-(C + 8) // BLK)
        s["pool"] = torch.empty(L, B * nb, 2, NKV, BLK, HD, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        s["table"] = torch.randperm(B * nb, generator=g, device="cuda").int().reshape(B, nb)
        s["lens"] = _ints([C - (b * 7919) % (C - C // 10 + 1) for b in range(B)])
        s["k"], s["v"] = (_randn(g, L, B * N, NKV * HD).bfloat16() for _ in range(2))
        count = _accepted(case)
        rng = random.Random(seed)
        s["count"] = _ints(count)
        s["path"] = _ints([[0] + sorted(rng.sample(range(1, N), c - 1)) + [-1] * (N - c) for c in count])
        if own:
            import codec_token_tts_gb300 as tts
            s["tts"], s["cache"] = tts, tts.KvCache(s["pool"], s["table"], layers=L)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)[s["op"]](s)


def _plain_attend(s):
    B, N, C = s["seqs"], s["nodes"], s["ctx"]
    # which nodes a node sees: itself, and what its parent sees
    see = torch.eye(N, dtype=torch.bool, device="cuda").repeat(B, 1, 1)
    at = torch.arange(B, device="cuda")
    for i in range(1, N):
        up = s["parents"][:, i].long()
        see[:, i] |= see[at, up.clamp(min=0)] & (up >= 0)[:, None]
    x = s["pool"][s["table"].long()].permute(2, 0, 3, 1, 4, 5).reshape(2, B, NKV, -1, HD)
    tree = torch.stack((s["k"], s["v"])).reshape(2, B, N, NKV, HD).transpose(2, 3)
    x = torch.cat((x, tree), 3).float()                                             # [2, B, 8, keys, 128]
    keys = x.shape[3] - N
    ok = (torch.arange(keys, device="cuda") < s["lens"][:, None])[:, None].expand(B, N, keys)
    ok = torch.cat((ok, see), -1)[:, None, :, None, :]                              # [B, 1, N, 1, keys]
    q = s["q"].float().reshape(B, N, NKV, 2, HD).transpose(1, 2).reshape(B, NKV, N * 2, HD)
    z = q @ x[0].transpose(-1, -2) / math.sqrt(HD)
    z = z.reshape(B, NKV, N, 2, -1).masked_fill(~ok, -math.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).reshape(B, NKV, N * 2, -1)
    o = (p @ x[1]).reshape(B, NKV, N, 2, HD).transpose(1, 2)
    live = torch.arange(N, device="cuda") < s["n"][:, None]
    o = torch.where(live[:, :, None, None, None], o, torch.zeros_like(o))
    return o.reshape(B * N, NQ * HD).to(s["out"].dtype)


def _plain_path(s, chosen):
    """The chosen nodes [B][N] (truth values) as counts and node lists, -1 behind the last."""
    B, N = chosen.shape
    count = chosen.sum(-1)
    order = torch.where(chosen, torch.arange(N, device="cuda"), N).sort(-1).values
    return count.int(), torch.where(order < N, order, -1).int()


def _plain_verify(s):
    B, N, V = s["seqs"], s["nodes"], s["vocab"]
    at = torch.arange(B, device="cuda")
    cur = torch.zeros(B, dtype=torch.long, device="cuda")
    chosen = torch.zeros(B, N, dtype=torch.bool, device="cuda")
    chosen[:, 0] = True
    parents, live = s["parents"].long(), torch.arange(N, device="cuda") < s["n"][:, None]
    if s["mode"] == "greedy":
        for j in range(1, N):
            hit = live[:, j] & (parents[:, j] == cur) & (s["tokens"][:, j] == s["best"][at, cur])
            chosen[:, j] = hit
            cur = torch.where(hit, j, cur)
        count, path = _plain_path(s, chosen)
        return {"count": count, "path": path, "next": s["best"][at, cur]}
    # decided in 64 bits: next to a border a 32-bit sum would pick another token
    drawn = s["mode"] == "drawn"
    p = s["target"][at * N, :V].double()                    # the rest of the current node's distribution, not normalised
    q = s["draft"][at * N, :V].double() if drawn else None
    r, mass = p, torch.ones(B, dtype=torch.float64, device="cuda")
    for j in range(1, N):
        mine = live[:, j] & (parents[:, j] == cur)
        x = s["tokens"][:, j].long()
        price = s["u"][:, j].double() * mass * (q[at, x] if drawn else 1.0)
        hit = mine & (price < r[at, x])
        miss = mine & ~hit
        chosen[:, j] = hit
        cur = torch.where(hit, j, cur)
        if drawn:
            rest = (r - mass[:, None] * q).clamp(min=0)
            left = rest.sum(-1)
        else:
            rest = r.scatter(1, x[:, None], 0.0)
            left = mass - r[at, x]
        row = at * N + cur
        fresh = s["target"][row, :V].double()
        r = torch.where(hit[:, None], fresh, torch.where(miss[:, None], rest, r))
        mass = torch.where(hit, torch.ones_like(mass), torch.where(miss, left, mass))
        p = torch.where(hit[:, None], fresh, p)
        if drawn:
            q = torch.where(hit[:, None], s["draft"][row, :V].double(), q)
    cdf = r.cumsum(-1)
    total = cdf[:, -1]
    token = (cdf <= (s["u_next"].double() * total)[:, None]).sum(-1).clamp(max=V - 1)
    ids = torch.arange(V, device="cuda")
    best = torch.where(p == p.amax(-1, keepdim=True), ids, V).amin(-1)
    count, path = _plain_path(s, chosen)
    return {"count": count, "path": path, "next": torch.where(total > 0, token, best).int()}


def _plain_commit(s):
    B, N = s["seqs"], s["nodes"]
    j = torch.arange(N, device="cuda")
    b, j = torch.nonzero(j < s["count"][:, None], as_tuple=True)
    row = b * N + s["path"][b, j].long()
    pos = s["lens"][b].long() + j
    page = s["table"][b, pos // BLK].long()
    for which, x in enumerate((s["k"], s["v"])):
        s["pool"][:, page, which, :, pos % BLK] = x[:, row].reshape(-1, len(row), NKV, HD).transpose(0, 1)
    return s["pool"]


def _own_attend(s):
    st = torch.cuda.current_stream().cuda_stream
    s["tts"].tts_bb_tree_attention(s["cache"], 0, s["seqs"], s["nodes"], s["q"], s["k"], s["v"], s["parents"], s["lens"], s["ctx"], s["out"], s["ws"],
                                   n_nodes=s["n"], stream=st)
    return s["out"]


def _own_verify(s):
    st = torch.cuda.current_stream().cuda_stream
    if s["mode"] == "greedy":
        s["tts"].tts_bb_tree_verify_greedy(s["seqs"], s["nodes"], s["tokens"], s["parents"], s["best"], s["count"], s["path"], s["next"],
                                           n_nodes=s["n"], stream=st)
    else:
        s["tts"].tts_bb_tree_verify(s["seqs"], s["nodes"], s["vocab"], s["tokens"], s["parents"], s["target"], s["u"], s["u_next"], s["count"],
                                    s["path"], s["next"], draft=s["draft"], n_nodes=s["n"], stream=st)
    return {"count": s["count"], "path": s["path"], "next": s["next"]}


def _own_commit(s):
    s["tts"].tts_bb_tree_commit(s["cache"], s["seqs"], s["nodes"], s["k"], s["v"], s["path"], s["count"], s["lens"],
                                stream=torch.cuda.current_stream().cuda_stream)
    return s["pool"]


_run_plain = {"attend": _plain_attend, "verify": _plain_verify, "commit": _plain_commit}
_run_own = {"attend": _own_attend, "verify": _own_verify, "commit": _own_commit}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "verify": _exact_verify, "commit": _exact_commit}[case["op"]](s)


def _ancestors(parents, i):
    line = []
    while i >= 0:
        line.append(i)
        i = parents[i]
    return line[::-1]


def _exact_attend(s):
    B, N = s["seqs"], s["nodes"]
    out = torch.zeros(B * N, NQ * HD, dtype=torch.float64, device="cuda")
    parents, lens, count = s["parents"].tolist(), s["lens"].tolist(), s["n"].tolist()
    for b in range(B):
        pages = s["pool"][s["table"][b, : -(-lens[b] // BLK)].long()]
        for g in range(NKV):
            old = [pages[:, w, g].reshape(-1, HD)[: lens[b]].double() for w in (0, 1)]
            new = [x[b * N : (b + 1) * N, g * HD : (g + 1) * HD].double() for x in (s["k"], s["v"])]
            q = s["q"][b * N : b * N + count[b], 2 * g * HD : (2 * g + 2) * HD].double().reshape(-1, HD)
            z = torch.cat((q @ old[0].T, q @ new[0].T), 1) / HD**0.5
            unseen = torch.ones(count[b], N, dtype=torch.bool)
            for i in range(count[b]):
                unseen[i, _ancestors(parents[b], i)] = False
            z[:, lens[b] :][unseen.cuda().repeat_interleave(2, 0)] = -math.inf
            o = torch.softmax(z, -1) @ torch.cat(old[1:] + new[1:])
            out[b * N : b * N + count[b], 2 * g * HD : (2 * g + 2) * HD] = o.reshape(count[b], 2 * HD)
    return out


def _exact_verify(s):
    B, N, V = s["seqs"], s["nodes"], s["vocab"]
    parents, count, tokens = s["parents"].tolist(), s["n"].tolist(), s["tokens"].tolist()
    out = {"count": [], "path": [], "next": []}
    for b in range(B):
        path, node = [], 0
        while node is not None:
            path.append(node)
            kids = [j for j in range(count[b]) if parents[b][j] == node]
            here, node = node, None
            if s["mode"] == "greedy":
                token = int(s["best"][b, here])
                node = next((j for j in kids if tokens[b][j] == token), None)
                continue
            p = s["target"][b * N + here, :V].double()
            q = s["draft"][b * N + here, :V].double() if s["mode"] == "drawn" else None
            removed, mass, rest = 0.0, 1.0, p.clone()     # the rest is p less `removed` times q, where that is positive
            for j in kids:
                x, u = tokens[b][j], float(s["u"][b, j])
                if u * mass * (float(q[x]) if q is not None else 1.0) < float(rest[x]):
                    node = j
                    break
                if q is not None:
                    removed += mass
                    rest = torch.relu(p - removed * q)
                    mass = float(rest.sum())
                else:
                    mass -= float(rest[x])
                    rest[x] = 0.0
            if node is None:
                sums = torch.cumsum(rest, 0)
                if float(sums[-1]) > 0:
                    token = int(torch.searchsorted(sums, float(s["u_next"][b]) * sums[-1:], right=True).clamp(max=V - 1))
                else:
                    token = int(torch.nonzero(p == p.max())[0])
        out["count"].append(len(path))
        out["path"].append(path + [-1] * (N - len(path)))
        out["next"].append(token)
    return {k: _ints(v) for k, v in out.items()}


def _exact_commit(s):
    N = s["nodes"]
    for b, (n, start) in enumerate(zip(s["count"].tolist(), s["lens"].tolist())):
        for j in range(n):
            block, tok, node = int(s["table"][b, (start + j) // BLK]), (start + j) % BLK, int(s["path"][b, j])
            for l in range(s["layers"]):
                s["pool"][l, block, 0, :, tok] = s["k"][l, b * N + node].view(NKV, HD)
                s["pool"][l, block, 1, :, tok] = s["v"][l, b * N + node].view(NKV, HD)
    return s["pool"]
