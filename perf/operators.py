"""Cases of the low-bit decode operators: their inputs, their plain forms and their definition in 64 bits.

Four operators that one decode step with 4-bit storage runs one after the other:

  append    q/k RMSNorm + half-rotate RoPE of fused QKV rows, keys and values appended in 4 bits to a
            paged cache, and the appended rows read back as the values they stand for
  attend    grouped-query attention (16 query / 8 KV heads of 128) over that cache, causal
  linear    y = x W^T with 4-bit weights and a scale (and zero point) for each group of input columns
  logprobs  log probabilities of given tokens, entropy, log-sum-exp and the top alternatives of logits rows

`run` computes the plain forms with elementary torch operations where `own` is false, and makes the calls of
codec_token_tts_gb300 where it is true. All sizes not in a case are the backbone's: 16 query and 8 KV heads of
128, 64-token cache blocks.
"""
import math

import torch

own = False

NQ, NKV, HD, BLK = 16, 8, 128, 64
QKV = (NQ + 2 * NKV) * HD
TILE = BLK * HD // 2 + BLK * 8          # 4-bit codes of 64 tokens, then (scale, offset) of 2 groups a token
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one stream's decode step: the smallest call, all latency
        {"name": "append_step_1", "op": "append", "seqs": 1, "tokens": 1, "ctx": 384, "io": "f32"},
        # a batched serving step, ragged positions
        {"name": "append_step_64", "op": "append", "seqs": 64, "tokens": 1, "ctx": 2000, "io": "f32"},
        # the prompts of a batch, ragged, padded to one length
        {"name": "append_prompt_16x2048", "op": "append", "seqs": 16, "tokens": 2048, "ctx": 2048, "io": "bf16"},
        # one stream a few seconds into an utterance
        {"name": "attend_1x333", "op": "attend", "seqs": 1, "tokens": 1, "ctx": 333, "ragged": False, "io": "bf16"},
        # a batched serving step over ragged caches, fp32 queries as the engine's own decode attention takes them
        {"name": "attend_64x2000", "op": "attend", "seqs": 64, "tokens": 1, "ctx": 2000, "ragged": True, "io": "f32"},
        # a few streams with very long caches
        {"name": "attend_8x65537", "op": "attend", "seqs": 8, "tokens": 1, "ctx": 65537, "ragged": False, "io": "bf16"},
        # the fused QKV projection of one token
        {"name": "linear_1x4096x1024", "op": "linear", "tokens": 1, "rows": 4096, "cols": 1024, "group": 128, "zeros": False, "io": "f32"},
        # the audio heads (an odd number of rows) on a few tokens
        {"name": "linear_7x8200x1024", "op": "linear", "tokens": 7, "rows": 8 * 1025, "cols": 1024, "group": 64, "zeros": True, "io": "f32"},
        # a large matrix, one token: bound by the weights' bytes
        {"name": "linear_1x16384x16384", "op": "linear", "tokens": 1, "rows": 16384, "cols": 16384, "group": 128, "zeros": True, "io": "bf16"},
        # the code just picked from one head's logits, with its nearest alternatives
        {"name": "logprobs_1x2048", "op": "logprobs", "rows": 1, "vocab": 2048, "pad": 0, "top": 5, "masked": False, "io": "f32"},
        # scoring a whole refinement pass: 8 items x 8 codebooks x 768 frames, the mask ids excluded
        {"name": "logprobs_49152x1025", "op": "logprobs", "rows": 8 * 8 * 768, "vocab": 1025, "pad": 0, "top": 5, "masked": True, "io": "f32"},
        # the text vocabulary, a batched step
        {"name": "logprobs_64x151676", "op": "logprobs", "rows": 64, "vocab": 151676, "pad": 4, "top": 20, "masked": False, "io": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("append", "attend", "linear", "logprobs"))
    io = rng.choice(("f32", "bf16"))
    if op == "append":
        if rng.random() < 0.5:
            return {"op": op, "seqs": _log(rng, 1, 64), "tokens": 1, "ctx": _log(rng, 64, 8192), "io": io}
        tokens = _log(rng, 2, 2048)
        return {"op": op, "seqs": rng.randint(1, 16 if io == "bf16" else 10), "tokens": tokens, "ctx": tokens + rng.randint(0, 500), "io": io}
    if op == "attend":
        ctx = _log(rng, 1, 65537)
        seqs = max(1, min(64, _log(rng, 1, 64), 8 * 65537 // ctx))
        return {"op": op, "seqs": seqs, "tokens": 1 if rng.random() < 0.6 or ctx < 8 or ctx * seqs > 131072 else rng.randint(2, 8), "ctx": ctx,
                "ragged": rng.random() < 0.6, "io": io}
    if op == "linear":
        group = rng.choice((32, 64, 128))
        cols = group * max(1, min(16384 // group, _log(rng, 128, 16384) // group))
        return {"op": op, "tokens": 1 if rng.random() < 0.5 else _log(rng, 2, 64), "rows": _log(rng, 16, 16384), "cols": cols, "group": group,
                "zeros": rng.random() < 0.5, "io": io}
    vocab = _log(rng, 2, 200000)
    rows = max(1, min(_log(rng, 1, 49152), 49152, 49152 * 1025 // vocab))
    return {"op": op, "rows": rows, "vocab": vocab, "pad": rng.choice((0, 0, 1, 3, 8)), "top": rng.choice((0, 1, 5, 20, 32)), "masked": rng.random() < 0.5, "io": io}


def _lens(case):
    """Keys of each sequence after the call (attend), or valid tokens of each sequence (append): by the case alone."""
    B, S, C = case["seqs"], case["tokens"], case["ctx"]
    if case["op"] == "append":
        return [1] * B if S == 1 else [S - (b * 7919) % (S // 2 + 1) for b in range(B)]
    lo = max(1, C // 10)
    return [C - (b * 7919) % (C - lo + 1) for b in range(B)] if case["ragged"] else [C] * B


def _starts(case):
    """Tokens cached before an append, for each sequence."""
    B, S, C = case["seqs"], case["tokens"], case["ctx"]
    return [(C - S) - (b * 613) % (max(1, (C - S) * 9 // 10) if S == 1 else C - S + 1) for b in range(B)]


def work(case):
    """The bytes read and written once, and the operations of the products."""
    e = 4 if case.get("io") == "f32" else 2
    if case["op"] == "append":
        n = sum(_lens(case))
        row = 2 * NKV * (HD // 2 + 8)
        return {"bytes": n * (QKV * e + NQ * HD * e + row + 2 * NKV * HD * 2 + 2 * 4 * HD // 2), "flops": 12.0 * n * QKV}
    if case["op"] == "attend":
        S, lens = case["tokens"], _lens(case)
        pairs = sum(max(0, n - s) for n in lens for s in range(S))
        return {"bytes": sum(lens) * 2 * NKV * (HD // 2 + 8) + 2 * len(lens) * S * NQ * HD * e, "flops": 4.0 * NQ * HD * pairs}
    if case["op"] == "linear":
        T, N, K, G = case["tokens"], case["rows"], case["cols"], case["group"]
        return {"bytes": N * K // 2 + N * (K // G) * (2.5 if case["zeros"] else 2) + T * (N + K) * e, "flops": 2.0 * T * N * K}
    R, V = case["rows"], case["vocab"]
    return {"bytes": R * V * e + R * (16 + 8 * case["top"]) + (V // 8 if case["masked"] else 0), "flops": 5.0 * R * V}


# ------------------------------------------------------------------ the 4-bit cache's format
def _unpack(pool):
    """uint8 [..., TILE] tiles -> the values they stand for, float32 [..., 64 tokens, 128].

    A token's 64 code bytes are 16 words; word w holds 8 dims of group w & 1, dims 64 (w & 1) + 8 (w >> 1) + i in
    nibble i. Behind the tile's codes stand two (bf16 scale, bf16 offset) pairs a token, one for each group of 64
    dims; a value is scale * (code + offset + 128)."""
    head = pool.shape[:-1]
    codes = pool[..., : BLK * HD // 2].reshape(*head, BLK, 8, 2, 4)
    codes = torch.stack((codes & 15, codes >> 4), -1).reshape(*head, BLK, 8, 2, 8)
    codes = codes.transpose(-3, -2).reshape(*head, BLK, 2, HD // 2)
    par = pool[..., BLK * HD // 2 :].contiguous().view(torch.bfloat16).reshape(*head, BLK, 2, 2, 1).float()
    return (par[..., 0, :] * (codes.float() + (par[..., 1, :] + 128))).flatten(-2)


def _quantise(x):
    """[..., 128] -> whole numbers 0..15 [..., 2, 64], scale and offset [..., 2, 1], all in x's type: the scale is a
    15th of a group's range (at least a 120th of its largest magnitude), rounded to bf16; codes count scales upward
    from the whole number next to the group's lowest value, and the offset is that number less 128."""
    x = x.reshape(*x.shape[:-1], 2, HD // 2)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = torch.maximum((hi - lo) / 15, torch.maximum(hi, -lo) / 120).float().bfloat16().to(x.dtype)
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    zero = torch.round(lo / safe)
    return (torch.round(x / safe) - zero).clamp(0, 15), scale, zero - 128


def _tiles(x):
    """float [..., 64 tokens, 128] -> uint8 [..., TILE]."""
    code, scale, offset = _quantise(x)
    head = x.shape[:-2]
    c = code.to(torch.uint8).reshape(*head, BLK, 2, 8, 8).transpose(-3, -2)
    c = c.reshape(*head, BLK, 8, 2, 4, 2)
    c = (c[..., 0] | (c[..., 1] << 4)).reshape(*head, BLK * HD // 2)
    par = torch.cat((scale, offset), -1).bfloat16().contiguous().view(torch.uint8).reshape(*head, BLK * 8)
    return torch.cat((c, par), -1)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    io = IO[case["io"]]
    if case["op"] == "append":
        B, S, C = case["seqs"], case["tokens"], case["ctx"]
        nb = -(-C // BLK)
        lens, starts = _lens(case), _starts(case)
        T = B * S
        b, i = torch.arange(T, device="cuda") // S, torch.arange(T, device="cuda") % S
        lens, starts = torch.tensor(lens, device="cuda"), torch.tensor(starts, device="cuda")
        s["seq"] = torch.where(i < lens[b], b, -1).int()
        s["pos"] = (starts[b] + i).int()
        # projections of normalised activations: a common size for each head and channel, some channels much larger
        chan = torch.exp(0.6 * _randn(g, 1, QKV))
        s["qkv"] = (_randn(g, T, QKV) * chan + 0.2 * _randn(g, 1, QKV)).to(io)
        s["gq"], s["gk"] = ((1 + 0.1 * _randn(g, HD)).bfloat16() for _ in range(2))
        s["table"] = torch.randperm(B * nb, generator=g, device="cuda").int().reshape(B, nb)
        s["pool"] = torch.zeros(B * nb, 2, NKV, TILE, dtype=torch.uint8, device="cuda")
        angle = torch.arange(C, device="cuda").double()[:, None] * 1e6 ** (-torch.arange(HD // 2, device="cuda").double() / (HD // 2))
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["q"] = torch.zeros(T, NQ, HD, dtype=io, device="cuda")
        s["k"], s["v"] = (torch.zeros(T, NKV, HD, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        if own:
            import codec_token_tts_gb300 as tts
            s["tts"], s["cache"] = tts, tts.Kv4Cache(s["pool"], s["table"])
    elif case["op"] == "attend":
        B, S, C = case["seqs"], case["tokens"], case["ctx"]
        nb = -(-C // BLK)
        # keys of unit RMS times a gain near 1, values with a size of their own for each channel
        kv = _randn(g, B * nb, 2, NKV, BLK, HD)
        kv[:, 1] *= torch.exp(0.5 * _randn(g, NKV, 1, HD))
        s["pool"] = _tiles(kv)
        s["table"] = torch.randperm(B * nb, generator=g, device="cuda").int().reshape(B, nb)
        s["lens"] = _ints(_lens(case))
        s["q"] = (1.5 * _randn(g, B * S, NQ, HD)).to(io)
        s["out"] = torch.zeros(B * S, NQ, HD, dtype=io, device="cuda")
        if own:
            import codec_token_tts_gb300 as tts
            s["tts"], s["cache"] = tts, tts.Kv4Cache(s["pool"], s["table"])
            s["ws"] = torch.empty(max(1, tts.tts_bb_kv4_attention_workspace(B, S, C)), dtype=torch.uint8, device="cuda")
    elif case["op"] == "linear":
        T, N, K, G = case["tokens"], case["rows"], case["cols"], case["group"]
        s["codes"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"] = (0.004 * torch.exp(0.3 * _randn(g, N, K // G))).bfloat16()
        s["zp"] = torch.randint(6, 11, (N, K // G), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
        s["x"] = _randn(g, T, K).to(io)
        s["y"] = torch.empty(T, N, dtype=io, device="cuda")
        if own:
            import codec_token_tts_gb300 as tts
            s["tts"] = tts
            s["w"] = torch.empty(tts.tts_bb_w4_packed_bytes(N, K, G), dtype=torch.uint8, device="cuda")
            tts.tts_bb_w4_pack(N, K, G, s["codes"], s["scales"], s["zp"], s["w"], torch.cuda.current_stream().cuda_stream)
    else:
        R, V = case["rows"], case["vocab"]
        z = 2.5 * _randn(g, R, V + case["pad"])
        z[:, :V] += 6.0 * (torch.rand(R, V, generator=g, device="cuda") < 3.0 / V)
        s["logits"] = z.to(io)
        s["target"] = torch.randint(0, V, (R,), generator=g, device="cuda").int()
        s["allowed"] = None
        if case["masked"]:  # the last id (a mask or pad id) and a few others are never answers
            ok = torch.rand(-(-V // 32) * 32, generator=g, device="cuda") < 0.98
            ok[V - 1 :] = False
            ok[0] = True
            s["allowed"] = ((ok.reshape(-1, 32).long() << torch.arange(32, device="cuda")).sum(1)).to(torch.uint32)
        s["lp"], s["ent"], s["lse"] = (torch.empty(R, device="cuda") for _ in range(3))
        k = case["top"]
        s["ids"] = torch.empty(R, k, dtype=torch.int32, device="cuda")
        s["tops"] = torch.empty(R, k, device="cuda")
        if own:
            import codec_token_tts_gb300 as tts
            s["tts"] = tts
            s["ws"] = torch.empty(max(1, tts.tts_bb_token_logprobs_workspace(R, V, k)), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)[s["op"]](s)


def _rope(x, c, n):
    h = HD // 2
    return torch.cat((x[..., :h] * c - x[..., h:] * n, x[..., h:] * c + x[..., :h] * n), -1)


def _plain_append(s):
    T = s["qkv"].shape[0]
    on = s["seq"] >= 0
    pos = s["pos"].long().clamp(max=s["cos"].shape[0] - 1)

    def rotated(x, gain, kind):
        x = x.to(kind)
        x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * gain.to(kind)
        return _rope(x, s["cos"][pos, None].to(kind), s["sin"][pos, None].to(kind))

    x = s["qkv"].reshape(T, NQ + 2 * NKV, HD)
    q = rotated(x[:, :NQ], s["gq"], torch.float32)
    k = rotated(x[:, NQ : NQ + NKV], s["gk"], torch.float64)      # next to the borders between codes
    v = x[:, NQ + NKV :].double()
    held = []
    for y in (k, v):
        code, scale, offset = _quantise(y)
        held.append((scale * (code + (offset + 128))).reshape(T, NKV, HD))
    rows = on[:, None, None]
    q, k, v = (torch.where(rows, y, torch.zeros_like(y)) for y in (q, *held))
    return {"q": q.to(s["q"].dtype), "k": k.bfloat16(), "v": v.bfloat16()}


def _plain_attend(s):
    B, S = s["seqs"], s["tokens"]
    x = _unpack(s["pool"][s["table"].long()])                       # [B, nb, 2, 8, 64, 128]
    x = x.permute(2, 0, 3, 1, 4, 5).reshape(2, B, NKV, -1, HD)      # [2, B, 8, L, 128]
    q = s["q"].float().reshape(B, S, NKV, 2, HD).transpose(1, 2).reshape(B, NKV, S * 2, HD)
    z = q @ x[0].transpose(-1, -2) / math.sqrt(HD)                  # [B, 8, S * 2, L]
    L = z.shape[-1]
    seen = s["lens"][:, None] - (S - 1) + torch.arange(S, device="cuda")            # [B, S] keys each query sees
    ok = (torch.arange(L, device="cuda") < seen[..., None])[:, None, :, None, :]
    z = z.reshape(B, NKV, S, 2, L).masked_fill(~ok, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    n = p.sum(-1, keepdim=True)
    p = (p / torch.where(n > 0, n, torch.ones_like(n))).reshape(B, NKV, S * 2, L)
    o = (p @ x[1]).reshape(B, NKV, S, 2, HD).transpose(1, 2)
    return o.reshape(B * S, NQ, HD).to(s["out"].dtype)


def _plain_linear(s):
    N, K, G = s["rows"], s["cols"], s["group"]
    c = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).reshape(N, K // G, G).float()
    zero = s["zp"][..., None].float() if s["zp"] is not None else 8.0
    w = ((c - zero) * s["scales"][..., None].float()).reshape(N, K)
    return (s["x"].float() @ w.T).to(s["y"].dtype)


def _plain_logprobs(s):
    R, V, k = s["rows"], s["vocab"], s["top"]
    z = s["logits"][:, :V].float()
    if s["allowed"] is not None:
        ok = ((s["allowed"].long()[:, None] >> torch.arange(32, device="cuda")) & 1).reshape(-1)[:V].bool()
        z = z.masked_fill(~ok, -math.inf)
    m = z.amax(-1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    total = e.sum(-1)
    lse = m[:, 0] + torch.log(total)
    ent = torch.log(total) - (e * d.masked_fill(d == -math.inf, 0.0)).sum(-1) / total
    lp = d.gather(1, s["target"].long()[:, None])[:, 0] - torch.log(total)
    out = {"logprob": lp, "entropy": ent, "lse": lse}
    if k:
        # value, then the lowest index: one whole number a place, all different; -inf is no alternative
        bits = (z + 0.0).view(torch.int32)
        order = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).long()
        key = (order << 32) | (0xFFFFFFFF - torch.arange(V, device="cuda"))
        n = min(k, V)
        ids = 0xFFFFFFFF - (key.topk(n, dim=-1).values & 0xFFFFFFFF)
        val = d.gather(1, ids) - torch.log(total)[:, None]
        ids = torch.where(val > -math.inf, ids, torch.full_like(ids, -1))
        pad = (0, k - n)
        out["ids"] = torch.nn.functional.pad(ids, pad, value=-1).int()
        out["top"] = torch.nn.functional.pad(val, pad, value=-math.inf)
    return out


def _own_append(s):
    t, st = s["tts"], torch.cuda.current_stream().cuda_stream
    n = s["qkv"].shape[0]
    t.tts_bb_kv4_append(s["cache"], n, s["qkv"], s["gq"], s["gk"], s["cos"], s["sin"], s["cos"].shape[0], s["seq"], s["pos"], s["q"], stream=st)
    t.tts_bb_kv4_read(s["cache"], n, s["seq"], s["pos"], s["k"], s["v"], stream=st)
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


def _own_attend(s):
    st = torch.cuda.current_stream().cuda_stream
    s["tts"].tts_bb_kv4_attention(s["cache"], s["seqs"], s["tokens"], s["q"], s["lens"], s["ctx"], s["out"], s["ws"], stream=st)
    return s["out"]


def _own_linear(s):
    st = torch.cuda.current_stream().cuda_stream
    s["tts"].tts_bb_w4_linear(s["tokens"], s["rows"], s["cols"], s["group"], s["x"], s["w"], s["y"], stream=st)
    return s["y"]


def _own_logprobs(s):
    st = torch.cuda.current_stream().cuda_stream
    s["tts"].tts_bb_token_logprobs(s["rows"], s["vocab"], s["logits"], s["target"], n_top=s["top"], logprob=s["lp"], entropy=s["ent"], lse=s["lse"],
                                   top_ids=s["ids"], top_logprobs=s["tops"], allowed=s["allowed"], workspace=s["ws"], stream=st)
    out = {"logprob": s["lp"], "entropy": s["ent"], "lse": s["lse"]}
    return {**out, "ids": s["ids"], "top": s["tops"]} if s["top"] else out


_run_plain = {"append": _plain_append, "attend": _plain_attend, "linear": _plain_linear, "logprobs": _plain_logprobs}
_run_own = {"append": _own_append, "attend": _own_attend, "linear": _own_linear, "logprobs": _own_logprobs}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "linear": _exact_linear, "logprobs": _exact_logprobs}[case["op"]](s)


def _exact_append(s):
    T = len(s["seq"])
    q = torch.zeros(T, NQ, HD, dtype=torch.float64, device="cuda")
    k, v = (torch.zeros(T, NKV, HD, dtype=torch.float64, device="cuda") for _ in range(2))
    live = torch.nonzero(s["seq"] >= 0)[:, 0]
    x = s["qkv"][live].double()
    turn = torch.complex(s["cos"][s["pos"][live].long()].double(), s["sin"][s["pos"][live].long()].double())

    def rotate(h, gain):  # pairs (i, i + 64) as complex numbers
        h = h / torch.sqrt((h * h).sum(-1, keepdim=True) / HD + 1e-6) * gain.double()
        w = torch.complex(h[..., : HD // 2], h[..., HD // 2 :]) * turn[:, None]
        return torch.cat((w.real, w.imag), -1)

    def held(y):
        out = torch.empty_like(y)
        for half in (slice(0, HD // 2), slice(HD // 2, HD)):
            p = y[..., half]
            low, high = p.min(-1).values, p.max(-1).values
            step = torch.max((high - low) / 15, p.abs().max(-1).values / 120).to(torch.float32).to(torch.bfloat16).double()
            safe = torch.where(step == 0, torch.ones_like(step), step)[..., None]
            first = torch.round(low[..., None] / safe)
            out[..., half] = step[..., None] * torch.minimum(torch.round(p / safe), first + 15)
        return out

    q[live] = rotate(x[:, : NQ * HD].view(-1, NQ, HD), s["gq"])
    k[live] = held(rotate(x[:, NQ * HD : (NQ + NKV) * HD].view(-1, NKV, HD), s["gk"]))
    v[live] = held(x[:, (NQ + NKV) * HD :].view(-1, NKV, HD))
    return {"q": q, "k": k, "v": v}


def _exact_attend(s):
    B, S = s["seqs"], s["tokens"]
    out = torch.zeros(B * S, NQ, HD, dtype=torch.float64, device="cuda")
    q = s["q"].double()
    for b, n in enumerate(s["lens"].tolist()):
        blocks = s["pool"][s["table"][b, : -(-n // BLK)].long()]
        words = blocks[..., : BLK * HD // 2].reshape(-1, 2, NKV, BLK, HD // 2)
        par = blocks[..., BLK * HD // 2 :].contiguous().view(torch.bfloat16).reshape(-1, 2, NKV, BLK, 2, 2).double()
        kv = torch.empty(2, NKV, len(blocks) * BLK, HD, dtype=torch.float64, device="cuda")
        for byte in range(HD // 2):
            w, t = byte // 4, byte % 4
            scale, off = (par[..., w % 2, j].permute(1, 2, 0, 3).reshape(2, NKV, -1) for j in (0, 1))
            col = words[..., byte].permute(1, 2, 0, 3).reshape(2, NKV, -1)
            d = 64 * (w % 2) + 8 * (w // 2) + 2 * t
            kv[..., d] = scale * ((col % 16).double() + off + 128)
            kv[..., d + 1] = scale * ((col // 16).double() + off + 128)
        for i in range(S):
            see = n - (S - 1 - i)
            if see > 0:
                y = q[b * S + i].view(NKV, 2, HD)
                a = torch.softmax(y @ kv[0, :, :see].transpose(1, 2) / HD**0.5, -1)
                out[b * S + i] = (a @ kv[1, :, :see]).view(NQ, HD)
    return out


def _exact_linear(s):
    y = torch.zeros(s["tokens"], s["rows"], dtype=torch.float64, device="cuda")
    G, x = s["group"], s["x"].double()
    for at in range(0, s["rows"], 2048):
        rows = slice(at, at + 2048)
        w = torch.empty(len(s["codes"][rows]), s["cols"], dtype=torch.float64, device="cuda")
        w[:, 0::2] = (s["codes"][rows] % 16).double()
        w[:, 1::2] = (s["codes"][rows] // 16).double()
        zero = s["zp"][rows].double() if s["zp"] is not None else torch.full_like(s["scales"][rows], 8.0, dtype=torch.float64)
        w = (w - zero.repeat_interleave(G, 1)) * s["scales"][rows].double().repeat_interleave(G, 1)
        y[:, rows] = x @ w.T
    return y


def _exact_logprobs(s):
    V, k = s["vocab"], s["top"]
    z = s["logits"][:, :V].double()
    if s["allowed"] is not None:
        i = torch.arange(V, device="cuda")
        bit = (s["allowed"].to(torch.int64)[i // 32] // 2 ** (i % 32)) % 2
        z[:, bit == 0] = -math.inf
    lse = torch.logsumexp(z, -1)
    lp = z - lse[:, None]
    p = torch.exp(lp)
    ent = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(-1)
    out = {"logprob": lp[torch.arange(len(lp), device="cuda"), s["target"].long()], "entropy": ent, "lse": lse}
    if k:
        val, ids = torch.sort(lp, dim=-1, descending=True, stable=True)
        val, ids = val[:, :k], ids[:, :k]
        ids = torch.where(val == -math.inf, -1, ids)
        short = k - val.shape[1]
        out["top"] = torch.cat((val, val.new_full((len(val), short), -math.inf)), 1)
        out["ids"] = torch.cat((ids, ids.new_full((len(ids), short), -1)), 1).int()
    return out
