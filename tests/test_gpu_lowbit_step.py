"""The low-bit operators as one decode step runs them: 4-bit QKV product -> q/k norm, RoPE and 4-bit append ->
attention over the 4-bit cache -> 4-bit output product and residual -> 4-bit head -> log probabilities, the picked token
fed back. Each stage is checked against its 64-bit form on what the stage before it left on the device, and the
step captured into a CUDA graph gives the bits of the eager one."""
import numpy as np
import pytest

from tests.gpu_util import tb
from tests.lowbit_util import (BLK, HD, NKV, NQ, U, attention, attention_tol, bf16_f64, decode, logprobs, make_pool, quantise, rotated,
                               unpack_w4)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

V, HID, LENS, STEPS, BPS = 2048, 1024, [0, 62, 127], 5, 3
SHAPES = {"qkv": (4096, HID, 64), "o": (HID, 2048, 128), "head": (V, HID, 32)}


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Step:
    def __init__(self):
        self.m = m = tb()
        rng = np.random.default_rng(77)
        B = len(LENS)
        self.w, self.packed = {}, {}
        for name, (N, K, G) in SHAPES.items():
            codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
            scales = bf16_f64(0.01 * np.exp(0.2 * rng.standard_normal((N, K // G))))
            zeros = rng.integers(6, 10, (N, K // G), dtype=np.uint8) if name != "o" else None
            self.w[name] = unpack_w4(codes, scales, zeros, G)
            self.packed[name] = torch.empty(m.tts_bb_w4_packed_bytes(N, K, G), dtype=torch.uint8, device="cuda")
            m.tts_bb_w4_pack(N, K, G, dev(codes), dev(scales).bfloat16(), None if zeros is None else dev(zeros), self.packed[name],
                             torch.cuda.current_stream().cuda_stream)
        self.emb = dev(rng.standard_normal((V, HID)).astype(np.float32))
        self.g = [bf16_f64(1 + 0.1 * rng.standard_normal(HD)) for _ in range(2)]
        self.gd = [dev(g).bfloat16() for g in self.g]
        self.cos, self.sin = m.tts_bb_rope_tables(1e6, BPS * BLK)
        self.cs = [dev(self.cos), dev(self.sin)]
        n = B * BPS
        self.table = rng.permutation(n).reshape(B, BPS).astype(np.int32)
        pool = make_pool(rng, n)
        self.pool = dev(pool)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cache = m.Kv4Cache(self.pool, dev(self.table), self.err)
        # the prompts' keys and values, appended as one ragged call
        seqs = np.concatenate([np.full(n, b) for b, n in enumerate(LENS)]).astype(np.int32)
        pos = np.concatenate([np.arange(n) for n in LENS]).astype(np.int32)
        self.append(dev(rng.standard_normal((len(seqs), 4096)).astype(np.float32)), dev(seqs), dev(pos), None)
        self.seqs = dev(np.arange(B, dtype=np.int32))
        self.pos, self.lens = dev(np.asarray(LENS, np.int32)), dev(np.asarray(LENS, np.int32) + 1)
        f = dict(dtype=torch.float32, device="cuda")
        self.tok = dev(np.array([5, 900, 2047], np.int32))
        self.x, self.qkv, self.q, self.attn = (torch.empty(B, k, **f) for k in (HID, 4096, 2048, 2048))
        self.o, self.h, self.logits = (torch.empty(B, k, **f) for k in (HID, HID, V))
        self.lp, self.ent, self.lse, self.top = (torch.empty(*s, **f) for s in ((B,), (B,), (B,), (B, 4)))
        self.ids = torch.empty(B, 4, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(max(1, m.tts_bb_kv4_attention_workspace(B, 1, BPS * BLK)), dtype=torch.uint8, device="cuda")
        self.ws2 = torch.empty(max(1, m.tts_bb_token_logprobs_workspace(B, V, 4)), dtype=torch.uint8, device="cuda")

    def append(self, qkv, seqs, pos, q):
        self.m.tts_bb_kv4_append(self.cache, len(seqs), qkv, *self.gd, *self.cs, BPS * BLK, seqs, pos, q,
                                 stream=torch.cuda.current_stream().cuda_stream)

    def linear(self, name, x, y):
        N, K, G = SHAPES[name]
        self.m.tts_bb_w4_linear(len(LENS), N, K, G, x, self.packed[name], y, torch.cuda.current_stream().cuda_stream)

    def step(self):
        st = torch.cuda.current_stream().cuda_stream
        torch.index_select(self.emb, 0, self.tok, out=self.x)
        self.linear("qkv", self.x, self.qkv)
        self.append(self.qkv, self.seqs, self.pos, self.q)
        self.m.tts_bb_kv4_attention(self.cache, len(LENS), 1, self.q, self.lens, BPS * BLK, self.attn, self.ws, stream=st)
        self.linear("o", self.attn, self.o)
        torch.add(self.x, self.o, out=self.h)
        self.linear("head", self.h, self.logits)
        self.m.tts_bb_token_logprobs(len(LENS), V, self.logits, self.tok, 4, self.lp, self.ent, self.lse, self.ids, self.top, workspace=self.ws2,
                                     stream=st)

    def feed(self):
        self.tok.copy_(self.ids[:, 0])
        self.pos.add_(1)
        self.lens.add_(1)

    def state(self):
        return [t.clone() for t in (self.qkv, self.q, self.attn, self.logits, self.lp, self.ent, self.lse, self.ids, self.top, self.pool)]


def lin_ok(w, x, y):
    x, y = x.double().cpu().numpy(), y.double().cpu().numpy()
    return (np.abs(y - x @ w.T) <= 2 * (w.shape[1] + 16) * U * (np.abs(x) @ np.abs(w).T)).all()


def test_a_step_stage_by_stage_and_captured():
    a = Step()
    seen = []
    for i in range(STEPS):
        tok = a.tok.cpu().numpy()
        a.step()
        seen.append(a.state())
        assert lin_ok(a.w["qkv"], a.x, a.qkv) and lin_ok(a.w["o"], a.attn, a.o) and lin_ok(a.w["head"], a.h, a.logits)
        pool = a.pool.cpu().numpy().reshape(len(LENS) * BPS, -1)
        qkv, q = a.qkv.double().cpu().numpy().reshape(-1, 32, HD), a.q.double().cpu().numpy().reshape(-1, NQ, HD)
        attn = a.attn.double().cpu().numpy().reshape(-1, NQ, HD)
        for b, n in enumerate(LENS):
            p = n + i
            c, s = a.cos[None, p].astype(np.float64), a.sin[None, p].astype(np.float64)
            eps = float(np.float32(1e-6))
            k = rotated(qkv[b : b + 1, NQ : NQ + NKV], a.g[1], c, s, eps)[0]
            for which, y in ((0, k), (1, qkv[b, NQ + NKV :])):
                code, scale, off = quantise(y)
                held = scale.repeat(64, -1) * (code + 128 + off.repeat(64, -1))
                got = np.array([decode(pool, a.table[b, p // BLK], which, h, p % BLK) for h in range(NKV)])
                assert np.array_equal(got, held)
            kv = [np.array([[decode(pool, a.table[b, j // BLK], which, h, j % BLK) for h in range(NKV)] for j in range(p + 1)]) for which in (0, 1)]
            want, mag, dots = attention(q[b], *kv, p + 1)
            assert (np.abs(attn[b] - want) <= attention_tol(want, mag, dots, p + 1, False)).all()
            z = a.logits[b].double().cpu().numpy()
            lp, ent, lse, ids, top, log_s, _ = logprobs(z, None, tok[b], 4)
            assert np.array_equal(a.ids[b].cpu().numpy(), ids)
            # sums of 2048 exponentials: (V / 32 + 64) U + 2^-21 of the sum, the differences U of themselves
            tol = (V / 32 + 64) * U + 2.0 ** -21 + 4 * U * (np.abs(z).max() - z.min())
            for g, w in ((a.lp[b], lp), (a.lse[b], lse), (a.top[b, 3], top[3])):
                assert abs(float(g) - w) <= tol
            assert abs(float(a.ent[b]) - ent) <= tol * (2 + np.abs(z - z.max()).max())
        a.feed()
    assert int(a.err) == 0

    b = Step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            b.step()
    for i in range(STEPS):
        with torch.cuda.stream(side):
            g.replay()
            got = b.state()
            b.feed()
        side.synchronize()
        assert all(torch.equal(x, y) or (x.dtype == torch.uint8 and np.array_equal(x.cpu().numpy(), y.cpu().numpy())) for x, y in zip(got, seen[i]))
