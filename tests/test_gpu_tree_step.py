"""The speculative decoding operators as a program runs them: drafts of a tree -> two layers of projections and tree attention over
the paged cache -> verification -> the accepted keys and values into both layers' caches -> the next drafts. The tokens are those
of plain greedy decoding, one a step, in 64 bits; each stage is checked on what the stage before it left; a captured step
gives the bits of the eager one."""
import numpy as np
import pytest

from tests.gpu_util import tb
from tests.lowbit_util import attention_tol, bf16_f64
from tests.tree_util import BLK, HD, NKV, NQ, tree_attention, verify, verify_greedy

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

V, HID, LAYERS, N, LENS, STEPS, BPS = 40, 64, 2, 7, [0, 62, 127], 6, 4
PARENTS = [-1, 0, 0, 1, 1, 3, 2]


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


class Model:
    def __init__(self):
        rng = np.random.default_rng(5)
        self.emb = rng.standard_normal((V, HID))
        self.wqkv = rng.standard_normal((LAYERS, 4096, HID)) / np.sqrt(HID)
        self.wo = 0.5 * rng.standard_normal((LAYERS, HID, 2048)) / np.sqrt(2048)
        self.head = rng.standard_normal((V, HID))
        self.cos, self.sin = (t.astype(np.float64) for t in tb().tts_bb_rope_tables(1e4, BPS * BLK))
        self.prompt = [bf16_f64(rng.standard_normal((LAYERS, 2, n, NKV, HD))) for n in LENS]
        self.first = [3, 17, 39]

    def rotated(self, x, pos):
        c, s = self.cos[pos], self.sin[pos]
        a, b = x[..., :64], x[..., 64:]
        return np.concatenate((a * c - b * s, b * c + a * s), -1)

    def greedy(self, b, count):
        """The tokens of plain decoding behind the first one, and the least margin of a choice."""
        kv = [[list(self.prompt[b][l, w]) for w in (0, 1)] for l in range(LAYERS)]
        token, out, margin = self.first[b], [], np.inf
        for i in range(count):
            pos, x = LENS[b] + i, self.emb[token]
            for l in range(LAYERS):
                y = (self.wqkv[l] @ x).reshape(32, HD)
                q = self.rotated(y[:NQ], pos).astype(np.float32).astype(np.float64)
                kv[l][0].append(bf16_f64(self.rotated(y[NQ : NQ + NKV], pos)))
                kv[l][1].append(bf16_f64(y[NQ + NKV :]))
                k, v = (np.array(t) for t in kv[l])
                o = tree_attention(q[None], k[:-1], v[:-1], k[-1:], v[-1:], [-1])[0][0]
                x = x + self.wo[l] @ o.reshape(-1)
            z = self.head @ x
            top = np.sort(z)
            margin = min(margin, top[-1] - top[-2])
            token = int(z.argmax())
            out.append(token)
        return out, margin


class Run:
    def __init__(self, m):
        t, self.m, self.B = tb(), m, len(LENS)
        self.t = t
        rng = np.random.default_rng(9)
        B = self.B
        nb = B * BPS + 2
        self.table = rng.permutation(nb)[: B * BPS].reshape(B, BPS).astype(np.int32)
        self.pool = torch.full((LAYERS, nb, 2, NKV, BLK, HD), float("nan"), dtype=torch.bfloat16, device="cuda")
        for b, n in enumerate(LENS):
            for j in range(n):
                self.pool[:, int(self.table[b, j // BLK]), :, :, j % BLK] = dev(m.prompt[b][:, :, j]).bfloat16()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cache = t.KvCache(self.pool, dev(self.table), self.err, layers=LAYERS)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.lens = dev(np.asarray(LENS, np.int32))
        self.parents = torch.tensor([PARENTS] * B, **i32)
        self.depth = torch.tensor([[0, 1, 1, 2, 2, 3, 2]] * B, device="cuda")
        self.tokens = torch.zeros(B, N, **i32)
        self.w = [dev(x) for x in (m.emb, m.wqkv, m.wo, m.head, m.cos, m.sin)]
        self.k, self.v = (torch.zeros(LAYERS, B * N, NKV * HD, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.q, self.o = (torch.zeros(LAYERS, B * N, NQ * HD, device="cuda") for _ in range(2))
        self.ids, self.path = (torch.zeros(B, N, **i32) for _ in range(2))
        self.count, self.next = (torch.zeros(B, **i32) for _ in range(2))
        self.logits = torch.zeros(B * N, V, dtype=torch.float64, device="cuda")
        self.ws = torch.empty(max(16, t.tts_bb_tree_attention_workspace(B, N, BPS * BLK)), dtype=torch.uint8, device="cuda")

    def step(self):
        t, B, st = self.t, self.B, torch.cuda.current_stream().cuda_stream
        emb, wqkv, wo, head, cos, sin = self.w
        x = emb[self.tokens.long().reshape(-1)]
        pos = (self.lens[:, None] + self.depth).reshape(-1)
        c, s = cos[pos][:, None], sin[pos][:, None]
        for l in range(LAYERS):
            y = (x @ wqkv[l].T).reshape(B * N, 32, HD)
            a, b = y[:, : NQ + NKV, :64], y[:, : NQ + NKV, 64:]
            qk = torch.cat((a * c - b * s, b * c + a * s), -1)
            self.q[l].copy_(qk[:, :NQ].reshape(B * N, -1))
            self.k[l].copy_(qk[:, NQ:].float().reshape(B * N, -1))
            self.v[l].copy_(y[:, NQ + NKV :].float().reshape(B * N, -1))
            t.tts_bb_tree_attention(self.cache, l, B, N, self.q[l], self.k[l], self.v[l], self.parents, self.lens, BPS * BLK, self.o[l], self.ws, stream=st)
            x = x + self.o[l].double() @ wo[l].T
        self.logits.copy_(x @ head.T)
        self.ids.copy_(self.logits.argmax(-1).reshape(B, N))
        t.tts_bb_tree_verify_greedy(B, N, self.tokens, self.parents, self.ids, self.count, self.path, self.next, err=self.err, stream=st)
        t.tts_bb_tree_commit(self.cache, B, N, self.k, self.v, self.path, self.count, self.lens, stream=st)
        self.lens.add_(self.count)

    def state(self):
        return [x.clone() for x in (self.k, self.v, self.q, self.o, self.logits, self.ids, self.count, self.path, self.next, self.lens, self.pool.view(torch.int16))]


def drafts(rng, truth, pending):
    """Node 0 the pending token; children that continue it rightly or not."""
    t = [pending] + [int(rng.integers(V)) for _ in range(N - 1)]
    for node, ahead in ((1, 0), (2, 0), (3, 1), (4, 1), (5, 2)):
        if rng.random() < 0.6 and ahead < len(truth):
            t[node] = truth[ahead]
    return t


def test_speculative_decoding_gives_the_tokens_of_plain_decoding():
    m = Model()
    want = [m.greedy(b, STEPS * 4 + 4) for b in range(len(LENS))]
    # attention in fp32 and one more rounding of keys in bf16 move a logit by 1e-3 at most; the oracle's choices are clearer
    assert min(w[1] for w in want) > 4e-3
    plans, seen = [], []
    for captured in (False, True):
        r, rng = Run(m), np.random.default_rng(1)
        out, pending = [[] for _ in LENS], list(m.first)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = None
        with torch.cuda.stream(side):
            if captured:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=side):
                    r.step()
            for i in range(STEPS):
                lens = r.lens.cpu().numpy()
                tokens = [drafts(rng, want[b][0][len(out[b]) :], pending[b]) for b in range(r.B)]
                r.tokens.copy_(dev(np.asarray(tokens, np.int32)))
                before = r.pool.clone()
                (g.replay if captured else r.step)()
                side.synchronize()
                if captured:
                    assert all(torch.equal(x, y) for x, y in zip(r.state(), seen[i]))
                else:
                    seen.append(r.state())
                    check(r, lens, np.asarray(tokens), before)
                path, count, nxt = r.path.cpu().numpy(), r.count.cpu().numpy(), r.next.cpu().numpy()
                for b in range(r.B):
                    out[b] += [tokens[b][j] for j in path[b, 1 : count[b]]] + [int(nxt[b])]
                    pending[b] = int(nxt[b])
                plans.append(count)
        for b in range(r.B):
            assert out[b] == want[b][0][: len(out[b])]
        assert int(r.err) == 0
    assert np.mean(plans) > 1.5 and np.max(plans) >= 3  # drafts were accepted


def check(r, lens, tokens, before):
    """Every stage against its plain form."""
    f = lambda x, h: x.double().cpu().numpy().reshape(r.B, N, h, HD)
    path, count = r.path.cpu().numpy(), r.count.cpu().numpy()
    want = before.clone()
    for b in range(r.B):
        pages = [int(r.table[b, j // BLK]) for j in range(lens[b])]
        for l in range(LAYERS):
            kv = [np.array([before[l, p, w, :, j % BLK].double().cpu().numpy() for j, p in enumerate(pages)]).reshape(-1, NKV, HD) for w in (0, 1)]
            o, mag, dots = tree_attention(f(r.q[l], NQ)[b], *kv, f(r.k[l], NKV)[b], f(r.v[l], NKV)[b], PARENTS)
            got = f(r.o[l], NQ)[b]
            for i in range(N):
                assert (np.abs(got[i] - o[i]) <= attention_tol(o[i], mag[i], dots[i], lens[b] + N, False)).all()
        nodes, token = verify_greedy(tokens[b], PARENTS, r.ids.cpu().numpy()[b])
        assert list(path[b]) == nodes + [-1] * (N - len(nodes)) and count[b] == len(nodes) and int(r.next[b]) == token
        for j, node in enumerate(nodes):
            p = lens[b] + j
            for w, x in ((0, r.k), (1, r.v)):
                want[:, int(r.table[b, p // BLK]), w, :, p % BLK] = x[:, b * N + node].reshape(LAYERS, NKV, HD)
    assert torch.equal(r.pool.view(torch.int16), want.view(torch.int16))
    assert np.array_equal(r.lens.cpu().numpy(), lens + count)
    # the same logits' probabilities, verified by given numbers as drafts that were chosen
    rng = np.random.default_rng(int(lens.sum()))
    p = torch.softmax(r.logits, -1).float()
    u, un = (rng.random(s).astype(np.float32) for s in ((r.B, N), r.B))
    c, nx = (torch.zeros(r.B, dtype=torch.int32, device="cuda") for _ in range(2))
    pa = torch.zeros(r.B, N, dtype=torch.int32, device="cuda")
    r.t.tts_bb_tree_verify(r.B, N, V, r.tokens, r.parents, p, dev(u), dev(un), c, pa, nx, stream=torch.cuda.current_stream().cuda_stream)
    ph = p.double().cpu().numpy().reshape(r.B, N, V)
    for b in range(r.B):
        nodes, token, _ = verify(tokens[b], PARENTS, ph[b], None, u[b].astype(np.float64), float(un[b]))
        assert pa[b].tolist() == nodes + [-1] * (N - len(nodes)) and int(c[b]) == len(nodes) and int(nx[b]) == token
