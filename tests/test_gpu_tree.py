"""Attention of trees of drafted tokens, their verification and their commit, against the plain forms in 64 bits."""
from fractions import Fraction

import numpy as np
import pytest

from tests.gpu_util import tb
from tests.lowbit_util import U, attention_tol
from tests.tree_util import BLK, BLOCK, HD, NKV, NQ, random_tree, tree_attention, verify, verify_exactly, verify_greedy

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
NAN = float("nan")


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def ints(x):
    return dev(np.asarray(x, np.int32))


def stream():
    return torch.cuda.current_stream().cuda_stream


class Case:
    """A cache whose every place is NaN but the sequences' own keys, and trees whose padding is NaN."""

    def __init__(self, seed, lens, N, io, nodes=None, parents=None, bps=None, layers=1, rows=None, kscale=1.0):
        rng = self.rng = np.random.default_rng(seed)
        B = self.B = len(lens)
        self.N, self.lens, self.io = N, list(lens), io
        self.nodes = [N] * B if nodes is None else list(nodes)
        bps = self.bps = bps or max(1, max(-(-max(n, 0) // BLK) for n in lens))
        rows = self.rows = list(range(B)) if rows is None else rows
        n_rows = max(rows) + 1
        self.n_blocks = n_rows * bps + 3
        self.table = rng.permutation(self.n_blocks)[: n_rows * bps].reshape(n_rows, bps).astype(np.int32)
        self.pool = torch.full((layers, self.n_blocks, 2, NKV, BLK, HD), NAN, dtype=torch.bfloat16, device="cuda")
        self.k = [None] * B
        self.v = [None] * B
        for b, n in enumerate(lens):
            if rows[b] < 0:
                continue
            n = min(max(n, 0), bps * BLK)
            x = dev(rng.standard_normal((2, max(n, 1), NKV, HD)) * np.array([kscale, 1.0])[:, None, None, None]).bfloat16()[:, :n]
            page = dev(self.table[rows[b]]).long()[torch.arange(n, device="cuda") // BLK]
            tok = torch.arange(n, device="cuda") % BLK
            for w in (0, 1):
                self.pool[layers - 1, page, w, :, tok] = x[w]
            self.k[b], self.v[b] = x.double().cpu().numpy()
        self.parents = np.full((B, N), 99, np.int32)
        for b in range(B):
            n = max(self.nodes[b], 0)
            self.parents[b, : min(n, N)] = (random_tree(rng, n) if parents is None else np.asarray(parents[b])[:n])[:N]
        # q, k and v as parts of wider rows
        dt = getattr(torch, io)
        self.qw = torch.full((B * N, 2048 + 8), NAN, dtype=dt, device="cuda")
        self.kvw = torch.full((B * N, 4096), NAN, dtype=torch.bfloat16, device="cuda")
        for b in range(B):
            n = min(max(self.nodes[b], 0), N)
            at = slice(b * N, b * N + n)
            self.qw[at, :2048] = dev(1.5 * rng.standard_normal((n, 2048))).to(dt)
            self.kvw[at, 2048:] = dev(rng.standard_normal((n, 2048))).bfloat16()
        self.q, (self.tk, self.tv) = self.qw[:, :2048], self.kvw[:, 2048:].split(1024, 1)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.layers = layers

    def run(self, out=None, seqs=None, max_len=None, table=None, ws=None, **kw):
        m = tb()
        max_len = max(max(self.lens), 0) if max_len is None else max_len
        out = torch.full((self.B * self.N, 2048), 7.0, dtype=self.q.dtype, device="cuda") if out is None else out
        if ws is None:
            # poisoned, and followed by bytes that have to stay
            need = m.tts_bb_tree_attention_workspace(self.B, self.N, max_len)
            ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
            tail = ws[need:]
            ws = ws[:need] if need else None
        else:
            tail = None
        cache = m.KvCache(self.pool, dev(self.table if table is None else table), self.err, layers=self.layers)
        self.keep = [cache, ws, ints(self.parents), ints(self.lens), ints(self.nodes)]
        m.tts_bb_tree_attention(cache, self.layers - 1, self.B, self.N, self.q, self.tk, self.tv, self.keep[2], self.keep[3], max_len, out, ws,
                                n_nodes=self.keep[4], seqs=None if seqs is None else ints(seqs), stream=stream(), **kw)
        if tail is not None:
            assert (tail == 0xFF).all()
        return out

    def want(self, b, keep=None):
        n = self.nodes[b]
        at = slice(b * self.N, b * self.N + n)
        f = lambda t, h: t[at].double().cpu().numpy().reshape(n, h, HD)
        k, v = self.k[b], self.v[b]
        if keep is not None:
            k, v = k[keep], v[keep]
        return tree_attention(f(self.q, NQ), k, v, f(self.tk, NKV), f(self.tv, NKV), self.parents[b, :n])

    def check(self, out, skip=(), keep=None):
        got = out.double().cpu().numpy().reshape(self.B, self.N, NQ, HD)
        for b in range(self.B):
            n = 0 if b in skip else self.nodes[b]
            assert (got[b, n:] == 7).all(), b
            if n:
                w, mag, dots = self.want(b, keep if b == 0 else None)
                tol = np.stack([attention_tol(w[i], mag[i], dots[i], self.lens[b] + n, self.io == "bfloat16") for i in range(n)])
                bad = ~(np.abs(got[b, :n] - w) <= tol)
                assert not bad.any(), (b, np.argwhere(bad)[:5], np.abs(got[b, :n] - w)[bad][:5], tol[bad][:5])


IO = pytest.mark.parametrize("io", ["float32", "bfloat16"])


@IO
@pytest.mark.parametrize("N, lens", [
    (1, [0]), (1, [1]), (3, [0, 1, 2]), (1, [63, 64, 65, 127, 128, 129]), (64, [0, 5, 200]), (17, [191, 192, 193]), (33, [1000]), (64, [64 * 9 + 3]), (5, [4097]),
    (2, [3000, 10, 0, 777])])
def test_attention_matches_the_definition(io, N, lens):
    rng = np.random.default_rng(N)
    c = Case(len(lens) * 100 + N, lens, N, io, nodes=[max(1, N - int(rng.integers(0, N))) if b else N for b in range(len(lens))])
    c.check(c.run())
    assert int(c.err) == 0


@IO
def test_attention_of_many_sequences(io):
    """More (sequence, head) pairs than blocks run at once, ragged, trees of every size, some sequences padding."""
    rng = np.random.default_rng(5)
    B = 40
    lens = [int(n) for n in rng.integers(0, 400, B)]
    c = Case(6, lens, 12, io, nodes=[int(n) for n in rng.integers(0, 13, B)])
    seqs = np.arange(B)
    seqs[[3, 17]] = -1
    c.check(c.run(seqs=seqs), skip=(3, 17))
    assert int(c.err) == 0


@IO
@pytest.mark.parametrize("B, longest", [(1, 256), (1, 257), (1, 576), (1, 577), (4, 320), (4, 641), (4, 769), (12, 641), (19, 1216), (19, 1217), (20, 65)])
def test_attention_of_few_sequences_whole_and_cut(io, B, longest):
    """On both sides of what decides whether a sequence is cut; one of no keys, padding, and a longest one last."""
    lens = [int(x) for x in np.random.default_rng(B + longest).integers(0, longest + 1, B)]
    lens[-1] = longest
    if B > 2:
        lens[1] = 0
    c = Case(40 + B, lens, 5, io, rows=[-1 if B > 3 and b == 2 else b for b in range(B)])
    c.check(c.run(seqs=c.rows), skip=[2] if B > 3 else ())


@IO
def test_attention_of_more_sequences_than_threads(io):
    """Lengths are summed in several turns of a block; every seventh sequence is padding or out of range."""
    rng = np.random.default_rng(51)
    B = 1100
    c = Case(52, [int(n) for n in rng.integers(0, 3, B) * rng.integers(1, 70, B)], 2, io, nodes=[int(n) for n in rng.integers(0, 3, B)])
    seqs = np.arange(B)
    seqs[::7] = np.where(np.arange(0, B, 7) % 2, -1, B)
    out = c.run(seqs=seqs, max_len=200 if c.bps * BLK >= 200 else c.bps * BLK)
    some = set(range(0, B, 7))
    c.check(out, skip=some)
    assert int(c.err) == tb().TREE_ERR_RANGE


@IO
def test_attention_and_commit_beyond_4_gigabytes(io):
    """Blocks whose bytes start above 2^32, of a pool whose other blocks are NaN."""
    c = Case(53, [100, 700], 5, io)
    far = 17000
    pool = torch.full((1, far + c.n_blocks, 2, NKV, BLK, HD), NAN, dtype=torch.bfloat16, device="cuda")
    pool[:, far:] = c.pool
    c.pool, c.table, c.n_blocks = pool, c.table + far, far + c.n_blocks
    c.check(c.run())
    m = tb()
    cache = m.KvCache(pool, dev(c.table[:, -1:]), c.err)
    x = torch.randn(2 * 5, 1024, device="cuda").bfloat16()
    m.tts_bb_tree_commit(cache, 2, 5, x, x, ints([[0, 3, -1, -1, -1], [4, -1, -1, -1, -1]]), ints([2, 1]), ints([62, 0]), stream=stream())
    for b, pos, row in ((0, 62, 0), (0, 63, 3), (1, 0, 9)):
        got = pool[0, int(c.table[b, -1]), :, :, pos].reshape(2, -1)
        assert torch.equal(got[0], x[row]) and torch.equal(got[1], x[row])
    assert int(c.err) == 0


@IO
def test_attention_split_over_a_long_cache(io):
    c = Case(7, [20000, 7], 3, io)
    c.check(c.run())


@IO
def test_attention_with_a_loose_bound(io):
    """max_len far above the lengths, blocks behind the keys named by nothing that may be read."""
    c = Case(8, [70, 3], 6, io, bps=300)
    t = c.table.copy()
    t[0, 2:], t[1, 1:] = -7, 2**31 - 1
    c.check(c.run(max_len=300 * BLK, table=t))
    assert int(c.err) == 0


@IO
def test_attention_chains_forests_and_stars(io):
    N = 9
    chain, star, forest = [-1, *range(8)], [-1] + [0] * 8, [-1, -1, 0, 1, -1, 4, 2, 3, -1]
    c = Case(9, [100, 100, 100], N, io, parents=[chain, star, forest])
    c.check(c.run())


@IO
def test_attention_of_one_layer_of_several_and_shared_rows(io):
    """Two sequences read the same cache row; layers below the one that is read are NaN."""
    c = Case(10, [130, 130], 4, io, layers=3, rows=[2, 2])
    c.k[0], c.v[0] = c.k[1], c.v[1]
    c.check(c.run(seqs=[2, 2]))


@IO
def test_attention_reports_what_it_skips(io):
    c = Case(11, [100, 100, 100, 100, 100, 100, 100], 4, io)
    c.nodes = [4, 5, -1, 4, 4, 4, 0]
    c.parents[3, 2] = 2          # its own parent
    c.parents[4, 1] = -2
    c.check(c.run(seqs=[0, 1, 2, 3, 4, 7, 6]), skip=(1, 2, 3, 4, 5))
    m = tb()
    assert int(c.err) == m.TREE_ERR_RANGE | m.TREE_ERR_TREE
    c = Case(12, [100, 100, 100], 2, io)
    c.lens[1], c.lens[2] = -1, 101
    c.check(c.run(max_len=100), skip=(1, 2))
    assert int(c.err) == m.TREE_ERR_RANGE


@IO
def test_attention_without_an_error_word(io):
    c = Case(13, [100, 100], 2, io)
    c.parents[1] = 5
    c.err = None
    c.check(c.run(), skip=(1,))


@IO
@pytest.mark.parametrize("where, entry", [(0, -1), (1, 10**6), (3, -5), (4, 2**31 - 1)])
def test_attention_leaves_out_keys_behind_bad_pages(io, where, entry):
    n = 64 * 4 + 10
    c = Case(14 + where, [n, 100], 3, io)
    t = c.table.copy()
    t[0, where] = entry
    keep = np.ones(n, bool)
    keep[where * BLK : (where + 1) * BLK] = False
    c.check(c.run(table=t), keep=keep)
    assert int(c.err) == tb().TREE_ERR_PAGE
    c = Case(15, [n], 3, io)   # every page of a sequence
    c.check(c.run(table=np.full_like(c.table, -1)), keep=np.zeros(n, bool))


@IO
def test_attention_keeps_what_is_masked_apart(io):
    """Infinities and NaN in the keys and values of a node reach that node and those below it alone, and values of such columns only."""
    parents = [-1, 0, 0, 1, 2, 3]
    for bad in (NAN, np.inf, -np.inf):
        c = Case(20, [70], 6, io, parents=[parents])
        want = c.want(0)[0]
        c.tv[2, 5] = bad
        c.tv[2, 1000] = bad
        c.tk[4] = NAN
        out = c.run().double().cpu().numpy().reshape(6, NQ, HD)
        clean = np.ones((6, NQ, HD), bool)
        clean[4] = False
        clean[2, 0:2, 5] = clean[2, 14:16, 1000 - 7 * HD] = False
        assert np.isfinite(out[clean]).all() and np.abs(out - want)[clean].max() < 0.05
        assert np.isnan(out[4]).all()
        x = out[2][[0, 1, 14, 15], [5, 5, 104, 104]]
        assert np.isnan(x).all() if np.isnan(bad) else (np.isnan(x) | (x == bad)).all()
        assert not np.isfinite(x).any()


@IO
def test_attention_of_large_and_small_scores(io):
    """Scores of hundreds (one key takes all), of nothing (all alike), and all far below zero."""
    c = Case(21, [300], 5, io, kscale=60.0)
    c.check(c.run())
    c = Case(22, [300], 5, io)
    c.q.zero_()
    c.check(c.run())
    c = Case(23, [200], 3, io)
    c.q.fill_(-3e4)
    page = dev(c.table[0]).long()
    c.pool[0, page, 0] = 1000.0
    c.tk.fill_(1000.0)
    c.k[0][:] = 1000.0
    # equal scores of -3.4e8 (magnitudes above the weights' own): the mean of what a node sees
    out = c.run().double().cpu().numpy().reshape(3, NQ, HD)
    w, mag, _ = c.want(0)
    assert (np.abs(out - w) <= 300 * U * mag + np.abs(w) * 2.0 ** -8 + mag * 2.0 ** -15).all()


@IO
@pytest.mark.parametrize("n", [70, 3000])
def test_attention_of_infinite_keys(io, n):
    """Scores of -inf: no weight beside others, NaN where a node sees nothing else. fp32 queries meet infinite keys in parts, whose signs may differ: or NaN."""
    c = Case(29, [n], 4, io, parents=[[-1, 0, 1, -1]])
    c.q.abs_()
    c.pool[0, dev(c.table[0]).long()[torch.arange(n, device="cuda") // BLK], 0, :, torch.arange(n, device="cuda") % BLK, 0] = -np.inf
    c.k[0][:, :, 0] = -np.inf
    c.tk.view(4, NKV, HD)[3, :, 0] = -np.inf
    out = c.run().double().cpu().numpy().reshape(4, NQ, HD)
    assert np.isnan(out[3]).all()
    w, mag, _ = c.want(0)
    assert np.isnan(w[3]).all()
    # scores of 128 products whose magnitudes add up to 200 at most, in fp32; bf16: weights in two parts, the result rounded
    near = np.abs(out - w) <= mag * (2 * 136 * 200 * U / np.sqrt(HD) + 2.0 ** -15) + np.abs(w) * 2.0 ** -8
    assert (near | (np.isnan(out).all(-1, keepdims=True) & (io == "float32")))[:3].all()


@IO
@pytest.mark.parametrize("N, lens", [(5, [100, 7]), (33, [5000, 130])])
@pytest.mark.parametrize("size", [13, 15, 17, 30, 59])
@pytest.mark.parametrize("shape", ["equal", "rising", "falling", "mixed"])
def test_attention_of_scores_far_from_zero(io, N, lens, size, shape):
    """Queries and keys of 2^size: scores of which the greatest take all, equally, whole sequences and cut ones. Keys are 2^size times one of
    few numbers of 8 bits, so equal keys' scores are equal and others' 2^18 apart at least."""
    c = Case(28, lens, N, io)
    rng = np.random.default_rng(size)
    pages = -(-max(lens) // BLK)
    of_page = {"equal": np.full(pages, 77), "rising": np.arange(pages) + 5, "falling": 120 - np.arange(pages), "mixed": rng.integers(0, 128, pages)}[shape]
    f = lambda i: 2.0 ** size * (1 + np.asarray(i) / 128)
    for b, n in enumerate(c.lens):
        page = np.arange(n) // BLK
        x = f(of_page[page])
        c.pool[0, dev(c.table[b]).long()[dev(page)], 0, :, dev(np.arange(n) % BLK)] = dev(x).bfloat16()[:, None, None]
        c.k[b][:] = x[:, None, None]
    q, tk = c.q.view(len(lens), N, NQ, HD), c.tk.view(len(lens), N, NKV, HD)
    q[:] = 2.0 ** size * (1 + 2.0 ** (-20 if io == "float32" else -6))
    q[:, :, 1::2] *= -1
    tk[:] = dev(f(np.full((len(lens), N), 77) if shape == "equal" else rng.integers(0, 128, (len(lens), N)))).bfloat16()[:, :, None, None]
    got = c.run().double().cpu().numpy().reshape(len(lens), N, NQ, HD)
    for b, n in enumerate(lens):
        w, mag, _ = c.want(b)
        # the exponentials of 0 and the sums; bf16: weights in two parts, the result rounded
        tol = mag * (2 * 2.0 ** -21 + (n + N + 32) * U) + (mag * 2.0 ** -15 + np.abs(w) * 2.0 ** -8 if io == "bfloat16" else 0)
        assert (np.abs(got[b] - w) <= tol).all(), (b, np.abs(got[b] - w).max())


@IO
@pytest.mark.parametrize("step", ["little", "much", "either", "once"])
@pytest.mark.parametrize("who", ["all", "last"])
def test_attention_of_scores_that_rise_from_page_to_page(io, step, who):
    """By less than the reference may lag, by more, up and down, and once: for all nodes, or for the last one alone."""
    c = Case(26, [64 * 21 + 20, 64 * 5, 64 * 2 + 1], 33, io)
    rng = np.random.default_rng(27)
    for b, n in enumerate(c.lens):
        page = np.arange(n) // BLK
        rise = {"little": 0.6 * page, "much": 3.0 * page, "either": rng.choice([-4.0, 0.0, 0.9, 4.0], page[-1] + 1)[page], "once": 9.0 * (page == page[-1] - 1)}[step]
        x = dev(rise * np.sqrt(HD) / 8).bfloat16()
        at = dev(c.table[b]).long()[dev(page)]
        c.pool[0, at, 0, :, dev(np.arange(n) % BLK), 0] = x[:, None]
        c.k[b][:, :, 0] = x.double().cpu().numpy()[:, None]
    q = c.q.view(3, 33, NQ, HD)
    q[:, :, :, 0] = 0.0
    q[:, 0 if who == "all" else 32 :, 0::3, 0] = 8.0
    q[:, 0 if who == "all" else 32 :, 1::3, 0] = -8.0
    c.check(c.run())


@IO
def test_attention_is_the_same_every_time_and_in_a_graph(io):
    """Bitwise, on another stream, in a captured graph that is replayed on other inputs, and two calls at once."""
    c = Case(24, [900, 40, 333], 7, io)
    first = c.run()
    for _ in range(3):
        assert torch.equal(c.run(), first)
    m = tb()
    need = m.tts_bb_tree_attention_workspace(c.B, c.N, 900)
    cache = m.KvCache(c.pool, dev(c.table), c.err)
    par, n = ints(c.parents), ints(c.nodes)
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.full_like(first, 7.0) for _ in range(2)]
    wss = [torch.empty(max(need, 16), dtype=torch.uint8, device="cuda") for _ in range(2)]
    lens = ints(c.lens)
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o, w in zip(sides, outs, wss):
            m.tts_bb_tree_attention(cache, 0, c.B, c.N, c.q, c.tk, c.tv, par, lens, 900, o, w, n_nodes=n, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(sides[0]), torch.cuda.graph(g, stream=sides[0]):
        m.tts_bb_tree_attention(cache, 0, c.B, c.N, c.q, c.tk, c.tv, par, lens, 900, outs[0], wss[0], n_nodes=n,
                                stream=torch.cuda.current_stream().cuda_stream)
    outs[0].fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first)
    c.lens = [500, 39, 1]
    lens.copy_(ints(c.lens))
    outs[0].fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], c.run(max_len=900))


def test_attention_does_not_need_node_counts_or_rows():
    c = Case(25, [90, 90], 3, "bfloat16")
    m = tb()
    out = torch.full((6, 2048), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(16, m.tts_bb_tree_attention_workspace(2, 3, 90)), dtype=torch.uint8, device="cuda")
    m.tts_bb_tree_attention(m.KvCache(c.pool, dev(c.table)), 0, 2, 3, c.q, c.tk, c.tv, ints(c.parents), ints(c.lens), 90, out, ws, stream=stream())
    c.check(out)


# ------------------------------------------------------------------ verification
class Trees:
    def __init__(self, seed, B, N, V, drawn, sharp=2.0, nodes=None, pad=0):
        rng = np.random.default_rng(seed)
        self.B, self.N, self.V = B, N, V
        self.nodes = [N] * B if nodes is None else nodes
        self.parents = np.stack([random_tree(rng, N, 4) for _ in range(B)])
        z = sharp * rng.standard_normal((B * N, V))
        d = z + 0.7 * rng.standard_normal((B * N, V))
        soft = lambda a: (lambda e: e / e.sum(-1, keepdims=True))(np.exp(a - a.max(-1, keepdims=True))).astype(np.float32)
        self.p, self.q = soft(z), soft(d) if drawn else None
        row = np.arange(B)[:, None] * N + np.maximum(self.parents, 0)
        cdf = np.cumsum(soft(d).astype(np.float64), -1)
        pick = rng.random((B, N))
        self.tokens = np.array([[int(np.searchsorted(cdf[row[b, j]], pick[b, j] * cdf[row[b, j], -1])) for j in range(N)] for b in range(B)], np.int32)
        self.u, self.un = rng.random((B, N)).astype(np.float32), rng.random(B).astype(np.float32)
        self.pad = pad

    def run(self, err=None, nodes=True):
        m = tb()
        wide = lambda x: torch.nn.functional.pad(dev(x), (0, self.pad), value=NAN)
        count, nxt = (torch.full((self.B,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
        path = torch.full((self.B, self.N), -9, dtype=torch.int32, device="cuda")
        m.tts_bb_tree_verify(self.B, self.N, self.V, ints(self.tokens), ints(self.parents), wide(self.p), dev(self.u), dev(self.un), count, path, nxt,
                             draft=None if self.q is None else wide(self.q), n_nodes=ints(self.nodes) if nodes else None, err=err, stream=stream())
        return count.cpu().numpy(), path.cpu().numpy(), nxt.cpu().numpy()

    def check(self, skip=(), least=1e-9):
        count, path, nxt = self.run()
        lengths = []
        for b in range(self.B):
            n = 0 if b in skip else self.nodes[b]
            if n == 0:
                assert count[b] == 0 and nxt[b] == -1 and (path[b] == -1).all()
                continue
            at = slice(b * self.N, b * self.N + n)
            f = lambda x: None if x is None else x[at].astype(np.float64)
            want, token, near = verify(self.tokens[b, :n], self.parents[b], f(self.p), f(self.q), self.u[b].astype(np.float64), float(self.un[b]))
            if near < least:
                continue  # closer to a border than the plain form itself resolves
            assert count[b] == len(want) and list(path[b]) == want + [-1] * (self.N - len(want)) and nxt[b] == token, b
            lengths.append(len(want))
        return lengths


DRAWN = pytest.mark.parametrize("drawn", [True, False])


@DRAWN
@pytest.mark.parametrize("B, N, V", [(1, 1, 1), (1, 1, 1000), (3, 5, 2), (70, 9, 33), (20, 64, 500), (5, 7, 2049), (40, 6, 4096), (3, 6, 30011), (2, 4, 151676),
                                     (700, 8, 70)])
def test_verify_matches_the_definition(drawn, B, N, V):
    t = Trees(B + N + V, B, N, V, drawn, nodes=[max(0, N - b % (N + 1)) if b % 4 == 3 else N for b in range(B)], pad=V % 3)
    lengths = t.check()
    if B >= 20 and N > 4 and drawn:  # the walks go somewhere (chosen drafts are accepted with p(x) alone: seldom, of many ids)
        assert 1 < np.mean(lengths) and max(lengths) > 2 and min(lengths) == 1
    if N > 1:
        count, path, nxt = t.run()
        for _ in range(2):
            again = t.run()
            assert all(np.array_equal(x, y) for x, y in zip(again, (count, path, nxt)))


@DRAWN
def test_verify_keeps_the_targets_distribution(drawn):
    """The token behind the root is distributed as the target's row, whatever the draft's: 5 standard deviations of 65000 trees'
    counts, the last id's and the likeliest's among them."""
    rng = np.random.default_rng(3)
    V, N, B = 6, 5, 13000
    counts, p = np.zeros(V), rng.dirichlet(np.ones(V)).astype(np.float32)
    d = rng.dirichlet(np.ones(V)).astype(np.float32)
    for turn in range(5):
        t = Trees(turn, 1, N, V, drawn)
        t.B, t.parents = B, np.tile(np.array([[-1, 0, 0, 0, 0]], np.int32), (B, 1))
        t.nodes = [N] * B
        t.p = np.tile(p, (B * N, 1))
        t.q = np.tile(d, (B * N, 1)) if drawn else None
        t.tokens = rng.choice(V, (B, N), p=d.astype(np.float64) / d.astype(np.float64).sum()).astype(np.int32)
        t.u, t.un = rng.random((B, N)).astype(np.float32), rng.random(B).astype(np.float32)
        count, path, nxt = t.run()
        first = np.where(count > 1, t.tokens[np.arange(B), path[:, 1]], nxt)
        counts += np.bincount(first, minlength=V)
    T = 5 * B
    assert (np.abs(counts - T * p) <= 5 * np.sqrt(T * p * (1 - p))).all(), (counts / T, p)


def test_verify_rows_of_every_alignment():
    """Rows that start at each of the four places of 16 bytes, the draft's like the target's or not."""
    m = tb()
    t = Trees(6, 12, 5, 5003, True)
    want = t.run()
    for dp in range(4):
        for dq in (dp, (dp + 1) % 4):
            def at(x, off):
                buf = torch.full((t.B * t.N, t.V + 5), NAN, device="cuda")
                buf[:, off : off + t.V] = dev(x)
                return buf[:, off : off + t.V]
            count, nxt = (torch.zeros(t.B, dtype=torch.int32, device="cuda") for _ in range(2))
            path = torch.zeros(t.B, t.N, dtype=torch.int32, device="cuda")
            m.tts_bb_tree_verify(t.B, t.N, t.V, ints(t.tokens), ints(t.parents), at(t.p, dp), dev(t.u), dev(t.un), count, path, nxt, draft=at(t.q, dq),
                                 stream=stream())
            assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip((count, path, nxt), want))


def test_verify_borders():
    """Numbers of 0 and next to 1, mass at one id, nothing left, equal rows, tokens out of range, the same token twice."""
    N, V = 4, 40
    t = Trees(1, 12, N, V, True)
    t.parents = np.tile(np.array([[-1, 0, 0, 1]], np.int32), (12, 1))
    one = lambda i: np.eye(V, dtype=np.float32)[i]
    below = np.float32(1 - 2.0 ** -24)
    p, q = t.p.reshape(12, N, V), t.q.reshape(12, N, V)
    t.u[0], t.un[0] = 0, 0
    t.u[1], t.un[1] = below, below
    p[2], q[2], t.tokens[2] = one(7), one(7), 7            # u 1 < 1: all accepted
    p[3], q[3], t.tokens[3] = one(V - 1), one(0), 0        # never accepted; the rest is p
    p[4], q[4], t.u[4] = q[4], q[4], below                 # equal rows: accepted but for rounding, else nothing is left
    p[5] = 0                                               # no mass at all: id 0
    p[6, 0], q[6, 0], t.tokens[6] = one(3) * np.float32(0.5), one(3), 3   # sum 1 / 2: r is 0 behind a rejection, id 3
    t.u[6] = below
    t.tokens[7], t.u[7] = [0, -1, V, 2**31 - 1], 0
    t.tokens[8], t.tokens[8, 2] = t.tokens[8, 1], t.tokens[8, 1]
    t.u[8] = below
    p[9, 0] = np.where(np.arange(V) < 2, np.float32(2.0 ** -30), 0)       # tiny rows
    p[10], q[10] = p[10] * np.float32(1.0005), q[10]
    t.un[11] = 1.0
    count, path, nxt = t.run()
    assert count[2] == 3 and list(path[2]) == [0, 1, 3, -1] and nxt[2] == 7
    assert count[3] == 1 and nxt[3] == V - 1 and nxt[5] == 0
    assert count[6] == 1 and nxt[6] == 3
    assert count[7] == 1
    assert nxt[9] in (0, 1) or count[9] > 1
    assert 0 <= nxt[11] < V
    t.p, t.q = p.reshape(-1, V), q.reshape(-1, V)
    t.un[11] = below
    t.check(skip=())
    t.q = None
    t.check()


def rounded_case(seed):
    """Rows p, q of 8 ids, a token x and a number u. Behind two rejections of id 0 the rest is (p - c q)^+ with c = 1 + sum (p - q)^+. Id 1's p is
    what c q rounds to in fp32, and above c q: u lies above the border of x for the sum of all rests, below it for the sum without id 1's."""
    rng = np.random.default_rng(seed)
    rests = lambda p, q, c: [max(x - c * y, 0) for x, y in zip(p, q)]
    while True:
        q = rng.dirichlet(np.full(8, 4.0)).astype(np.float32)
        p = (q * (1 + 0.02 * rng.standard_normal(8))).astype(np.float32)
        p[0] = q[0] * np.float32(0.9)
        P, Q = [Fraction(float(x)) for x in p], [Fraction(float(x)) for x in q]
        for _ in range(30):  # c moves with id 1's p
            c = 1 + sum(rests(P, Q, 1))
            same = p[1] == np.float32(float(c * Q[1]))
            if same:
                break
            p[1] = np.float32(float(c * Q[1]))
            P[1] = Fraction(float(p[1]))
        if not same or P[1] <= c * Q[1]:
            continue
        r = rests(P, Q, c)
        for x in range(2, 8):
            low, high = (r[x] / (Q[x] * z) for z in (sum(r), sum(r) - r[1]))
            u = np.float32(float((low + high) / 2))
            if r[x] > 0 and u < 1 and low * (1 + Fraction(1, 2 ** 40)) < Fraction(float(u)) < high * (1 - Fraction(1, 2 ** 40)):
                return p, q, x, u


def test_verify_counts_a_rest_below_the_rounding_of_its_product():
    t = Trees(2, 4, 4, 8, True)
    t.parents = np.tile(np.array([[-1, 0, 0, 0]], np.int32), (4, 1))
    t.u[:, 1:3] = 1 - 2.0 ** -10
    for b in range(4):
        t.p[4 * b], t.q[4 * b], x, t.u[b, 3] = rounded_case(b)
        t.tokens[b] = [0, 0, 0, x]
    count, path, nxt = t.run()
    assert list(count) == [1, 1, 1, 1]


@pytest.mark.parametrize("V", [2, 70, 5000])
@pytest.mark.parametrize("top", [1.0, 0.98])
def test_verify_of_stars_whose_draft_repeats_one_token(V, top):
    """17 to 63 children of the root, all (but for one at the end) of the token that the draft gives `top`, all rejected: c, the sum of
    what the rejections leave, passes 16 (and with that what 64 bits hold of c q in 2^-60) and 32."""
    N, likely, nexts = 64, (0.06, 0.3, 0.45), (0.0, 0.004, 0.01, 0.05, 0.4)
    todo = [(p0, n, un) for p0 in likely for n in range(18, N + 1) for un in nexts]
    t = Trees(1, len(todo), N, 2, True)
    rng = np.random.default_rng(V)
    t.V = V
    t.parents[:] = [-1] + [0] * (N - 1)
    t.nodes = [n for _, n, _ in todo]
    t.tokens[:] = 0
    t.u[:] = 0.9
    t.un = np.array([un for _, _, un in todo], np.float32)
    others = rng.dirichlet(np.ones(V - 1), len(todo))
    root = np.arange(len(todo)) * N
    t.p, t.q = (np.zeros((len(todo) * N, V), np.float32) for _ in range(2))
    t.p[root, 0] = [p0 for p0, _, _ in todo]
    t.p[root, 1:] = (1 - np.array([[p0] for p0, _, _ in todo])) * others
    t.q[root, 0] = top
    t.q[root, 1:] = (1 - top) / (V - 1)
    for b, n in enumerate(t.nodes):
        if b % 3 == 0:
            t.tokens[b, n - 1] = V - 1
    assert len(t.check(least=1e-7)) > 0.9 * len(todo)


@pytest.mark.parametrize("V, steps", [(64, 1), (64, 40), (1500, 3), (5003, 60)])
def test_verify_of_a_draft_next_to_the_target(V, steps):
    """Rows that differ by a few steps of fp32: what the first rejection of a node leaves is of the size of 2^-24, and the rejections and
    the next token behind it are of that. Masses are held to some 2^-46 for each rejection (seven here), whatever their size."""
    B, N = 24, 20
    t = Trees(V + steps, B, N, V, True, sharp=1.0)
    rng = np.random.default_rng(V)
    t.parents[:] = [-1] + [0] * 7 + [1] * 3 + [2] * 3 + [3, 4, 5, 6, 7, 7]
    t.p[:: N] = np.where(rng.random((B, V)) < 0.02, t.p[:: N] * np.float32(1 + 2.0 ** -20), t.p[:: N])
    off = rng.integers(-steps, steps + 1, t.p.shape) * np.spacing(t.p)
    t.q = (t.p + off).astype(np.float32)
    below = 1 - 2.0 ** -24
    for b in range(B):  # the root's first child is rejected: its draft lies above the target; a third of the trees end there, behind seven such
        above = np.nonzero(t.q[b * N] * below >= t.p[b * N].astype(np.float64))[0]
        t.tokens[b, 1:8] = rng.choice(above, 7) if b % 3 == 0 else rng.integers(0, V, 7)
        t.tokens[b, 1], t.u[b, 1] = rng.choice(above), below
    count, path, nxt = t.run()
    seen, rejected = 0, 0
    for b in range(B):
        at = slice(b * N, (b + 1) * N)
        want, token, near = verify_exactly(t.tokens[b], t.parents[b], t.p[at], t.q[at], t.u[b], t.un[b])
        if near < 8 * 2.0 ** -46:
            continue
        assert count[b] == len(want) and list(path[b]) == want + [-1] * (N - len(want)) and nxt[b] == token, b
        seen += 1
        rejected += len(want) == 1
    assert seen > 0.8 * B and rejected >= 6


@DRAWN
def test_verify_with_values_that_are_no_probabilities(drawn):
    """NaN, infinities, negative and large values: some path and some token, and no other sequence's changes."""
    t = Trees(2, 30, 6, 3000, drawn)
    good = t.run()
    bad = [NAN, np.inf, -np.inf, -1.0, 7.0, 3e38]
    for i, x in enumerate(bad):
        t.p[(5 * i) * 6 : (5 * i + 1) * 6, :: i + 1] = x
    t.u[2], t.un[2] = NAN, NAN
    t.u[3], t.un[3] = -1, 5
    count, path, nxt = t.run()
    assert (count >= 1).all() and (count <= 6).all() and (nxt >= 0).all() and (nxt < 3000).all()
    same = [b for b in range(30) if b % 5 and b not in (2, 3)]
    for a, b in zip(good, (count, path, nxt)):
        assert np.array_equal(a[same], b[same])


@DRAWN
def test_verify_reports_what_it_skips(drawn):
    t = Trees(4, 8, 5, 100, drawn, nodes=[5, 6, -1, 5, 5, 0, 1, 5])
    t.parents[3, 2], t.parents[4, 0] = 2, 0
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t.run(err)
    assert int(err) == tb().TREE_ERR_RANGE | tb().TREE_ERR_TREE
    t.check(skip=(1, 2, 3, 4))
    t = Trees(5, 6, 5, 100, drawn)
    t.check()
    a, b = t.run(), t.run(nodes=False)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))


@DRAWN
def test_verify_in_a_graph_and_two_at_once(drawn):
    m = tb()
    t = Trees(8, 20, 8, 9000, drawn)
    want = t.run()
    a = [ints(t.tokens), ints(t.parents), dev(t.p), dev(t.u), dev(t.un)]
    q = dev(t.q) if drawn else None
    outs = [[torch.zeros(t.B, dtype=torch.int32, device="cuda"), torch.zeros(t.B, t.N, dtype=torch.int32, device="cuda"),
             torch.zeros(t.B, dtype=torch.int32, device="cuda")] for _ in range(2)]
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    call = lambda o, st: m.tts_bb_tree_verify(t.B, t.N, t.V, *a, *o, draft=q, stream=st)
    for _ in range(5):
        for o, s in zip(outs, sides):
            call(o, s.cuda_stream)
    torch.cuda.synchronize()
    for o in outs:
        assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(o, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(sides[0]), torch.cuda.graph(g, stream=sides[0]):
        call(outs[0], torch.cuda.current_stream().cuda_stream)
    for x in outs[0]:
        x.fill_(-9)
    g.replay()
    torch.cuda.synchronize()
    assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(outs[0], want))
    t.u = np.random.default_rng(9).random(t.u.shape).astype(np.float32)
    a[3].copy_(dev(t.u))
    g.replay()
    torch.cuda.synchronize()
    assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(outs[0], t.run()))


@pytest.mark.parametrize("B, N", [(1, 1), (3, 64), (130, 33), (1000, 6)])
def test_greedy_matches_the_definition(B, N):
    rng = np.random.default_rng(B)
    parents = np.stack([random_tree(rng, N, 5) for _ in range(B)])
    tokens, ids = (rng.integers(-1, 3, (B, N)).astype(np.int32) for _ in range(2))
    nodes = [int(n) for n in rng.integers(0, N + 1, B)]
    nodes[0] = N
    bad = set()
    if B > 5:
        parents[1, 0], nodes[1] = 1, N
        nodes[2], nodes[3] = N + 1, -1
        bad = {1, 2, 3}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    count, nxt = (torch.full((B,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    path = torch.full((B, N), -9, dtype=torch.int32, device="cuda")
    tb().tts_bb_tree_verify_greedy(B, N, ints(tokens), ints(parents), ints(ids), count, path, nxt, n_nodes=ints(nodes), err=err, stream=stream())
    count, path, nxt = (x.cpu().numpy() for x in (count, path, nxt))
    for b in range(B):
        n = 0 if b in bad else nodes[b]
        want, token = verify_greedy(tokens[b, :n], parents[b], ids[b]) if n else ([], -1)
        assert count[b] == len(want) and list(path[b]) == want + [-1] * (N - len(want)) and nxt[b] == token
    assert int(err) == (3 << 1 if bad else 0)


# ------------------------------------------------------------------ commit
@pytest.mark.parametrize("L, B, N, strided", [(1, 1, 1, False), (3, 5, 7, True), (28, 3, 64, False), (2, 130, 4, True)])
def test_commit_writes_the_paths_and_nothing_else(L, B, N, strided):
    rng = np.random.default_rng(L + B + N)
    m = tb()
    bps, n_rows = 3, B + 2
    nb = n_rows * bps + 1
    pool = torch.randn(L, nb, 2, NKV, BLK, HD, device="cuda").bfloat16()
    table = rng.permutation(nb)[: n_rows * bps].reshape(n_rows, bps).astype(np.int32)
    seqs = rng.permutation(n_rows)[:B].astype(np.int32)
    lens = rng.integers(0, bps * BLK - 64, B).astype(np.int32)
    count = rng.integers(0, N + 1, B).astype(np.int32)
    path = np.full((B, N), -1, np.int32)
    for b in range(B):
        path[b, : count[b]] = np.sort(rng.permutation(N)[: count[b]])
    flags = 0
    if B >= 5:
        lens[0], count[0], path[0] = bps * BLK - 2, N, np.arange(N)         # runs over the end of its row
        seqs[1] = -1
        seqs[2] = n_rows
        count[3], path[3] = 2, [1, N] + [-1] * (N - 2)                      # a node out of range
        lens[4], count[4], path[4] = 60, N, np.arange(N)
        table[seqs[4], 1] = nb                                              # a page out of range
        flags = m.TREE_ERR_RANGE | m.TREE_ERR_TREE | (m.TREE_ERR_PAGE if 60 + N > BLK else 0)  # only a path that gets there meets it
    if B >= 130:
        lens[10], count[11], count[12] = -1, -1, N + 1
    k, v = (torch.randn(L, B * N + 3, 2048, device="cuda").bfloat16()[:, : B * N, 512:1536] for _ in range(2))
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    want = pool.clone()
    for b in range(B):
        if not 0 <= seqs[b] < n_rows or lens[b] < 0 or not 0 <= count[b] <= N:
            continue
        for j in range(count[b]):
            pos, node = lens[b] + j, path[b, j]
            if pos < bps * BLK and 0 <= node < N and 0 <= table[seqs[b], pos // BLK] < nb:
                for w, x in ((0, k), (1, v)):
                    want[:, int(table[seqs[b], pos // BLK]), w, :, int(pos % BLK)] = x[:, b * N + int(node)].reshape(L, NKV, HD)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = m.KvCache(pool, dev(table), err, layers=L)
    m.tts_bb_tree_commit(cache, B, N, k, v, ints(path), ints(count), ints(lens), seqs=ints(seqs), stream=stream())
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))
    assert int(err) == flags


def test_commit_at_positions_beyond_31_bits():
    """A row whose table is that long (of pages that all but the last two are one): K and V from position 2^31 - 3 on."""
    m = tb()
    bps, N = 2 ** 25 + 1, 6
    pool = torch.randn(4, 2, NKV, BLK, HD, device="cuda").bfloat16()
    table = torch.zeros(1, bps, dtype=torch.int32, device="cuda")
    table[0, -2], table[0, -1] = 2, 1
    k, v = (torch.randn(1, N, 1024, device="cuda").bfloat16() for _ in range(2))
    want = pool.clone()
    for j in range(N):
        for w, x in ((0, k), (1, v)):
            want[2 if j < 3 else 1, w, :, (61 + j) % BLK] = x[0, j].reshape(NKV, HD)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.tts_bb_tree_commit(m.KvCache(pool, table, err), 1, N, k, v, ints(np.arange(N)), ints([N]), ints([2 ** 31 - 3]), stream=stream())
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))
    assert int(err) == 0
