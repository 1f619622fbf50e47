"""The 4-bit paged cache: append, read-back and attention against their plain forms in 64 bits."""
import numpy as np
import pytest

from tests.gpu_util import tb
from tests.lowbit_util import (BLK, BLOCK, HD, NKV, NQ, U, attention, attention_tol, bf16_f64, code_bytes, decode, fill, make_pool,
                               par_bytes, quantise, rotated)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
EPS = 1e-6


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def stream():
    return torch.cuda.current_stream().cuda_stream


class Setup:
    """A cache of n_seqs rows, its blocks scattered over the pool, with gains and rope tables."""

    def __init__(self, seed, n_seqs, bps, n_pos=None, spare=3):
        self.rng = np.random.default_rng(seed)
        self.n_blocks = n_seqs * bps + spare
        self.table = self.rng.permutation(self.n_blocks)[: n_seqs * bps].reshape(n_seqs, bps).astype(np.int32)
        self.gq, self.gk = (bf16_f64(1 + 0.1 * self.rng.standard_normal(HD)) for _ in range(2))
        m = tb()
        self.cos, self.sin = m.tts_bb_rope_tables(1e6, n_pos or bps * BLK)
        self.pool_h = make_pool(self.rng, self.n_blocks)
        self.pool = dev(self.pool_h)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cache = m.Kv4Cache(self.pool, dev(self.table), self.err)

    def append(self, qkv, seqs, positions, q_out=None, **kw):
        args = [dev(self.gq, torch.bfloat16), dev(self.gk, torch.bfloat16), dev(self.cos), dev(self.sin)]
        return tb().tts_bb_kv4_append(self.cache, len(seqs), qkv, *args, len(self.cos), dev(np.asarray(seqs, np.int32)),
                                      dev(np.asarray(positions, np.int32)), q_out, eps=EPS, stream=stream(), **kw)

    def expect(self, x, seqs, positions):
        """The pool's bytes and the queries after appending x [T][4096] (float64)."""
        pool = self.pool_h.copy()
        x = x.reshape(len(x), 32, HD)
        pos = np.clip(positions, 0, len(self.cos) - 1)
        c, s = self.cos[pos].astype(np.float64), self.sin[pos].astype(np.float64)
        eps = float(np.float32(EPS))
        q, k = rotated(x[:, :NQ], self.gq, c, s, eps), rotated(x[:, NQ : NQ + NKV], self.gk, c, s, eps)
        for which, y in enumerate((k, x[:, NQ + NKV :])):
            code, scale, off = quantise(y)
            by, par = code_bytes(code), par_bytes(scale, off)
            for t, (b, p) in enumerate(zip(seqs, positions)):
                if b >= 0:
                    tile, tok = pool[self.table[b, p // BLK], which], p % BLK
                    tile[:, tok * 64 : tok * 64 + 64] = by[t]
                    tile[:, 4096 + tok * 8 : 4096 + tok * 8 + 8] = par[t]
        return pool, q


def same_pool(got, want):
    """Bytes equal; a NaN scale is any bf16 NaN, and its codes and offset do not matter."""
    got, want = got.reshape(want.shape), want
    for a, b in zip(got, want):
        if np.array_equal(a, b):
            continue
        pa, pb = (torch.from_numpy(t[..., 4096:].copy()).view(torch.bfloat16).float().numpy().reshape(2, NKV, BLK, 2, 2) for t in (a, b))
        nan = np.isnan(pb[..., 0])
        assert np.array_equal(nan, np.isnan(pa[..., 0]))
        assert np.array_equal(pa[~nan], pb[~nan])
        ca, cb = (t[..., :4096].reshape(2, NKV, BLK, 8, 2, 4) for t in (a, b))
        live = ~np.broadcast_to(nan[..., None, :, None], ca.shape)
        assert np.array_equal(ca[live], cb[live])


@pytest.mark.parametrize("io", ["float32", "bfloat16"])
@pytest.mark.parametrize("T", [1, 5, 130, 700])
def test_append_writes_the_definitions_bytes(io, T):
    """Every byte of the pool, the untouched ones too: codes and parameters are those of 64-bit arithmetic."""
    s = Setup(T, 3, 5)
    dt = getattr(torch, io)
    x = s.rng.standard_normal((T, 4096)) * np.exp(0.6 * s.rng.standard_normal((1, 4096))) + 0.3 * s.rng.standard_normal((1, 4096))
    xd = torch.zeros(T, 4096 + 8, dtype=dt, device="cuda")[:, :4096]  # rows further apart than they are long
    xd.copy_(dev(x))
    x = xd.double().cpu().numpy()
    cells = s.rng.permutation(3 * 5 * BLK)[:T]
    seqs, pos = (cells // (5 * BLK)).astype(np.int32), (cells % (5 * BLK)).astype(np.int32)
    if T > 1:
        seqs[T // 2] = -1
    q_out = torch.full((T + 1, NQ, HD), 7.0, dtype=dt, device="cuda")
    assert s.append(xd, seqs, pos, q_out) == 0
    pool, q = s.expect(x, seqs, pos)
    same_pool(s.pool.cpu().numpy(), pool)
    got = q_out.double().cpu().numpy()
    assert (got[T] == 7).all() and (T == 1 or (got[T // 2] == 7).all())
    live = seqs >= 0
    # norm, gain and rotation: 16 U of |x cos| + |x' sin| <= sqrt 2 of the pair, then one rounding of the type
    pair = np.sqrt(q[..., :64] ** 2 + q[..., 64:] ** 2)
    tol = 16 * U * np.sqrt(2) * np.concatenate((pair, pair), -1) + (np.abs(q) * 2.0 ** -8 if io == "bfloat16" else 0)
    assert (np.abs(got[:T] - q) <= tol)[live].all()
    assert int(s.err) == 0


def test_append_without_queries_and_long_positions():
    """q_out may be absent, and positions far along rotate by their own table row."""
    s = Setup(2, 1, 40)
    x = s.rng.standard_normal((4, 4096)).astype(np.float32)
    pos = np.array([2559, 2496, 0, 1000], np.int32)
    assert s.append(dev(x), [0] * 4, pos) == 0
    same_pool(s.pool.cpu().numpy(), s.expect(x.astype(np.float64), [0] * 4, pos)[0])


def test_append_special_groups():
    """Constant groups, zeros, an offset far from zero, tiny and huge magnitudes, and values that are not finite."""
    s = Setup(4, 1, 1)
    x = s.rng.standard_normal((10, 4096))
    v = x.reshape(10, 32, HD)[:, 24:]
    v[0] = 0.0
    v[1] = 3.25
    v[2] = 100 + 0.01 * v[2]
    v[3] *= 1e-30
    v[4] *= 1e35
    v[5, :, 3], v[6, :, 70], v[7, :, 127] = np.nan, np.inf, -np.inf
    v[8] *= 1e-38
    v[9] = -np.abs(v[9])
    x = x.astype(np.float32)
    assert s.append(dev(x), [0] * 10, np.arange(10)) == 0
    want, _ = s.expect(x.astype(np.float64), [0] * 10, np.arange(10))
    same_pool(s.pool.cpu().numpy(), want)
    k, vv = (torch.empty(10, NKV, HD, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tb().tts_bb_kv4_read(s.cache, 10, dev(np.zeros(10, np.int32)), dev(np.arange(10, dtype=np.int32)), k, vv, stream=stream())
    vv = vv.double().cpu().numpy()
    assert (vv[0] == 0).all() and np.isfinite(vv[[1, 2, 3, 4, 8, 9]]).all()
    assert np.isnan(vv[5, :, :64]).all() and np.isfinite(vv[5, :, 64:]).all()
    assert np.isnan(vv[6:8, :, 64:]).all() and np.isfinite(vv[6:8, :, :64]).all()
    xv = x.reshape(10, 32, HD)[:, 24:].astype(np.float64)
    # half a scale (plus what the scale's own rounding, 2^-9 of 15 scales, clips), then bf16
    for t in (1, 2, 3, 4, 9):
        g = xv[t].reshape(NKV, 2, 64)
        step = np.maximum((g.max(-1) - g.min(-1)) / 15, np.abs(g).max(-1) / 120) * (1 + 2.0 ** -8)
        assert (np.abs(vv[t].reshape(NKV, 2, 64) - g) <= 0.54 * step[..., None] + np.abs(g) * 2.0 ** -8).all()


def test_read_gives_the_held_values():
    s = Setup(5, 2, 3)
    x = s.rng.standard_normal((100, NKV, HD))
    val = [fill(s.pool_h, s.table[1], x, w) for w in (0, 1)]
    s.pool.copy_(dev(s.pool_h))
    seqs, pos = np.ones(100, np.int32), s.rng.permutation(100).astype(np.int32)
    seqs[7] = -1
    k, v = (torch.full((100, NKV, HD), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tb().tts_bb_kv4_read(s.cache, 100, dev(seqs), dev(pos), k, v, stream=stream())
    for y, w in ((k, val[0]), (v, val[1])):
        y = y.double().cpu().numpy()
        assert (y[7] == 9).all()
        live = np.arange(100) != 7
        assert np.array_equal(y[live], bf16_f64(w)[pos][live])
    assert np.array_equal(val[0][3, 2], decode(s.pool_h.reshape(-1, BLOCK), s.table[1, 0], 0, 2, 3))


def test_out_of_range_tokens_are_skipped_and_reported():
    s = Setup(6, 2, 2, n_pos=100)
    m = tb()
    x = dev(s.rng.standard_normal((5, 4096)).astype(np.float32))
    before = s.pool.clone()
    q = torch.full((5, NQ, HD), 3.0, device="cuda")
    for seqs, pos, bit in (([2, -1, -1, -1, -1], [0] * 5, m.KV4_ERR_RANGE), ([0, -1, -1, -1, -1], [100, 0, 0, 0, 0], m.KV4_ERR_RANGE),
                           ([1, -1, -1, -1, -1], [-1] * 5, m.KV4_ERR_RANGE), ([0, -1, -1, -1, -1], [2**31 - 1] * 5, m.KV4_ERR_RANGE)):
        s.err.zero_()
        assert s.append(x, seqs, pos, q) == 0
        assert int(s.err) == bit
        assert torch.equal(s.pool, before) and bool((q == 3).all())
    for page in (-1, s.n_blocks, 2**31 - 1):
        table = s.table.copy()
        table[0, 1] = page
        bad = m.Kv4Cache(s.pool, dev(table), s.err)
        keep, s.cache = s.cache, bad
        s.err.zero_()
        assert s.append(x, [0, -1, -1, -1, -1], [70] * 5, q) == 0
        assert int(s.err) == m.KV4_ERR_PAGE and torch.equal(s.pool, before)
        k = torch.full((1, NKV, HD), 3.0, dtype=torch.bfloat16, device="cuda")
        v = k.clone()
        s.err.zero_()
        m.tts_bb_kv4_read(bad, 1, dev(np.zeros(1, np.int32)), dev(np.array([70], np.int32)), k, v, stream=stream())
        assert int(s.err) == m.KV4_ERR_PAGE and bool((k == 3).all()) and bool((v == 3).all())
        s.cache = keep


def filled(seed, lens, bps, sharp=1.0, spare=3):
    """A cache holding len[b] random tokens for each row, NaN parameters everywhere else."""
    s = Setup(seed, len(lens), bps, spare=spare)
    s.k, s.v = [], []
    for b, n in enumerate(lens):
        s.k.append(fill(s.pool_h, s.table[b], sharp * s.rng.standard_normal((n, NKV, HD)), 0))
        s.v.append(fill(s.pool_h, s.table[b], s.rng.standard_normal((n, NKV, HD)) + 0.5 * s.rng.standard_normal((1, NKV, HD)), 1))
    s.pool.copy_(dev(s.pool_h))
    return s


def attend(s, q, lens, S, max_len, rows=None, out=None, ws=None):
    m = tb()
    B = len(lens)
    out = torch.full_like(q, 5.0) if out is None else out
    n = m.tts_bb_kv4_attention_workspace(B, S, max_len)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
    rows = None if rows is None else dev(np.asarray(rows, np.int32))
    assert m.tts_bb_kv4_attention(s.cache, B, S, q, dev(np.asarray(lens, np.int32)), max_len, out, ws if n else None, rows, stream=stream()) == 0
    return out


def check(s, q, lens, S, out, rows=None):
    bf = out.dtype == torch.bfloat16
    qh, got = q.double().cpu().numpy(), out.double().cpu().numpy()
    for b, n in enumerate(lens):
        row = b if rows is None else rows[b]
        for i in range(S):
            if row < 0:
                assert (got[b * S + i] == 5).all()
                continue
            seen = max(0, n - (S - 1 - i))
            want, mag, dots = attention(qh[b * S + i], s.k[row], s.v[row], seen)
            off = np.abs(got[b * S + i] - want)
            assert (off <= attention_tol(want, mag, dots, seen, bf)).all(), (b, i, n, off.max())


CASES = [([1], 1, 1.0), ([0, 1, 2, 15, 16, 17], 1, 1.0), ([63, 64, 65, 127, 128, 129], 1, 1.0), ([333], 1, 1.0), ([200, 777, 31], 1, 1.0),
         ([0, 1, 2, 3, 70], 3, 1.0), ([5, 130, 64], 8, 1.0), ([66, 10], 64, 1.0), ([900, 411], 2, 6.0)]


@pytest.mark.parametrize("io", ["float32", "bfloat16"])
@pytest.mark.parametrize("lens,S,sharp", CASES)
def test_attention_against_64_bits(lens, S, sharp, io):
    """Lengths around the tile and block sizes, empty rows, chunks longer than their cache, sharp softmaxes; what lies
    behind the keys is NaN, and the outputs of the next rows stay as they were."""
    s = filled(len(lens) * 100 + S, lens, (max(lens) + 70) // BLK + 1, sharp)
    q = dev(1.5 * s.rng.standard_normal((len(lens) * S, NQ, HD))).to(getattr(torch, io))
    out = torch.full((len(lens) * S + 1, NQ, HD), 5.0, dtype=q.dtype, device="cuda")
    attend(s, q, lens, S, max(max(lens), 1), out=out)
    check(s, q, lens, S, out)
    assert bool((out[-1] == 5).all()) and int(s.err) == 0
    loose = attend(s, q, lens, S, s.table.shape[1] * BLK)  # another split, the same values to the same bound
    check(s, q, lens, S, loose)
    assert torch.equal(loose, attend(s, q, lens, S, s.table.shape[1] * BLK))


@pytest.mark.parametrize("io", ["float32", "bfloat16"])
@pytest.mark.parametrize("lens,S,bps,max_len", [([700, 0, 65, 300], 1, 260, 16640), ([0, 130, 0, 2, 515, 0], 3, 260, 16640), ([20000, 9001], 1, 313, 20000),
                                                ([1], 1, 300, 19200), ([0, 0], 2, 300, 19200), ([40] * 70, 1, 40, 2560), ([90, 5], 64, 130, 8320),
                                                ([5000, 2100], 1, 90, 5760), ([10000, 33, 9000], 1, 160, 10240), ([2100], 2, 34, 2176), ([30000], 1, 470, 30080)])
def test_attention_dealt_over_all_blocks(lens, S, bps, max_len, io):
    """Long bounds, where the keys of all rows are dealt evenly to the launch: rows in several shares, several rows in one,
    rows that see nothing, and shares that get nothing."""
    s = filled(sum(lens) + S, lens, bps)
    q = dev(1.5 * s.rng.standard_normal((len(lens) * S, NQ, HD))).to(getattr(torch, io))
    out = attend(s, q, lens, S, max_len)
    check(s, q, lens, S, out)
    assert torch.equal(out, attend(s, q, lens, S, max_len)) and int(s.err) == 0
    rows = list(range(len(lens)))[::-1]
    rows[0] = -1
    check(s, q, lens[::-1], S, attend(s, q, lens[::-1], S, max_len, rows), rows)
    if len(lens) > 1:
        s.err.zero_()
        bad = list(lens)
        bad[1] = max_len + 1
        out = attend(s, q, bad, S, max_len)
        assert int(s.err) == tb().KV4_ERR_RANGE and bool((out.view(len(lens), -1)[1] == 5).all())
        check(s, q[:S], lens[:1], S, out[:S])


@pytest.mark.parametrize("B", [24, 40])
def test_attention_of_very_many_rows(B):
    """More rows than a block's threads in the even deal, and more than it sums over: one block each, at any length."""
    lens = [70] * B
    s = filled(21, lens, 130)
    q = dev(s.rng.standard_normal((B * 64, NQ, HD))).bfloat16()
    out = attend(s, q, lens, 64, 8320)
    check(s, q, lens, 64, out)


def test_attention_rows_and_padding():
    lens = [40, 300, 7]
    s = filled(11, lens, 6)
    q = dev(s.rng.standard_normal((4, NQ, HD)).astype(np.float32))
    rows = [2, -1, 1, 1]  # a row may be read twice
    out = attend(s, q, [7, 50, 300, 123], 1, 300, rows)
    check(s, q, [7, 50, 300, 123], 1, out, rows)


def test_attention_out_of_range():
    """Rows and key counts out of range leave their output; keys behind a bad page stay out of the sums."""
    m = tb()
    lens = [200, 100]
    s = filled(12, lens, 4)
    q = dev(s.rng.standard_normal((2, NQ, HD)).astype(np.float32))
    for rows, kl in (([0, 2], [200, 100]), ([0, 1], [200, 201]), ([0, 1], [200, -1]), ([0, 2**31 - 1], [200, 100])):
        s.err.zero_()
        out = attend(s, q, kl, 1, 200, rows)
        assert int(s.err) == m.KV4_ERR_RANGE and bool((out[1] == 5).all())
        check(s, q, kl[:1], 1, out[:1], rows[:1])
    for page in (-1, s.n_blocks):
        table = s.table.copy()
        table[0, 1] = page
        keep, s.cache = s.cache, m.Kv4Cache(s.pool, dev(table), s.err)
        s.err.zero_()
        out = attend(s, q, lens, 1, 200)
        assert int(s.err) == m.KV4_ERR_PAGE
        s.cache = keep
        k, v = (np.delete(a, np.s_[64:128], 0) for a in (s.k[0], s.v[0]))
        want, mag, dots = attention(q[0].double().cpu().numpy(), k, v, len(k))
        assert (np.abs(out[0].double().cpu().numpy() - want) <= attention_tol(want, mag, dots, len(k), False)).all()
        check(s, q[1:], lens[1:], 1, out[1:], [1])
        table[:] = page  # nothing at all is left: zeros
        s.cache = m.Kv4Cache(s.pool, dev(table), s.err)
        assert bool((attend(s, q, lens, 1, 200) == 0).all())
        s.cache = keep


def test_attention_nan_in_a_seen_key_reaches_the_output():
    """A value that is not finite is not hidden: its group's outputs are NaN, and a NaN key makes the row NaN."""
    s = filled(13, [90, 90], 2)
    tiles = s.pool_h.reshape(-1, 2, NKV, 4608)
    tiles[s.table[0, 1], 1, 2, 4096 + 8 * 5 : 4096 + 8 * 5 + 2] = (0xC0, 0x7F)  # the scale of V, head 2, group 0, key 69
    tiles[s.table[1, 0], 0, 3, 4096 + 8 * 9 + 4 : 4096 + 8 * 9 + 6] = (0xC0, 0x7F)  # of K, head 3, key 9
    s.pool.copy_(dev(s.pool_h))
    q = dev(s.rng.standard_normal((2, NQ, HD)).astype(np.float32))
    out = attend(s, q, [90, 90], 1, 128).cpu().numpy()
    nan = np.isnan(out)
    want = np.zeros_like(nan)
    want[0, 4:6, :64] = True
    want[1, 6:8] = True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("io", ["float32", "bfloat16"])
@pytest.mark.parametrize("S,max_len", [(2, 128), (3, 128), (2, 16640), (5, 16640)])
def test_attention_nan_in_a_later_key_stays_with_the_later_queries(S, max_len, io):
    """The last query's own key is NaN, and its value: the queries before it do not see either; nor do queries that are not
    finite reach one another."""
    lens = [90, 65, 49]
    s = filled(14, lens, 260)
    tiles = s.pool_h.reshape(-1, 2, NKV, 4608)
    for b, which in ((0, 0), (1, 1)):
        n = lens[b] - 1
        tiles[s.table[b, n // BLK], which, :, 4096 + 8 * (n % BLK) : 4104 + 8 * (n % BLK)] = (0xC0, 0x7F, 0x00, 0xC3) * 2
    s.pool.copy_(dev(s.pool_h))
    q = dev(s.rng.standard_normal((3 * S, NQ, HD))).to(getattr(torch, io))
    q[3 * S - 1, 5, 77] = float("inf")
    q[2 * S, 4, 3] = float("nan")
    out = attend(s, q, lens, S, max_len)
    nan = out.isnan().view(3, S, NQ, HD).cpu().numpy()
    want = np.zeros_like(nan)
    want[:2, S - 1] = True
    want[2, S - 1, 5] = want[2, 0, 4] = True
    assert np.array_equal(nan, want)
    s.v[1][lens[1] - 1] = s.k[0][lens[0] - 1] = 0.0
    out.view(3, S, NQ, HD)[:2, S - 1] = 0.0
    got, qh = out.view(3, S, NQ, HD).double().cpu().numpy(), q.view(3, S, NQ, HD).double().cpu().numpy()
    for b in range(2):
        for i in range(S - 1):
            seen = lens[b] - (S - 1 - i)
            ref, mag, dots = attention(qh[b, i], s.k[b], s.v[b], seen)
            assert (np.abs(got[b, i] - ref) <= attention_tol(ref, mag, dots, seen, io == "bfloat16")).all()


def test_attention_matches_the_bf16_entry_point():
    """The same values in a bf16 pool through tts_bb_gqa_decode_attention_static."""
    m = tb()
    lens = [150, 64, 321]
    s = filled(14, lens, 6)
    q = dev(s.rng.standard_normal((3, NQ, HD))).bfloat16()
    out = attend(s, q, lens, 1, 321)
    pool = torch.zeros(s.n_blocks, 2, NKV, BLK, HD, dtype=torch.bfloat16, device="cuda")
    for b, n in enumerate(lens):
        k, v = (torch.zeros(n, NKV, HD, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        m.tts_bb_kv4_read(s.cache, n, dev(np.full(n, b, np.int32)), dev(np.arange(n, dtype=np.int32)), k, v, stream=stream())
        for j in range(-(-n // BLK)):
            z = min(n, j * BLK + BLK)
            pool[int(s.table[b, j]), 0, :, : z - j * BLK] = k[j * BLK : z].transpose(0, 1)
            pool[int(s.table[b, j]), 1, :, : z - j * BLK] = v[j * BLK : z].transpose(0, 1)
    ref = torch.empty_like(q)
    pos = dev(np.asarray(lens, np.int32) - 1)
    assert m.tts_bb_gqa_decode_attention_static(q, pool, s.cache.page_table, 6, pos, 3, 320, ref, stream()) == 0
    # K and V rounded to bf16: scores move by 2^-9 sum |q k| / sqrt(128) (about 0.02 here), values by 2^-9; outputs twice rounded
    assert float((out.float() - ref.float()).abs().max()) <= 0.08 * float(ref.float().abs().max())


def test_attention_on_two_streams_and_in_graphs():
    """Calls that overlap with workspaces of their own, and a captured step replayed on new lengths and queries."""
    m = tb()
    lens = [700, 65, 300]
    s = filled(15, lens, 12)
    q = [dev(s.rng.standard_normal((3, NQ, HD)).astype(np.float32)) for _ in range(2)]
    want = [attend(s, x, lens, 1, 700) for x in q]
    torch.cuda.synchronize()
    n = m.tts_bb_kv4_attention_workspace(3, 1, 700)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q[0]) for _ in range(2)]
    ws = [torch.empty(max(n, 1), dtype=torch.uint8, device="cuda") for _ in range(2)]
    kl = dev(np.asarray(lens, np.int32))
    torch.cuda.synchronize()
    for _ in range(20):
        for x, o, w, st in zip(q, outs, ws, streams):
            m.tts_bb_kv4_attention(s.cache, 3, 1, x, kl, 700, o, w, stream=st.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x, o, w = q[0].clone(), outs[0], ws[0]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            m.tts_bb_kv4_attention(s.cache, 3, 1, x, kl, 700, o, w, stream=torch.cuda.current_stream().cuda_stream)
    for new in ([700, 65, 300], [1, 0, 17], [64, 64, 299]):
        kl.copy_(dev(np.asarray(new, np.int32)))
        x.copy_(q[1])
        g.replay()
        torch.cuda.synchronize()
        check(s, q[1], new, 1, o)


def test_offsets_past_two_gib():
    """A sequence whose blocks lie behind the first 2^31 (and 2^32) bytes of the pool."""
    m = tb()
    n_blocks = 2**32 // BLOCK + 40
    s = Setup(16, 1, 3)
    pool = torch.zeros(n_blocks, BLOCK, dtype=torch.uint8, device="cuda")
    table = np.array([[2**31 // BLOCK + 5, n_blocks - 1, 2**32 // BLOCK + 1]], np.int32)
    s.cache, s.table = m.Kv4Cache(pool, dev(table), s.err), table
    x = s.rng.standard_normal((150, 4096)).astype(np.float32)
    q = torch.zeros(150, NQ, HD, device="cuda")
    s.append(dev(x), [0] * 150, np.arange(150), q)
    seen = pool[table[0].tolist()].cpu().numpy()
    s.pool_h = np.zeros((3, 2, NKV, 4608), np.uint8)
    s.table = np.array([[0, 1, 2]], np.int32)
    want, _ = s.expect(x.astype(np.float64), [0] * 150, np.arange(150))
    same_pool(seen, want)
    flat = want.reshape(3, BLOCK)
    s.k = [np.array([[decode(flat, p // BLK, 0, h, p % BLK) for h in range(NKV)] for p in range(150)])]
    s.v = [np.array([[decode(flat, p // BLK, 1, h, p % BLK) for h in range(NKV)] for p in range(150)])]
    check(s, q[149:], [150], 1, attend(s, q[149:], [150], 1, 150))
    assert int(s.err) == 0


@pytest.mark.parametrize("S,n", [(1, 48), (2, 49)])
def test_bf16_attention_has_no_bias(S, n):
    """Outputs of values above zero that round to another bf16 number than the exact ones do so upward as often as downward: weights
    that are all taken too low would move them all downward."""
    B = 64
    s = Setup(7, B, 1)
    s.k, s.v = [], []
    for b in range(B):
        s.k.append(fill(s.pool_h, s.table[b], s.rng.standard_normal((n, NKV, HD)), 0))
        s.v.append(fill(s.pool_h, s.table[b], np.abs(s.rng.standard_normal((n, NKV, HD))) + 0.5, 1))
    s.pool.copy_(dev(s.pool_h))
    q = dev(1.5 * s.rng.standard_normal((B * S, NQ, HD))).bfloat16()
    got = attend(s, q, [n] * B, S, n).double().cpu().numpy().reshape(B, S, NQ, HD)
    qh = q.double().cpu().numpy().reshape(B, S, NQ, HD)
    want = bf16_f64([[attention(qh[b, i], s.k[b], s.v[b], n - (S - 1 - i))[0] for i in range(S)] for b in range(B)])
    low, high = int((got < want).sum()), int((got > want).sum())
    # six deviations of a fair coin's difference; and fp32 sums by truncation, at most 4 steps of 2^-23, move 2^-21 of the
    # outputs' 2^-8 steps
    assert abs(low - high) <= 6 * np.sqrt(low + high) + got.size * 2.0 ** -13, (low, high)


@pytest.mark.parametrize("io", ["float32", "bfloat16"])
@pytest.mark.parametrize("S,max_len", [(1, 70), (2, 70), (1, 1000), (1, 16640), (2, 16640)])
def test_attention_of_very_low_scores(S, max_len, io):
    """Scores around -1e32, all of them: the largest one's key has the whole weight."""
    s = Setup(8, 2, 260)
    lens = [70, 66]
    s.k, s.v = [], []
    for b, n in enumerate(lens):
        k = 1e15 * (1 + 0.1 * s.rng.standard_normal((n, NKV, HD)))
        k[11 + b] *= 0.5
        s.k.append(fill(s.pool_h, s.table[b], k, 0))
        s.v.append(fill(s.pool_h, s.table[b], s.rng.standard_normal((n, NKV, HD)), 1))
    s.pool.copy_(dev(s.pool_h))
    q = dev(-1e16 * (1 + 0.1 * s.rng.standard_normal((2 * S, NQ, HD)))).to(getattr(torch, io))
    out = attend(s, q, lens, S, max_len).double().cpu().numpy()
    for b in range(2):
        want = s.v[b][11 + b].repeat(2, 0)
        for i in range(S):
            assert (np.abs(out[b * S + i] - want) <= np.abs(want) * (2.0 ** -8 if io == "bfloat16" else 4 * U)).all()


def queries_ok(got, q, rows, bf16):
    """As in test_append_writes_the_definitions_bytes: 16 U of the pair's |x cos| + |x' sin|, then one rounding of the type."""
    pair = np.sqrt(q[..., :64] ** 2 + q[..., 64:] ** 2)
    tol = 16 * U * np.sqrt(2) * np.concatenate((pair, pair), -1) + (np.abs(q) * 2.0 ** -8 if bf16 else 0)
    return (np.abs(got - q) <= tol)[rows].all()


@pytest.mark.parametrize("io", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,q_io", [(1900, "float32"), (1900, "bfloat16"), (4099, "float32"), (4099, "bfloat16"), (4099, None)])
def test_append_of_prompts(T, q_io, io):
    """More tokens than blocks, so that a block goes on with further ones, and enough of fp32 for two launches; padding before, among and
    behind the tokens, one token out of range among them, queries of either type or none."""
    s = Setup(T, 3, 24)
    x = s.rng.standard_normal((T, 4096)) * np.exp(0.6 * s.rng.standard_normal((1, 4096))) + 0.3 * s.rng.standard_normal((1, 4096))
    xd = dev(x).to(getattr(torch, io))
    x = xd.double().cpu().numpy()
    cells = s.rng.permutation(3 * 24 * BLK)[:T]
    seqs, pos = (cells // (24 * BLK)).astype(np.int32), (cells % (24 * BLK)).astype(np.int32)
    seqs[s.rng.random(T) < 0.2] = -1
    seqs[[0, 912, 1023, T - 1]] = -1
    seqs[1024] = 3
    q_out = None if q_io is None else torch.full((T + 1, NQ, HD), 7.0, dtype=getattr(torch, q_io), device="cuda")
    assert s.append(xd, seqs, pos, q_out) == 0
    assert int(s.err) == tb().KV4_ERR_RANGE
    seqs[1024] = -1
    pool, q = s.expect(x, seqs, pos)
    same_pool(s.pool.cpu().numpy(), pool)
    if q_out is not None:
        got, live = q_out.double().cpu().numpy(), seqs >= 0
        assert (got[:T][~live] == 7).all() and (got[T] == 7).all()
        assert queries_ok(got[:T], q, live, q_io == "bfloat16")


@pytest.mark.parametrize("io,q_io", [("float32", "bfloat16"), ("bfloat16", "float32")])
def test_append_with_queries_of_the_other_type(io, q_io):
    s = Setup(31, 2, 2)
    xd = dev(s.rng.standard_normal((50, 4096))).to(getattr(torch, io))
    seqs, pos = np.repeat([0, 1], 25).astype(np.int32), np.tile(np.arange(25), 2).astype(np.int32) * 5
    q_out = torch.zeros(50, NQ, HD, dtype=getattr(torch, q_io), device="cuda")
    assert s.append(xd, seqs, pos, q_out) == 0
    pool, q = s.expect(xd.double().cpu().numpy(), seqs, pos)
    same_pool(s.pool.cpu().numpy(), pool)
    assert queries_ok(q_out.double().cpu().numpy(), q, np.arange(50), q_io == "bfloat16")


def test_append_of_rows_far_apart():
    """Rows of QKV more than 2^32 bytes from one another."""
    s = Setup(32, 1, 1)
    far = 2**29 + 8
    xd = torch.empty(2 * far + 4096, dtype=torch.float32, device="cuda").as_strided((3, 4096), (far, 1))
    xd.copy_(dev(s.rng.standard_normal((3, 4096)).astype(np.float32)))
    assert s.append(xd, [0] * 3, np.arange(3)) == 0
    same_pool(s.pool.cpu().numpy(), s.expect(xd.double().cpu().numpy(), [0] * 3, np.arange(3))[0])


def test_read_of_prompts():
    """Enough tokens for four a thread, with a remainder of three, padding and a row out of range among them."""
    T, n = 4867, 300
    s = Setup(9, 1, 5)
    val = [fill(s.pool_h, s.table[0], s.rng.standard_normal((n, NKV, HD)), w) for w in (0, 1)]
    s.pool.copy_(dev(s.pool_h))
    seqs, pos = np.zeros(T, np.int32), s.rng.integers(0, n, T).astype(np.int32)
    seqs[s.rng.random(T) < 0.2] = -1
    seqs[[T - 1, 17]] = 0, 1
    k, v = (torch.full((T + 4, NKV, HD), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert tb().tts_bb_kv4_read(s.cache, T, dev(seqs), dev(pos), k, v, stream=stream()) == 0
    assert int(s.err) == tb().KV4_ERR_RANGE
    live = seqs == 0
    for y, w in ((k, val[0]), (v, val[1])):
        y = y.double().cpu().numpy()
        assert (y[T:] == 9).all() and (y[:T][~live] == 9).all() and np.array_equal(y[:T][live], bf16_f64(w)[pos][live])


def test_attention_of_the_most_sequences():
    """As many query tokens as a call takes, over a few cache rows that many of them read."""
    B = 65535
    lens = [3, 70, 1]
    s = filled(33, lens, 2)
    rows = (np.arange(B) % 4 - 1).astype(np.int32)
    kl = np.array([0] + lens, np.int32)[rows + 1]
    q = torch.randn(B, NQ, HD, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16()
    out = attend(s, q, kl, 1, 70, rows)
    some = [0, 1, 2, 3, 30000, 30001, 30002, B - 3, B - 2, B - 1]
    check(s, q[some], kl[some], 1, out[some], rows[some])
    assert bool((out[::4] == 5).all()) and int(s.err) == 0


@pytest.mark.parametrize("io", ["float32", "bfloat16"])
@pytest.mark.parametrize("S,max_len", [(1, 200), (3, 200), (1, 16640)])
def test_attention_of_large_magnitudes(S, max_len, io):
    """Keys and values of 1e25, queries of 1e-25 (scores near 1), and small keys and values with large queries."""
    for big in (1e25, 1e-25):
        s = Setup(34, 2, 260)
        lens = [200, 67]
        s.k, s.v = ([fill(s.pool_h, s.table[b], big * s.rng.standard_normal((n, NKV, HD)), w) for b, n in enumerate(lens)] for w in (0, 1))
        s.pool.copy_(dev(s.pool_h))
        q = dev(s.rng.standard_normal((2 * S, NQ, HD)) / big).to(getattr(torch, io))
        check(s, q, lens, S, attend(s, q, lens, S, max_len))
