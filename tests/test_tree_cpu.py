"""Refusals of the speculative decoding operators, and their tests' plain forms: no GPU needed (every refusal returns before
the device is touched)."""
import ctypes as C

import numpy as np
import pytest

from tests.gpu_util import tb
from tests.test_lowbit_cpu import On, refused
from tests.tree_util import lineage, random_tree, tree_attention, verify, verify_greedy

P = 0x1000  # stands for a device address: never read


def cache(m, **kw):
    d = dict(pool=P, page_table=P, err=None, layer_stride=4 * 131072, n_layers=3, n_blocks=4, n_seqs=2, blocks_per_seq=2)
    d.update(kw)
    return C.byref(m.tts_bb_kv_cache(*d.values()))


def bad_caches(m):
    bad = [dict(pool=None), dict(page_table=None), dict(n_blocks=0), dict(n_blocks=2**20 + 1, layer_stride=2**60), dict(n_seqs=0), dict(blocks_per_seq=0),
           dict(pool=P + 8), dict(n_layers=0), dict(layer_stride=0), dict(layer_stride=4 * 131072 - 8), dict(layer_stride=4 * 131072 + 4),
           dict(layer_stride=-8), dict(page_table=P + 2), dict(err=P + 1)]
    return [None] + [cache(m, **b) for b in bad]


def test_attention_refuses():
    m = tb()
    need = max(m.tts_bb_tree_attention_workspace(2, 5, 128), 16)
    good = dict(cache=cache(m), layer=0, B=2, N=5, q=P, type=0, q_stride=2048, k=P, v=P, kv_stride=1024, parents=P, n_nodes=P, seqs=None, lens=P,
                max_len=128, out=P, ws=P, n=need, stream=None)
    refused(m.lib.tts_bb_tree_attention, good, dict(
        cache=bad_caches(m), layer=[-1, 3], B=[0, -1, 3, 2**31 - 1], N=[0, -1, 65], q=[None, P + 8], type=[-1, 2], q_stride=[0, 2047, 2050, -2048],
        k=[None, P + 8], v=[None, P + 2], kv_stride=[0, 1020, 1028, -1024], parents=[None, P + 1], n_nodes=[P + 2], seqs=[P + 3], lens=[None, P + 1],
        max_len=[-1, 129, 2**31 - 1], out=[None, P + 4]))
    refused(m.lib.tts_bb_tree_attention, {**good, "type": 1}, dict(q_stride=[2052]))
    assert m.lib.tts_bb_tree_attention(*{**good, "seqs": P, "B": 1024, "N": 64, "n": 2**62}.values()) == -1  # B * N = 65536
    # short sequences need no workspace, long ones do
    assert m.tts_bb_tree_attention_workspace(2, 5, 128) == 0
    need = m.tts_bb_tree_attention_workspace(2, 5, 6400)
    assert 0 < need < 2**25
    long = {**good, "cache": cache(m, blocks_per_seq=100), "max_len": 6400, "n": need}
    refused(m.lib.tts_bb_tree_attention, long, dict(ws=[None, P + 8], n=[need - 1, 0]))
    big = {**good, "cache": cache(m, blocks_per_seq=2**25), "seqs": P, "B": 9, "N": 1, "max_len": 2**30, "n": 2**62}
    assert m.lib.tts_bb_tree_attention(*big.values()) == -1 and m.tts_bb_tree_attention_workspace(9, 1, 2**30) == 0  # B * max_len above 2^33
    for args in ((0, 1, 1), (1, 0, 1), (1, 65, 1), (1, 1, -1), (1, 1, 2**30 + 1), (1024, 64, 64), (2**31 - 1, 64, 64)):
        assert m.tts_bb_tree_attention_workspace(*args) == 0


def test_verify_refuses():
    m = tb()
    good = dict(B=2, N=5, V=100, tokens=P, parents=P, n=P, target=P, ps=100, draft=P, qs=100, u=P, un=P, count=P, path=P, next=P, err=P, stream=None)
    off = [P + 1, P + 2, P + 3]
    refused(m.lib.tts_bb_tree_verify, good, dict(
        B=[0, -1, 13108], N=[0, 65, -1], V=[0, -1, 2**30 + 1], tokens=[None] + off, parents=[None] + off, n=off, target=[None] + off, ps=[99, 0, -100],
        draft=off, qs=[99, 0, -1], u=[None] + off, un=[None] + off, count=[None] + off, path=[None] + off, next=[None] + off, err=off))
    good = dict(B=2, N=5, tokens=P, parents=P, n=P, ids=P, count=P, path=P, next=P, err=P, stream=None)
    refused(m.lib.tts_bb_tree_verify_greedy, good, dict(
        B=[0, -1, 13108], N=[0, 65, -1], tokens=[None] + off, parents=[None] + off, n=off, ids=[None] + off, count=[None] + off, path=[None] + off,
        next=[None] + off, err=off))


def test_commit_refuses():
    m = tb()
    good = dict(cache=cache(m), B=2, N=5, k=P, v=P, rs=1024, ls=10240, path=P, count=P, seqs=None, lens=P, stream=None)
    refused(m.lib.tts_bb_tree_commit, good, dict(
        cache=bad_caches(m), B=[0, -1, 3, 65536], N=[0, 65], k=[None, P + 8], v=[None, P + 2], rs=[0, 1016, 1028, -1024], ls=[-8, 10244], path=[None, P + 1],
        count=[None, P + 2], seqs=[P + 3], lens=[None, P + 1]))


def test_wrappers_check_tensors(monkeypatch):
    """Types, devices, strides and sizes, and tensors of another device than the current one, whichever argument it is."""
    torch = pytest.importorskip("torch")
    m = tb()
    x = torch.zeros(2, 2048)
    with pytest.raises(TypeError):
        m.tts_bb_tree_attention(None, 0, 1, 2, x, x, x, x, x, 0, x.bfloat16())
    with pytest.raises(ValueError):
        m.KvCache(torch.zeros(131072, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32))
    monkeypatch.setattr(m, "_here", lambda: 1)
    calls = []
    monkeypatch.setattr(m, "lib", type("Lib", (), {"__getattr__": lambda self, name: lambda *a: calls.append((name, a)) or 0})())
    i32, u8, bf, f32 = torch.int32, torch.uint8, torch.bfloat16, torch.float32
    z = lambda *n, dt=f32: On(torch.zeros(*n, dtype=dt), 1)
    for n, layers in ((131072, 0), (131072, 2), (131073, 1)):
        with pytest.raises(ValueError):
            m.KvCache(z(n, dt=bf), z(1, 2, dt=i32), layers=layers)
    with pytest.raises(TypeError):
        m.KvCache(z(131072), z(1, 2, dt=i32))
    kv = m.KvCache(z(262144, dt=bf), z(1, 2, dt=i32), z(1, dt=i32), layers=2)
    assert (kv.struct.n_layers, kv.struct.n_blocks, kv.struct.layer_stride, kv.struct.n_seqs, kv.struct.blocks_per_seq) == (2, 1, 131072, 1, 2)
    here = {
        "tts_bb_tree_attention": dict(cache=kv, layer=1, B=1, N=2, q=z(2, 2048), k=z(2, 1024, dt=bf), v=z(2, 1024, dt=bf), parents=z(2, dt=i32), kv_lens=z(1, dt=i32),
                                      max_len=64, out=z(2, 2048), workspace=z(16, dt=u8), n_nodes=z(1, dt=i32), seqs=z(1, dt=i32)),
        "tts_bb_tree_verify": dict(B=1, N=2, V=5, tokens=z(2, dt=i32), parents=z(2, dt=i32), target=z(2, 5), u=z(2), u_next=z(1), n_accepted=z(1, dt=i32),
                                   path=z(2, dt=i32), next_token=z(1, dt=i32), draft=z(2, 6), n_nodes=z(1, dt=i32), err=z(1, dt=i32)),
        "tts_bb_tree_verify_greedy": dict(B=1, N=2, tokens=z(2, dt=i32), parents=z(2, dt=i32), target_ids=z(2, dt=i32), n_accepted=z(1, dt=i32), path=z(2, dt=i32),
                                          next_token=z(1, dt=i32), n_nodes=z(1, dt=i32), err=z(1, dt=i32)),
        "tts_bb_tree_commit": dict(cache=kv, B=1, N=2, k=z(2, 2, 1024, dt=bf), v=z(2, 2, 1024, dt=bf), path=z(2, dt=i32), n_accepted=z(1, dt=i32),
                                   kv_lens=z(1, dt=i32), seqs=z(1, dt=i32)),
    }
    for name, args in here.items():
        f = getattr(m, name)
        f(**args)
        assert calls and calls.pop()[0] == name
        for key, t in args.items():
            if isinstance(t, On):
                with pytest.raises(ValueError, match="current device"):
                    f(**{**args, key: On(t.t, 0)})
                small = t.t.reshape(-1)[:0]
                if key != "workspace":
                    with pytest.raises(ValueError):
                        f(**{**args, key: On(small, 1)})
                with pytest.raises(TypeError):
                    f(**{**args, key: On(t.t.double(), 1)})
        assert not calls
    # strided rows, and the strides that have to agree
    wide = lambda *shape: On(torch.zeros(*shape, 4096, dtype=bf)[..., 2048:][..., :1024], 1)
    a = here["tts_bb_tree_attention"]
    m.tts_bb_tree_attention(**{**a, "k": wide(2), "v": wide(2)})
    assert calls.pop()[1][9] == 4096
    with pytest.raises(ValueError, match="row stride"):
        m.tts_bb_tree_attention(**{**a, "k": wide(2)})
    c = here["tts_bb_tree_commit"]
    m.tts_bb_tree_commit(**{**c, "k": wide(2, 2), "v": wide(2, 2)})
    assert calls.pop()[1][5:7] == (4096, 8192)
    m.tts_bb_tree_commit(**c)
    assert calls.pop()[1][5:7] == (1024, 2048)
    with pytest.raises(ValueError, match="strides"):
        m.tts_bb_tree_commit(**{**c, "v": wide(2, 2)})
    monkeypatch.setattr(m, "_here", lambda: 0)
    for name in ("tts_bb_tree_attention", "tts_bb_tree_commit"):
        with pytest.raises(ValueError, match="current device"):
            getattr(m, name)(**{k: On(t.t, 0) if isinstance(t, On) else t for k, t in here[name].items()})
    assert not calls


def test_the_plain_forms():
    """The tests' own forms: what a node sees, the marginal of the verified tokens, and a planted mistake is seen."""
    rng = np.random.default_rng(0)
    parents = np.array([-1, 0, 0, 1, 3, -1], np.int32)
    assert lineage(parents, 4) == [4, 3, 1, 0] and lineage(parents, 5) == [5]
    q, k, v, tk, tv = (rng.standard_normal((n, h, 128)) for n, h in ((6, 16), (9, 8), (9, 8), (6, 8), (6, 8)))
    out, mag, _ = tree_attention(q, k, v, tk, tv, parents)
    tv2 = tv.copy()
    tv2[2] += 1  # no ancestor of the others
    other = tree_attention(q, k, v, tk, tv2, parents)[0]
    assert np.array_equal(np.delete(out, 2, 0), np.delete(other, 2, 0)) and not np.array_equal(out[2], other[2])
    assert (np.abs(out) <= mag + 1e-12).all()
    # root with three drawn children over 5 ids: the token behind the root is distributed as p, whatever q is
    p, d = rng.dirichlet(np.ones(5)), rng.dirichlet(np.ones(5))
    wrong, right, T = np.zeros(5), np.zeros(5), 20000
    par = np.array([-1, 0, 0, 0], np.int32)
    for _ in range(T):
        tok = np.concatenate(([0], rng.choice(5, 3, p=d)))
        pp, qq = np.tile(p, (4, 1)), np.tile(d, (4, 1))
        u, un = rng.random(4), rng.random()
        path, token, _ = verify(tok, par, pp, qq, u, un)
        right[tok[path[1]] if len(path) > 1 else token] += 1
        tok = np.concatenate(([0], rng.integers(0, 5, 3)))  # drawn from another distribution than q: biased
        path, token, _ = verify(tok, par, pp, qq, u, un)
        wrong[tok[path[1]] if len(path) > 1 else token] += 1
    sigma = np.sqrt(T * p * (1 - p))
    assert (np.abs(right - T * p) <= 5 * sigma).all() and (np.abs(wrong - T * p) > 5 * sigma).any()
    assert verify_greedy([9, 4, 4, 7], [-1, 0, 0, 2], [4, 7, 7, 1]) == ([0, 1], 7)
    assert random_tree(rng, 5).shape == (5,)
