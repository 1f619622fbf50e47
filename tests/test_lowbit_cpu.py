"""Refusals of the low-bit decode operators and their host-side functions: no GPU needed (every refusal returns before
the device is touched)."""
import ctypes as C

import numpy as np
import pytest

from tests.gpu_util import tb
from tests.lowbit_util import bf16_f64, code_bytes, quantise

P = 0x1000  # stands for a device address: never read


def cache(m, **kw):
    d = dict(pool=P, page_table=P, err=None, n_blocks=4, n_seqs=2, blocks_per_seq=2)
    d.update(kw)
    return m.tts_bb_kv4(d["pool"], d["page_table"], d["err"], d["n_blocks"], d["n_seqs"], d["blocks_per_seq"])


BAD_CACHES = [dict(pool=None), dict(page_table=None), dict(n_blocks=0), dict(n_seqs=0), dict(blocks_per_seq=0), dict(pool=P + 8)]


def refused(f, good, bad):
    for name, values in bad.items():
        for v in values:
            args = dict(good)
            assert name in args
            args[name] = v
            assert f(*args.values()) == -1, (name, v)


def test_append_and_read_refuse():
    m = tb()
    good = dict(cache=C.byref(cache(m)), T=1, qkv=P, qkv_type=0, stride=4096, gq=P, gk=P, eps=1e-6, cos=P, sin=P, n_pos=1, seqs=P, pos=P, q=P, q_type=0,
                stream=None)
    bad_cache = [None] + [C.byref(cache(m, **b)) for b in BAD_CACHES]
    refused(m.lib.tts_bb_kv4_append, good, dict(
        cache=bad_cache, T=[0, -1], qkv=[None, P + 8], qkv_type=[-1, 2, 3], stride=[4095, 0, -4096, 4098], gq=[None, P + 4], gk=[None, P + 2],
        eps=[-1.0, float("nan")], cos=[None, P + 8], sin=[None, P + 4], n_pos=[0, -5], seqs=[None], pos=[None], q=[P + 8], q_type=[2, -1]))
    good = dict(cache=C.byref(cache(m)), T=1, seqs=P, pos=P, k=P, v=P, stream=None)
    refused(m.lib.tts_bb_kv4_read, good, dict(cache=bad_cache, T=[0], seqs=[None], pos=[None], k=[None, P + 4], v=[None, P + 2]))


def test_attention_refuses():
    m = tb()
    n = m.tts_bb_kv4_attention_workspace(2, 1, 128)
    good = dict(cache=C.byref(cache(m)), B=2, S=1, q=P, type=0, seqs=None, lens=P, max_len=128, out=P, ws=P, n=n, stream=None)
    bad = dict(cache=[None] + [C.byref(cache(m, **b)) for b in BAD_CACHES], B=[0, -1, 3, 65536], S=[0, m.KV4_MAX_QUERIES + 1], q=[None, P + 8],
               type=[-1, 2], lens=[None], max_len=[0, -1, 129, 2**31 - 1], out=[None, P + 4])
    if n:
        bad.update(ws=[None, P + 8], n=[n - 1, 0])
    refused(m.lib.tts_bb_kv4_attention, good, bad)
    good.update(seqs=P, B=1024, S=64, n=2**62)
    assert m.lib.tts_bb_kv4_attention(*good.values()) == -1  # B * S = 65536
    good = dict(cache=C.byref(cache(m, blocks_per_seq=2**25)), B=1, S=1, q=P, type=0, seqs=None, lens=P, max_len=2**30 + 1, out=P, ws=P, n=2**62, stream=None)
    assert m.lib.tts_bb_kv4_attention(*good.values()) == -1
    for args in ((0, 1, 1), (1, 0, 1), (1, 1, 2**30 + 1), (1, 65, 1), (1, 1, 0), (1024, 64, 64), (2**31 - 1, 64, 64)):
        assert m.tts_bb_kv4_attention_workspace(*args) == 0


def test_w4_refuses():
    m = tb()
    for args in ((0, 128, 128), (1, 0, 128), (1, 128, 16), (1, 128, 256), (1, 100, 32), (1, 64, 128), (2**20 + 1, 128, 128), (1, 2**20 + 128, 128), (1, 2**18 + 128, 128), (-1, 128, 64)):
        assert m.tts_bb_w4_packed_bytes(*args) == 0
        assert m.lib.tts_bb_w4_pack(*args, P, P, P, P, None) == -1
        assert m.lib.tts_bb_w4_linear(1, *args, P, 0, 2**21, P, P, None) == -1
    refused(m.lib.tts_bb_w4_pack, dict(N=16, K=128, G=64, codes=P, scales=P, zeros=None, packed=P, stream=None),
            dict(codes=[None], scales=[None, P + 1], packed=[None, P + 8]))
    refused(m.lib.tts_bb_w4_linear, dict(T=1, N=16, K=128, G=64, x=P, type=0, stride=128, packed=P, y=P, stream=None),
            dict(T=[0, -1, 65], x=[None, P + 4], type=[2, -1], stride=[127, 130, 0], packed=[None, P + 4], y=[None, P + 2]))
    refused(m.lib.tts_bb_w4_linear, dict(T=1, N=16, K=128, G=64, x=P, type=1, stride=128, packed=P, y=P, stream=None), dict(stride=[132], y=[P + 1]))


def test_logprobs_refuses():
    m = tb()
    good = dict(R=2, V=100, z=P, type=0, stride=100, targets=P, allowed=P, a_stride=4, k=2, lp=P, ent=None, lse=None, ids=P, top=P, ws=P, n=2**40, stream=None)
    refused(m.lib.tts_bb_token_logprobs, good, dict(R=[0, -1, 2**27 + 1], V=[0, -3, 2**30 + 1], z=[None, P + 2], type=[-1, 3], stride=[99, 0, -1], a_stride=[3, 1, -4], k=[-1, 33],
                                                    lp=[None], ids=[None], top=[None]))
    good.update(V=300000, stride=300000, a_stride=0, n=0)
    if m.tts_bb_token_logprobs_workspace(2, 300000, 2):
        assert m.lib.tts_bb_token_logprobs(*good.values()) == -1
        good.update(n=2**40, ws=None)
        assert m.lib.tts_bb_token_logprobs(*good.values()) == -1


def test_rope_tables():
    m = tb()
    for theta, n in ((1e6, 300), (1e4, 5)):
        c, s = m.tts_bb_rope_tables(theta, n)
        a = np.arange(n)[:, None] * theta ** (-2.0 * np.arange(64) / 128)
        # an angle in 64 bits is off by 2^-52 of itself or less; then half a step of fp32
        for got, want in ((c, np.cos(a)), (s, np.sin(a))):
            assert got.shape == (n, 64) and (np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 1e-12).all()
    buf = np.zeros(64, np.float32).ctypes.data
    for args in ((1e6, 0, buf, buf), (0.0, 1, buf, buf), (-1.0, 1, buf, buf), (float("nan"), 1, buf, buf), (1e6, 1, None, buf), (1e6, 1, buf, None)):
        assert m.lib.tts_bb_rope_tables(*args) == -1


def test_wrappers_check_tensors():
    """Types, devices, strides and sizes are refused before the library is called."""
    torch = pytest.importorskip("torch")
    m = tb()
    x = torch.zeros(2, 128)
    with pytest.raises(TypeError):
        m.tts_bb_w4_linear(2, 16, 128, 64, x, x, x)
    with pytest.raises(TypeError):
        m.tts_bb_w4_linear(2, 16, 128, 64, x, x, x.bfloat16())
    with pytest.raises(TypeError):
        m.Kv4Cache(x, torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        m.Kv4Cache(x, torch.zeros(1, dtype=torch.int32))


class On:
    """Stands for a tensor on another device than the current one."""

    def __init__(self, t, device):
        self.t, self.device, self.is_cuda, self.dtype = t, f"cuda:{device}", True, t.dtype
        self.get_device = lambda: device

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_wrappers_refuse_another_device(monkeypatch):
    """A tensor that is not on the current device is refused, whichever argument it is, and a cache made on another."""
    torch = pytest.importorskip("torch")
    m = tb()
    monkeypatch.setattr(m, "_here", lambda: 1)
    calls = []
    monkeypatch.setattr(m, "lib", type("Lib", (), {"__getattr__": lambda self, name: lambda *a: calls.append(name) or 0})())
    z = lambda n, dt=torch.float32: On(torch.zeros(n, dtype=dt), 1)
    i32, u8, bf = torch.int32, torch.uint8, torch.bfloat16
    cache = m.Kv4Cache(z(m.KV4_BLOCK_BYTES, u8), On(torch.zeros(1, 2, dtype=i32), 1), z(1, i32))
    here = {
        "tts_bb_kv4_append": dict(cache=cache, T=1, qkv=z(4096), q_norm=z(128, bf), k_norm=z(128, bf), cos_table=z(64), sin_table=z(64), n_pos=1,
                                  seqs=z(1, i32), positions=z(1, i32), q_out=z(2048)),
        "tts_bb_kv4_read": dict(cache=cache, T=1, seqs=z(1, i32), positions=z(1, i32), k_out=z(1024, bf), v_out=z(1024, bf)),
        "tts_bb_kv4_attention": dict(cache=cache, B=1, S=1, q=z(2048), kv_lens=z(1, i32), max_len=64, out=z(2048), workspace=z(16, u8), seqs=z(1, i32)),
        "tts_bb_w4_pack": dict(N=16, K=64, group=64, codes=z(512, u8), scales=z(16, bf), zeros=z(16, u8), packed=z(576, u8)),
        "tts_bb_w4_linear": dict(T=1, N=16, K=64, group=64, x=z(64), packed=z(576, u8), y=z(16)),
        "tts_bb_token_logprobs": dict(R=1, V=64, logits=z(64), targets=z(1, i32), n_top=1, logprob=z(1), entropy=z(1), lse=z(1), top_ids=z(1, i32),
                                      top_logprobs=z(1), allowed=z(2, i32), workspace=z(16, u8)),
    }
    monkeypatch.setattr(m, "tts_bb_w4_packed_bytes", lambda *a: 576)
    for name, args in here.items():
        f = getattr(m, name)
        f(**args)
        assert calls and calls.pop() == name
        for k, v in args.items():
            if isinstance(v, On):
                with pytest.raises(ValueError, match="current device"):
                    f(**{**args, k: On(v.t, 0)})
        assert not calls
    monkeypatch.setattr(m, "_here", lambda: 0)
    for name in ("tts_bb_kv4_append", "tts_bb_kv4_read", "tts_bb_kv4_attention"):
        with pytest.raises(ValueError, match="current device"):
            getattr(m, name)(**{k: On(v.t, 0) if isinstance(v, On) else v for k, v in here[name].items()})
    assert not calls


def test_the_plain_quantiser():
    """The tests' own quantiser: at most half a scale off (plus what the scale's rounding clips), its ends at codes 0
    and 15, and a planted mistake (the bits of a word in another order) is seen in the bytes."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 128)) * np.exp(rng.standard_normal((50, 1)))
    code, scale, off = quantise(x)
    val = scale.repeat(64, -1) * (code + 128 + off.repeat(64, -1))
    assert (np.abs(val - x) <= 0.54 * scale.repeat(64, -1)).all()
    g = code.reshape(50, 2, 64)
    assert (g.min(-1) == 0).all() and (g.max(-1) >= 14).all()
    assert np.array_equal(scale, bf16_f64(scale)) and np.array_equal(off, np.rint(off))
    swapped = code.copy()
    swapped[:, [0, 64]] = swapped[:, [64, 0]]
    assert not np.array_equal(code_bytes(code), code_bytes(swapped))


def test_misaligned_words_are_refused():
    """32-bit arrays off a 4-byte boundary, which a kernel would fault on."""
    m = tb()
    off = [P + 1, P + 2, P + 3]
    bad_cache = [C.byref(cache(m, **{k: v})) for k in ("page_table", "err") for v in off]
    refused(m.lib.tts_bb_kv4_append, dict(cache=C.byref(cache(m)), T=1, qkv=P, qkv_type=0, stride=4096, gq=P, gk=P, eps=1e-6, cos=P, sin=P, n_pos=1, seqs=P,
                                          pos=P, q=P, q_type=0, stream=None), dict(cache=bad_cache, seqs=off, pos=off))
    refused(m.lib.tts_bb_kv4_read, dict(cache=C.byref(cache(m)), T=1, seqs=P, pos=P, k=P, v=P, stream=None), dict(cache=bad_cache, seqs=off, pos=off))
    refused(m.lib.tts_bb_kv4_attention, dict(cache=C.byref(cache(m)), B=2, S=1, q=P, type=0, seqs=None, lens=P, max_len=128, out=P, ws=P, n=2**40, stream=None),
            dict(cache=bad_cache, seqs=off, lens=off))
    refused(m.lib.tts_bb_token_logprobs, dict(R=2, V=100, z=P, type=0, stride=100, targets=P, allowed=P, a_stride=4, k=2, lp=P, ent=P, lse=P, ids=P, top=P, ws=P,
                                              n=2**40, stream=None), {k: off for k in ("targets", "allowed", "lp", "ent", "lse", "ids", "top")})
