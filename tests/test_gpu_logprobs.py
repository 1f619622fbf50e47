"""Log probabilities, entropy and top alternatives against their plain form in 64 bits."""
import numpy as np
import pytest

from tests.gpu_util import tb
from tests.lowbit_util import U, logprobs

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def words(ok):
    n = -(-len(ok) // 32) * 32
    b = np.zeros(n, np.uint64)
    b[: len(ok)] = ok
    return (b.reshape(-1, 32) << np.arange(32, dtype=np.uint64)).sum(1).astype(np.uint32).view(np.int32)


def call(z, V, targets, k, allowed=None):
    m = tb()
    R = len(z)
    o = {n: torch.full((R + 1,), 7.0, device="cuda") for n in ("logprob", "entropy", "lse")}
    ids = torch.full((R * k + 1,), 7, dtype=torch.int32, device="cuda")
    top = torch.full((R * k + 1,), 7.0, device="cuda")
    ws = torch.full((max(1, m.tts_bb_token_logprobs_workspace(R, V, k)),), 0xFF, dtype=torch.uint8, device="cuda")
    m.tts_bb_token_logprobs(R, V, z, None if targets is None else dev(np.asarray(targets, np.int32)), k,
                            None if targets is None else o["logprob"], o["entropy"], o["lse"], ids if k else None, top if k else None,
                            allowed, ws, stream=torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert all(float(x[R]) == 7 for x in o.values()) and int(ids[-1]) == 7 and float(top[-1]) == 7
    return [o[n][:R].double().cpu().numpy() for n in ("logprob", "entropy", "lse")] + [
        ids[:-1].reshape(R, k).cpu().numpy(), top[:-1].reshape(R, k).double().cpu().numpy()]


def near(got, want, tol):
    got, want = np.asarray(got), np.asarray(want)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    assert (np.abs(got - want)[fine] <= np.broadcast_to(tol, got.shape)[fine]).all(), (got, want, tol)


def check(z, V, targets, k, ok=None, allowed=None):
    """z: device tensor [R][>= V]; ok: bool [V] or [R][V]."""
    lp, ent, lse, ids, top = call(z, V, targets, k, allowed)
    zh = z.double().cpu().numpy()[:, :V]
    for r in range(len(zh)):
        okr = None if ok is None else ok if ok.ndim == 1 else ok[r]
        t = -1 if targets is None else targets[r]
        wlp, went, wlse, wids, wtop, log_s, mx = logprobs(zh[r], okr, t, k)
        # a difference z - m: U of it; an exponential: 2^-21 and U |z - m| of itself; a sum over V: (V / 32 + 64) U of it
        # (each adds V / (32 or more) terms in turn); the logarithm of 1 + r: 2^-22 of itself
        s_rel = (V / 32 + 64) * U + 2.0 ** -21
        fin = zh[r][np.isfinite(zh[r])] if okr is None else zh[r][okr & np.isfinite(zh[r])]
        d = np.sort(fin)[:-1] - mx if len(fin) and np.isfinite(wlse) else np.zeros(0)
        e = np.exp(d)
        r_err = (e * (s_rel + U * np.abs(d))).sum()
        t_err = (e * np.abs(d) * (s_rel + U * np.abs(d) + U)).sum()
        log_err = r_err / (1 + e.sum()) + log_s * 2.0 ** -22
        ent_err = log_err + (t_err + (e * np.abs(d)).sum() * r_err / (1 + e.sum())) / (1 + e.sum()) + 2 * U * (log_s + abs(went) if np.isfinite(went) else 0)
        if targets is not None:
            near(lp[r], wlp, log_err + 2 * U * (abs(wlp) + log_s if np.isfinite(wlp) else 0) + 1e-37)
        near(ent[r], went, ent_err + 1e-37)
        near(lse[r], wlse, log_err + 2 * U * (abs(mx) + log_s))
        assert np.array_equal(ids[r], wids), (r, ids[r], wids)
        with np.errstate(invalid="ignore"):
            near(top[r], wtop, log_err + 2 * U * np.where(np.isfinite(wtop), np.abs(wtop) + log_s, 0) + 1e-37)


TYPES = ["float32", "bfloat16", "float16"]
SIZES = [(1, 1, 1), (1, 2048, 5), (3, 2, 5), (5, 31, 32), (4, 32, 0), (7, 33, 3), (130, 1025, 5), (65, 1056, 20), (9, 4097, 32), (33, 3000, 1), (6, 20011, 20),
         (3, 70000, 32), (2, 151676, 20), (2, 600007, 5), (650, 200, 4), (700, 1025, 5), (620, 1900, 20), (610, 3001, 32), (612, 3105, 7), (609, 1025, 32), (610, 2048, 28), (612, 3000, 32), (620, 1088, 24), (3, 256, 32), (640, 97, 32), (640, 96, 30), (330, 24001, 32)]


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("R,V,k", SIZES)
def test_rows_against_64_bits(R, V, k, io):
    rng = np.random.default_rng(V + k)
    z = 3.0 * rng.standard_normal((R, V + 5)) + 8.0 * (rng.random((R, V + 5)) < 2 / V)
    zd = dev(z).to(getattr(torch, io))
    zd[:, V:] = float("nan")  # behind the row: not read into it
    check(zd[:, :V], V, rng.integers(0, V, R), k)
    check(zd[:, :V].contiguous(), V, rng.integers(0, V, R), k)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("R,V,k", [(4, 1025, 5), (3, 3001, 20), (2, 40000, 32), (5, 40, 32), (2, 23000, 20), (609, 1025, 5), (608, 2047, 3), (2, 500001, 4), (9, 1025, 20), (4, 520, 32), (3, 9000, 32), (620, 3300, 9), (611, 1025, 32), (608, 300, 32), (608, 2100, 29)])
def test_masked_places_do_not_count(R, V, k, io):
    """Masked NaN, infinities and the type's lowest value; one mask for all rows, and one a row; a row with nothing
    left, with one id left, and targets that are masked or out of range."""
    rng = np.random.default_rng(V)
    dt = getattr(torch, io)
    z = dev(3.0 * rng.standard_normal((R, V))).to(dt)
    for fill in (float("nan"), float("inf"), float("-inf"), torch.finfo(dt).min, torch.finfo(dt).max):
        ok = rng.random(V) < 0.6
        ok[3] = True
        y = z.clone()
        y[:, dev(~ok)] = fill
        targets = rng.integers(0, V, R)
        targets[0] = 3
        check(y, V, targets, k, ok, dev(words(ok)))
    ok = rng.random((R, V)) < 0.5
    ok[0] = False
    ok[1] = False
    ok[1, V // 2] = True
    targets = rng.integers(0, V, R)
    targets[1] = V // 2
    check(z, V, targets, k, ok, dev(np.stack([words(o) for o in ok])))
    check(z[:5], V, [-1, V, 2**31 - 1, -2**31, 0][:R], k)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("V,times", [(50, 1), (1025, 1), (3000, 1), (66000, 1), (420000, 1), (1025, 50), (2001, 44), (2900, 44)])
def test_ties_and_special_rows(V, times, io):
    dt = getattr(torch, io)
    rng = np.random.default_rng(V)
    rows = [np.zeros(V), np.where(np.arange(V) % 2, 0.0, -0.0), np.round(rng.standard_normal(V)), np.arange(V) * 2.0 ** -6, -np.arange(V) * 2.0 ** -6,
            np.full(V, -np.inf), np.where(np.arange(V) == V - 2, 1.5, -np.inf), np.where(np.arange(V) % 7, rng.standard_normal(V), -np.inf),
            np.full(V, float(torch.finfo(dt).min)), np.where(np.arange(V) == 9, 40.0, rng.standard_normal(V)), np.full(V, 60000.0),
            np.where(np.arange(V) == 4, np.nan, 0.0), np.where(np.arange(V) == V - 1, np.inf, 0.0), np.where(np.arange(V) < V // 2, 1.0, 2.0)]
    rows = rows * times
    z = dev(np.stack(rows)).to(dt)
    check(z, V, np.full(len(rows), 9), 32)
    check(z, V, np.full(len(rows), V - 2), 1)


def test_a_sure_row_keeps_its_digits():
    """log p of a token with all but 1e-9 of the probability, and its entropy, to a relative bound."""
    z = np.zeros((2, 2000))
    z[:, 77] = 28.0
    z[1] -= 5000.0
    zd = dev(z.astype(np.float32))
    lp, ent, _, _, _ = call(zd, 2000, [77, 77], 1)
    zh = zd.double().cpu().numpy()
    for r in range(2):
        wlp, went = logprobs(zh[r], None, 77, 1)[:2]
        assert abs(lp[r] - wlp) <= 1e-5 * abs(wlp) and abs(ent[r] - went) <= 1e-5 * went


def test_unwanted_outputs_may_be_absent():
    m = tb()
    z = dev(np.random.default_rng(0).standard_normal((4, 500)).astype(np.float32))
    full = call(z, 500, [1, 2, 3, 4], 3)
    e = torch.empty(4, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    n = m.tts_bb_token_logprobs_workspace(4, 500, 3)
    ws = torch.empty(max(1, n), dtype=torch.uint8, device="cuda")
    m.tts_bb_token_logprobs(4, 500, z, entropy=e, workspace=ws, stream=st)
    assert np.array_equal(e.double().cpu().numpy(), full[1])
    m.tts_bb_token_logprobs(4, 500, z, targets=dev(np.array([1, 2, 3, 4], np.int32)), logprob=e, workspace=ws, stream=st)
    assert np.array_equal(e.double().cpu().numpy(), full[0])


def test_two_streams_and_a_captured_graph():
    m = tb()
    rng = np.random.default_rng(5)
    R, V, k = 3, 100000, 20
    zs = [dev(rng.standard_normal((R, V)).astype(np.float32)) for _ in range(2)]
    n = max(1, m.tts_bb_token_logprobs_workspace(R, V, k))
    want = [call(z, V, [5] * R, k) for z in zs]
    t = dev(np.full(R, 5, np.int32))
    bufs = [(torch.empty(R, device="cuda"), torch.empty(R, k, dtype=torch.int32, device="cuda"), torch.empty(R, k, device="cuda"),
             torch.empty(n, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()) for _ in zs]
    torch.cuda.synchronize()
    for _ in range(10):
        for z, (lp, ids, top, ws, st) in zip(zs, bufs):
            m.tts_bb_token_logprobs(R, V, z, t, k, logprob=lp, top_ids=ids, top_logprobs=top, workspace=ws, stream=st.cuda_stream)
    torch.cuda.synchronize()
    for w, (lp, ids, top, _, _) in zip(want, bufs):
        assert np.array_equal(lp.double().cpu().numpy(), w[0]) and np.array_equal(ids.cpu().numpy(), w[3])
    lp, ids, top, ws, side = bufs[0]
    z = zs[0].clone()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            m.tts_bb_token_logprobs(R, V, z, t, k, logprob=lp, top_ids=ids, top_logprobs=top, workspace=ws,
                                    stream=torch.cuda.current_stream().cuda_stream)
    z.copy_(zs[1])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(lp.double().cpu().numpy(), want[1][0]) and np.array_equal(ids.cpu().numpy(), want[1][3])
    assert np.array_equal(top.double().cpu().numpy(), want[1][4])


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("R,V,k", [(1, 20000, 5), (3, 70000, 20), (2, 250001, 32), (305, 26000, 5), (2, 420000, 3)])
def test_lowest_values_that_are_not_masked(R, V, k, io):
    """Ids at the type's lowest value that no mask excludes: whole slices of a row of them, behind, before and around the others."""
    rng = np.random.default_rng(V)
    dt = getattr(torch, io)
    for others in (slice(0, V // 2), slice(V // 2, V), slice(V // 3, V // 3 + 3), slice(V - 1, V)):
        z = torch.full((R, V), torch.finfo(dt).min, dtype=dt, device="cuda")
        z[:, others] = dev(3.0 * rng.standard_normal((R, others.stop - others.start)) - 5.0).to(dt)
        targets = rng.integers(0, V, R)
        targets[0] = others.start
        check(z, V, targets, k)


@pytest.mark.parametrize("io", ["float32", "bfloat16"])
@pytest.mark.parametrize("R,V,k", [(6, 200, 20), (608, 200, 32), (609, 1025, 5), (608, 1900, 20), (610, 3001, 32), (6, 3001, 20), (6, 100, 8)])
def test_alternatives_of_very_low_logits(R, V, k, io):
    """Allowed ids around -1e30 (a common fill) are alternatives as long as they are finite; masked ones are not, whatever their logit."""
    rng = np.random.default_rng(V)
    dt = getattr(torch, io)
    z = torch.full((R, V), -1e30, dtype=dt, device="cuda")
    z[0::6, 7:10] = dev(rng.standard_normal((len(z[0::6]), 3))).to(dt)
    z[1::6] = dev(rng.uniform(-1e30, -9e29, (len(z[1::6]), V))).to(dt)
    z[2::6, ::2] = dev(rng.uniform(-1.1e30, -8e29, (len(z[2::6]), (V + 1) // 2))).to(dt)
    z[3::6, 5:] = -9.5e29
    z[4::6, V // 2] = 0.0
    z[5::6] = -9e29
    targets = rng.integers(0, V, R)
    check(z, V, targets, k)
    ok = rng.random(V) < 0.3
    ok[8] = True
    z[:, dev(~ok)] = 1.0
    check(z, V, targets, k, ok, dev(words(ok)))


@pytest.mark.parametrize("V,R", [(200, 3), (40000, 3), (420000, 2)])
def test_rows_far_apart(V, R):
    """Rows of logits and of masks more than 2^32 bytes from one another."""
    rng = np.random.default_rng(V)
    far, mask_far = 2**30 + 4, 2**30 + 3
    z = torch.empty((R - 1) * far + V, dtype=torch.float32, device="cuda").as_strided((R, V), (far, 1))
    z.copy_(dev(3.0 * rng.standard_normal((R, V)).astype(np.float32)))
    ok = rng.random((R, V)) < 0.7
    n = -(-V // 32)
    allowed = torch.empty((R - 1) * mask_far + n, dtype=torch.int32, device="cuda").as_strided((R, n), (mask_far, 1))
    allowed.copy_(dev(np.stack([words(o) for o in ok])))
    check(z, V, rng.integers(0, V, R), 7, ok, allowed)
