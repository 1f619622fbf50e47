"""Products with 4-bit weights against their plain form in 64 bits."""
import numpy as np
import pytest

from tests.gpu_util import tb
from tests.lowbit_util import U, bf16_f64, unpack_w4

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def weights(rng, N, K, G, zeros):
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = bf16_f64(0.02 * np.exp(0.5 * rng.standard_normal((N, K // G))) * rng.choice([1, -1], (N, K // G)))
    z = rng.integers(0, 16, (N, K // G), dtype=np.uint8) if zeros else None
    return codes, scales, z


def pack(N, K, G, codes, scales, z):
    m = tb()
    n = m.tts_bb_w4_packed_bytes(N, K, G)
    p = torch.full((n + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    m.tts_bb_w4_pack(N, K, G, dev(codes), dev(scales).bfloat16(), None if z is None else dev(z), p,
                     torch.cuda.current_stream().cuda_stream)
    assert bool((p[n:] == 0xAB).all())
    return p[:n]


def run(N, K, G, T, io, zeros, seed=0, spread=1.0):
    m = tb()
    rng = np.random.default_rng(seed + N + K + T)
    codes, scales, z = weights(rng, N, K, G, zeros)
    packed = pack(N, K, G, codes, scales, z)
    dt = getattr(torch, io)
    pad = 8
    x = torch.full((T, K + pad), float("nan"), dtype=dt, device="cuda")[:, :K]  # rows further apart than they are long
    x.copy_(dev(rng.standard_normal((T, K)) * np.exp(spread * rng.standard_normal((T, K)))))
    y = torch.full((T * N + 16,), 7.0, dtype=dt, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    m.tts_bb_w4_linear(T, N, K, G, x, packed, y, st)
    assert bool((y[T * N :] == 7).all())
    w, xh = unpack_w4(codes, scales, z, G), x.double().cpu().numpy()
    want, mag = xh @ w.T, np.abs(xh) @ np.abs(w).T
    # exact products, K (+ parts, scales, warps) additions in fp32, each off by at most 2 U (an accumulator that
    # truncates) of the magnitudes; then one rounding of the type
    tol = 2 * (K + 16) * U * mag + (np.abs(want) * 2.0 ** -8 if io == "bfloat16" else 0) + 1e-37
    got = y[: T * N].reshape(T, N).double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol)
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel <= (2.0 ** -8 if io == "bfloat16" else 64 * U), rel
    again = torch.empty(T * N, dtype=dt, device="cuda")
    m.tts_bb_w4_linear(T, N, K, G, x, packed, again, st)
    assert torch.equal(again, y[: T * N])
    return w, xh


@pytest.mark.parametrize("io", ["float32", "bfloat16"])
@pytest.mark.parametrize("N,K,G,zeros", [(1, 32, 32, True), (16, 64, 64, False), (17, 96, 32, True), (33, 128, 128, True), (1025, 1024, 128, False),
                                         (100, 2080, 32, True), (48, 4160, 64, True), (31, 16384, 128, True)])
def test_single_token(N, K, G, zeros, io):
    run(N, K, G, 1, io, zeros)


@pytest.mark.parametrize("io", ["float32", "bfloat16"])
@pytest.mark.parametrize("T", [2, 3, 5, 7, 8, 9, 16, 17, 21, 22, 31, 32, 33, 42, 43, 63, 64])
def test_token_counts(T, io):
    run(39, 1152, (32, 64, 128)[T % 3], T, io, T % 2 == 0)


def test_values_of_every_code_and_zero():
    """One-hot rows read the weights out: every (code, zero) pair, exactly."""
    m = tb()
    N, K, G = 16, 64, 32
    codes = np.tile(np.arange(16, dtype=np.uint8), 2 * K // 32)[None].repeat(N, 0).reshape(N, K)
    packed_codes = codes[:, 0::2] | codes[:, 1::2] << 4
    scales = np.full((N, K // G), 0.5)
    z = np.arange(16, dtype=np.uint8)[:, None].repeat(K // G, 1)
    p = pack(N, K, G, packed_codes, scales, z)
    x = torch.eye(K, device="cuda")
    y = torch.empty(K, N, device="cuda")
    m.tts_bb_w4_linear(K, N, K, G, x, p, y, torch.cuda.current_stream().cuda_stream)
    assert np.array_equal(y.cpu().numpy(), unpack_w4(packed_codes, scales, z, G).T)


def test_extreme_values_of_x():
    """fp32 rows far from 1, where three truncated parts still hold all of x; infinities and NaN reach their row only."""
    m = tb()
    run(40, 256, 64, 2, "float32", True, spread=8.0)
    rng = np.random.default_rng(3)
    codes, scales, z = weights(rng, 20, 128, 64, True)
    p = pack(20, 128, 64, codes, scales, z)
    x = rng.standard_normal((4, 128)).astype(np.float32)
    x[1, 5], x[2, 70] = np.inf, np.nan
    x[3] *= 1e-40
    y = torch.empty(4, 20, device="cuda")
    m.tts_bb_w4_linear(4, 20, 128, 64, dev(x), p, y, torch.cuda.current_stream().cuda_stream)
    y = y.double().cpu().numpy()
    w = unpack_w4(codes, scales, z, 64)
    assert np.isfinite(y[[0, 3]]).all() and not np.isfinite(y[1:3]).any()
    assert np.allclose(y[0], x[0].astype(np.float64) @ w.T, atol=1e-4)


def test_two_streams_and_a_captured_graph():
    m = tb()
    rng = np.random.default_rng(9)
    N, K, G = 257, 1024, 128
    codes, scales, z = weights(rng, N, K, G, True)
    p = pack(N, K, G, codes, scales, z)
    xs = [dev(rng.standard_normal((3, K)).astype(np.float32)) for _ in range(2)]
    want = []
    for x in xs:
        y = torch.empty(3, N, device="cuda")
        m.tts_bb_w4_linear(3, N, K, G, x, p, y, torch.cuda.current_stream().cuda_stream)
        want.append(y)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in xs], [torch.empty(3, N, device="cuda") for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, y, st in zip(xs, outs, streams):
            m.tts_bb_w4_linear(3, N, K, G, x, p, y, st.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    side = torch.cuda.Stream()
    x, y = xs[0].clone(), outs[0]
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            m.tts_bb_w4_linear(3, N, K, G, x, p, y, torch.cuda.current_stream().cuda_stream)
    x.copy_(xs[1])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[1])


@pytest.mark.parametrize("io", ["float32", "bfloat16"])
@pytest.mark.parametrize("N,K,G,T", [(70, 8192, 128, 5), (33, 16384, 64, 9), (16, 4096, 32, 64), (17, 16384, 128, 40), (5000, 256, 64, 2), (9000, 64, 32, 1),
                                         (300, 4224, 128, 64), (40, 65536, 128, 3), (2100, 4096, 64, 33), (16, 262144, 128, 1), (17, 3168, 32, 64)])
def test_many_and_long_rows_of_x(N, K, G, T, io):
    """Rows of x in slices of a cluster's blocks, uneven ones too, and in chunks; more tiles than blocks."""
    run(N, K, G, T, io, True)


def test_pack_and_product_back_to_back():
    """The product right behind the packing on one stream, again and again on one buffer, sees the new weights."""
    m = tb()
    rng = np.random.default_rng(8)
    N, K, G = 2048, 512, 64
    st = torch.cuda.current_stream().cuda_stream
    sets = [weights(rng, N, K, G, True) for _ in range(4)]
    on = [(dev(c), dev(s).bfloat16(), dev(z)) for c, s, z in sets]
    x = dev(rng.standard_normal((1, K)).astype(np.float32))
    p = torch.empty(m.tts_bb_w4_packed_bytes(N, K, G), dtype=torch.uint8, device="cuda")
    ys = [torch.empty(1, N, device="cuda") for _ in sets]
    torch.cuda.synchronize()
    for (c, s, z), y in zip(on, ys):
        m.tts_bb_w4_pack(N, K, G, c, s, z, p, st)
        m.tts_bb_w4_linear(1, N, K, G, x, p, y, st)
    for (c, s, z), y in zip(sets, ys):
        w = unpack_w4(c, s, z, G)
        xh = x.double().cpu().numpy()
        assert (np.abs(y.double().cpu().numpy() - xh @ w.T) <= 2 * (K + 16) * U * (np.abs(xh) @ np.abs(w).T)).all()


@pytest.mark.parametrize("N,K,G,T", [(257, 4096, 128, 8), (1030, 2048, 64, 33)])
def test_slices_of_a_cluster_captured(N, K, G, T):
    """A call that splits K, captured as the first of its kind, and replayed beside another on a stream of its own."""
    m = tb()
    rng = np.random.default_rng(N)
    codes, scales, z = weights(rng, N, K, G, True)
    p = pack(N, K, G, codes, scales, z)
    xs = [dev(rng.standard_normal((T, K))).bfloat16() for _ in range(3)]
    x, y = xs[2].clone(), torch.zeros(T, N, device="cuda", dtype=torch.bfloat16)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        m.tts_bb_w4_linear(T, N, K, G, x, p, y, torch.cuda.current_stream().cuda_stream)
    want = []
    for v in xs:
        want.append(torch.empty(T, N, device="cuda", dtype=torch.bfloat16))
        m.tts_bb_w4_linear(T, N, K, G, v, p, want[-1], torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    other, out = torch.cuda.Stream(), torch.empty(T, N, device="cuda", dtype=torch.bfloat16)
    for v, w in zip(xs, want):
        x.copy_(v)
        torch.cuda.synchronize()
        for _ in range(10):
            with torch.cuda.stream(side):
                g.replay()
            m.tts_bb_w4_linear(T, N, K, G, xs[0], p, out, other.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(y, w) and torch.equal(out, want[0])


@pytest.mark.parametrize("N", [2**20, 2**20 - 15, 2**20 - 16])
def test_most_rows_of_weights(N):
    """The largest matrices that are not refused: more tiles of 16 rows than a grid's second dimension may have."""
    run(N, 32, 32, 1, "float32", True)


@pytest.mark.parametrize("io", ["float32", "bfloat16"])
@pytest.mark.parametrize("K,T", [(32, 32), (4096, 8)])
def test_tiny_rows_of_x(K, T, io):
    """Rows whose largest value lies near the least numbers of the type, subnormal ones too, keep their digits."""
    m = tb()
    rng = np.random.default_rng(K)
    N, G = 48, 32
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales, z = np.full((N, K // G), 2.0 ** 30), rng.integers(0, 16, (N, K // G), dtype=np.uint8)
    p = pack(N, K, G, codes, scales, z)
    w = unpack_w4(codes, scales, z, G)
    for top in (2.0 ** -100, 2.0 ** -104, 2.0 ** -113, 2.0 ** -114, 2.0 ** -120, 1.7e-38, 1e-40, 2.0 ** -149):
        x = torch.zeros(T, K, dtype=getattr(torch, io), device="cuda")
        x[torch.arange(T), torch.arange(T) * (K // T)] = dev(top * (1 + rng.random(T))).to(x.dtype)
        y = torch.empty(T, N, dtype=x.dtype, device="cuda")
        m.tts_bb_w4_linear(T, N, K, G, x, p, y, torch.cuda.current_stream().cuda_stream)
        want = x.double().cpu().numpy() @ w.T
        # one value a row: within one step (2 U), its two parts' products added (U); the scale is a power of two
        tol = (2.0 ** -8 + 6 * U if io == "bfloat16" else 6 * U) * np.abs(want)
        assert (np.abs(y.double().cpu().numpy() - want) <= tol).all(), top


def test_rows_of_x_far_apart():
    """Rows more than 2^32 bytes from one another."""
    m = tb()
    rng = np.random.default_rng(4)
    N, K, G, far = 40, 256, 64, 2**29 + 4
    codes, scales, z = weights(rng, N, K, G, True)
    p = pack(N, K, G, codes, scales, z)
    x = torch.empty(4 * far + K, dtype=torch.float32, device="cuda").as_strided((3, K), (2 * far, 1))
    x.copy_(dev(rng.standard_normal((3, K)).astype(np.float32)))
    y = torch.empty(3, N, device="cuda")
    m.tts_bb_w4_linear(3, N, K, G, x, p, y, torch.cuda.current_stream().cuda_stream)
    xh, w = x.double().cpu().numpy(), unpack_w4(codes, scales, z, G)
    assert (np.abs(y.double().cpu().numpy() - xh @ w.T) <= 2 * (K + 16) * U * (np.abs(xh) @ np.abs(w).T)).all()
