"""Plain 64-bit forms of the low-bit decode operators (numpy / CPU torch), shared by their tests."""
import numpy as np
import torch

NQ, NKV, HD, BLK = 16, 8, 128, 64
TILE, PAR, BLOCK = 4608, 4096, 73728
U = 2.0 ** -24  # half a step of fp32, relative


def bf16_f64(x):
    """float64 -> nearest bf16 (through float32, as every conversion here), as float64."""
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().double().numpy()


def rotated(x, gain, cos, sin, eps):
    """x [T][H][128] float64, gain [128], cos / sin [T][64]: RMSNorm with gain, then the pairs (i, i + 64) rotated."""
    x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * gain
    a, b = x[..., :64], x[..., 64:]
    c, s = cos[:, None], sin[:, None]
    return np.concatenate((a * c - b * s, b * c + a * s), -1)


def quantise(x):
    """x [..., 128] float64 -> codes [..., 128] uint8, scale and offset [..., 2] float64."""
    g = x.reshape(*x.shape[:-1], 2, 64)
    lo, hi = g.min(-1), g.max(-1)
    with np.errstate(invalid="ignore", over="ignore"):
        scale = bf16_f64(np.maximum((hi - lo) / 15, np.maximum(hi, -lo) / 120))
    bad = ~np.isfinite(g).all(-1)
    safe = np.where((scale > 0) & ~bad, scale, 1.0)
    zero = np.where((scale > 0) & ~bad, np.rint(np.where(bad, 0.0, lo) / safe), 0.0)
    code = np.clip(np.rint(np.where(bad[..., None], 0.0, g) / safe[..., None]) - zero[..., None], 0, 15)
    code = np.where((scale > 0)[..., None] & ~bad[..., None], code, 0.0)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, np.nan, scale), zero - 128


def code_bytes(code):
    """[..., 128] codes of a token's head -> its 64 bytes."""
    out = np.zeros((*code.shape[:-1], 64), np.uint8)
    for d in range(128):
        w, i = 2 * ((d % 64) // 8) + d // 64, d % 8
        out[..., 4 * w + i // 2] |= code[..., d] << (4 * (i % 2))
    return out


def par_bytes(scale, offset):
    """[..., 2] -> the 8 parameter bytes of a token's head."""
    p = torch.from_numpy(np.stack((scale, offset), -1).astype(np.float32)).bfloat16()
    return p.contiguous().view(torch.uint8).numpy().reshape(*scale.shape[:-1], 8)


def decode(pool, block, which, head, tok):
    """The 128 values held at one place of a pool (numpy uint8 [n][BLOCK])."""
    t = pool[block].reshape(2, NKV, TILE)[which, head]
    by, p = t[tok * 64 : tok * 64 + 64], t[PAR + tok * 8 : PAR + tok * 8 + 8].copy()
    p = torch.from_numpy(p).view(torch.bfloat16).double().numpy().reshape(2, 2)
    out = np.zeros(128)
    for d in range(128):
        w, i = 2 * ((d % 64) // 8) + d // 64, d % 8
        out[d] = p[d // 64, 0] * ((by[4 * w + i // 2] >> (4 * (i % 2)) & 15) + 128 + p[d // 64, 1])
    return out


def make_pool(rng, n_blocks, garbage=True):
    """A pool whose every byte is set: random codes, and parameters that are NaN where nothing is written later."""
    pool = rng.integers(0, 256, (n_blocks, 2, NKV, TILE), dtype=np.uint8)
    pool[..., PAR:] = 0xFF if garbage else 0  # bf16 0xFFFF: NaN
    return pool


def fill(pool, blocks, x, which):
    """Quantises x [n][8][128] into positions 0 .. n - 1 of a sequence whose cache blocks are `blocks`."""
    if not len(x):
        return x
    code, scale, off = quantise(x)
    by, par = code_bytes(code), par_bytes(scale, off)
    val = scale.repeat(64, -1) * (code + 128 + off.repeat(64, -1))
    for n in range(len(x)):
        t = pool[blocks[n // BLK], which]
        tok = n % BLK
        t[:, tok * 64 : tok * 64 + 64] = by[n]
        t[:, PAR + tok * 8 : PAR + tok * 8 + 8] = par[n]
    return val


def attention(q, k, v, seen):
    """q [16][128], k and v [n][8][128], the first `seen` keys -> out [16][128], and a bound of sum p |v|, max sum |q k|."""
    out, mag, dots = np.zeros((NQ, HD)), np.zeros((NQ, HD)), np.zeros(NQ)
    if seen <= 0:
        return out, mag, dots
    for h in range(NQ):
        kk, vv = k[:seen, h // 2], v[:seen, h // 2]
        z = kk @ q[h] / np.sqrt(HD)
        p = np.exp(z - z.max())
        p /= p.sum()
        out[h], mag[h] = p @ vv, p @ np.abs(vv)
        dots[h] = (np.abs(kk) @ np.abs(q[h])).max() / np.sqrt(HD)
    return out, mag, dots


def attention_tol(out, mag, dots, seen, bf16):
    """Bound of an fp32 kernel's error. A score: 128 products summed in fp32, (128 + 8) U of sum |q k| / sqrt(128);
    the exponential 2^-21; each weight is off by twice that relative to the sum of weights, and sums over the keys
    by (seen + 32) U of sum p |v|. bf16: weights as two truncated bf16 parts (2^-15), the result rounded once (2^-8... of
    the value at half a step 2^-9, doubled for a tie moved by the error)."""
    rel = 2 * (136 * U * dots + 2.0 ** -21) + (seen + 32) * U
    tol = mag * rel[:, None] + 1e-30
    return tol + mag * 2.0 ** -15 + np.abs(out) * 2.0 ** -8 if bf16 else tol


def unpack_w4(codes, scales, zeros, group):
    """uint8 [N][K / 2], [N][K / G] float, [N][K / G] or None -> float64 [N][K]."""
    N, half = codes.shape
    c = np.empty((N, 2 * half))
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    z = np.full(scales.shape, 8.0) if zeros is None else zeros.astype(np.float64)
    return (c - z.repeat(group, 1)) * scales.astype(np.float64).repeat(group, 1)


def logprobs(z, allowed, target, k):
    """One row in 64 bits: (logprob, entropy, lse, ids[k], top[k], log_s, m)."""
    z = np.asarray(z, np.float64).copy()
    if allowed is not None:
        z[~allowed] = -np.inf
    ids, top = np.full(k, -1), np.full(k, -np.inf)
    if np.isnan(z).any() or np.isposinf(z).any():
        return np.nan, np.nan, np.nan, ids, np.full(k, np.nan), 0.0, 0.0
    if not np.isfinite(z).any():
        return -np.inf, 0.0, -np.inf, ids, top, 0.0, 0.0
    m = z.max()
    i0 = int(np.argmax(z))
    rest = np.delete(z, i0)
    e = np.exp(rest - m)
    log_s = np.log1p(e.sum())
    d = np.where(np.isfinite(rest), rest - m, 0.0)
    ent = log_s - (e * d).sum() / (1 + e.sum())
    lp = (z[target] - m) - log_s if 0 <= target < len(z) else -np.inf
    order = np.argsort(-z, kind="stable")[:k]
    order = order[np.isfinite(z[order])]
    ids[: len(order)], top[: len(order)] = order, (z[order] - m) - log_s
    return lp, ent, m + log_s, ids, top, log_s, m
