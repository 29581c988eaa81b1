"""Plain 64-bit implementation of the FP4 cache rows (E2M1 codes with a
power-of-two scale for every 32 values, in 320 bytes) for the tests: encoding
by search over the eight magnitudes, decoding bit by bit, appending, and the
attention of a query over given rows."""
import numpy as np

import oracle as O

ROW_BYTES, CODE_BYTES, BLOCKS = 320, 288, 18
MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def encode(x):
    """[n, 576] bf16 values (as float64) to rows uint8 [n, 320]."""
    x = np.asarray(x, np.float64)
    n = x.shape[0]
    out = np.zeros((n, ROW_BYTES), np.uint8)
    for r in range(n):
        words = np.zeros(72, np.uint64)
        for j in range(BLOCKS):
            block = x[r, 32 * j:32 * j + 32]
            if not np.all(np.isfinite(block)):
                out[r, CODE_BYTES + j] = 255
                continue
            top = np.abs(block).max()
            e = -127
            while top > 6 * 2.0 ** e:
                e += 1
            out[r, CODE_BYTES + j] = e + 127
            for i, v in enumerate(block):
                off = np.abs(abs(v) / 2.0 ** e - MAGNITUDES)
                best = np.flatnonzero(off == off.min())
                code = int(best[best % 2 == 0][0] if len(best) > 1 else best[0])
                w, k = divmod(32 * j + i, 8)
                words[w] |= np.uint64(code << (4 * k))
                if np.signbit(v):
                    words[w] |= np.uint64(1 << (8 * k + 7 if k < 4 else 8 * (k - 4) + 3))
        out[r, :CODE_BYTES] = words.astype("<u4").view(np.uint8)
    return out


def decode_rows(rows):
    """Rows uint8 [n, 320] to values [n, 576] in float64."""
    n = rows.shape[0]
    words = np.ascontiguousarray(rows[:, :CODE_BYTES]).view("<u4").astype(np.int64)
    out = np.zeros((n, 576))
    for k in range(8):
        mag = MAGNITUDES[(words >> (4 * k)) & 7]
        neg = (words >> (8 * k + 7 if k < 4 else 8 * (k - 4) + 3)) & 1
        out[:, k::8] = np.where(neg, -mag, mag)
    byte = rows[:, CODE_BYTES:CODE_BYTES + BLOCKS].astype(np.float64)
    scale = np.where(byte == 255, np.nan, 2.0 ** (byte - 127))
    return out * np.repeat(scale, 32, axis=1)


def through_e5m2(x):
    """Values as the decode reads them: rounded to E5M2 (multiples of 2^-16
    below 2^-14), saturated at 57,344."""
    a = np.abs(x)
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -14))) - 2)
    with np.errstate(invalid="ignore"):
        y = np.minimum(np.rint(a / step) * step, 57344.0)
    return np.where(np.isnan(x), np.nan, np.copysign(y, x))


def rotated(k_pe, positions, theta):
    """bf16 values (as float64) of RoPE keys [n, 64] at their positions: rounded to
    fp32 and then to bf16."""
    if not theta > 0:
        return np.asarray(k_pe, np.float64)
    x = O.rope_rotate(np.asarray(k_pe, np.float64), np.asarray(positions), theta).astype(np.float32)
    return O.bf16_bits_to_f64(O.f64_to_bf16_bits(x.astype(np.float64)))


def appended(cache, table, seq_ids, positions, c_kv, k_pe, theta, page):
    """A copy of cache uint8 [pages, P, 320] with the tokens' rows written."""
    cache = cache.copy()
    rows = encode(np.concatenate([c_kv, rotated(k_pe, positions, theta)], axis=1))
    for b, pos, row in zip(seq_ids, positions, rows):
        cache[table[b, pos // page], pos % page] = row
    return cache


def gathered(cache, table, b, length, page):
    """Values [length, 576] of a sequence's rows, as the decode reads them."""
    if length == 0:
        return np.zeros((0, 576))
    pos = np.arange(length)
    return through_e5m2(decode_rows(cache[table[b, pos // page], pos % page]))


def attend(q_nope, q_pe, rows, W_UK, W_UV, scale):
    """(out [H, 128], lse [H]) of one query token over rows [n, 576]."""
    H = q_nope.shape[0]
    out, lse = np.zeros((H, 128)), np.full(H, -np.inf)
    if len(rows):
        for h in range(H):
            s = scale * (rows[:, :512] @ (W_UK[h].T @ q_nope[h]) + rows[:, 512:] @ q_pe[h])
            m = s.max()
            p = np.exp(s - m)
            lse[h] = m + np.log(p.sum())
            out[h] = W_UV[h] @ ((p / p.sum()) @ rows[:, :512])
    return out, lse
