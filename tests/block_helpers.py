"""64-bit references of the calls on caches with block scales, written from
their definition in numpy: e4m3 codes by a table, scales by search."""
import numpy as np

D, TILE = 128, 16
LOW, HIGH = -50, 30
NAN = 0x7F


def _table():
    v = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if c & 127 == 127 else -x if c & 128 else x
    return v


VALUES = _table()
_MAGS = VALUES[:127]
_MIDS = (_MAGS[1:] + _MAGS[:-1]) / 2


def encode(x):
    """e4m3 codes of float64 values: nearest, ties to even, saturating, NaN as 0x7F."""
    a = np.minimum(np.abs(x), 448.0)
    lo = np.searchsorted(_MIDS, a, side="left")   # codes below `a`'s nearest: ties go to the lower one
    hi = np.searchsorted(_MIDS, a, side="right")  # .. to the upper one
    c = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))
    return np.where(np.isnan(x), NAN, c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def exponent(top):
    """The least e in the range with top <= 448 2^e, by search."""
    e = np.full(np.shape(top), LOW)
    for x in range(LOW, HIGH):
        e = np.where(top > 448.0 * 2.0 ** x, x + 1, e)
    return e


def clamped(scales):
    return np.clip(scales.astype(int) - 127, LOW, HIGH)


def bf16(x):
    """float64 of bf16 torch tensors."""
    import torch
    return x.detach().cpu().to(torch.float64).numpy()


def finite_top(x, axis):
    return np.max(np.where(np.isfinite(x), np.abs(x), 0.0), axis=axis, initial=0.0)


def write_tile(pool, scales, page, h, tile, kv, x, t0):
    """New values x [n][D] of one tile of K (kv 0) or V (kv 1) at slots t0 .. ; pool [P][H][tpp][2][16 D]."""
    n = len(x)
    old = int(clamped(scales[page, h, tile, kv])) if t0 > 0 else LOW
    e = max(old, int(exponent(finite_top(x, None))))
    block = pool[page, h, tile, kv]
    view = block.reshape(TILE, D) if kv == 0 else block.reshape(D, TILE).T
    if t0 > 0 and e > old:
        view[:t0] = encode(VALUES[view[:t0]] * 2.0 ** (old - e))
    view[t0:t0 + n] = encode(x * 2.0 ** -e)
    scales[page, h, tile, kv] = e + 127


def write_tokens(pool, scales, table, first, k, v, ps):
    """One request's consecutive tokens k, v [n][H][D] (float64) from position `first`."""
    n, H, _ = k.shape
    for a in range(first // TILE, -(-(first + n) // TILE)):
        p0, p1 = max(first, a * TILE), min(first + n, a * TILE + TILE)
        page, tile = table[p0 // ps], p0 % ps // TILE
        for h in range(H):
            write_tile(pool, scales, page, h, tile, 0, k[p0 - first:p1 - first, h], p0 % TILE)
            write_tile(pool, scales, page, h, tile, 1, v[p0 - first:p1 - first, h], p0 % TILE)


def context(pool, scales, table, L, h, ps):
    """K and V [L][D] of one request and kv head, float64; and V's exponents [L]."""
    n = -(-L // ps)
    x = VALUES[pool[table[:n], h]]
    e = clamped(scales[table[:n], h])
    x = x * 2.0 ** e[..., None]
    k = x[:, :, 0].reshape(-1, D)[:L]
    v = x[:, :, 1].reshape(-1, D, TILE).transpose(0, 2, 1).reshape(-1, D)[:L]
    return k, v, np.repeat(e[:, :, 1].reshape(-1), TILE)[:L]


def attend(q, k, v, ev, limit, sm):
    """Rows q [N][D] over the first limit[i] tokens: (out, lse, |weights| |V| sums, score bound, weight unit).

    score bound: sm * sum |q| |k| of the row's largest token, what errors of fp32 score sums go with;
    weight unit: the largest weight times 2^ev over the sum, what f16 weights are relative to."""
    N = len(q)
    out, lse = np.zeros((N, D)), np.full(N, -np.inf)
    size, sbound, unit = np.zeros((N, D)), np.zeros(N), np.zeros(N)
    s = q @ k.T * sm
    sabs = np.abs(q) @ np.abs(k).T * abs(sm)
    for i in range(N):
        n = limit[i]
        if n <= 0:
            continue
        x = s[i, :n]
        m = np.max(x)
        p = np.exp(x - m)
        z = p.sum()
        lse[i] = m + np.log(z)
        out[i] = p @ v[:n] / z
        size[i] = p @ np.abs(v[:n]) / z
        sbound[i] = sabs[i, :n].max()
        unit[i] = (p * 2.0 ** ev[:n]).max() / z
    return out, lse, size, sbound, unit
