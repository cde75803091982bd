"""References in 64 bits for the latent-cache and block operators, written from
the layouts and formulas of include/dsa.h (numpy, element by element where that
is affordable; no code shared with the library or the oracle)."""
import numpy as np

BF16, FP8, Q4 = 1, 2, 3                   # dsa_dtype values of the cache formats

E4M3 = np.zeros(256)
for _c in range(256):
    _e, _m = (_c >> 3) & 15, _c & 7
    _v = _m / 512.0 if _e == 0 else (8 + _m) * 2.0 ** (_e - 10)
    if (_c & 127) == 127:
        _v = np.nan
    E4M3[_c] = -_v if _c & 128 else _v


def bf16(x):
    """Round to the nearest bf16 (ties to even), as float64."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        m, e = np.frexp(x)
        return np.where(np.isfinite(x), np.ldexp(np.rint(m * 256.0), e - 8), x)


def row_bytes(fmt, dc, dr):
    if fmt == BF16:
        return 2 * (dc + dr)
    if fmt == FP8:
        return dc + dc // 32 + 2 * dr
    return -(-(dc // 2 + 2 * dr + dc // 16) // 16) * 16


def _u16_as_bf16(lo, hi):
    w = (lo.astype(np.uint32) | hi.astype(np.uint32) << 8) << 16
    return w.view(np.float32).astype(np.float64)


def decode_rows(rows, fmt, dc, dr):
    """The values of byte rows [..., row_bytes] as float64 [..., dc + dr]."""
    rows = np.asarray(rows, np.uint8)
    at = {BF16: 2 * dc, FP8: dc + dc // 32, Q4: dc // 2}[fmt]
    pe = _u16_as_bf16(rows[..., at:at + 2 * dr:2], rows[..., at + 1:at + 2 * dr:2])
    if fmt == BF16:
        c = _u16_as_bf16(rows[..., 0:2 * dc:2], rows[..., 1:2 * dc:2])
    elif fmt == FP8:
        s = np.ascontiguousarray(rows[..., dc:at]).view(np.float32).astype(np.float64)
        # the library's product is a single-precision one, then rounded to bf16
        c = (E4M3[rows[..., :dc]] * np.repeat(s, 128, -1)).astype(np.float32)
        c = bf16(c)
    else:
        c = np.empty(rows.shape[:-1] + (dc,))
        sa = dc // 2 + 2 * dr
        s = _u16_as_bf16(rows[..., sa:sa + dc // 16:2], rows[..., sa + 1:sa + dc // 16:2])
        for v in range(dc):
            nib = (v % 8) // 2 + 4 * (v % 2)
            byte = rows[..., v // 8 * 4 + nib // 2]
            n = (byte >> (4 * (nib % 2)) & 15).astype(np.float64) - 8
            c[..., v] = bf16(n * s[..., v // 32])
    return np.concatenate([c, pe], -1)


def prologue(kv, norm_w, eps, cs, interleaved, dc):
    """Norm and rotation of kv [B,S,dc+dr] in 64 bits."""
    kv = np.asarray(kv, np.float64)
    c, p = kv[..., :dc].copy(), kv[..., dc:].copy()
    dr = p.shape[-1]
    if norm_w is not None:
        c = c / np.sqrt((c * c).mean(-1, keepdims=True) + eps) * np.asarray(norm_w, np.float64)
    if cs is not None:
        z = np.asarray(cs, np.float64)
        z = z[..., 0] + 1j * z[..., 1]
        a = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, dr // 2), slice(dr // 2, None))
        y = (p[..., a[0]] + 1j * p[..., a[1]]) * z
        p[..., a[0]], p[..., a[1]] = y.real, y.imag
    return np.concatenate([c, p], -1)


def q4_groups(c):
    """(codes minus 8, scales) of c [..., dc] by the 4-bit rule, in 64 bits."""
    g = np.asarray(c, np.float64).reshape(*c.shape[:-1], -1, 32)
    s = bf16(np.maximum(np.abs(g).max(-1), np.float32(1e-4)).astype(np.float32) / np.float32(7))
    n = np.clip(np.rint(g / s[..., None]), -7, 7)
    return n.reshape(c.shape), s


def attend(q, rows, positions, sm_scale, dc):
    """q [Hq, d], rows [t, d] float64, positions (distinct) -> out [Hq, dc], lse [Hq]."""
    q = np.asarray(q, np.float64)
    if len(positions) == 0:
        return np.zeros((q.shape[0], dc)), np.full(q.shape[0], -np.inf)
    c = rows[np.asarray(positions)]
    z = sm_scale * (q @ c.T)
    m = z.max(-1, keepdims=True)
    p = np.exp(z - m)
    l = p.sum(-1, keepdims=True)
    return p @ c[:, :dc] / l, (m + np.log(l))[:, 0]


def block_positions(blk, block, i):
    """Positions that a query at position i attends to by its block list."""
    done = (i + 1) // block
    out = list(range(done * block, i + 1))
    for e in blk:
        if 0 <= e < done:
            out += range(int(e) * block, (int(e) + 1) * block)
    return out


def block_keys(codes, scales, block, D):
    """Means of whole blocks of decoded keys: codes [T, D], scales [T] -> [T // block, D]."""
    n = codes.shape[0] // block
    k = E4M3[codes[:n * block]] * np.asarray(scales[:n * block], np.float64)[:, None]
    return k.reshape(n, block, D).mean(1)
