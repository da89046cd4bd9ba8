"""Plain 64-bit forms that the tests of the FP4 layers and of expert routing compare with."""
import numpy as np

import oracle
from _layout import untile_scales


def block(fmt) -> int:
    return 16 if fmt == "nvfp4" else 32


def quantized(h: np.ndarray, fmt, amax: float = 0.0):
    """(scale codes, E2M1 codes, row scales) of the fp32 rows h, each row with its own second-level scale."""
    h = np.ascontiguousarray(h, np.float32)
    scales, codes, rows = [], [], []
    for r in h:
        enc, dec = oracle.tensor_scale(amax or float(np.max(np.abs(r)))) if fmt == "nvfp4" else (1.0, 1.0)
        s, c = oracle.quant_blocks(r, block(fmt), fmt, enc)
        scales.append(s)
        codes.append(c)
        rows.append(dec)
    return np.stack(scales), np.stack(codes), np.array(rows, np.float32)


def read_matrix(m):
    """(scale codes, E2M1 codes, row scales) of a GPU FP4Matrix, experts stacked along the rows."""
    fmt = "nvfp4" if m.fmt == 1 else "mxfp4"
    raw = m.codes.cpu().numpy()[: m.experts * m.rows * m.k // 2].reshape(m.experts * m.rows, m.k // 2)
    codes = np.stack([raw & 15, raw >> 4], axis=-1).reshape(raw.shape[0], m.k)
    per = m.k // block(fmt)
    size = (m.rows + 127) // 128 * ((per + 3) // 4) * 512
    buf = m.scales.cpu().numpy()
    scales = np.concatenate([untile_scales(buf[e * size : (e + 1) * size], m.rows, per) for e in range(m.experts)])
    return scales, codes, m.row_scale.cpu().numpy()


def padded_scales(m):
    """The places of every row past its last scale, up to a multiple of four."""
    per = m.k // (16 if m.fmt == 1 else 32)
    wide = (per + 3) // 4 * 4
    size = (m.rows + 127) // 128 * (wide // 4) * 512
    buf = m.scales.cpu().numpy()
    return np.concatenate([untile_scales(buf[e * size : (e + 1) * size], m.rows, wide)[:, per:] for e in range(m.experts)])


def values(m) -> np.ndarray:
    scales, codes, rows = read_matrix(m)
    fmt = "nvfp4" if m.fmt == 1 else "mxfp4"
    return oracle.dequant_blocks(scales, codes, fmt) * rows.astype(np.float64)[:, None]


def check_product(y: np.ndarray, xv: np.ndarray, wv: np.ndarray, bf16: bool, what: str = ""):
    """y against xv wv^T in 64 bits.

    Every product of two FP4 elements and their block scales is exact in fp32 (2 x 2 bits times 4 x 4 bits).
    They are added in fp32 in some order: at most k - 1 additions, each off by at most 2^-23 of a partial sum
    (round to nearest is 2^-24; the tensor core may cut off), which no partial sum of magnitudes exceeds.
    A dot product of length k inside the core counts as one addition for each 16 elements at least, so
    k / 16 + 16 steps are allowed, not k.  Then two products with the row scales (2^-24 each) and one rounding
    to bf16 (2^-8) or none.  Where the magnitudes add up to 2^128 or more, a partial sum in fp32 may be infinite
    whatever the whole sum is: such values are outside the operator's range and only have to be non-finite or right."""
    k = xv.shape[1]
    ref = xv @ wv.T
    mag = np.abs(xv) @ np.abs(wv).T
    tol = (k / 16 + 16) * 2.0**-23 * mag + 2 * 2.0**-24 * np.abs(ref)
    if bf16:
        tol = tol + 2.0**-8 * (np.abs(ref) + tol)
    with np.errstate(invalid="ignore"):
        near = (np.abs(y.astype(np.float64) - ref) <= tol) | ((mag >= 2.0**128) & ~np.isfinite(y))
    bad = np.argwhere(~near)
    assert bad.size == 0, (f"{what}: {len(bad)} of {y.size} values off, first at {bad[0].tolist()}: "
                           f"{y[tuple(bad[0])]} for {ref[tuple(bad[0])]}")


def routed(logits, top_k, score="softmax", bias=None, groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0):
    """ids and weights (64 bits) of every token, one token and one choice at a time."""
    t, n = logits.shape
    ids = np.full((t, top_k), -1, np.int64)
    weights = np.zeros((t, top_k))
    per = n // groups
    for i in range(t):
        z = logits[i].astype(np.float64)
        on = z > -np.inf  # NaN compares false
        p = np.zeros(n)
        if score == "softmax" and on.any():
            m = z[on].max()
            with np.errstate(invalid="ignore"):
                e = np.where(z[on] == m, 1.0, np.exp(z[on] - m))
            p[on] = e / e.sum()
        elif score == "sigmoid":
            with np.errstate(over="ignore"):
                p[on] = 1.0 / (1.0 + np.exp(-z[on]))
        c = p + (0.0 if bias is None else bias.astype(np.float64))
        c = np.where(on & (c > -np.inf), c, -np.inf)
        if groups > 1:
            value = [sum(sorted((v for v in c[g * per : (g + 1) * per] if v > -np.inf), reverse=True)[:group_top])
                     if (c[g * per : (g + 1) * per] > -np.inf).any() else -np.inf for g in range(groups)]
            kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
            for g in range(groups):
                if g not in kept:
                    c[g * per : (g + 1) * per] = -np.inf
        by = np.where(c > -np.inf, z if bias is None else c, -np.inf)
        order = [e for e in sorted(range(n), key=lambda e: (-by[e] if c[e] > -np.inf else np.inf, e)) if c[e] > -np.inf]
        order = order[:top_k]
        w = p[order]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        ids[i, : len(order)] = order
        weights[i, : len(order)] = w * scale
    return ids, weights


def laid_out(ids, experts, capacity):
    """rows, offsets and slots of an assignment, one place at a time."""
    rows, slots = np.full(capacity, -1, np.int64), np.full(ids.shape, -1, np.int64)
    offsets = [0]
    for e in range(experts):
        at = offsets[-1]
        for t, j in np.argwhere(ids == e):
            rows[at], slots[t, j] = t, at
            at += 1
        offsets.append((at + 127) // 128 * 128)
    return rows, np.array(offsets), slots
