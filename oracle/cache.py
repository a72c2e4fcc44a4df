"""fp64 oracle of the generation path: rotary positions with several axes, the
append to the paged cache and the attention of a chunk over it.  numpy only,
one sequence, head and pair at a time; shares no code with the library."""
import numpy as np


def rope_pairs(D, n_axes, sections, base, per_axis):
    """(axis, frequency) of every pair j < D / 2."""
    out = []
    if sections is None:
        return [(j % n_axes, base ** (-2.0 * j / D)) for j in range(D // 2)]
    for ax, n in enumerate(sections):
        for i in range(n):
            out.append((ax, base ** (-i / n) if per_axis else base ** (-2.0 * len(out) / D)))
    return out


def rotate(x, pos, pairs, sign=1.0):
    """x [T, H, D] fp64; pair (j, j + D/2) of row t turned by sign * pos[t, axis] * freq."""
    y = np.empty_like(x)
    h = x.shape[-1] // 2
    for j, (ax, f) in enumerate(pairs):
        a = pos[:, ax].astype(np.float64) * f * sign
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        y[..., j] = x[..., j] * c - x[..., j + h] * s
        y[..., j + h] = x[..., j + h] * c + x[..., j] * s
    return y


def rms_norm(x, w, eps):
    return w * x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def gather(pages, table, length):
    """The first `length` positions of a sequence: [length, Hkv, D] from
    pages [n, page_size, Hkv, D] and its row of the table."""
    ps = pages.shape[1]
    return np.stack([pages[table[t // ps], t % ps] for t in range(length)]) if length else \
        np.zeros((0,) + pages.shape[2:])


def attend(q, k, v, last, scale):
    """q [n, Hq, D], k, v [L, Hkv, D], last [n] (last visible position, -1:
    none).  Returns o [n, Hq, D], lse [Hq, n] and a = sum_j p_j |v_j| [n, Hq, D]."""
    n, Hq, D = q.shape
    g = Hq // k.shape[1]
    o, a, lse = np.zeros((n, Hq, D)), np.zeros((n, Hq, D)), np.full((Hq, n), -np.inf)
    for i in range(n):
        e = min(int(last[i]), len(k) - 1)
        if e < 0:
            continue
        for h in range(Hq):
            s = scale * (k[:e + 1, h // g] @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            z = p.sum()
            o[i, h] = (p / z) @ v[:e + 1, h // g]
            a[i, h] = (p / z) @ np.abs(v[:e + 1, h // g])
            lse[h, i] = m + np.log(z)
    return o, lse, a
