"""The arithmetic of gfx950's matrix-core operation under the routed experts in
4 bits (v_mfma_scale_f32_16x16x128_f8f6f4, E2M1 by E4M3 with E8M0 scales),
measured through moe_mxfp4_mma_tiles and pinned by
tests/test_gpu_mx4_matrix_cores.py: in groups of eight consecutive K every exact
product is cut toward zero to a multiple of 2^(E - 13), E the largest sum of the
operands' exponents in the group (the rule of the 32x32x64 form too, see
tests/mma_rules.py).  Two neighbouring groups' sums at a time are then added to
the accumulator, in eight steps in the order of K: each step aligns its three
terms 24 bits below the largest, a group by its E, whatever is left of its sum
(512 - 512 in a group cuts an accumulator of 2^-16 off, which lies below
2^(9 - 24)), and rounds the sum to fp32.  The model allows a step three such
quanta, one for each term, and half an fp32 step of its sum."""
import numpy as np

from oracle import moe_oracle as O
from tests import mx_ref as R

U = 2.0 ** -24


def exponents(codes, mant, bias):
    """Exponents of element codes (sign cut off); that of a subnormal or zero is
    the smallest normal one's."""
    return np.maximum(codes.astype(np.int64) >> mant, 1) - bias


def operands4(codes, scale):
    """(values [r][K], exponents [r][K]) of E2M1 codes [r][K/2], scales [r][K/32]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    s = np.repeat(scale.astype(np.int64) - 127, 32, axis=1)
    return np.where(c & 8, -1.0, 1.0) * R.E2M1[c & 7] * np.ldexp(1.0, s), exponents(c & 7, 1, 1) + s


def operands8(codes, scale):
    """The same of E4M3 codes [r][K], scales [r][K/32]."""
    s = np.repeat(scale.astype(np.int64) - 127, 32, axis=1)
    return O.e4m3_decode(codes) * np.ldexp(1.0, s), exponents(codes & 127, 3, 7) + s


def group_tops(p, e):
    """E of the groups of eight [..., K/8] of products p [..., K] with their
    operands' exponents' sums e; far below any where a group has none."""
    q = p.reshape(*p.shape[:-1], -1, 8)
    return np.where(q != 0, e.reshape(q.shape), -1000).max(-1)


def cut(p, e):
    """What the groups keep of each product."""
    q = p.reshape(*p.shape[:-1], -1, 8)
    grid = np.ldexp(1.0, group_tops(p, e) - 13)[..., None]
    return (np.trunc(q / grid) * grid).reshape(p.shape)


def operation(p, e, acc, err):
    """The operation on products p [..., 128] (their operands' exponents' sums
    e), whose accumulator is acc, off by at most err: the same of its result."""
    g = cut(p, e).reshape(*p.shape[:-1], 16, 8).sum(-1)
    lead = np.maximum(np.abs(g), np.ldexp(1.0, group_tops(p, e)))
    for s in range(0, 16, 2):
        top = np.maximum(np.abs(acc) + err, np.maximum(lead[..., s], lead[..., s + 1]))
        acc = acc + g[..., s] + g[..., s + 1]
        err = err + 3 * U * top
        err = err + U * (np.abs(acc) + err)
    return acc, err


def product(w, we, x, xe):
    """Weights [n][K] times one token [K] (values, exponents) as the kernels sum
    them: four chains of pairs of 128, added in order."""
    p, e = w * x, we + xe
    total, off = np.zeros(len(w)), np.zeros(len(w))
    for chain in range(4):
        acc, err = np.zeros(len(w)), np.zeros(len(w))
        for pair in range(chain, (p.shape[1] // 128 + 1) // 2, 4):
            for k in range(256 * pair, min(256 * pair + 256, p.shape[1]), 128):
                acc, err = operation(p[:, k:k + 128], e[:, k:k + 128], acc, err)
        total = total + acc
        off = off + err
        off = off + U * (np.abs(total) + off)
    return total, off


def routed_ffn(x, x_scale, idx, tw, weights, add):
    """(y [T][d], bound [T][d]) of the routed experts with the operation's own
    arithmetic.  x [T][d] codes, x_scale; weights: for gate, up and down (codes
    [E][rows][cols/2], scales [cols/128][E*rows][4]); numpy arrays."""
    xv, xe = operands8(x, x_scale)
    T, d = xv.shape
    y = np.zeros((T, d)) if add is None else add.copy()
    err, mag = np.zeros((T, d)), np.abs(y)
    E = len(weights[0][0])

    def expert(m, i):
        codes, scale = weights[m]
        rows = codes.shape[1]
        return operands4(codes[i], scale[:, i * rows:(i + 1) * rows].transpose(1, 0, 2).reshape(rows, -1))

    for i in range(E):
        at = [(t, j) for t in range(T) for j in range(idx.shape[1]) if idx[t, j] == i]
        if not at:
            continue
        gate, up, (dv, de) = expert(0, i), expert(1, i), expert(2, i)
        for t, j in at:
            G, eg = product(*gate, xv[t], xe[t])
            V, ev = product(*up, xv[t], xe[t])
            h = O.silu(G) * V
            # as in mx_ref.routed_ffn
            eh = 1.1 * eg * np.abs(V) + np.abs(O.silu(G)) * ev + eg * ev * 1.1 + (8 + np.abs(G)) * U * np.abs(h)
            q, off = R.round_h(h[None], eh[None])
            q, off = q[0], off[0]
            eb = np.repeat(O.mx_scale_exponent(np.abs(h).reshape(-1, 32).max(-1)), 32)
            qe = np.maximum(np.where(q != 0, np.frexp(q)[1] - 1, -1000), eb - 6)
            o, eo = product(dv, de, q, qe)
            # where an element may have been rounded the other way, its group may be cut otherwise
            top = np.abs(dv * (np.abs(q) + off)).reshape(d, -1, 8).max(-1)
            eo = eo + np.abs(dv) @ off + (top * (off.reshape(-1, 8).max(-1) > 0)).sum(-1) * 8 * 2.0 ** -12
            y[t] += tw[t, j] * o
            err[t] += np.abs(tw[t, j]) * eo
            mag[t] += np.abs(tw[t, j]) * (np.abs(o) + eo)
    err = err + 20 * U * mag                      # as in mx_ref.routed_ffn
    return y, err + 2.0 ** -8 * (np.abs(y) + err) + 1e-38
