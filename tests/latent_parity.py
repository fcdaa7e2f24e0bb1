"""Error bounds of the latent-space operators, element by element, from the fp64 oracle's own quantities.

u = 2^-8 is half a step of bf16 relative to the value, f = 2^-24 that of fp32. With e the error of a score
(natural units), a softmax weight is off by the factor exp(+-2 e) at most: e enters the weight and the
normaliser.

  e  <= scale * sum|q||k| * (d + 16) f      fp32 products and sums of d terms in any order, fp32 cos and sin
      + scale * sum_rope |q||k| * (2u + u^2)  bf16: both rotated rope slices are rounded to bf16 operands
      + (|s| + |lse|) 2 f                     scaling by log2(e) in fp32
  P  : factor exp(2 e) (1 + 2^-20)            2^x to 2 units of the last place; a bf16 operand adds u
  O  : sum P|c| (ep + (n + 8) f) + u |O|
  dP : sum|dO||c| (d + 8) f;  D = sum P dP: sum P (ep |dP| + eP) with the same sums
  dS : scale (ep P|dP - D| + P (err dP + err D)), + u |dS| as a bf16 operand
  dq : sum_k err(dS)|k| + |dS||k_rope| u + n f sum|dS||k|, then rounded (the rope part turned back: both
       elements of a pair share the larger error)
  dc, dkr: the same over the rows, fp32 sums of n_rows terms in any order.
"""
import numpy as np

from oracle import latent as ol

BLOCK = 5
F = 2.0 ** -24


def _pairmax(e):
    """Elements of a rope pair after a turn: |cos| e0 + |sin| e1 <= e0 + e1."""
    s = e[..., 0::2] + e[..., 1::2]
    return np.repeat(s, 2, axis=-1)


def _weights(x, k, d_l, scale, u, lse=None, extra=0.0, mask=None):
    """P, LSE, the weights' relative error and the scores' error for rows x [r, d], keys k [n, d]."""
    s = x @ k.T * scale
    if mask is not None:
        s = np.where(mask, s, -np.inf)
    p, z = ol._softmax(s)
    d = x.shape[-1]
    ax, ak = np.abs(x), np.abs(k)
    # an operand's rotated slice is rounded from the exact turn, pair by pair
    e = scale * (ax @ ak.T) * (d + 16) * F + scale * (ax[:, d_l:] @ ak[:, d_l:].T) * (2 * u + u * u + extra)
    fin = np.isfinite(s)
    zz = np.where(np.isfinite(z), z, 0.0)
    e = e + (np.abs(np.where(fin, s, 0.0)) + np.abs(zz)[:, None]) * 2 * F
    if mask is not None:
        e = np.where(mask, e, 0.0)
    em = e.max(-1, keepdims=True) if e.shape[1] else np.zeros((e.shape[0], 1))
    ep = np.expm1(e + em) * (1 + 2.0 ** -20) + 2.0 ** -20
    return p, z, ep, em[:, 0]


def fwd_block(x, k, d_l, scale, bf16, extra=0.0, mask=None):
    """Oracle and bounds of rows x over keys k: (o, err o, lse, err lse)."""
    u = 2.0 ** -8 if bf16 else 0.0
    p, z, ep, em = _weights(x, k, d_l, scale, u, extra=extra, mask=mask)
    c = k[:, :d_l]
    o = p @ c
    n = k.shape[0]
    eo = (p * (ep + u + (n + 8) * F)) @ np.abs(c)
    eo = eo * (1 + u) + (u if bf16 else F) * np.abs(o) + 1e-38
    return o, eo, z, em + (np.abs(np.where(np.isfinite(z), z, 0)) + n + 8) * 4 * F


def attn(q, c, kr, an, kp, S, W, scale, base, bf16, dout=None, lse_err=True):
    """(values, bounds) of o, lse and, with dout, dq, dc, dkr."""
    q, c, kr = (np.asarray(t, np.float64) for t in (q, c, kr))
    B, H, R, d = q.shape
    d_l = c.shape[-1]
    u = 2.0 ** -8 if bf16 else 0.0
    r = u if bf16 else F  # of the outputs
    val = dict(o=np.zeros((B, H, R, d_l)), lse=np.full((B, H, R), -np.inf))
    err = dict(o=np.zeros((B, H, R, d_l)), lse=np.zeros((B, H, R)))
    if dout is not None:
        dout = np.asarray(dout, np.float64)
        for n, t in (("dq", q), ("dc", c), ("dkr", kr)):
            val[n], err[n] = np.zeros(t.shape), np.zeros(t.shape)
    terms = np.zeros(c.shape[:2])  # rows that add to a key
    for b, n, a, idx, k, pos in ol.blocks(c, kr, an, kp, S, W, base):
        rows = slice(BLOCK * n, BLOCK * n + BLOCK)
        x = ol._block_q(q, b, n, a, d_l, base).reshape(H * BLOCK, d)
        o, eo, z, ez = fwd_block(x, k, d_l, scale, bf16)
        for nm, t, w in (("o", o, eo), ("lse", z, ez)):
            sh = (H, BLOCK) + t.shape[1:]
            val[nm][b, :, rows], err[nm][b, :, rows] = t.reshape(sh), w.reshape(sh)
        if dout is None:
            continue
        g = dout[b, :, rows].reshape(H * BLOCK, d_l)
        p, z, ep, em = _weights(x, k, d_l, scale, u)
        ep = ep + np.expm1(2 * ez)[:, None]  # the lse that the backward is given has the forward's error
        cc = k[:, :d_l]
        dp = g @ cc.T
        edp = np.abs(g) @ np.abs(cc).T * (d_l + 8) * F
        D = (p * dp).sum(-1, keepdims=True)
        m = k.shape[0]
        eD = (p * (ep * np.abs(dp) + (1 + ep) * edp + (m + 8) * F * np.abs(dp))).sum(-1, keepdims=True)
        ds = scale * p * (dp - D)
        eds = scale * p * (ep * np.abs(dp - D) + (1 + ep) * (edp + eD)) + 4 * F * np.abs(ds)
        ak, ax = np.abs(k), np.abs(x)
        rk = ak.copy()
        rk[:, :d_l] = 0
        rx = ax.copy()
        rx[:, :d_l] = 0
        eds_op = eds * (1 + u) + u * np.abs(ds)
        y = ds @ k
        ey = eds_op @ ak * (1 + u) + (np.abs(ds) @ rk) * u + (np.abs(ds) @ ak) * (m + 8) * F
        dq = np.concatenate([y[:, :d_l], ol.turn(y[:, d_l:].reshape(H, BLOCK, -1), np.broadcast_to(
            a + np.arange(BLOCK), (H, BLOCK)), base, True).reshape(H * BLOCK, -1)], 1)
        ey = np.concatenate([ey[:, :d_l], _pairmax(ey[:, d_l:])], 1)
        val["dq"][b, :, rows] = dq.reshape(H, BLOCK, d)
        err["dq"][b, :, rows] = (ey * (1 + r) + r * np.abs(dq)).reshape(H, BLOCK, d)
        gk = ds.T @ x
        nr = x.shape[0]
        egk = eds_op.T @ ax * (1 + u) + np.abs(ds).T @ rx * u + np.abs(ds).T @ ax * (nr + 8) * F
        gc = gk[:, :d_l] + p.T @ g
        egc = egk[:, :d_l] + (p * (ep + u + (nr + 8) * F)).T @ np.abs(g)
        val["dc"][b, idx] += gc
        val["dkr"][b, idx] += ol.turn(gk[:, d_l:], pos, base, True)
        # sums over blocks: one more fp32 rounding of the running sum for each
        terms[b, idx] += 1
        err["dc"][b, idx] += egc + np.abs(gc) * F
        err["dkr"][b, idx] += _pairmax(egk[:, d_l:]) + np.abs(gk[:, d_l:]) * F
    if dout is not None:
        for nm in ("dc", "dkr"):
            err[nm] = err[nm] * (1 + terms.max() * 2 * F) * (1 + r) + r * np.abs(val[nm])
    return val, err


def check(name, got, ref, err):
    g = got.detach().double().cpu().numpy() if hasattr(got, "detach") else np.asarray(got, np.float64)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    ninf = np.isneginf(ref)
    assert np.array_equal(np.isneginf(g), ninf), "%s: -inf pattern differs" % name
    g, r, e = g[~ninf], ref[~ninf], err[~ninf]
    assert np.all(np.isfinite(g)), "%s: values that are not finite" % name
    if g.size == 0:
        return
    over = np.abs(g - r) - (e + 1e-30)
    w = int(np.argmax(over))
    assert over[w] <= 0, "%s: |%.6g - %.6g| = %.3g > %.3g (at %d of %d)" % (name, g[w], r[w], abs(g[w] - r[w]), e[w],
                                                                           w, g.size)
