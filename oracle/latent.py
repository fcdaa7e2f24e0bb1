"""fp64 oracle of the latent-space operators (NumPy): the draft attention over latents and its
gradients, the rows of the latent cache, and the attention of new tokens over the paged cache.

TEST INFRASTRUCTURE ONLY: nothing in the product imports it.

Definitions (page "GLM 5.2 DSpark speculative-training design", §3 for the mask, §4 for MLA and RoPE):
a key is k_p = [c_p ; R(p) kr_p], a query row at position t is [q_l ; R(t) q_r], R the rotation of
adjacent pairs by t * base^(-2i/d_r); s = scale * q . k over the row's visible keys, P = softmax(s),
O = P C, LSE = logsumexp(s). With dP = dO C^T, D = sum_k P dP, dS = scale * P (dP - D):
dq = dS K, dc = dS^T q_l + P^T dO, dkr = R^T (dS^T q_r), the rope part of dq turned back as well.

Pinned by tests/test_oracle_latent.py: the expanded oracle through the absorbed identity, finite
differences, and brute force over the representable values of the 8-bit format.
"""
import numpy as np

BLOCK = 5


def turn(x, pos, base, back=False):
    """x [..., d_r] turned (back: by the inverse) to positions pos [...]."""
    d_r = x.shape[-1]
    x = np.asarray(x, np.float64)
    if d_r == 0:
        return x.copy()
    th = float(base) ** (-2.0 * np.arange(d_r // 2) / d_r)
    z = (x[..., 0::2] + 1j * x[..., 1::2]) * np.exp((-1j if back else 1j) * np.asarray(pos, np.float64)[..., None] * th)
    out = np.empty_like(x)
    out[..., 0::2], out[..., 1::2] = z.real, z.imag
    return out


def _softmax(s):
    """P and LSE of score rows; -inf entries are masked, a row of them gives P = 0, LSE = -inf."""
    m = s.max(axis=-1, initial=-np.inf)
    live = m > -np.inf
    e = np.exp(s - np.where(live, m, 0.0)[..., None])
    l = e.sum(-1)
    with np.errstate(divide="ignore"):
        lse = np.where(live, m + np.log(np.where(live, l, 1.0)), -np.inf)
    return e / np.where(live, l, 1.0)[..., None], lse


def blocks(c, kr, anchors, keep, S, W, base):
    """Per kept block (b, n): its key indices, keys [m, d_l + d_r] and the keys' positions."""
    B, N = anchors.shape
    for b in range(B):
        for n in range(N):
            if not keep[b, n]:
                continue
            a = int(anchors[b, n])
            idx = np.concatenate([np.arange(max(0, a - W + 1), a), S + BLOCK * n + np.arange(BLOCK)])
            pos = np.concatenate([np.arange(max(0, a - W + 1), a), a + np.arange(BLOCK)])
            yield b, n, a, idx, np.concatenate([c[b, idx], turn(kr[b, idx], pos, base)], 1), pos


def _block_q(q, b, n, a, d_l, base):
    """Rows (head, offset) of block n, rope part turned: [n_h, 5, d]."""
    x = np.asarray(q[b, :, BLOCK * n:BLOCK * n + BLOCK], np.float64)
    return np.concatenate([x[..., :d_l], turn(x[..., d_l:], np.broadcast_to(a + np.arange(BLOCK), x.shape[:2]), base)], -1)


def attn_fwd(q, c, kr, anchors, keep, S, W, scale, base):
    B, H, R, _ = q.shape
    d_l = c.shape[-1]
    o, lse = np.zeros((B, H, R, d_l)), np.full((B, H, R), -np.inf)
    for b, n, a, idx, k, _ in blocks(c, kr, anchors, keep, S, W, base):
        p, z = _softmax(_block_q(q, b, n, a, d_l, base) @ k.T * scale)
        o[b, :, BLOCK * n:BLOCK * n + BLOCK] = p @ k[:, :d_l]
        lse[b, :, BLOCK * n:BLOCK * n + BLOCK] = z
    return o, lse


def attn_bwd(q, c, kr, anchors, keep, dout, S, W, scale, base):
    d_l = c.shape[-1]
    dq, dc, dkr = np.zeros(q.shape), np.zeros(c.shape), np.zeros(kr.shape)
    for b, n, a, idx, k, pos in blocks(c, kr, anchors, keep, S, W, base):
        rows = slice(BLOCK * n, BLOCK * n + BLOCK)
        x, g = _block_q(q, b, n, a, d_l, base), np.asarray(dout[b, :, rows], np.float64)
        p, _ = _softmax(x @ k.T * scale)
        dp = g @ k[:, :d_l].T
        ds = scale * p * (dp - (p * dp).sum(-1, keepdims=True))
        y = ds @ k
        dq[b, :, rows, :d_l] = y[..., :d_l]
        dq[b, :, rows, d_l:] = turn(y[..., d_l:], np.broadcast_to(a + np.arange(BLOCK), y.shape[:2]), base, True)
        gk = np.einsum("hjk,hjd->kd", ds, x)
        dc[b, idx] += gk[:, :d_l] + np.einsum("hjk,hjd->kd", p, g)
        dkr[b, idx] += turn(gk[:, d_l:], pos, base, True)
    return dq, dc, dkr


# ---- the cache's rows ------------------------------------------------------------------------
GROUP = 128


def norm_rows(c, w, eps):
    c = np.asarray(c, np.float64)
    if w is None:
        return c
    return c / np.sqrt((c * c).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def e4m3_values():
    """The values of codes 0 .. 126 (positive, finite)."""
    k = np.arange(127)
    e, f = k >> 3, k & 7
    return np.where(e > 0, (1 + f / 8.0) * 2.0 ** (e - 7.0), f / 8.0 * 2.0 ** -6)


def fp8_scale(amax):
    """Least 2^e, e >= -117, with amax <= 448 * 2^e; 1 for amax = 0."""
    if amax == 0:
        return 1.0
    e = -117
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def fp8_round(y):
    """Rows y [T, d_l] as (values that the 8-bit row stands for, scales [T, d_l / 128])."""
    vals = e4m3_values()
    out, scales = np.empty(y.shape), np.empty((y.shape[0], y.shape[1] // GROUP))
    for t in range(y.shape[0]):
        for g in range(scales.shape[1]):
            x = y[t, g * GROUP:(g + 1) * GROUP]
            fin = np.isfinite(x)
            s = fp8_scale(np.abs(x[fin]).max(initial=0.0))
            a = np.where(fin, np.abs(x), 0.0) / s
            hi = np.searchsorted(vals, a).clip(0, 126)
            lo = (hi - 1).clip(0)
            up, dn = vals[hi] - a, a - vals[lo]
            pick = np.where((up < dn) | ((up == dn) & (hi % 2 == 0)), hi, lo)
            out[t, g * GROUP:(g + 1) * GROUP] = np.where(fin, np.copysign(vals[pick], np.where(fin, x, 0.0)) * s, np.nan)
            scales[t, g] = s
    return out, scales


# ---- new tokens over the paged cache -----------------------------------------------------------
def paged(q, lat, rope, table, q_start, kv_len, page_size, scale, causal, window, base, o=None, lse=None):
    """q [T, n_h, d_l + d_r]; lat [slots, d_l] and rope [slots, d_r] the values of the cache's rows (rope
    already turned). Rows of o and lse behind the last sequence keep what they hold."""
    T, H, _ = q.shape
    d_l = lat.shape[1]
    o = np.zeros((T, H, d_l)) if o is None else np.array(o, np.float64)
    lse = np.full((T, H), -np.inf) if lse is None else np.array(lse, np.float64)
    for s in range(len(kv_len)):
        n_q, kv = int(q_start[s + 1] - q_start[s]), int(kv_len[s])
        ctx = kv - n_q
        for i in range(n_q):
            t = ctx + i
            hi = min(t + 1, kv) if causal else kv
            lo = max(0, (t if causal else ctx) - window + 1) if window > 0 else 0
            keys = np.arange(lo, max(lo, hi))
            tok = int(q_start[s]) + i
            if keys.size == 0:
                o[tok], lse[tok] = 0.0, -np.inf
                continue
            slot = table[s, keys // page_size].astype(np.int64) * page_size + keys % page_size
            k = np.concatenate([lat[slot], rope[slot]], 1)
            x = np.concatenate([q[tok, :, :d_l], turn(q[tok, :, d_l:], np.full(H, t), base)], -1)
            p, lse[tok] = _softmax(x @ k.T * scale)
            o[tok] = p @ lat[slot]
    return o, lse
