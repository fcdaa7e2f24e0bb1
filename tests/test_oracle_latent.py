"""Pins of the latent-space oracle (oracle/latent.py).

- The absorbed identity: with keys and values expanded from the latents by per-head linear maps and the maps
  folded into queries and outputs, the expanded oracle gives the same attention and, by the chain rule, the same
  gradients.
- Central differences of sum(dO * O) along random directions of every input.
- The 8-bit rounding against brute force over all representable values, and torch's e4m3 conversion.
- The paged attention of a draft block against the draft attention of the same tokens.
"""
import numpy as np
import pytest
import torch

from oracle import latent as ol

BASE = 10000.0


def _case(seed, B=1, S=30, N=3, W=7, H=2, d_l=12, d_r=6, keep=1.0):
    g = np.random.default_rng(seed)
    an = g.integers(0, S - 1, (B, N)).astype(np.int32)
    kp = (g.random((B, N)) < keep).astype(np.uint8)
    L = S + 5 * N
    return (g.standard_normal((B, H, 5 * N, d_l + d_r)), g.standard_normal((B, L, d_l)),
            g.standard_normal((B, L, d_r)), an, kp, g.standard_normal((B, H, 5 * N, d_l)))


@pytest.mark.parametrize("seed,kw", [(1, {}), (2, dict(B=2, W=50, keep=0.5)), (3, dict(W=1))])
def test_absorbed_equals_expanded(oracle_mod, seed, kw):
    q, c, kr, an, kp, _ = _case(seed, **kw)
    S, W = kw.get("S", 30), kw.get("W", 7)
    B, H, R, _ = q.shape
    d_l, d_r, d_c, d_v = c.shape[-1], kr.shape[-1], 5, 4
    g = np.random.default_rng(seed + 100)
    uk, uv = g.standard_normal((H, d_c, d_l)), g.standard_normal((H, d_v, d_l))
    qc = g.standard_normal((B, H, R, d_c))
    kc, v = np.einsum("hcl,bpl->bhpc", uk, c), np.einsum("hvl,bpl->bhpv", uv, c)
    qr = q[..., d_l:]
    ro, rl = oracle_mod.attn_fwd(np.concatenate([qc, qr], -1), kc, kr, v, an, kp, S, W, BASE)
    qa = np.concatenate([np.einsum("bhrc,hcl->bhrl", qc, uk), qr], -1)
    o, lse = ol.attn_fwd(qa, c, kr, an, kp, S, W, (d_c + d_r) ** -0.5, BASE)
    np.testing.assert_allclose(np.einsum("bhrl,hvl->bhrv", o, uv), ro, atol=1e-12)
    np.testing.assert_allclose(lse, rl, atol=1e-12)
    # gradients by the chain rule
    go = g.standard_normal(ro.shape)
    edq, edkc, edkr, edv = oracle_mod.attn_bwd(np.concatenate([qc, qr], -1), kc, kr, v, an, kp, go, S, W, BASE)
    dq, dc, dkr = ol.attn_bwd(qa, c, kr, an, kp, np.einsum("bhrv,hvl->bhrl", go, uv), S, W, (d_c + d_r) ** -0.5, BASE)
    np.testing.assert_allclose(np.einsum("bhrl,hcl->bhrc", dq[..., :d_l], uk), edq[..., :d_c], atol=1e-11)
    np.testing.assert_allclose(dq[..., d_l:], edq[..., d_c:], atol=1e-11)
    np.testing.assert_allclose(dc, np.einsum("bhpc,hcl->bpl", edkc, uk) + np.einsum("bhpv,hvl->bpl", edv, uv),
                               atol=1e-10)
    np.testing.assert_allclose(dkr, edkr, atol=1e-11)


@pytest.mark.parametrize("seed", [5, 6])
def test_finite_differences(seed):
    q, c, kr, an, kp, dout = _case(seed, keep=0.8)
    grads = ol.attn_bwd(q, c, kr, an, kp, dout, 30, 7, 0.3, BASE)
    g = np.random.default_rng(seed + 50)
    args = [q, c, kr]
    for i in range(3):
        u = g.standard_normal(args[i].shape)
        f = []
        for e in (1e-5, -1e-5):
            a = list(args)
            a[i] = a[i] + e * u
            f.append((ol.attn_fwd(*a, an, kp, 30, 7, 0.3, BASE)[0] * dout).sum())
        assert abs((f[0] - f[1]) / 2e-5 - (grads[i] * u).sum()) < 1e-6 * (1 + abs((grads[i] * u).sum()))


def test_fp8_rounding_brute_force():
    g = np.random.default_rng(7)
    vals = np.concatenate([-ol.e4m3_values()[::-1], ol.e4m3_values()])
    y = g.standard_normal((6, 128)) * np.exp(g.uniform(-20, 20, (6, 1)))
    y[3] = 0
    y[4, :100] *= 1e-4  # below the normal range of the group's scale
    out, sc = ol.fp8_round(y)
    for t in range(6):
        s = sc[t, 0]
        assert np.log2(s) == round(np.log2(s))
        if np.any(y[t]):
            assert np.abs(y[t]).max() <= 448 * s and (np.abs(y[t]).max() > 224 * s)
        best = np.abs(y[t][:, None] - vals[None] * s).min(1)
        np.testing.assert_allclose(np.abs(out[t] - y[t]), best, atol=0)
    x = torch.from_numpy(y / sc).float()  # exact in 32 bits? only compare where it is
    same = (x.double().numpy() == y / sc)
    ref = x.to(torch.float8_e4m3fn).double().numpy() * sc
    assert np.array_equal(out[same], ref[same])
    assert ol.fp8_scale(448.0 * 2.0 ** -117) == 2.0 ** -117 and ol.fp8_scale(1e-45) == 2.0 ** -117
    assert ol.fp8_scale(np.nextafter(448.0, 449)) == 2.0


@pytest.mark.parametrize("W", [1, 9, 40])
def test_paged_draft_block_is_the_draft_attention(W):
    """A sequence whose context is positions 0 .. A-1 and whose 5 new tokens are a block at anchor A."""
    g = np.random.default_rng(W)
    S, H, d_l, d_r, A, page = 33, 3, 8, 4, 21, 4
    c, kr = g.standard_normal((1, S + 5, d_l)), g.standard_normal((1, S + 5, d_r))
    q = g.standard_normal((1, H, 5, d_l + d_r))
    o, lse = ol.attn_fwd(q, c, kr, np.array([[A]]), np.array([[1]]), S, W, 0.4, BASE)
    pos = np.arange(A + 5)
    src = np.concatenate([np.arange(A), S + np.arange(5)])
    order = g.permutation(9)
    lat, rope = np.full((9 * page, d_l), np.nan), np.full((9 * page, d_r), np.nan)
    slot = order[pos // page] * page + pos % page
    lat[slot], rope[slot] = c[0, src], ol.turn(kr[0, src], pos, BASE)
    po, pl = ol.paged(q[0].transpose(1, 0, 2), lat, rope, order[None, :7], [0, 5], [A + 5], page, 0.4, False, W, BASE)
    np.testing.assert_allclose(po.transpose(1, 0, 2), o[0], atol=1e-13)
    np.testing.assert_allclose(pl.T, lse[0], atol=1e-13)


def test_paged_causal_is_one_token_at_a_time():
    g = np.random.default_rng(9)
    H, d_l, d_r, page, kv = 2, 8, 4, 4, 19
    lat, rope = g.standard_normal((24, d_l)), g.standard_normal((24, d_r))
    table = g.permutation(6)[None]
    q = g.standard_normal((4, H, d_l + d_r))
    for w in (0, 1, 6):
        o, lse = ol.paged(q, lat, rope, table, [0, 4], [kv], page, 0.4, True, w, BASE)
        for i in range(4):
            o1, l1 = ol.paged(q[i:i + 1], lat, rope, table, [0, 1], [kv - 3 + i], page, 0.4, True, w, BASE)
            np.testing.assert_allclose(o[i], o1[0], atol=1e-13)
            np.testing.assert_allclose(lse[i], l1[0], atol=1e-13)
    # more new tokens than keys: the first tokens see nothing
    o, lse = ol.paged(q, lat, rope, table, [0, 4], [2], page, 0.4, True, 0, BASE)
    assert np.all(o[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.all(np.isfinite(lse[2:]))
