"""The bounds that test_gpu_latent_rope.py holds the kernels to, on the CPU: results formed in 64 bits from rope slices
split as hi + lo keep them, results with one of the lo parts left out do not."""
import numpy as np
import pytest
import torch

import latent_parity as lp
from oracle import latent as ol
from speculative_draft_mla_b200 import capi
from test_gpu_latent_attn import make
from test_gpu_latent_rope import SPLIT_BOTH, SPLIT_QUERY, rope_heavy, tight  # noqa: F401 (a fixture)

BASE, SCALE = 10000.0, capi.LATENT_SCALE


def split(x):
    hi = torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()
    return hi, torch.from_numpy(x - hi).to(torch.bfloat16).double().numpy()


def scores(x, k, d_l, terms):
    """Rows x over keys k, the rope slices (turned, exact) as the given products of their parts."""
    q, r = dict(zip("hl", split(x[:, d_l:]))), dict(zip("hl", split(k[:, d_l:])))
    s = x[:, :d_l] @ k[:, :d_l].T
    for a, b in terms:
        s = s + q[a] @ r[b].T
    return s * SCALE


def draft(terms, terms_bwd):
    """lse, dq, dc with the scores of forward and backward formed from these products; what the kernels round besides
    is left out."""
    S, N, W, H, d_l = 300, 6, 128, 23, 512
    t = make(S, 1, S, N, H, d_l, 64, "bf16")
    rope_heavy(t["q"], d_l)
    q, c, kr, dout = (t[n].double().numpy() for n in ("q", "c", "kr", "dout"))
    an, kp = t["an"].numpy(), t["kp"].numpy()
    out = dict(lse=np.full(q.shape[:3], -np.inf), dq=np.zeros(q.shape), dc=np.zeros(c.shape))
    for b, n, a, idx, k, pos in ol.blocks(c, kr, an, kp, S, W, BASE):
        rows = slice(5 * n, 5 * n + 5)
        x = ol._block_q(q, b, n, a, d_l, BASE).reshape(H * 5, -1)
        _, z = ol._softmax(scores(x, k, d_l, terms))
        out["lse"][b, :, rows] = z.reshape(H, 5)
        p = np.exp(scores(x, k, d_l, terms_bwd) - z[:, None])
        g = dout[b, :, rows].reshape(H * 5, d_l)
        dp = g @ k[:, :d_l].T
        ds = SCALE * p * (dp - (p * dp).sum(-1, keepdims=True))
        y = (ds @ k).reshape(H, 5, -1)
        out["dq"][b, :, rows, :d_l] = y[..., :d_l]
        out["dq"][b, :, rows, d_l:] = ol.turn(y[..., d_l:], np.broadcast_to(a + np.arange(5), (H, 5)), BASE, True)
        out["dc"][b, idx] += ds.T @ x[:, :d_l] + p.T @ g
    val, err = lp.attn(q, c, kr, an, kp, S, W, SCALE, BASE, True, dout)
    for name, x in out.items():
        lp.check(name, x, val[name], err[name])


def paged(terms):
    g = torch.Generator().manual_seed(31)
    q = rope_heavy(torch.randn(4, 40, 576, generator=g).to(torch.bfloat16), 512).double().numpy()
    k = torch.randn(300, 576, generator=g).to(torch.bfloat16).double().numpy()  # (the cache's keys are bf16 numbers)
    for i in range(4):
        x = np.concatenate([q[i, :, :512], ol.turn(q[i, :, 512:], np.full(40, 299), BASE)], -1)
        ro, eo, rz, ez = lp.fwd_block(x, k, 512, SCALE, True, extra=2.0 ** -20)
        p, z = ol._softmax(scores(x, k, 512, terms))
        lp.check("o", p @ k[:, :512], ro, eo)
        lp.check("lse", z, rz, ez)


ALL = ("hh", "lh", "hl")


def test_draft_split_keeps_the_bounds(tight):
    tight(SPLIT_BOTH)
    draft(ALL, ALL)


@pytest.mark.parametrize("gone", ["lh", "hl"])
@pytest.mark.parametrize("where", ["forward", "backward"])
def test_draft_a_product_left_out_does_not(gone, where, tight):
    tight(SPLIT_BOTH)
    less = tuple(t for t in ALL if t != gone)
    with pytest.raises(AssertionError):
        draft(less, less) if where == "forward" else draft(ALL, less)


def test_paged_split_keeps_the_bounds(tight):
    tight(SPLIT_QUERY)
    paged(("hh", "lh"))


def test_paged_the_remainder_left_out_does_not(tight):
    tight(SPLIT_QUERY)
    with pytest.raises(AssertionError):
        paged(("hh",))
