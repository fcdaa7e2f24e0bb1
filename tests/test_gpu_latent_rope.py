"""Scores that their rope part makes up: what the split of the turned slices into hi + lo of two bf16 promises.

With u = 2^-8 a turned value is hi + lo to u^2 of it; the draft attention forms hi hi + lo hi + hi lo, so that a score
is off by 3 u^2 = 3 2^-16 of its sum of |q_r||k_r|, where one bf16 for each slice would leave up to 2 u. Over the cache
the keys are exact operands: u^2. The bounds of latent_parity allow 2 u + u^2; here they are taken with these instead.
In fp32 kernels (other widths) the turns are not split at all, which the same bounds hold for.

With queries' rope slices six times the rest, dropping one lo moves a score by 4e-3 or so and the LSE with it; the
bound is 1e-3."""
import pytest
import torch

import latent_parity as lp
from speculative_draft_mla_b200 import build as dbuild
from speculative_draft_mla_b200 import capi
from test_gpu_latent_attn import compare, make, run
from test_gpu_latent_cache import filled, plan, reference

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
SPLIT_BOTH, SPLIT_QUERY = 3 * U * U - (2 * U + U * U), U * U - (2 * U + U * U)


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dbuild.build()
    return capi.load()


@pytest.fixture
def tight(monkeypatch):
    """Takes the allowance for the rope slices' operands: from 2 u + u^2 to that plus the given."""
    def take(change):
        loose = lp._weights
        monkeypatch.setattr(lp, "_weights", lambda *a, extra=0.0, **kw: loose(*a, extra=extra + change, **kw))
    return take


def rope_heavy(q, d_l):
    q[..., :d_l] *= 1 / 16
    q[..., d_l:] *= 6
    return q


# S, N, W, n_h, d_l, d_r
@pytest.mark.parametrize("S,N,W,n_h,d_l,d_r", [(300, 12, 128, 23, 512, 64), (90, 6, 30, 64, 512, 64),
                                               (300, 4, 150, 5, 512, 64), (70, 5, 20, 4, 64, 32)])
def test_draft_attention(S, N, W, n_h, d_l, d_r, tight):
    t = make(S, 1, S, N, n_h, d_l, d_r, "bf16")
    rope_heavy(t["q"], d_l)
    tight(SPLIT_BOTH)
    compare(t, run(t, S, W), S, W)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 128), (True, 300)])
def test_paged_attention(kind, causal, window, tight):
    q_lens, kv_lens, page, n_h = [5, 1, 9], [700, 133, 260], 16, 40
    n_pages, table, qs, kv = plan(11, q_lens, kv_lens, page)
    cache, lat, rope = filled(12, kind, n_pages, page, 512, 64)
    q = rope_heavy(torch.randn(15, n_h, 576, generator=torch.Generator().manual_seed(13)).to(torch.bfloat16), 512)
    tight(SPLIT_QUERY)
    val, err = reference(q.double().numpy(), lat, rope, table.numpy(), qs.numpy(), kv.numpy(), page, capi.LATENT_SCALE,
                         causal, window, True)
    o, lse, ws = capi.latent_attn_paged(q.cuda(), cache, table.cuda(), qs.cuda(), kv.cuda(), causal=causal,
                                        window=window)
    capi.get_error(ws)
    lp.check("o", o, val["o"], err["o"])
    lp.check("lse", lse, val["lse"], err["lse"])


def test_rope_key_gradient_of_queries_that_cancel():
    """dS exact and equal in three heads, whose queries' rope slices are x, 2.5 x and -3.5 x: the rope keys' gradients
    are 0, and what is left of them shows how the queries were rounded: u^2 of the terms as hi + lo (and fp32 sums and
    turns, 24 units), u with hi alone, 2^-9 of each term on the average.

    Keys' rope slices of 0 make all scores 0: over 8 keys (W = 4) P = 1 / 8. dO = (1, 0, ..) and latents (a_p, 0, ..)
    with the mean of a_p over a block's keys 0 make dP = a_p, D = 0, dS = scale a_p / 8, exact in bf16."""
    S, N, W, H = 64, 3, 4, 3
    g = torch.Generator().manual_seed(21)
    # five bits of mantissa, so that 2.5 x and 3.5 x are bf16 numbers
    x = torch.randint(16, 32, (1, 1, 5 * N, 64), generator=g).float() * 2.0 ** torch.randint(-5, -2, (1, 1, 5 * N, 64),
                                                                                             generator=g)
    x *= torch.randint(0, 2, x.shape, generator=g) * 2 - 1
    q = torch.zeros(1, H, 5 * N, 576)
    for h, f in enumerate((1.0, 2.5, -3.5)):
        q[:, h:h + 1, :, 512:] = f * x
    assert torch.equal(q, q.to(torch.bfloat16).float())
    anchors = [20, 40, 62]
    c = torch.zeros(1, S + 5 * N, 512)
    for n, a in enumerate(anchors):
        c[0, a - 3:a, 0] = torch.tensor([1.0, -2.0, 3.0])
        c[0, S + 5 * n:S + 5 * n + 5, 0] = torch.tensor([2.0, -1.0, -3.0, 1.0, -1.0])
    kr = torch.zeros(1, S + 5 * N, 64)
    dout = torch.zeros(1, H, 5 * N, 512)
    dout[..., 0] = 1
    d = [t.to(torch.bfloat16).cuda() for t in (q, c, kr)]
    an, kp = torch.tensor([anchors], dtype=torch.int32).cuda(), torch.ones(1, N, dtype=torch.uint8).cuda()
    o, lse, ws = capi.latent_attn_fwd(*d, an, kp, S, W)
    assert torch.allclose(lse, torch.full_like(lse, 3 * 0.6931471805599453), rtol=2.0 ** -22, atol=0)
    dq, dc, dkr = capi.latent_attn_bwd(*d, an, kp, lse, dout.to(torch.bfloat16).cuda(), S, W, workspace=ws)
    capi.get_error(ws)
    # terms of a key: dS of its block's 15 rows (5 offsets, 3 heads) times both elements of a pair, both ways
    pair = (x[..., 0::2].abs() + x[..., 1::2].abs()).repeat_interleave(2, -1)
    pair = (pair[..., 0::2] + pair[..., 1::2]).repeat_interleave(2, -1)[0, 0].view(N, 5, 64).sum(1) * 7.0
    bound = torch.zeros(1, S + 5 * N, 64)
    for n, a in enumerate(anchors):
        for keys in (slice(a - 3, a), slice(S + 5 * n, S + 5 * n + 5)):
            ds = capi.LATENT_SCALE / 8 * c[0, keys, :1].abs()
            bound[0, keys] = ds * pair[n] * (U * U + 24 * 2.0 ** -24)
    assert (dkr.float().cpu().abs() <= bound).all(), (dkr.float().cpu().abs() / bound.clamp_min(1e-30)).max()
    # one head alone has the gradient
    only = [d[0][:, :1].contiguous(), d[1], d[2]]
    _, l1, ws = capi.latent_attn_fwd(*only, an, kp, S, W)
    _, _, dk1 = capi.latent_attn_bwd(*only, an, kp, l1, dout[:, :1].contiguous().to(torch.bfloat16).cuda(), S, W,
                                     workspace=ws)
    assert dk1.float().abs().max() > 100 * bound.max()
