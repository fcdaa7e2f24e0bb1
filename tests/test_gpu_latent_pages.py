"""Pages and lengths that are out of range, in every kernel of the paged attention: the keys of such pages are skipped
and reported, the other sequences are as without them. The long kernel brings keys in steps of 64, in groups of 8
where pages hold whole groups and row by row elsewhere, and shares a sequence's steps between pairs of CTAs; the short
one takes sequences of up to 144 keys."""
import numpy as np
import pytest
import torch

import latent_parity as lp
from oracle import latent as ol
from speculative_draft_mla_b200 import build as dbuild
from speculative_draft_mla_b200 import capi
from test_gpu_latent_cache import filled, plan

pytestmark = pytest.mark.gpu
ERR_PAGE = 10
BASE = 10000.0


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dbuild.build()
    return capi.load()


def expected(q, lat, rope, table, n_pages, page, ctx, kv, bf16):
    """Rows q [n, n_h, 576] of one sequence at positions ctx .. over its keys on pages within range (causal)."""
    out = []
    for i in range(q.shape[0]):
        p = np.arange(min(ctx + i + 1, kv))
        p = p[(table[p // page] >= 0) & (table[p // page] < n_pages)]
        if p.size == 0:
            z = np.zeros((q.shape[1], 512))
            out.append((z, z, np.full(q.shape[1], -np.inf), np.zeros(q.shape[1])))
            continue
        slot = table[p // page].astype(np.int64) * page + p % page
        k = np.concatenate([lat[slot], rope[slot]], 1)
        x = np.concatenate([q[i, :, :512], ol.turn(q[i, :, 512:], np.full(q.shape[1], ctx + i), BASE)], -1)
        out.append(lp.fwd_block(x, k, 512, capi.LATENT_SCALE, bf16, extra=2.0 ** -20))
    return [np.stack(t) for t in zip(*out)]


# q_lens, kv_lens, {sequence: pages of its table that are bad}
LAYOUTS = {
    "short": ([2, 3, 1], [140, 90, 33], {0: (1, 8), 1: (5,)}),
    "long": ([2, 6, 1, 3], [700, 333, 90, 200], {0: (1, 9, 43), 1: (20,), 3: (0, 12)}),
    "one long sequence": ([1], [3000], {0: (0, 37, 38, 39, 100, 187)}),
    "every page": ([3, 2], [400, 300], {0: tuple(range(25))}),
}


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_bad_pages(name, page, kind):
    q_lens, kv_lens, bad = LAYOUTS[name]
    n_h = 24
    n_pages, table, qs, kv = plan(3, q_lens, kv_lens, page, 1)
    cache, lat, rope = filled(4, kind, n_pages, page, 512, 64)
    T = sum(q_lens)
    q = torch.randn(T, n_h, 576, generator=torch.Generator().manual_seed(5))
    q = q.to(torch.float32 if kind == "f32" else torch.bfloat16)
    wrong = [n_pages, -1, 2 ** 31 - 1, -2 ** 31, n_pages + 3, -17]
    worse = table.clone()
    for s, pages in bad.items():
        for j, at in enumerate(pages if name == "every page" and page == 16 else [x * 16 // page for x in pages]):
            worse[s, at] = wrong[j % len(wrong)]
        if name == "every page":
            worse[s, :] = -1
    clean, cl, ws = capi.latent_attn_paged(q.cuda(), cache, table.cuda(), qs.cuda(), kv.cuda())
    capi.get_error(ws)
    o, lse, ws = capi.latent_attn_paged(q.cuda(), cache, worse.cuda(), qs.cuda(), kv.cuda(), workspace=ws)
    with pytest.raises(capi.DsparkError) as e:
        capi.get_error(ws)
    assert e.value.status == ERR_PAGE
    for s, (n, k) in enumerate(zip(q_lens, kv_lens)):
        a, b = int(qs[s]), int(qs[s + 1])
        if s not in bad:
            assert torch.equal(o[a:b], clean[a:b]) and torch.equal(lse[a:b], cl[a:b])
        ro, eo, rz, ez = expected(q[a:b].double().numpy(), lat, rope, worse[s].numpy(), n_pages, page, k - n, k,
                                  kind != "f32")
        lp.check("o", o[a:b], ro, eo)
        lp.check("lse", lse[a:b], rz, ez)
    # the workspace serves the next call
    o, lse, ws = capi.latent_attn_paged(q.cuda(), cache, table.cuda(), qs.cuda(), kv.cuda(), workspace=ws)
    capi.get_error(ws)
    assert torch.equal(o, clean) and torch.equal(lse, cl)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("wrong", [-1, -2 ** 31, 801, 2 ** 31 - 1])
def test_bad_lengths_in_a_wide_table(wrong, kind):
    q_lens, kv_lens, page, n_h = [2, 3, 1], [800, 500, 300], 16, 24
    n_pages, table, qs, kv = plan(6, q_lens, kv_lens, page, 1)
    cache, _, _ = filled(7, kind, n_pages, page, 512, 64)
    q = torch.randn(6, n_h, 576, generator=torch.Generator().manual_seed(8))
    q = q.to(torch.float32 if kind == "f32" else torch.bfloat16).cuda()
    kv[1] = 0
    clean, cl, ws = capi.latent_attn_paged(q, cache, table.cuda(), qs.cuda(), kv.cuda())
    capi.get_error(ws)
    kv[1] = wrong
    out = torch.full_like(clean, 3.0), torch.full_like(cl, 3.0)
    o, lse, ws = capi.latent_attn_paged(q, cache, table.cuda(), qs.cuda(), kv.cuda(), out=out)
    with pytest.raises(capi.DsparkError) as e:
        capi.get_error(ws)
    assert e.value.status == ERR_PAGE
    assert torch.count_nonzero(o[2:5]) == 0 and torch.isneginf(lse[2:5]).all()
    assert torch.equal(o, clean) and torch.equal(lse, cl)  # (steps are shared out as for a length of 0)
