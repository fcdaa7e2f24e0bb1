"""Sequences of the paged attention that q_start gets wrong: they attend nothing and are reported, the others are as
without them."""
import pytest
import torch

import latent_parity as lp
from speculative_draft_mla_b200 import build as dbuild
from speculative_draft_mla_b200 import capi
from test_gpu_latent_cache import filled, reference

pytestmark = pytest.mark.gpu
ERR_PAGE = 10
PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dbuild.build()
    return capi.load()


def reported(ws):
    with pytest.raises(capi.DsparkError) as e:
        capi.get_error(ws)
    assert e.value.status == ERR_PAGE
    capi.get_error(ws)


# q_start, T, sequences that attend
WRONG = {
    "one range three times, then another": ([0, 8, 0, 8, 0, 8, 12], 12, (0, 5)),
    "begins within an earlier one": ([0, 4, 2, 6, 9], 9, (0, 3)),
    "within one that is refused": ([0, 5, 3, 8, 6, 9, 11], 11, (0, 5)),
    "past the tokens": ([0, 3, 20, 3, 6], 6, (0, 3)),
    "negative": ([-2, 3, 5], 5, (1,)),
    "an empty one above": ([5, 5, 0, 3], 5, (2,)),
}


@pytest.mark.parametrize("kv_len,window", [(60, 0), (300, 0), (300, 40), (300, 145)])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("name", sorted(WRONG))
def test_wrong_starts_leave_the_others(name, kind, kv_len, window):
    starts, T, good = WRONG[name]
    n, n_h = len(starts) - 1, 64
    per = -(-kv_len // PAGE)
    cache, lat, rope = filled(5, kind, 40, PAGE, 512, 64)
    g = torch.Generator().manual_seed(6)
    table = torch.randint(0, 40, (n, per), generator=g, dtype=torch.int32).cuda()
    q = torch.randn(T, n_h, 576, generator=g).to(torch.float32 if kind == "f32" else torch.bfloat16).cuda()
    kv = (kv_len - torch.arange(n, dtype=torch.int32)).cuda()
    out = torch.full((T, n_h, 512), 5.0, dtype=q.dtype, device="cuda"), torch.full((T, n_h), 9.0, device="cuda")
    o, lse, ws = capi.latent_attn_paged(q, cache, table, torch.tensor(starts, dtype=torch.int32).cuda(), kv,
                                        window=window, out=out)
    reported(ws)
    left = torch.ones(T, dtype=torch.bool)
    for s in good:
        a, b = starts[s], starts[s + 1]
        left[a:b] = False
        val, err = reference(q[a:b].double().cpu().numpy(), lat, rope, table[s:s + 1].cpu().numpy(), [0, b - a],
                             kv[s:s + 1].cpu().numpy(), PAGE, capi.LATENT_SCALE, True, window, kind != "f32")
        lp.check("o", o[a:b], val["o"], err["o"])
        lp.check("lse", lse[a:b], val["lse"], err["lse"])
    assert bool((o[left] == 5).all()) and bool((lse[left] == 9).all())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["behind a thousand", "empty ones first"])
def test_wrong_starts_far_down_the_list(name, kind):
    """More sequences than the plan's threads: what came before is carried on."""
    if name == "behind a thousand":
        starts, good = list(range(1031)) + [500, 503, 1030, 1033], list(range(1030)) + [1033]
    else:
        starts, good = [5] * 1030 + [0, 3, 3, 4, 5], [1030, 1032, 1033]
    n, T, n_h = len(starts) - 1, max(starts), 3
    cache, lat, rope = filled(15, kind, 12, PAGE, 512, 64)
    g = torch.Generator().manual_seed(16)
    table = torch.randint(0, 12, (n, 10), generator=g, dtype=torch.int32)
    q = torch.randn(T, n_h, 576, generator=g).to(torch.float32 if kind == "f32" else torch.bfloat16)
    kv = torch.randint(1, 30, (n,), generator=g, dtype=torch.int32)
    out = torch.full((T, n_h, 512), 5.0, dtype=q.dtype, device="cuda"), torch.full((T, n_h), 9.0, device="cuda")
    o, lse, ws = capi.latent_attn_paged(q.cuda(), cache, table.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(),
                                        kv.cuda(), out=out)
    reported(ws)
    left = torch.ones(T, dtype=torch.bool)
    for s in good:
        a, b = starts[s], starts[s + 1]
        left[a:b] = False
        if a % 97 and s + 4 < n:
            continue
        val, err = reference(q[a:b].double().numpy(), lat, rope, table[s:s + 1].numpy(), [0, b - a], kv[s:s + 1].numpy(),
                             PAGE, capi.LATENT_SCALE, True, 0, kind != "f32")
        lp.check("o", o[a:b], val["o"], err["o"])
        lp.check("lse", lse[a:b], val["lse"], err["lse"])
    assert bool((o[left] == 5).all()) and bool((lse[left] == 9).all()) and not bool((lse[~left] == 9).any())


def test_ranges_repeated_until_their_tiles_pass_32_bits():
    """2^17 sequences over the same 128 tokens of 16385 heads: 2.2e9 row tiles if all of them attended. The first does."""
    T, n_h, n, kv_len = 128, 16385, 1 << 18, 150
    cache, lat, rope = filled(9, "bf16", 10, PAGE, 512, 64)
    q = torch.randn(T, n_h, 576, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(10, dtype=torch.int32, device="cuda").repeat(n, 1)
    starts = torch.tensor([0, T], dtype=torch.int32).repeat(n // 2 + 1)[:n + 1].cuda()
    kv = torch.full((n,), kv_len, dtype=torch.int32, device="cuda")
    o, lse, ws = capi.latent_attn_paged(q, cache, table, starts, kv)
    reported(ws)
    heads = [0, 1, 127, 128, 8191, 16383, 16384]
    val, err = reference(q[:, heads].double().cpu().numpy(), lat, rope, table[:1].cpu().numpy(), [0, T], [kv_len], PAGE,
                         capi.LATENT_SCALE, True, 0, True)
    lp.check("o", o[:, heads], val["o"], err["o"])
    lp.check("lse", lse[:, heads], val["lse"], err["lse"])
