"""Waits of the long paged kernel do not grow with the context: a prompt over a million keys within limits of 20 ms."""
import numpy as np
import pytest
import torch

from oracle import latent as ol
from speculative_draft_mla_b200 import build as dbuild
from speculative_draft_mla_b200 import capi
from test_gpu_latent_cache import filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dbuild.build()
    return capi.load()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_tiles_that_take_longer_than_a_wait(kind):
    """80 tiles of 16384 steps, each longer than the limit: what waits for a tile's end has to allow for its steps."""
    page, n_pages, n_h, T, kv_len = 64, 32, 64, 160, 1 << 20
    cache, lat, rope = filled(41, kind, n_pages, page, 512, 64)
    g = torch.Generator().manual_seed(42)
    table = torch.randint(0, n_pages, (1, kv_len // page), generator=g, dtype=torch.int32)
    q = torch.randn(T, n_h, 576, generator=g).to(torch.bfloat16)
    args = (q.cuda(), cache, table.cuda(), torch.tensor([0, T], dtype=torch.int32).cuda(),
            torch.tensor([kv_len], dtype=torch.int32).cuda())
    want, wl, ws = capi.latent_attn_paged(*args)
    capi.get_error(ws)
    prev = capi.set_wait_limit_ns(20_000_000)
    try:
        o, lse, ws = capi.latent_attn_paged(*args)
        capi.get_error(ws)
    finally:
        capi.set_wait_limit_ns(prev)
    assert torch.equal(o, want) and torch.equal(lse, wl)
    # the last token sees every key: its 2048 rows of the cache, each as often as the table names its page
    often = np.repeat(np.bincount(table[0].numpy(), minlength=n_pages), page)
    k = np.concatenate([lat, rope], 1)
    x = q[-1].double().numpy()
    x = np.concatenate([x[:, :512], ol.turn(x[:, 512:], np.full(n_h, kv_len - 1), 10000.0)], -1)
    s = x @ k.T * capi.LATENT_SCALE
    m = s.max(-1, keepdims=True)
    e = np.exp(s - m) * often
    ref, rl = e / e.sum(-1, keepdims=True) @ lat, m[:, 0] + np.log(e.sum(-1))
    # fp32 sums of 16384 steps and 64 keys each, P rounded to bf16: 2^-8 and 2^14 2^-24 of the terms
    assert np.all(np.abs(lse[-1].double().cpu().numpy() - rl) <= 2.0 ** -9)
    assert np.all(np.abs(o[-1].double().cpu().numpy() - ref) <= 2.0 ** -7 * (e / e.sum(-1, keepdims=True) @ np.abs(lat)))
