"""Values that are not finite in long sequences of the paged attention: they reach the rows that see them and no
others, and a call that meets them ends as any other call does. The waits of the kernels are limited to 20 ms here, a
hundred times what a step of a call of this size takes: work that keeps a kernel's other warps waiting shows as a
device error."""
import pytest
import torch

import latent_parity as lp
from speculative_draft_mla_b200 import build as dbuild
from speculative_draft_mla_b200 import capi
from test_gpu_latent_cache import filled, reference

pytestmark = pytest.mark.gpu
PAGE, N_PAGES, N_SEQ, Q_LEN, N_H = 64, 300, 16, 6, 64
BAD = 3                                                      # the sequence that holds the bad row
KV = [16384 - 701 * s for s in range(N_SEQ)]                 # 16384 .. 5869


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dbuild.build()
    return capi.load()


@pytest.fixture
def short_waits():
    prev = capi.set_wait_limit_ns(20_000_000)
    yield
    capi.set_wait_limit_ns(prev)


def problem(kind):
    """Sequences that share their pages, but for the bad sequence's first and last, which nobody else has."""
    cache, lat, rope = filled(7, kind, N_PAGES, PAGE, 512, 64)
    g = torch.Generator().manual_seed(8)
    table = torch.randint(0, N_PAGES - 2, (N_SEQ, KV[0] // PAGE), generator=g, dtype=torch.int32)
    last = (KV[BAD] - 1) // PAGE
    table[BAD, 0], table[BAD, last] = N_PAGES - 2, N_PAGES - 1
    q = torch.randn(N_SEQ * Q_LEN, N_H, 576, generator=g).to(torch.bfloat16)
    qs = torch.arange(N_SEQ + 1, dtype=torch.int32) * Q_LEN
    return cache, lat, rope, table, q, qs, torch.tensor(KV, dtype=torch.int32)


def slot(table, key):
    return int(table[BAD, key // PAGE]) * PAGE + key % PAGE


def spoil(cache, kind, at, value):
    row = cache.view(N_PAGES * PAGE, -1)[at]
    if kind == "fp8":
        row.fill_(0xff)  # NaN in e4m3, bf16 and fp32
    elif value == "nan":
        row.fill_(float("nan"))
    else:
        row[3] = float(value)


@pytest.mark.parametrize("kind,value", [("bf16", "nan"), ("bf16", "inf"), ("fp8", "nan")])
@pytest.mark.parametrize("where", ["own", "later token", "both"])
def test_one_bad_row_among_long_sequences(kind, value, where, short_waits):
    cache, lat, rope, table, q, qs, kv = problem(kind)
    args = (q.cuda(), cache, table.cuda(), qs.cuda(), kv.cuda())
    clean, cl, ws = capi.latent_attn_paged(*args)
    capi.get_error(ws)
    n = KV[BAD]
    if where != "later token":
        spoil(cache, kind, slot(table, 17), value)      # seen by all rows of the sequence
    if where != "own":
        spoil(cache, kind, slot(table, n - 1), value)   # seen by its last token, not by the one in the same tile
    out = torch.full_like(clean, 7.0), torch.full_like(cl, 7.0)
    o, lse, ws = capi.latent_attn_paged(*args, out=out)
    capi.get_error(ws)
    rows = slice(BAD * Q_LEN, (BAD + 1) * Q_LEN)
    others = torch.ones(N_SEQ * Q_LEN, dtype=torch.bool)
    others[rows] = False
    assert torch.equal(o[others], clean[others]) and torch.equal(lse[others], cl[others])
    free = 0 if where != "later token" else Q_LEN - 1   # tokens that see no bad row
    if free:
        val, err = reference(q[rows].double().numpy(), lat, rope, table[BAD:BAD + 1].numpy(), [0, Q_LEN], [n], PAGE,
                             capi.LATENT_SCALE, True, 0, True)
        lp.check("o", o[rows][:free], val["o"][:free], err["o"][:free])
        lp.check("lse", lse[rows][:free], val["lse"][:free], err["lse"][:free])
    if value == "nan":
        assert torch.isnan(o[rows][free:]).all() and torch.isnan(lse[rows][free:]).all()
    else:
        # A score of +inf leaves no softmax (NaN); one of -inf has weight 0, and 0 x inf only in its own column.
        s = q[rows][free:, :, 3].float()
        up, down = s > 0, s < 0
        got, gl = o[rows][free:].float().cpu(), lse[rows][free:].cpu()
        assert torch.isnan(got[up]).all() and torch.isnan(gl[up]).all()
        rest = [c for c in range(512) if c != 3]
        assert torch.isfinite(got[down][:, rest]).all() and torch.isfinite(gl[down]).all()
        assert torch.isnan(got[down][:, 3]).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_a_bad_row_at_the_beginning_of_a_window(kind, short_waits):
    """The first token's window begins with it, the second's, in the same tile, behind it."""
    cache, lat, rope, table, q, qs, kv = problem(kind)
    n, window = KV[BAD], 1000
    key = n - Q_LEN - window + 1
    table[BAD, key // PAGE] = N_PAGES - 2
    spoil(cache, kind, slot(table, key), "nan")
    o, lse, ws = capi.latent_attn_paged(q.cuda(), cache, table.cuda(), qs.cuda(), kv.cuda(), window=window)
    capi.get_error(ws)
    for s in range(N_SEQ):
        a = s * Q_LEN
        val, err = reference(q[a:a + Q_LEN].double().numpy(), lat, rope, table[s:s + 1].numpy(), [0, Q_LEN], KV[s:s + 1],
                             PAGE, capi.LATENT_SCALE, True, window, True)
        if s == BAD:
            assert torch.isnan(o[a]).all() and torch.isnan(lse[a]).all()
        f = 1 if s == BAD else 0
        lp.check("o", o[a + f:a + Q_LEN], val["o"][f:], err["o"][f:])
        lp.check("lse", lse[a + f:a + Q_LEN], val["lse"][f:], err["lse"][f:])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_rows_of_two_calls_with_a_bad_row_are_the_same(kind, short_waits):
    cache, _, _, table, q, qs, kv = problem(kind)
    spoil(cache, kind, slot(table, KV[BAD] - 3), "nan")
    args = (q.cuda(), cache, table.cuda(), qs.cuda(), kv.cuda())
    o, lse, ws = capi.latent_attn_paged(*args)
    for _ in range(3):
        o2, lse2, _ = capi.latent_attn_paged(*args, workspace=ws)
        capi.get_error(ws)
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16))
        assert torch.equal(lse.view(torch.int32), lse2.view(torch.int32))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_a_bad_row_in_a_prompt(kind, short_waits):
    """Tiles that one pair works on alone, and more of them than pairs: half of the tokens see the bad row."""
    page, n_h, n, kv_len = 16, 32, 900, 1000
    cache, lat, rope = filled(17, kind, 63, page, 512, 64)
    g = torch.Generator().manual_seed(18)
    table = torch.randperm(63, generator=g).to(torch.int32)[None]
    q = torch.randn(n, n_h, 576, generator=g).to(torch.bfloat16)
    key = 550
    at = int(table[0, key // page]) * page + key % page
    cache.view(63 * page, -1)[at] = 0xff if kind == "fp8" else float("nan")
    qs, kv = torch.tensor([0, n], dtype=torch.int32), torch.tensor([kv_len], dtype=torch.int32)
    o, lse, ws = capi.latent_attn_paged(q.cuda(), cache, table.cuda(), qs.cuda(), kv.cuda())
    capi.get_error(ws)
    first = key - (kv_len - n)  # the first token that sees it
    assert torch.isnan(o[first:]).all() and torch.isnan(lse[first:]).all()
    assert torch.isfinite(o[:first].float()).all() and torch.isfinite(lse[:first]).all()
    near = slice(first - 8, first)  # tokens whose tile holds rows that see it, and some beside
    val, err = reference(q[near].double().numpy(), lat, rope, table.numpy(), [0, 8], [key], page, capi.LATENT_SCALE,
                         True, 0, True)
    lp.check("o", o[near], val["o"], err["o"])
    lp.check("lse", lse[near], val["lse"], err["lse"])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("n_seq", [2, 200])
def test_a_bad_row_in_the_short_kernel(kind, n_seq):
    """Windows that keep sequences within 144 keys, more sequences than CTAs too: a token's own row is bad, the token
    beside it in its tile does not see it, the later ones do. Limits of 3 ms, for calls of less than 0.1."""
    page, n_h, q_len, window, kv_len, hit = 16, 64, 20, 100, 300, 5
    n_pages, per = 80 + n_seq * 3, -(-kv_len // page)
    cache, lat, rope = filled(27, kind, n_pages, page, 512, 64)
    g = torch.Generator().manual_seed(28)
    table = torch.randint(0, 80, (n_seq, per), generator=g, dtype=torch.int32)
    table[:, -3:] = 80 + torch.arange(3 * n_seq, dtype=torch.int32).view(n_seq, 3)  # the new tokens' pages
    q = torch.randn(n_seq * q_len, n_h, 576, generator=g).to(torch.bfloat16)
    qs = torch.arange(n_seq + 1, dtype=torch.int32) * q_len
    kv = torch.full((n_seq,), kv_len, dtype=torch.int32)
    key = kv_len - q_len + hit
    rows = cache.view(n_pages * page, -1)
    spoiled = list(range(0, n_seq, 2))
    for s in spoiled:
        rows[int(table[s, key // page]) * page + key % page] = 0xff if kind == "fp8" else float("nan")
    prev = capi.set_wait_limit_ns(3_000_000)
    try:
        o, lse, ws = capi.latent_attn_paged(q.cuda(), cache, table.cuda(), qs.cuda(), kv.cuda(), window=window)
        capi.get_error(ws)
    finally:
        capi.set_wait_limit_ns(prev)
    for s in (0, 1, n_seq - 2, n_seq - 1):
        a = s * q_len
        val, err = reference(q[a:a + q_len].double().numpy(), lat, rope, table[s:s + 1].numpy(), [0, q_len], [kv_len], page,
                             capi.LATENT_SCALE, True, window, True)
        free = hit if s in spoiled else q_len
        lp.check("o", o[a:a + free], val["o"][:free], err["o"][:free])
        lp.check("lse", lse[a:a + free], val["lse"][:free], err["lse"][:free])
        assert torch.isnan(o[a + free:a + q_len]).all() and torch.isnan(lse[a + free:a + q_len]).all()
