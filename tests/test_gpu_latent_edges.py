"""The latent operators at their edges: waits that run out, calls at the same time on two streams, pages shared by
sequences, bounds of kv_len that choose other kernels, refused tensors."""
import pytest
import torch

import latent_parity as lp
from speculative_draft_mla_b200 import build as dbuild
from speculative_draft_mla_b200 import capi
from test_gpu_latent_attn import make, run
from test_gpu_latent_cache import filled, plan, reference

pytestmark = pytest.mark.gpu
ERR_DEVICE = 7


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dbuild.build()
    return capi.load()


def _runs_out(call):
    """call (returning its workspace) with waits of 1 ns: the device error, and only once. (A wait looks at the time
    after 64 polls of up to a few microseconds each; the sizes here make some wait for longer.)"""
    prev = capi.set_wait_limit_ns(1)
    try:
        ws = call()
        with pytest.raises(capi.DsparkError) as e:
            capi.get_error(ws)
        assert e.value.status == ERR_DEVICE
    finally:
        assert capi.set_wait_limit_ns(prev) == 1
    capi.get_error(ws)


def _close(a, b):
    # fp32 sums of tiles' contributions in any order, rounded to bf16
    a, b = a.float(), b.float()
    assert ((a - b).abs() <= torch.maximum(a.abs(), b.abs()) * 2.0 ** -7 + 1e-5).all()


def test_draft_waits_run_out_and_the_context_recovers():
    S, W = 300, 128
    t = make(5, 1, S, 300, 64, 512, 64, "bf16")
    before = run(t, S, W)
    d = {k: v.cuda() for k, v in t.items()}
    _runs_out(lambda: capi.latent_attn_fwd(d["q"], d["c"], d["kr"], d["an"], d["kp"], S, W)[2])

    def bwd():
        ws = capi.alloc_latent_workspace(capi.latent_problem(1, 64, S, 300, W), "cuda")
        capi.latent_attn_bwd(d["q"], d["c"], d["kr"], d["an"], d["kp"], before["lse"], d["dout"], S, W, workspace=ws)
        return ws

    _runs_out(bwd)
    after = run(t, S, W)
    for k in ("o", "lse", "dq"):
        assert torch.equal(before[k], after[k]), k
    for k in ("dc", "dkr"):
        _close(before[k], after[k])


@pytest.mark.parametrize("name,kind", [("long", "bf16"), ("short", "bf16"), ("short", "fp8")])
def test_paged_waits_run_out_and_the_context_recovers(name, kind):
    n_seq, q_len, kv_len, window = (2, 20, 120000, 0) if name == "long" else (300, 5, 200, 128)
    cache, _, _ = filled(72, kind, 64, 16, 512, 64)
    g = torch.Generator().manual_seed(73)
    table = torch.randint(0, 64, (n_seq, -(-kv_len // 16)), generator=g, dtype=torch.int32)
    qs = torch.arange(n_seq + 1, dtype=torch.int32) * q_len
    kv = torch.full((n_seq,), kv_len, dtype=torch.int32)
    q = torch.randn(n_seq * q_len, 64, 576, generator=g).to(torch.bfloat16).cuda()
    args = (q, cache, table.cuda(), qs.cuda(), kv.cuda())
    o, lse, ws = capi.latent_attn_paged(*args, window=window)
    capi.get_error(ws)
    _runs_out(lambda: capi.latent_attn_paged(*args, window=window)[2])
    o2, lse2, ws = capi.latent_attn_paged(*args, window=window)
    capi.get_error(ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("causal", [True, False])
def test_bounds_of_kv_len_choose_kernels_not_results(kind, causal):
    """Sequences of up to 144 keys without a window: by the table's width, by a bound, by a wrong bound."""
    q_lens, kv_lens, page, n_h = [1, 5, 0, 7, 144, 2], [144, 9, 33, 7, 144, 0], 16, 24
    n_pages, table, qs, kv = plan(81, q_lens, kv_lens, page)
    cache, lat, rope = filled(82, kind, n_pages, page, 512, 64)
    q = torch.randn(sum(q_lens), n_h, 576, generator=torch.Generator().manual_seed(83)).to(torch.bfloat16)
    val, err = reference(q.double().numpy(), lat, rope, table.numpy(), qs.numpy(), kv.numpy(), page,
                         capi.LATENT_SCALE, causal, 0, True)
    wide = torch.full((len(kv_lens), 40), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    for t, bound in ((table, 0), (table, 144), (wide, 0), (wide, 144), (wide, 20), (wide, 145)):
        o, lse, ws = capi.latent_attn_paged(q.cuda(), cache, t.cuda(), qs.cuda(), kv.cuda(), bound, causal=causal)
        capi.get_error(ws)
        lp.check("o", o, val["o"], err["o"])
        lp.check("lse", lse, val["lse"], err["lse"])


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("window", [0, 100])
def test_sequences_share_pages(kind, window):
    """A common beginning stored once, a page named twice within a sequence's table too."""
    page, n_h = 16, 16
    cache, lat, rope = filled(92, kind, 24, page, 512, 64)
    table = torch.tensor([[3, 7, 5, 11, 3, 9, 2, 1, 0, 20, 21, 8], [3, 7, 5, 11, 3, 9, 2, 1, 0, 22, 23, 4]],
                         dtype=torch.int32)
    qs, kv = torch.tensor([0, 3, 4], dtype=torch.int32), torch.tensor([190, 170], dtype=torch.int32)
    q = torch.randn(4, n_h, 576, generator=torch.Generator().manual_seed(93))
    q = q.to(torch.float32 if kind == "f32" else torch.bfloat16)
    val, err = reference(q.double().numpy(), lat, rope, table.numpy(), qs.numpy(), kv.numpy(), page,
                         capi.LATENT_SCALE, True, window, kind != "f32")
    o, lse, ws = capi.latent_attn_paged(q.cuda(), cache, table.cuda(), qs.cuda(), kv.cuda(), window=window)
    capi.get_error(ws)
    lp.check("o", o, val["o"], err["o"])
    lp.check("lse", lse, val["lse"], err["lse"])


def test_calls_at_the_same_time_on_two_streams():
    """Different problems of every operator, each stream with workspaces of its own."""
    S, W = 260, 100
    drafts = [make(100 + i, 1, S, 30 + i, 20 + 6 * i, 512, 64, "bf16") for i in range(2)]
    page = 16
    n_pages, table, qs, kv = plan(101, [2, 5], [300, 180], page)
    cache, _, _ = filled(102, "fp8", n_pages, page, 512, 64)
    q = [torch.randn(7, 64, 576, generator=torch.Generator().manual_seed(103 + i)).to(torch.bfloat16).cuda()
         for i in range(2)]
    args = (cache, table.cuda(), qs.cuda(), kv.cuda())

    def work(i):
        out = run(drafts[i], S, W)
        out["p"], out["pl"], ws = capi.latent_attn_paged(q[i], *args, window=130 * i)
        return out, ws

    alone = [work(i)[0] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    dev = [{k: v.cuda() for k, v in t.items()} for t in drafts]
    torch.cuda.synchronize()
    for rep in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                d = dev[i]
                o, lse, ws = capi.latent_attn_fwd(d["q"], d["c"], d["kr"], d["an"], d["kp"], S, W)
                dq, dc, dkr = capi.latent_attn_bwd(d["q"], d["c"], d["kr"], d["an"], d["kp"], lse, d["dout"], S, W,
                                                   workspace=ws, flags=capi.FLAG_REUSE_DESCRIPTOR)
                p, pl, pws = capi.latent_attn_paged(q[i], *args, window=130 * i)
                got[i] = dict(o=o, lse=lse, dq=dq, dc=dc, dkr=dkr, p=p, pl=pl, ws=ws, pws=pws)
        torch.cuda.synchronize()
        for i in range(2):
            capi.get_error(got[i].pop("ws"))
            capi.get_error(got[i].pop("pws"))
            for k, x in got[i].items():
                if k in ("dc", "dkr"):
                    _close(x, alone[i][k])
                else:
                    assert torch.equal(x, alone[i][k]), k


def test_repeated_tokens_or_heads_are_refused():
    cache = capi.latent_cache(4, 16)
    table = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    qs, kv = torch.tensor([0, 2], dtype=torch.int32).cuda(), torch.tensor([20], dtype=torch.int32).cuda()
    one = torch.zeros(1, 1, 576, dtype=torch.bfloat16, device="cuda")
    for q in (one.expand(2, 8, 576), one.expand(1, 8, 576), one.expand(2, 1, 576)):
        with pytest.raises(ValueError):
            capi.latent_attn_paged(q, cache, table, qs, kv)
    q = torch.zeros(2, 8, 576, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(1, 1, 512, dtype=torch.bfloat16, device="cuda").expand(2, 8, 512)
    with pytest.raises(ValueError):
        capi.latent_attn_paged(q, cache, table, qs, kv, out=(o, torch.zeros(2, 8, device="cuda")))


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
def test_nothing_to_do(kind):
    """No tokens, no sequences, no pages: calls that write what they have to and nothing else."""
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    cache, _, _ = filled(111, kind, 3, 8, 512, 64)
    before = cache.clone()
    i32 = dict(dtype=torch.int32, device="cuda")
    none = torch.empty(0, 64, 576, dtype=dt, device="cuda")
    o, lse, ws = capi.latent_attn_paged(none, cache, torch.zeros(2, 3, **i32), torch.zeros(3, **i32),
                                        torch.full((2,), 20, **i32))
    capi.get_error(ws)
    assert o.shape == (0, 64, 512) and lse.shape == (0, 64)
    q = torch.randn(4, 64, 576, device="cuda").to(dt)
    out = (torch.full((4, 64, 512), 3.0, dtype=dt, device="cuda"), torch.full((4, 64), 2.0, device="cuda"))
    _, _, ws = capi.latent_attn_paged(q, cache, torch.zeros(0, 3, **i32), torch.zeros(1, **i32),
                                      torch.zeros(0, **i32), out=out)
    capi.get_error(ws)
    assert bool((out[0] == 3).all()) and bool((out[1] == 2).all())
    # sequences without keys: zero rows
    no_pages = torch.empty((0, 8) + cache.shape[2:], dtype=cache.dtype, device="cuda")
    _, _, ws = capi.latent_attn_paged(q, no_pages, torch.zeros(2, 0, **i32), torch.tensor([0, 1, 4], **i32),
                                      torch.zeros(2, **i32), out=out)
    capi.get_error(ws)
    assert torch.count_nonzero(out[0]) == 0 and torch.isneginf(out[1]).all()
    # no rows, and rows of slots out of range
    empty = torch.empty(0, dtype=torch.int64, device="cuda")
    capi.latent_cache_write(cache, none[:, 0, :512].contiguous(), none[:, 0, 512:].contiguous(), empty.int(), empty)
    slots = torch.tensor([-1, 24, 1 << 40, -(1 << 40)], device="cuda")
    capi.latent_cache_write(cache, q[:, 0, :512].contiguous(), q[:, 0, 512:].contiguous(), slots.int(), slots)
    assert torch.equal(cache, before)
    c, kr = capi.latent_cache_read(cache, empty)
    assert c.shape == (0, 512) and kr.shape == (0, 64)
    c, kr = capi.latent_cache_read(cache, slots)
    assert torch.count_nonzero(c) == 0 and torch.count_nonzero(kr) == 0


@pytest.mark.parametrize("n_h", [100, 128, 129, 256])
@pytest.mark.parametrize("kind,window", [("bf16", 0), ("fp8", 90)])
def test_head_counts_around_a_tile(n_h, kind, window):
    """Heads that just fill a tile of rows, leave some, need one of the next chunk, or fill two."""
    q_lens, kv_lens, page = [2, 1], [170, 60], 16
    n_pages, table, qs, kv = plan(121, q_lens, kv_lens, page)
    cache, lat, rope = filled(122, kind, n_pages, page, 512, 64)
    q = torch.randn(3, n_h, 576, generator=torch.Generator().manual_seed(123)).to(torch.bfloat16)
    val, err = reference(q.double().numpy(), lat, rope, table.numpy(), qs.numpy(), kv.numpy(), page,
                         capi.LATENT_SCALE, True, window, True)
    o, lse, ws = capi.latent_attn_paged(q.cuda(), cache, table.cuda(), qs.cuda(), kv.cuda(), window=window)
    capi.get_error(ws)
    lp.check("o", o, val["o"], err["o"])
    lp.check("lse", lse, val["lse"], err["lse"])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,N", [(0, 3), (2, 0)])
def test_empty_batches(B, N, dt):
    S, n_h = 20, 64
    q = torch.zeros(B, n_h, 5 * N, 576, dtype=dt, device="cuda")
    c, kr = (torch.ones(B, S + 5 * N, d, dtype=dt, device="cuda") for d in (512, 64))
    an, kp = (torch.ones(B, N, dtype=t, device="cuda") for t in (torch.int32, torch.uint8))
    o, lse, ws = capi.latent_attn_fwd(q, c, kr, an, kp, S, 8)
    capi.get_error(ws)
    dq, dc, dkr = capi.latent_attn_bwd(q, c, kr, an, kp, lse, o, S, 8, workspace=ws)
    capi.get_error(ws)
    assert dq.shape == q.shape and torch.count_nonzero(dc) == 0 and torch.count_nonzero(dkr) == 0
