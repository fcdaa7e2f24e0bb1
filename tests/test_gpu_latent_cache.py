"""The paged latent cache (write, read) and the attention over it, on the GPU against the fp64 oracle.

Written rows: the norm is formed in 64 bits and rounded once, so 16- and 8-bit rows are the nearest values of the
oracle's rows. The oracle's own 64-bit sum may differ in its last bits, which moves a value across a rounding
border only when it lies within 2^-40 of it: such values may take either neighbour.
"""
import numpy as np
import pytest
import torch

import latent_parity as lp
from oracle import latent as ol
from speculative_draft_mla_b200 import build as dbuild
from speculative_draft_mla_b200 import capi

pytestmark = pytest.mark.gpu
BASE = 10000.0
KINDS = {"f32": capi.CACHE_F32, "bf16": capi.CACHE_BF16, "fp8": capi.CACHE_FP8}


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dbuild.build()
    return capi.load()


def to_bf16(x):
    """fp64 to bf16, rounded once (through fp32 with the lost bits kept sticky)."""
    x = np.asarray(x, np.float64)
    f = x.astype(np.float32)
    with np.errstate(invalid="ignore"):
        toward = np.where(np.abs(f.astype(np.float64)) > np.abs(x), np.nextafter(f, np.float32(0)), f)
    bits = toward.view(np.uint32) | (toward.astype(np.float64) != x).astype(np.uint32)
    return torch.from_numpy(bits.view(np.float32).copy()).to(torch.bfloat16)


def near(got, want, exact, what):
    """Equal, or one of the neighbours when the value sits on a rounding border."""
    g, w = np.asarray(got, np.float64), np.asarray(want, np.float64)
    same = (g == w) | (np.isnan(g) & np.isnan(w))
    if same.all():
        return
    mid = (g + w) / 2
    assert np.all(np.abs(exact - mid)[~same] <= 2.0 ** -40 * np.abs(exact)[~same]), what


def rows_of(kind, seed, T, d_l, d_r, dtype):
    g = torch.Generator().manual_seed(seed)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    c = (torch.randn(T, d_l, generator=g) * 3).to(dt)
    kr = torch.randn(T, d_r, generator=g).to(dt)
    w = (1 + 0.1 * torch.randn(d_l, generator=g)).to(dt)
    pos = torch.randint(0, 200000, (T,), generator=g, dtype=torch.int32)
    return c, kr, w, pos


# T, n_pages, page_size, d_l, d_r
SIZES = [(1, 1, 1, 512, 64), (7, 3, 4, 512, 64), (131, 20, 16, 512, 64), (9, 4, 5, 128, 8), (5, 2, 3, 384, 0),
         (33, 3, 64, 256, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("size", SIZES)
def test_write_and_read(size, kind, norm, dtype):
    T, n_pages, page, d_l, d_r = size
    c, kr, w, pos = rows_of(kind, T + d_l, T, d_l, d_r, dtype)
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int64)
    T = slots.numel()
    c, kr, pos = c[:T], kr[:T], pos[:T]
    if T > 3:
        slots[1], slots[2] = -1, n_pages * page  # padded tokens
        c[1], c[2] = float("nan"), float("inf")
    cache = capi.latent_cache(n_pages, page, d_l, d_r, KINDS[kind])
    cache.view(torch.uint8).fill_(0x5a)
    before = cache.cpu().clone()
    capi.latent_cache_write(cache, c.cuda(), kr.cuda(), pos.cuda(), slots.cuda(),
                            norm_weight=w.cuda() if norm else None, eps=1e-5)
    ok = ((slots >= 0) & (slots < n_pages * page)).numpy()
    # rows that no token names stay as they were
    after = cache.cpu().view(n_pages * page, -1)
    other = np.ones(n_pages * page, bool)
    other[slots.numpy()[ok]] = False
    assert torch.equal(after[other].view(torch.uint8), before.view(n_pages * page, -1)[other].view(torch.uint8))
    for out_dt in (torch.float32, torch.bfloat16):
        cg, kg = capi.latent_cache_read(cache, slots.cuda(), d_l, d_r, dtype=out_dt)
        assert torch.count_nonzero(cg[~ok]) == 0 and torch.count_nonzero(kg[~ok]) == 0
        y = ol.norm_rows(c.double().numpy()[ok], w.double().numpy() if norm else None, 1e-5)
        r = ol.turn(kr.double().numpy()[ok], pos.numpy()[ok], BASE)
        cg, kg = cg.cpu()[ok], kg.cpu()[ok]
        if kind == "fp8":
            near(cg.double().numpy(), ol.fp8_round(y)[0], y, "fp8 rows")
        elif kind == "bf16" or out_dt == torch.bfloat16:
            # f32 rows read as bf16 are rounded twice: half a step of each
            if kind == "bf16":
                near(cg.double().numpy(), to_bf16(y).double().numpy(), y, "bf16 rows")
            else:
                assert np.all(np.abs(cg.double().numpy() - y) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(y))
        else:
            assert np.all(np.abs(cg.double().numpy() - y) <= 2.0 ** -24 * np.abs(y))
        # the turn is formed in fp32 from an angle brought into [-pi, pi] in 64 bits: the angle's rounding, sine
        # and cosine (2 units) and the two products give 8 * 2^-24 of the pair's size
        half = 2.0 ** -24 if kind == "f32" and out_dt == torch.float32 else 2.0 ** -8
        size_ = lp._pairmax(np.abs(kr.double().numpy()[ok]))
        assert np.all(np.abs(kg.double().numpy() - r) <= half * np.abs(r) * 1.001 + 8 * 2.0 ** -24 * size_ + (
            2.0 ** -24 * size_ if kind == "f32" else 0))


def test_fp8_special_values():
    """Zeros, subnormal and huge groups, ties, values that are not finite."""
    c = torch.zeros(6, 512)
    c[1, :128] = torch.linspace(-1, 1, 128) * 1e30
    c[1, 128:256] = torch.linspace(-1, 1, 128) * 1e-38
    c[1, 256:384] = 2.0 ** -120
    c[2] = torch.arange(512).float() - 256.5           # ties among them
    c[3, 5], c[3, 130], c[3, 260] = float("nan"), float("inf"), float("-inf")
    c[3, 6], c[3, 131] = 3.0, -2.0
    c[4] = 448.0
    c[5] = torch.nextafter(torch.tensor(448.0), torch.tensor(1e9))
    kr = torch.zeros(6, 64)
    cache = capi.latent_cache(1, 8, kind=capi.CACHE_FP8)
    slots = torch.arange(6).cuda()
    capi.latent_cache_write(cache, c.cuda(), kr.cuda(), torch.zeros(6, dtype=torch.int32).cuda(), slots)
    cg, _ = capi.latent_cache_read(cache, slots, dtype=torch.float32)
    want, sc = ol.fp8_round(c.double().numpy())
    assert np.array_equal(cg.cpu().double().numpy(), want, equal_nan=True)
    rows = cache.cpu().view(8, -1)[:6]
    assert np.array_equal(rows[:, 640:656].contiguous().view(torch.float32).double().numpy(), sc)
    # a second write of what was read gives the same bytes: the values it stands for are kept exactly
    fin = torch.tensor([0, 1, 2, 4, 5])
    cache2 = capi.latent_cache(1, 8, kind=capi.CACHE_FP8)
    capi.latent_cache_write(cache2, cg[fin.cuda()].contiguous(), kr[fin].cuda(), torch.zeros(5, dtype=torch.int32).cuda(),
                            slots[fin.cuda()])
    c2, _ = capi.latent_cache_read(cache2, slots[fin.cuda()], dtype=torch.float32)
    assert torch.equal(c2, cg[fin.cuda()])


def test_rows_of_a_long_cache():
    """Slots whose byte offset passes 2^32."""
    n_pages = 60000  # x 64 rows x 1152 B = 4.4 GB
    cache = torch.empty(n_pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    cache[0].fill_(7.0)
    c, kr, w, pos = rows_of("bf16", 5, 40, 512, 64, "bf16")
    slots = torch.arange(n_pages * 64 - 40, n_pages * 64).cuda()
    capi.latent_cache_write(cache, c.cuda(), kr.cuda(), pos.cuda(), slots)
    assert torch.equal(cache.view(-1, 576)[-40:, :512].cpu(), c)
    cg, _ = capi.latent_cache_read(cache, slots)
    assert torch.equal(cg.cpu(), c)
    assert bool((cache[0] == 7).all())
    # attention over pages at both ends of it
    q = torch.randn(2, 64, 576, device="cuda").to(torch.bfloat16)
    cache[-2].normal_()
    cache[-1, :, 512:].normal_()
    cache[-1, :24, :512].normal_()
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device="cuda")
    qs, kv = torch.tensor([0, 2], dtype=torch.int32).cuda(), torch.tensor([100], dtype=torch.int32).cuda()
    o, lse, ws = capi.latent_attn_paged(q, cache, table, qs, kv)
    capi.get_error(ws)
    low = cache[-2:].clone()
    o2, lse2, _ = capi.latent_attn_paged(q, low, table - (n_pages - 2), qs, kv)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


# ---- attention over the cache ------------------------------------------------------------------
def filled(seed, kind, n_pages, page, d_l, d_r):
    g = torch.Generator().manual_seed(seed)
    n = n_pages * page
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    cache = capi.latent_cache(n_pages, page, d_l, d_r, KINDS[kind])
    capi.latent_cache_write(cache, torch.randn(n, d_l, generator=g).to(dt).cuda(),
                            torch.randn(n, d_r, generator=g).to(dt).cuda(),
                            torch.randint(0, 9000, (n,), generator=g, dtype=torch.int32).cuda(),
                            torch.arange(n).cuda())
    c, kr = capi.latent_cache_read(cache, torch.arange(n).cuda(), d_l, d_r, dtype=torch.float32)
    return cache, c.cpu().double().numpy(), kr.cpu().double().numpy()


def plan(seed, q_lens, kv_lens, page, spare=2):
    g = torch.Generator().manual_seed(seed)
    need = [-(-k // page) for k in kv_lens]
    order = torch.randperm(sum(need) + spare, generator=g).to(torch.int32)
    table = torch.full((len(need), max(need + [1])), -7, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    qs = torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32)
    return sum(need) + spare, table, qs, torch.tensor(kv_lens, dtype=torch.int32)


def reference(q, lat, rope, table, qs, kv, page, scale, causal, window, bf16):
    """Oracle and bounds; scores against keys of any position (the turned queries' angles in 64 bits, then fp32:
    2^-20 of the rope products)."""
    T, H, _ = q.shape
    d_l = lat.shape[1]
    val = dict(o=np.zeros((T, H, d_l)), lse=np.full((T, H), -np.inf))
    err = dict(o=np.zeros((T, H, d_l)), lse=np.zeros((T, H)))
    for s in range(len(kv)):
        n_q, k_n = int(qs[s + 1] - qs[s]), int(kv[s])
        for i in range(n_q):
            t, tok = k_n - n_q + i, int(qs[s]) + i
            hi = min(t + 1, k_n) if causal else k_n
            lo = max(0, (t if causal else k_n - n_q) - window + 1) if window else 0
            keys = np.arange(lo, max(lo, hi))
            if keys.size == 0:
                continue
            slot = table[s, keys // page].astype(np.int64) * page + keys % page
            k = np.concatenate([lat[slot], rope[slot]], 1)
            x = np.concatenate([q[tok, :, :d_l], ol.turn(q[tok, :, d_l:], np.full(H, t), BASE)], -1)
            o, eo, z, ez = lp.fwd_block(x, k, d_l, scale, bf16, extra=2.0 ** -20)
            val["o"][tok], err["o"][tok], val["lse"][tok], err["lse"][tok] = o, eo, z, ez
    return val, err


# name: q_lens, kv_lens, page, n_h, d_l, d_r, causal, window, kinds
PAGED = {
    "one_token": ([1], [1], 16, 64, 512, 64, True, 0, ("bf16", "fp8", "f32")),
    "one_token_long": ([1], [1500], 64, 64, 512, 64, True, 0, ("bf16", "fp8")),
    "decode_ragged": ([1, 1, 1, 1], [5, 64, 65, 700], 16, 64, 512, 64, True, 0, ("bf16", "fp8", "f32")),
    "causal_chunks": ([3, 6, 1, 8], [130, 6, 900, 257], 64, 64, 512, 64, True, 0, ("bf16", "fp8")),
    "causal_window": ([4, 7, 1], [300, 90, 64], 32, 16, 512, 64, True, 50, ("bf16", "fp8", "f32")),
    "causal_window_wide": ([6, 2], [900, 500], 32, 40, 512, 64, True, 300, ("bf16", "fp8")),
    "causal_window_one": ([4, 3], [40, 3], 32, 16, 512, 64, True, 1, ("bf16", "fp8")),
    "draft_block": ([5, 5, 5], [700, 5, 133], 64, 64, 512, 64, False, 128, ("bf16", "fp8")),
    "draft_block_whole": ([5, 5], [200, 777], 128, 64, 512, 64, False, 0, ("bf16", "fp8")),
    "draft_window_one": ([5, 2], [70, 2], 16, 8, 512, 64, False, 1, ("bf16", "fp8")),
    # windows of which some sequences see more keys together than others: both kernels of one call
    "mixed_window_draft": ([5, 40, 1, 25, 20], [400, 300, 7, 160, 20], 16, 64, 512, 64, False, 120, ("bf16", "fp8")),
    "mixed_window_causal": ([3, 60, 1, 30], [400, 300, 7, 160], 16, 20, 512, 64, True, 110, ("bf16", "fp8")),
    "short_window_many_heads": ([2, 1], [100, 70], 16, 160, 512, 64, True, 33, ("bf16", "fp8")),
    "short_window_odd_pages": ([7, 3, 2], [77, 123, 300], 5, 20, 512, 64, True, 140, ("bf16", "fp8")),
    "short_many_sequences": ([2] * 170, [30 + i for i in range(170)], 16, 16, 512, 64, False, 40, ("bf16", "fp8")),
    "odd_pages": ([2, 5], [77, 123], 5, 20, 512, 64, True, 0, ("bf16", "fp8")),
    "page_of_one": ([2], [70], 1, 3, 512, 64, True, 0, ("bf16", "fp8")),
    "many_heads": ([2, 3], [100, 70], 16, 160, 512, 64, True, 0, ("bf16", "fp8")),
    "one_head": ([130, 3], [200, 150], 16, 1, 512, 64, True, 0, ("bf16", "fp8")),
    "heads_48_long_chunk": ([33, 40], [700, 333], 16, 48, 512, 64, True, 0, ("bf16", "fp8")),
    "narrow": ([3, 1], [40, 17], 4, 2, 128, 8, True, 0, ("bf16", "fp8", "f32")),
    "no_rope": ([3, 1], [40, 17], 4, 2, 256, 0, False, 9, ("bf16", "fp8", "f32")),
    "empty_sequences": ([0, 2, 0, 3, 0], [0, 30, 12, 3, 0], 8, 16, 512, 64, True, 0, ("bf16", "fp8")),
    "tokens_before_position_zero": ([4, 3], [2, 0], 8, 16, 512, 64, True, 0, ("bf16", "fp8", "f32")),
}


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("name", sorted(PAGED))
def test_paged_against_oracle(name, kind):
    q_lens, kv_lens, page, n_h, d_l, d_r, causal, window, kinds = PAGED[name]
    if kind not in kinds:
        pytest.skip("not a case of this kind")
    n_pages, table, qs, kv = plan(len(name), q_lens, kv_lens, page)
    cache, lat, rope = filled(len(name) + 1, kind, n_pages, page, d_l, d_r)
    g = torch.Generator().manual_seed(len(name) + 2)
    T = sum(q_lens)
    tail = 3  # padded tokens behind the last sequence
    q = torch.randn(T + tail, n_h, d_l + d_r, generator=g).to(torch.float32 if kind == "f32" else torch.bfloat16)
    o = torch.full((T + tail, n_h, d_l), 5.0, dtype=q.dtype).cuda()
    lse = torch.full((T + tail, n_h), 9.0).cuda()
    _, _, ws = capi.latent_attn_paged(q.cuda(), cache, table.cuda(), qs.cuda(), kv.cuda(), max(kv_lens), d_l=d_l,
                                      d_r=d_r, causal=causal, window=window, out=(o, lse))
    capi.get_error(ws)
    assert bool((o[T:] == 5).all()) and bool((lse[T:] == 9).all())
    val, err = reference(q[:T].double().numpy(), lat, rope, table.numpy(), qs.numpy(), kv.numpy(), page,
                         capi.LATENT_SCALE, causal, window, kind != "f32")
    lp.check("o", o[:T], val["o"], err["o"])
    lp.check("lse", lse[:T], val["lse"], err["lse"])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_paged_strides_bounds_and_capture(kind):
    """q and o as slices of wider tensors and head-major; any max_kv_len; a captured call replayed with other
    lengths, tables and queries."""
    page, n_h = 16, 64
    n_pages, table, qs, kv = plan(31, [3, 2, 6], [400, 33, 800], page)
    cache, lat, rope = filled(32, kind, n_pages, page, 512, 64)
    g = torch.Generator().manual_seed(33)
    wide = torch.randn(11, n_h, 640, generator=g).to(torch.bfloat16).cuda()
    q = wide[:, :, 32:608]
    args = (cache, table.cuda(), qs.cuda(), kv.cuda())
    ref, rl, _ = capi.latent_attn_paged(q.contiguous(), *args, 800)
    val, err = reference(q.double().cpu().numpy(), lat, rope, table.numpy(), qs.numpy(), kv.numpy(), page,
                         capi.LATENT_SCALE, True, 0, True)
    lp.check("o", ref, val["o"], err["o"])
    lp.check("lse", rl, val["lse"], err["lse"])
    wo = torch.full((11, n_h, 768), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(11, n_h, device="cuda")
    capi.latent_attn_paged(q, *args, 800, out=(wo[:, :, 128:640], lse))
    assert torch.equal(wo[:, :, 128:640], ref) and torch.equal(lse, rl)
    assert bool((wo[:, :, :128] == 3).all()) and bool((wo[:, :, 640:] == 3).all())
    hm = q.transpose(0, 1).contiguous().transpose(0, 1)
    oh = torch.empty(n_h, 11, 512, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    capi.latent_attn_paged(hm, *args, 800, out=(oh, lse))
    assert torch.equal(oh, ref) and torch.equal(lse, rl)
    for bound in (0, 1, 100, 10 ** 6):  # only how the keys are split: other roundings, the same bounds
        o2, l2, ws = capi.latent_attn_paged(q, *args, bound)
        capi.get_error(ws)
        lp.check("o", o2, val["o"], err["o"])
        lp.check("lse", l2, val["lse"], err["lse"])
    # capture
    qc = q.contiguous().clone()
    tb, qd, kd = table.cuda().clone(), qs.cuda().clone(), kv.cuda().clone()
    ws = capi.alloc_latent_paged_workspace(qc, cache, tb, 800)
    o, lse = torch.empty_like(ref), torch.empty_like(rl)
    capi.latent_attn_paged(qc, cache, tb, qd, kd, 800, workspace=ws, out=(o, lse))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.latent_attn_paged(qc, cache, tb, qd, kd, 800, workspace=ws, out=(o, lse))
    n2, table2, qs2, kv2 = plan(34, [1, 8, 2], [799, 300, 150], page, 0)
    assert n2 <= n_pages
    qc.copy_(torch.randn(11, n_h, 576, generator=g).to(torch.bfloat16))
    tb.fill_(-1)
    tb[:, :table2.shape[1]].copy_(table2)
    qd.copy_(qs2)
    kd.copy_(kv2)
    val, err = reference(qc.double().cpu().numpy(), lat, rope, tb.cpu().numpy(), qs2.numpy(), kv2.numpy(), page,
                         capi.LATENT_SCALE, True, 0, True)
    for _ in range(2):
        o.fill_(float("nan"))
        lse.fill_(float("nan"))
        graph.replay()
        capi.get_error(ws)
        lp.check("o", o, val["o"], err["o"])
        lp.check("lse", lse, val["lse"], err["lse"])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 128), (True, 40)])
def test_paged_values_outside_the_mask_do_not_matter(kind, causal, window):
    """NaN in every row that no token of a sequence sees: behind its last key, before its window, spare pages."""
    page, n_h = 32, 16
    q_lens, kv_lens = [5, 2, 1], [201, 75, 33]
    n_pages, table, qs, kv = plan(41, q_lens, kv_lens, page)
    cache, lat, rope = filled(42, kind, n_pages, page, 512, 64)
    q = torch.randn(8, n_h, 576, generator=torch.Generator().manual_seed(43))
    q = q.to(torch.float32 if kind == "f32" else torch.bfloat16).cuda()
    args = (table.cuda(), qs.cuda(), kv.cuda(), 201)
    o, lse, _ = capi.latent_attn_paged(q, cache, *args, causal=causal, window=window)
    seen = torch.zeros(n_pages * page, dtype=torch.bool)
    for s, (a, k) in enumerate(zip(q_lens, kv_lens)):
        lo = max(0, k - a - window + 1) if window else 0
        p = np.arange(lo, k)
        seen[torch.from_numpy(table.numpy()[s, p // page].astype(np.int64) * page + p % page)] = True
    rows = cache.view(n_pages * page, -1)
    rows[(~seen).cuda()] = 0xff if kind == "fp8" else float("nan")  # 0xff: NaN in e4m3, bf16 and fp32
    o2, lse2, _ = capi.latent_attn_paged(q, cache, *args, causal=causal, window=window)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
def test_paged_later_tokens_do_not_matter(kind):
    """Causal: a NaN or an infinity in a token's own row reaches that token and the later ones, not the earlier."""
    page, n_h = 16, 64
    n_pages, table, qs, kv = plan(51, [6, 3], [150, 40], page)
    cache, lat, rope = filled(52, kind, n_pages, page, 512, 64)
    q = torch.randn(9, n_h, 576, generator=torch.Generator().manual_seed(53))
    q = q.to(torch.float32 if kind == "f32" else torch.bfloat16).cuda()
    args = (table.cuda(), qs.cuda(), kv.cuda(), 150)
    val, err = reference(q.double().cpu().numpy(), lat, rope, table.numpy(), qs.numpy(), kv.numpy(), page,
                         capi.LATENT_SCALE, True, 0, kind != "f32")
    rows = cache.view(n_pages * page, -1)
    for s, p in ((0, 147), (1, 38)):
        rows[int(table[s, p // page]) * page + p % page] = 0xff if kind == "fp8" else float("nan")
    o, lse, _ = capi.latent_attn_paged(q, cache, *args)
    # positions 144 .. 146 of the first, 37 of the second: the values they have without the bad rows. (Not the same
    # bits: such rows are summed in another order, both within the bounds of the exact result.)
    for a, b in ((0, 3), (6, 7)):
        lp.check("o", o[a:b], val["o"][a:b], err["o"][a:b])
        lp.check("lse", lse[a:b], val["lse"][a:b], err["lse"][a:b])
    for a, b in ((3, 6), (7, 9)):
        assert torch.isnan(o[a:b].float()).all()


def test_paged_bad_pages_and_lengths():
    """What only the device sees: reported, and nothing outside the cache is read."""
    page, n_h = 16, 16
    n_pages, table, qs, kv = plan(61, [2, 2, 2], [50, 70, 40], page, 1)
    cache, lat, rope = filled(62, "bf16", n_pages, page, 512, 64)
    q = torch.randn(6, n_h, 576, generator=torch.Generator().manual_seed(63)).to(torch.bfloat16)
    good, gl, ws = capi.latent_attn_paged(q.cuda(), cache, table.cuda(), qs.cuda(), kv.cuda(), 70)
    capi.get_error(ws)

    def call(t, a, k):
        out = capi.latent_attn_paged(q.cuda(), cache, t.cuda(), a.cuda(), k.cuda(), 70, workspace=ws,
                                     out=(torch.zeros_like(good), torch.zeros_like(gl)))
        with pytest.raises(capi.DsparkError) as e:
            capi.get_error(ws)
        assert e.value.status == 10
        capi.get_error(ws)
        return out

    bad = table.clone()
    bad[1, 2], bad[0, 1] = n_pages, -3
    o, lse, _ = call(bad, qs, kv)
    assert torch.equal(o[4:], good[4:])
    # the page's keys are skipped: the oracle over the others
    for s, gone in ((0, (16, 32)), (1, (32, 48))):
        for i in range(2):
            tok, t = 2 * s + i, int(kv[s]) - 2 + i
            p = np.array([x for x in range(t + 1) if not gone[0] <= x < gone[1]])
            slot = table.numpy()[s, p // page].astype(np.int64) * page + p % page
            k = np.concatenate([lat[slot], rope[slot]], 1)
            x = q[tok].double().numpy()
            x = np.concatenate([x[:, :512], ol.turn(x[:, 512:], np.full(n_h, t), BASE)], -1)
            ro, eo, rz, ez = lp.fwd_block(x, k, 512, capi.LATENT_SCALE, True, extra=2.0 ** -20)
            lp.check("o", o[tok], ro, eo)
            lp.check("lse", lse[tok], rz, ez)
    for wrong in (-1, table.shape[1] * page + 1):
        k = kv.clone()
        k[1] = wrong
        o, lse, _ = call(table, qs, k)
        assert torch.equal(o[:2], good[:2]) and torch.equal(o[4:], good[4:])
        assert torch.count_nonzero(o[2:4]) == 0 and torch.isneginf(lse[2:4]).all()
    for wrong in ([0, 4, 2, 6], [0, 2, 4, 7], [-1, 2, 4, 6]):
        o, lse, _ = call(table, torch.tensor(wrong, dtype=torch.int32), kv)


def test_a_serving_step(oracle_mod):
    """Write, draft and verify as a serving loop runs them: a prefix and a draft block go into the cache, the block
    attends over it (draft mask), the block's latents are overwritten by the verified tokens', which attend
    causally; the draft result equals the training operator's for the same tokens."""
    S, A, W, H, page = 90, 61, 128, 64, 16
    g = torch.Generator().manual_seed(71)
    c, kr = torch.randn(1, S + 5, 512, generator=g).to(torch.bfloat16), torch.randn(1, S + 5, 64, generator=g).to(
        torch.bfloat16)
    q = torch.randn(1, H, 5, 576, generator=g).to(torch.bfloat16)
    an, kp = torch.tensor([[A]], dtype=torch.int32), torch.ones(1, 1, dtype=torch.uint8)
    o, lse, ws = capi.latent_attn_fwd(q.cuda(), c.cuda(), kr.cuda(), an.cuda(), kp.cuda(), S, W)
    cache = capi.latent_cache(8, page)
    table = torch.tensor([[5, 2, 7, 0, 1]], dtype=torch.int32)
    src = torch.cat([torch.arange(A), S + torch.arange(5)])
    pos = torch.arange(A + 5)
    slots = table[0, pos // page].long() * page + pos % page
    capi.latent_cache_write(cache, c[0, src].cuda(), kr[0, src].cuda(), pos.int().cuda(), slots.cuda())
    args = (cache, table.cuda(), torch.tensor([0, 5], dtype=torch.int32).cuda(),
            torch.tensor([A + 5], dtype=torch.int32).cuda(), A + 5)
    qt = q[0].transpose(0, 1).contiguous()
    po, pl, ws = capi.latent_attn_paged(qt.cuda(), *args, causal=False, window=W)
    capi.get_error(ws)
    f = [x.double().numpy() for x in (q, c, kr)]
    val, err = lp.attn(*f, an.numpy(), kp.numpy(), S, W, capi.LATENT_SCALE, BASE, True)
    lp.check("training o", o, val["o"], err["o"])
    lp.check("paged o", po.transpose(0, 1)[None], val["o"], err["o"] * (1 + 2.0 ** -10))
    lp.check("paged lse", pl.T[None], val["lse"], err["lse"] + 2.0 ** -14)
    # the verified tokens take the block's places
    new = torch.arange(A, A + 5)
    capi.latent_cache_write(cache, c[0, new].cuda(), kr[0, new].cuda(), new.int().cuda(), slots[A:].cuda())
    vo, vl, ws = capi.latent_attn_paged(qt.cuda(), *args, causal=True)
    capi.get_error(ws)
    lat, rope = capi.latent_cache_read(cache, torch.arange(8 * page).cuda(), dtype=torch.float32)
    val, err = reference(qt.double().numpy(), lat.cpu().double().numpy(), rope.cpu().double().numpy(), table.numpy(),
                         np.array([0, 5]), np.array([A + 5]), page, capi.LATENT_SCALE, True, 0, True)
    lp.check("verified o", vo, val["o"], err["o"])
    lp.check("verified lse", vl, val["lse"], err["lse"])


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_read_of_many_tokens(kind):
    """From 9472 tokens on a warp reads several: every slot, repeated and padded ones too, in any order."""
    cache, lat, rope = filled(81, kind, 40, 16, 256, 32)
    g = torch.Generator().manual_seed(82)
    slots = torch.randint(-3, 40 * 16 + 3, (9473,), generator=g)
    c, kr = capi.latent_cache_read(cache, slots.cuda(), 256, 32, dtype=torch.float32)
    ok = ((slots >= 0) & (slots < 640)).numpy()
    at = slots.numpy()[ok]
    assert np.array_equal(c.cpu().double().numpy()[ok], lat[at]) and np.array_equal(kr.cpu().double().numpy()[ok], rope[at])
    assert torch.count_nonzero(c.cpu()[~ok]) == 0 and torch.count_nonzero(kr.cpu()[~ok]) == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("size", [1e-18, 1e-30, 1e17, 1e30])
def test_write_far_from_one(kind, size):
    """Rows whose squares or products leave the middle of fp32's range: the same nearest values."""
    g = torch.Generator().manual_seed(83)
    c = (torch.randn(40, 512, generator=g) * size).to(torch.bfloat16)
    w = (torch.randn(512, generator=g) * 3).to(torch.bfloat16)
    cache = capi.latent_cache(3, 16, kind=KINDS[kind])
    slots = torch.arange(40).cuda()
    z = torch.zeros(40, 64, dtype=torch.bfloat16)
    capi.latent_cache_write(cache, c.cuda(), z.cuda(), torch.zeros(40, dtype=torch.int32).cuda(), slots,
                            norm_weight=w.cuda(), eps=1e-70)
    got, _ = capi.latent_cache_read(cache, slots, dtype=torch.float32)
    y = ol.norm_rows(c.double().numpy(), w.double().numpy(), 1e-70)
    want = ol.fp8_round(y)[0] if kind == "fp8" else to_bf16(y).double().numpy()
    near(got.cpu().double().numpy(), want, y, "rows")
