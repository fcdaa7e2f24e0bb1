"""Workloads of the latent-space operators: the draft attention over latent keys and values (forward
and backward), the paged latent cache (write, read) and the attention that reads it.

``run`` computes a case with elementary torch operations, or, with ``own`` set, through the package's
public entry points. ``exact`` computes the same from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

BLOCK = 5        # draft block length
D_L, D_R = 512, 64  # latent width and rope width of the page's MLA
SCALE = 256 ** -0.5  # of the expanded head (192 + 64), which the absorbed form keeps
BASE = 10000.0
EPS = 1e-5
GROUP = 128      # latent values per scale of the 8-bit cache


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    draft = dict(n_h=64, W=128, d_l=D_L, d_r=D_R, dtype="bf16")
    return [
        # the reference-sized problem in fp32: a latency-bound call
        dict(name="fwd_tiny_f32", op="fwd", B=1, S=64, N=4, W=16, n_h=4, d_l=32, d_r=16, dtype="f32", drop=0.0),
        # a short training batch: one sequence of 2048 tokens
        dict(name="fwd_s2048_n128", op="fwd", B=1, S=2048, N=128, drop=0.0, **draft),
        # the benchmark's training batch
        dict(name="fwd_s8192_n512_b2", op="fwd", B=2, S=8192, N=512, drop=0.0, **draft),
        # backward of the short batch
        dict(name="bwd_s2048_n128", op="bwd", B=1, S=2048, N=128, drop=0.0, **draft),
        # backward of the largest training batch, a tenth of its blocks padding
        dict(name="bwd_s4096_n512_b4_pad", op="bwd", B=4, S=4096, N=512, drop=0.1, **draft),
        # serving one user: one new token over an 8192-token context (latency)
        dict(name="paged_decode_1x1_8192", op="paged", n_seq=1, q_len=1, kv=8192, ragged=False, n_h=64, d_l=D_L,
             d_r=D_R, window=0, causal=True, page=64, cache="bf16"),
        # drafting for a batch of users: 5-token blocks over the draft's own window, 8-bit cache
        dict(name="paged_draft_128x5_w128", op="paged", n_seq=128, q_len=5, kv=4096, ragged=True, n_h=64, d_l=D_L,
             d_r=D_R, window=128, causal=False, page=64, cache="fp8"),
        # verifying drafted tokens over the whole context: ragged chunks, causal
        dict(name="paged_chunk_16x6_16384", op="paged", n_seq=16, q_len=6, kv=16384, ragged=True, n_h=64, d_l=D_L,
             d_r=D_R, window=0, causal=True, page=64, cache="bf16"),
        # one decoding step's tokens into the 8-bit cache
        dict(name="write_fp8_160", op="write", T=160, n_pages=512, page=64, d_l=D_L, d_r=D_R, cache="fp8", norm=True),
        # a prefill's tokens into the 16-bit cache
        dict(name="write_bf16_16384", op="write", T=16384, n_pages=512, page=64, d_l=D_L, d_r=D_R, cache="bf16",
             norm=True),
        # one draft window back out of the 8-bit cache
        dict(name="read_fp8_127", op="read", T=127, n_pages=512, page=64, d_l=D_L, d_r=D_R, cache="fp8"),
        # whole contexts back out of the 8-bit cache
        dict(name="read_fp8_32768", op="read", T=32768, n_pages=1024, page=64, d_l=D_L, d_r=D_R, cache="fp8"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "paged", "paged", "write", "read"])
    if op in ("fwd", "bwd"):
        if rng.random() < 0.2:
            S = _log_int(rng, 16, 256)
            return dict(op=op, B=rng.randint(1, 2), S=S, N=_log_int(rng, 1, 12), W=_log_int(rng, 2, 64),
                        n_h=rng.randint(1, 6), d_l=rng.choice([32, 64, 96]), d_r=rng.choice([8, 16, 32]),
                        dtype="f32", drop=rng.choice([0.0, 0.2]))
        B = rng.randint(1, 3)
        return dict(op=op, B=B, S=_log_int(rng, 512, 8192), N=_log_int(rng, 32, 400), W=_log_int(rng, 24, 128),
                    n_h=rng.choice([16, 20, 32, 48, 64, 64]), d_l=D_L, d_r=D_R, dtype="bf16",
                    drop=rng.choice([0.0, 0.1]))
    if op == "paged":
        causal = rng.random() < 0.6
        windowed = rng.random() < 0.4
        kv = _log_int(rng, 256, 16384)
        q_len = rng.randint(1, 8) if rng.random() < 0.8 else rng.randint(9, 48)
        most = max(1, min(96, 16 * 6 * 16384 // (kv * q_len)))
        return dict(op=op, n_seq=_log_int(rng, 1, most), q_len=q_len, kv=kv, ragged=rng.random() < 0.7,
                    n_h=rng.choice([16, 32, 40, 64, 64]), d_l=D_L, d_r=D_R, window=_log_int(rng, 16, 512) if windowed else 0,
                    causal=causal, page=rng.choice([16, 32, 64, 128]), cache=rng.choice(["bf16", "fp8"]))
    T = _log_int(rng, 1, 16384)
    page = rng.choice([16, 64, 128])
    return dict(op=op, T=T, n_pages=-(-T // page) + rng.randint(1, 256), page=page, d_l=D_L, d_r=D_R,
                cache=rng.choice(["bf16", "fp8", "fp8"]), **({"norm": rng.random() < 0.7} if op == "write" else {}))


def _lens(case):
    """New tokens and keys (the new ones among them) of every sequence of a paged case."""
    rng = random.Random(case["n_seq"] * 1000003 + case["q_len"] * 1009 + case["kv"])
    q, kv = [], []
    for s in range(case["n_seq"]):
        ql = case["q_len"]
        if case["ragged"] and case["causal"] and s:
            ql = rng.randint(1, case["q_len"])
        k = case["kv"]
        if case["ragged"] and s:
            k = rng.randint(max(ql, case["kv"] // 4), case["kv"])
        q.append(ql)
        kv.append(max(k, ql))
    return q, kv


def _span(case, q, kv):
    """First visible key over a sequence's rows and the visible pairs of row and key."""
    w = case["window"]
    ctx = kv - q
    lo = max(0, ctx - w + 1) if w else 0
    if not case["causal"]:
        return lo, q * (kv - lo)
    pairs = sum(ctx + i + 1 - (max(0, ctx + i - w + 1) if w else 0) for i in range(q))
    return lo, pairs


def _row_bytes(case):
    if case["cache"] == "fp8":
        n = case["d_l"] + 2 * case["d_r"] + 4 * (case["d_l"] // GROUP)
        return (n + 15) // 16 * 16
    return (case["d_l"] + case["d_r"]) * 2


def work(case):
    op, dl, dr = case["op"], case["d_l"], case["d_r"]
    dk = dl + dr
    if op in ("fwd", "bwd"):
        es = 4 if case["dtype"] == "f32" else 2
        B, S, N, H = case["B"], case["S"], case["N"], case["n_h"]
        rows = B * H * BLOCK * N
        kept = B * (N - int(N * case["drop"])) * H * BLOCK
        keys = min(case["W"] - 1, S) + BLOCK
        ckv = B * (S + BLOCK * N) * dk * es
        if op == "fwd":
            return {"bytes": kept * dk * es + ckv + rows * (dl * es + 4), "flops": 2 * kept * keys * (dk + dl)}
        return {"bytes": kept * (dk + dl) * es + kept * 4 + rows * dk * es + 2 * ckv,
                "flops": 2 * kept * keys * (3 * dk + 2 * dl)}
    if op == "paged":
        qs, kvs = _lens(case)
        byt = fl = 0
        for q, kv in zip(qs, kvs):
            lo, pairs = _span(case, q, kv)
            byt += q * case["n_h"] * ((dk + dl) * 2 + 4) + (kv - lo) * _row_bytes(case)
            fl += 2 * pairs * case["n_h"] * (dk + dl)
        return {"bytes": byt, "flops": fl}
    T = case["T"]
    if op == "write":
        back = T * dk * 2 if case["cache"] == "fp8" else 0  # the values read back
        return {"bytes": T * (dk * 2 + _row_bytes(case)) + back, "flops": T * (4 * dl + 6 * dr)}
    return {"bytes": T * (_row_bytes(case) + dk * 2), "flops": T * dk}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _dt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _rows_fp8(lat, rope, dl, dr, nbytes):
    """Rows of the 8-bit cache for latents [n, dl] that fit e4m3 times a power of two, and ropes [n, dr]."""
    n = lat.shape[0]
    g = lat.float().view(n, dl // GROUP, GROUP)
    amax = g.abs().amax(-1).clamp_min(1e-20)
    scale = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
    rows = torch.zeros(n, nbytes, dtype=torch.uint8, device=lat.device)
    rows[:, :dl] = (g / scale[..., None]).view(n, dl).to(torch.float8_e4m3fn).view(torch.uint8)
    rows[:, dl:dl + 2 * dr] = rope.contiguous().view(torch.uint8)
    rows[:, dl + 2 * dr:dl + 2 * dr + 4 * (dl // GROUP)] = scale.contiguous().view(torch.uint8)
    return rows


def _make_cache(case, g, dev):
    n = case["n_pages"] * case["page"]
    dl, dr = case["d_l"], case["d_r"]
    lat = torch.randn(n, dl, generator=g, device=dev)
    rope = torch.randn(n, dr, generator=g, device=dev).to(torch.bfloat16)
    if case["cache"] == "fp8":
        rows = _rows_fp8(lat, rope, dl, dr, _row_bytes(case))
    else:
        rows = torch.cat([lat.to(torch.bfloat16), rope], 1)
    return rows.view(case["n_pages"], case["page"], -1)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    hg = torch.Generator().manual_seed(seed)
    op, dl, dr = case["op"], case["d_l"], case["d_r"]
    st = dict(case=case)
    if op in ("fwd", "bwd"):
        B, S, N, H = case["B"], case["S"], case["N"], case["n_h"]
        dt = _dt(case["dtype"])
        pool = S - 1
        an = torch.stack([torch.randperm(pool, generator=hg)[:N] if pool >= N else
                          torch.randint(0, pool, (N,), generator=hg) for _ in range(B)]).to(torch.int32)
        kp = torch.ones(B, N, dtype=torch.uint8)
        for b in range(B):
            kp[b, torch.randperm(N, generator=hg)[:int(N * case["drop"])]] = 0
        st["anchors"], st["keep"] = an.to(dev), kp.to(dev)
        # absorbed queries times unit-norm latents: scores of a few units
        st["q"] = torch.randn(B, H, BLOCK * N, dl + dr, generator=g, device=dev).to(dt)
        st["c"] = torch.randn(B, S + BLOCK * N, dl, generator=g, device=dev).to(dt)
        st["kr"] = torch.randn(B, S + BLOCK * N, dr, generator=g, device=dev).to(dt)
        if op == "bwd":
            st["lse"] = _plain_fwd(st)[1]
            st["dout"] = torch.randn(B, H, BLOCK * N, dl, generator=g, device=dev).to(dt)
        if own:
            from speculative_draft_mla_b200 import capi
            prob = capi.latent_problem(B, H, S, N, case["W"], dl, dr, SCALE, BASE, capi.dtype_code(dt))
            st["ws"] = capi.alloc_latent_workspace(prob, torch.device(dev))
        return st
    if op == "paged":
        qs, kvs = _lens(case)
        need = [-(-kv // case["page"]) for kv in kvs]
        case = dict(case, n_pages=sum(need) + 3)
        st["case"] = case
        st["cache"] = _make_cache(case, g, dev)
        order = torch.randperm(case["n_pages"], generator=hg)
        table = torch.full((len(qs), max(need)), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = order[at:at + n].to(torch.int32)
            at += n
        st["table"] = table.to(dev)
        st["q_start"] = torch.tensor([0] + torch.tensor(qs).cumsum(0).tolist(), dtype=torch.int32, device=dev)
        st["kv_len"] = torch.tensor(kvs, dtype=torch.int32, device=dev)
        st["qs"], st["kvs"] = qs, kvs
        st["q"] = torch.randn(sum(qs), case["n_h"], dl + dr, generator=g, device=dev).to(torch.bfloat16)
        if own:
            from speculative_draft_mla_b200 import capi
            st["ws"] = capi.alloc_latent_paged_workspace(st["q"], st["cache"], st["table"], max(kvs), d_l=dl, d_r=dr,
                                                         window=case["window"])
        return st
    st["cache"] = _make_cache(case, g, dev)
    slots = torch.randperm(case["n_pages"] * case["page"], generator=hg)[:case["T"]]
    if op == "write":
        T = case["T"]
        slots[torch.rand(T, generator=hg) < 0.02] = -1  # padded tokens of the batch
        st["c"] = torch.randn(T, dl, generator=g, device=dev).mul_(3.0).to(torch.bfloat16)
        st["kr"] = torch.randn(T, dr, generator=g, device=dev).to(torch.bfloat16)
        st["pos"] = torch.randint(0, 131072, (T,), generator=hg, dtype=torch.int32).to(dev)
        st["w"] = (1.0 + 0.1 * torch.randn(dl, generator=g, device=dev)).to(torch.bfloat16) if case["norm"] else None
    st["slots"] = slots.to(torch.int64).to(dev)
    return st


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _angles(pos, dr):
    """cos and sin [..., dr/2] of pos * base^(-2i/dr), angles in 64 bits."""
    f = torch.exp(torch.arange(dr // 2, device=pos.device, dtype=torch.float64) * (-2.0 * math.log(BASE) / dr))
    a = pos.double()[..., None] * f
    return torch.cos(a), torch.sin(a)


def _rotate(x, cos, sin):
    """Adjacent pairs of the last axis turned by the angles."""
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2)


def _plain_gather(st):
    """Per block: its keys' positions [B, N, K], their visibility, the keys [B, N, K, d_l + d_r]."""
    case = st["case"]
    S, N, W = case["S"], case["N"], case["W"]
    A = st["anchors"].long()
    dev = A.device
    B = A.shape[0]
    i = torch.arange(W - 1, device=dev)
    ctx = A[..., None] - (W - 1) + i
    own_keys = S + BLOCK * torch.arange(N, device=dev)[None, :, None] + torch.arange(BLOCK, device=dev)
    idx = torch.cat([ctx, own_keys.expand(B, N, BLOCK)], -1)
    vis = (idx >= 0) & st["keep"].bool()[..., None]
    idx = idx.clamp_min(0)
    pos = torch.arange(S, device=dev)[None].expand(B, S)
    pos = torch.cat([pos, (A[..., None] + torch.arange(BLOCK, device=dev)).flatten(1)], 1)
    cos, sin = _angles(pos, case["d_r"])
    k = torch.cat([st["c"].float(), _rotate(st["kr"].float(), cos.float(), sin.float())], -1)
    b = torch.arange(B, device=dev)[:, None, None]
    return idx, vis, k[b, idx], (cos.float(), sin.float())


def _plain_q(st):
    """Queries [B, N, H * 5, d_l + d_r] in 32 bits, the rope part turned."""
    case = st["case"]
    B, H, N, dl, dr = case["B"], case["n_h"], case["N"], case["d_l"], case["d_r"]
    pos = (st["anchors"].long()[..., None] + torch.arange(BLOCK, device=st["q"].device)).flatten(1)
    cos, sin = _angles(pos, dr)
    q = st["q"].float()
    q = torch.cat([q[..., :dl], _rotate(q[..., dl:], cos.float()[:, None], sin.float()[:, None])], -1)
    return q.view(B, H, N, BLOCK, dl + dr).permute(0, 2, 1, 3, 4).reshape(B, N, H * BLOCK, dl + dr)


def _rows_back(x, case):
    """[B, N, H * 5, d] to [B, H, 5N, d]."""
    B, N = x.shape[:2]
    return x.view(B, N, case["n_h"], BLOCK, -1).permute(0, 2, 1, 3, 4).reshape(B, case["n_h"], N * BLOCK, -1)


def _plain_fwd(st):
    case = st["case"]
    _, vis, k, _ = _plain_gather(st)
    s = torch.matmul(_plain_q(st), k.transpose(-1, -2)) * SCALE
    s = torch.where(vis[:, :, None], s, -torch.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m.isinf(), 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, k[..., :case["d_l"]]) / torch.where(l > 0, l, 1.0)
    lse = torch.where(l > 0, m + torch.log(l), -torch.inf)
    return _rows_back(o, case).to(st["q"].dtype), _rows_back(lse, case)[..., 0].contiguous()


def _plain_bwd(st):
    case = st["case"]
    B, H, N, S, dl, dr = (case[x] for x in ("B", "n_h", "N", "S", "d_l", "d_r"))
    idx, vis, k, (cos, sin) = _plain_gather(st)
    q = _plain_q(st)

    def rows(x):
        return x.view(B, H, N, BLOCK, -1).permute(0, 2, 1, 3, 4).reshape(B, N, H * BLOCK, -1).float()

    lse, do = rows(st["lse"]), rows(st["dout"])
    s = torch.matmul(q, k.transpose(-1, -2)) * SCALE
    p = torch.exp(torch.where(vis[:, :, None], s - torch.where(lse.isinf(), 0.0, lse), -torch.inf))
    dp = torch.matmul(do, k[..., :dl].transpose(-1, -2))
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * SCALE
    dq = _rows_back(torch.matmul(ds, k), case)
    dk = torch.matmul(ds.transpose(-1, -2), q)
    dk[..., :dl] += torch.matmul(p.transpose(-1, -2), do)
    flat = (idx + torch.arange(B, device=idx.device)[:, None, None] * (S + BLOCK * N)).flatten()
    dkf = torch.zeros(B * (S + BLOCK * N), dl + dr, device=dk.device)
    dkf.index_add_(0, flat, dk.flatten(0, 2))
    dkf = dkf.view(B, S + BLOCK * N, dl + dr)
    dkr = _rotate(dkf[..., dl:], cos, -sin)
    qc, qs = cos[:, None, S:], sin[:, None, S:]
    dq = torch.cat([dq[..., :dl], _rotate(dq[..., dl:], qc, -qs)], -1)
    dt = st["q"].dtype
    return dq.to(dt), dkf[..., :dl].to(dt), dkr.to(dt)


def _plain_values(rows, case, dtype=torch.float32):
    """Latent and rope parts of cache rows [..., row] as the values that they stand for."""
    dl, dr = case["d_l"], case["d_r"]
    if case["cache"] != "fp8":
        return rows[..., :dl].to(dtype), rows[..., dl:].to(dtype)
    lead = rows.shape[:-1]
    v = rows[..., :dl].contiguous().view(torch.float8_e4m3fn).to(torch.float32)
    r = rows[..., dl:dl + 2 * dr].contiguous().view(torch.bfloat16)
    s = rows[..., dl + 2 * dr:dl + 2 * dr + 4 * (dl // GROUP)].contiguous().view(torch.float32)
    v = (v.view(*lead, dl // GROUP, GROUP) * s[..., None]).flatten(-2)
    return v.to(dtype), r.to(dtype)


def _plain_paged(st):
    case = st["case"]
    H, dl, dr, page, w = case["n_h"], case["d_l"], case["d_r"], case["page"], case["window"]
    dev = st["q"].device
    q0 = st["q_start"].long()
    ql, kl = q0[1:] - q0[:-1], st["kv_len"].long()
    Q = max(st["qs"])
    ctx = kl - ql
    first = (ctx - w + 1).clamp_min(0) if w else torch.zeros_like(ctx)
    K = max(kv - _span(case, q, kv)[0] for q, kv in zip(st["qs"], st["kvs"]))
    key = first[:, None] + torch.arange(K, device=dev)  # [n_seq, K]
    live = key < kl[:, None]
    pg = st["table"].long().gather(1, (key // page).clamp_max(st["table"].shape[1] - 1))
    slot = torch.where(live, pg * page + key % page, 0)
    lat, rope = _plain_values(st["cache"].flatten(0, 1)[slot], case)
    k = torch.cat([lat, rope], -1)
    i = torch.arange(Q, device=dev)
    pos = ctx[:, None] + i  # [n_seq, Q]
    tok = (q0[:-1, None] + i).clamp_max(st["q"].shape[0] - 1)
    q = st["q"][tok].float()  # [n_seq, Q, H, d]
    cos, sin = _angles(pos, dr)
    q = torch.cat([q[..., :dl], _rotate(q[..., dl:], cos.float()[:, :, None], sin.float()[:, :, None])], -1)
    s = torch.matmul(q.flatten(1, 2), k.transpose(-1, -2)) * SCALE
    if case["causal"]:
        vis = key[:, None, :] <= pos[..., None]
        if w:
            vis &= key[:, None, :] > pos[..., None] - w
    else:
        vis = live[:, None, :].expand(-1, Q, -1)
    vis = (vis & live[:, None, :]).repeat_interleave(H, 1)
    s.masked_fill_(~vis, -torch.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m.isinf(), 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, lat) / torch.where(l > 0, l, 1.0)
    lse = torch.where(l > 0, m + torch.log(l), -torch.inf)
    n = ql.shape[0]
    keep = (i < ql[:, None]).flatten()
    return (o.view(n * Q, H, dl)[keep].to(st["q"].dtype), lse.view(n * Q, H)[keep])


def _e4m3(v):
    """Nearest e4m3 values (ties to even) of 64-bit values within +-448."""
    _, ex = torch.frexp(v)
    step = torch.exp2((ex - 1).clamp_min(-6).double() - 3)
    return torch.round(v / step) * step


def _plain_write(st):
    case = st["case"]
    dl, dr = case["d_l"], case["d_r"]
    x = st["c"].double()  # the 8-bit borders need more than 32 bits
    if st["w"] is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * st["w"].double()
    cos, sin = _angles(st["pos"], dr)
    r = _rotate(st["kr"].double(), cos, sin).to(torch.bfloat16)
    ok = st["slots"] >= 0
    if case["cache"] != "fp8":
        rows = st["cache"].view(-1, dl + dr)
        rows[st["slots"][ok]] = torch.cat([x.to(torch.bfloat16), r], -1)[ok]
        return st["cache"]
    g = x.view(-1, dl // GROUP, GROUP)
    man, ex = torch.frexp(g.abs().amax(-1))
    e = torch.where(man <= 0.875, ex - 9, ex - 8)  # the least power with amax <= 448 * 2^e
    e = torch.where(man == 0, 0, e).clamp_min(-117)
    scale = torch.exp2(e.double())
    v = (_e4m3(g / scale[..., None]) * scale[..., None]).view(-1, dl)
    # the cache's own bytes, then the written rows as the values that they stand for
    rows = st["cache"].view(-1, _row_bytes(case))
    new = torch.zeros(v.shape[0], rows.shape[1], dtype=torch.uint8, device=v.device)
    new[:, :dl] = (v.view_as(g) / scale[..., None]).view(-1, dl).float().to(torch.float8_e4m3fn).view(torch.uint8)
    new[:, dl:dl + 2 * dr] = r.contiguous().view(torch.uint8)
    new[:, dl + 2 * dr:dl + 2 * dr + 4 * (dl // GROUP)] = scale.float().contiguous().view(torch.uint8)
    rows[st["slots"][ok]] = new[ok]
    return _plain_read(st)


def _plain_read(st):
    case = st["case"]
    ok = st["slots"] >= 0
    rows = st["cache"].flatten(0, 1)[st["slots"].clamp_min(0)]
    lat, rope = _plain_values(rows, case, torch.bfloat16)
    return torch.where(ok[:, None], lat, 0), torch.where(ok[:, None], rope, 0)


def run(state):
    st, case = state, state["case"]
    op = case["op"]
    if not own:
        if op == "fwd":
            return _plain_fwd(st)
        if op == "bwd":
            return _plain_bwd(st)
        if op == "paged":
            return _plain_paged(st)
        return _plain_write(st) if op == "write" else _plain_read(st)
    from speculative_draft_mla_b200 import capi
    if op == "fwd":
        o, lse, _ = capi.latent_attn_fwd(st["q"], st["c"], st["kr"], st["anchors"], st["keep"], case["S"], case["W"],
                                         scale=SCALE, rope_base=BASE, workspace=st["ws"])
        return o, lse
    if op == "bwd":
        dq, dc, dkr = capi.latent_attn_bwd(st["q"], st["c"], st["kr"], st["anchors"], st["keep"], st["lse"],
                                           st["dout"], case["S"], case["W"], scale=SCALE, rope_base=BASE,
                                           workspace=st["ws"])
        return dq, dc, dkr
    if op == "paged":
        o, lse, _ = capi.latent_attn_paged(st["q"], st["cache"], st["table"], st["q_start"], st["kv_len"],
                                           max(st["kvs"]), d_l=case["d_l"], d_r=case["d_r"], scale=SCALE,
                                           causal=case["causal"], window=case["window"], rope_base=BASE,
                                           workspace=st["ws"])
        return o, lse
    if op == "write":
        capi.latent_cache_write(st["cache"], st["c"], st["kr"], st["pos"], st["slots"], norm_weight=st["w"], eps=EPS,
                                rope_base=BASE)
        if case["cache"] != "fp8":
            return st["cache"]
    return capi.latent_cache_read(st["cache"], st["slots"], d_l=case["d_l"], d_r=case["d_r"])


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _turn64(x, pos, back=False):
    """The rope slice x [n, ..., dr] of positions pos [n] as complex numbers times e^{i angle}."""
    dr = x.shape[-1]
    z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], dr // 2, 2).contiguous())
    f = torch.tensor([BASE ** (-2.0 * i / dr) for i in range(dr // 2)], dtype=torch.float64, device=x.device)
    a = torch.outer(pos.double(), f).view(pos.shape[0], *([1] * (x.dim() - 2)), dr // 2)
    z = z * torch.polar(torch.ones_like(a), -a if back else a)
    return torch.view_as_real(z).flatten(-2)


def _exact_draft(st, grad):
    case = st["case"]
    B, H, N, S, W, dl = (case[x] for x in ("B", "n_h", "N", "S", "W", "d_l"))
    dev = st["q"].device
    anchors, keep = st["anchors"].tolist(), st["keep"].tolist()
    five = torch.arange(BLOCK, device=dev)
    o = torch.zeros(B, H, BLOCK * N, dl, dtype=torch.float64, device=dev)
    lse = torch.full((B, H, BLOCK * N), -math.inf, dtype=torch.float64, device=dev)
    dq = torch.zeros(st["q"].shape if grad else (0,), dtype=torch.float64, device=dev)
    dc = torch.zeros(st["c"].shape if grad else (0,), dtype=torch.float64, device=dev)
    dkr = torch.zeros(st["kr"].shape if grad else (0,), dtype=torch.float64, device=dev)
    for b in range(B):
        kr = _turn64(st["kr"][b, :S], torch.arange(S, device=dev))
        for n in range(N):
            if not keep[b][n]:
                continue
            A = anchors[b][n]
            lo, d0 = max(0, A - W + 1), S + BLOCK * n
            pos = A + five
            keys = torch.cat([torch.cat([st["c"][b, lo:A], st["c"][b, d0:d0 + BLOCK]]).double(),
                              torch.cat([kr[lo:A], _turn64(st["kr"][b, d0:d0 + BLOCK], pos)])], 1)
            qb = st["q"][b, :, BLOCK * n:BLOCK * n + BLOCK].transpose(0, 1)  # [5, H, d]
            qb = torch.cat([qb[..., :dl].double(), _turn64(qb[..., dl:], pos)], -1).flatten(0, 1)
            sc = qb @ keys.T * SCALE
            z = torch.logsumexp(sc, 1)
            p = torch.exp(sc - z[:, None])
            rows = slice(BLOCK * n, BLOCK * n + BLOCK)
            if not grad:
                o[b, :, rows] = (p @ keys[:, :dl]).view(BLOCK, H, dl).transpose(0, 1)
                lse[b, :, rows] = z.view(BLOCK, H).T
                continue
            do = st["dout"][b, :, rows].transpose(0, 1).flatten(0, 1).double()
            dp = do @ keys[:, :dl].T
            ob = p @ keys[:, :dl]
            ds = p * (dp - (do * ob).sum(1, keepdim=True)) * SCALE
            gq = (ds @ keys).view(BLOCK, H, -1)
            dq[b, :, rows, :dl] = gq[..., :dl].transpose(0, 1)
            dq[b, :, rows, dl:] = _turn64(gq[..., dl:], pos, True).transpose(0, 1)
            gk = ds.T @ qb
            gc = gk[:, :dl] + p.T @ do
            m = A - lo
            dc[b, lo:A] += gc[:m]
            dc[b, d0:d0 + BLOCK] += gc[m:]
            dkr[b, lo:A] += gk[:m, dl:]
            dkr[b, d0:d0 + BLOCK] += _turn64(gk[m:, dl:], pos, True)
        if grad:
            dkr[b, :S] = _turn64(dkr[b, :S], torch.arange(S, device=dev), True)
    return (dq, dc, dkr) if grad else (o, lse)


def _exact_rows(rows, case):
    """Cache rows as 64-bit values: e4m3 codes by their definition, sign, exponent and fraction."""
    dl, dr = case["d_l"], case["d_r"]
    if case["cache"] != "fp8":
        return rows[..., :dl].double(), rows[..., dl:].double()
    code = rows[..., :dl].int()
    e, f = (code >> 3) & 15, (code & 7).double()
    mag = torch.where(e > 0, (1 + f / 8) * torch.exp2(e.double() - 7), f / 8 * 2.0 ** -6)
    v = torch.where(code >= 128, -mag, mag)
    s = rows[..., dl + 2 * dr:dl + 2 * dr + 4 * (dl // GROUP)].contiguous().view(torch.float32).double()
    v = v * s.repeat_interleave(GROUP, -1)
    return v, rows[..., dl:dl + 2 * dr].contiguous().view(torch.bfloat16).double()


def _exact_paged(st):
    case = st["case"]
    dl, page, w = case["d_l"], case["page"], case["window"]
    dev = st["q"].device
    flat = st["cache"].flatten(0, 1)
    outs, lses, at = [], [], 0
    for s, (ql, kv) in enumerate(zip(st["qs"], st["kvs"])):
        pages = st["table"][s, :-(-kv // page)].long()
        slots = (pages[:, None] * page + torch.arange(page, device=dev)).flatten()[:kv]
        lat, rope = _exact_rows(flat[slots], case)
        ctx = kv - ql
        for i in range(ql):
            t = ctx + i
            hi = t + 1 if case["causal"] else kv
            lo = max(0, (t if case["causal"] else ctx) - w + 1) if w else 0
            q = st["q"][at + i]
            pos = torch.full((q.shape[0],), t, device=dev)
            qr = _turn64(q[:, dl:], pos)
            sc = (q[:, :dl].double() @ lat[lo:hi].T + qr @ rope[lo:hi].T) * SCALE
            z = torch.logsumexp(sc, 1)
            outs.append(torch.exp(sc - z[:, None]) @ lat[lo:hi])
            lses.append(z)
        at += ql
    return torch.stack(outs), torch.stack(lses)


def _exact_write(st):
    case = st["case"]
    dl, dr = case["d_l"], case["d_r"]
    x = st["c"].double()
    if st["w"] is not None:
        ms = torch.linalg.vector_norm(x, dim=1) ** 2 / dl
        x = x * st["w"].double() * ((ms + EPS) ** -0.5)[:, None]
    r = _turn64(st["kr"], st["pos"])
    keep = st["slots"] >= 0
    if case["cache"] != "fp8":
        out = st["cache"].double()
        out.view(-1, dl + dr)[st["slots"][keep]] = torch.cat([x, r], 1)[keep]
        return out
    # nearest of the representable magnitudes, ties to the even code
    codes = torch.arange(127, device=x.device)
    mags = torch.where(codes >= 8, (1 + (codes % 8) / 8.0).double() * torch.exp2((codes // 8).double() - 7),
                       codes.double() / 512)
    out = torch.empty_like(x)
    for g0 in range(0, dl, GROUP):
        g = x[:, g0:g0 + GROUP]
        amax = g.abs().amax(1)
        pows = torch.exp2(torch.arange(-117, 121, device=x.device).double())
        scale = pows[torch.searchsorted(448.0 * pows, amax.contiguous()).clamp_max(237)]
        scale = torch.where(amax == 0, 1.0, scale)[:, None]
        a = (g.abs() / scale).contiguous()
        hi = torch.searchsorted(mags, a).clamp_max(126)
        lo = (hi - 1).clamp_min(0)
        up, down = mags[hi] - a, a - mags[lo]
        pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        out[:, g0:g0 + GROUP] = torch.copysign(mags[pick], g) * scale
    out[~keep] = 0
    r[~keep] = 0
    return out, r


def exact(case, seed):
    op = case["op"]
    if op in ("fwd", "bwd") and case["B"] * case["N"] > 4096:
        return None
    st = prepare(case, seed)
    if op in ("fwd", "bwd"):
        return _exact_draft(st, op == "bwd")
    if op == "paged":
        return _exact_paged(st)
    if op == "write":
        return _exact_write(st)
    rows = st["cache"].flatten(0, 1)[st["slots"]]
    return _exact_rows(rows, case)
