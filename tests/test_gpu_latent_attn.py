"""The latent draft attention on the GPU against the fp64 oracle, within the bounds of latent_parity."""
import numpy as np
import pytest
import torch

import latent_parity as lp
from oracle import latent as ol
from speculative_draft_mla_b200 import build as dbuild
from speculative_draft_mla_b200 import capi

pytestmark = pytest.mark.gpu
BASE = 10000.0


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dbuild.build()
    return capi.load()


def make(seed, B, S, N, n_h, d_l, d_r, dtype, keep=1.0, spread=False):
    g = torch.Generator().manual_seed(seed)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    an = torch.randint(0, S - 1, (B, N), generator=g, dtype=torch.int32)
    if B and N and S >= 3:
        an[0, 0] = 0
        an[-1, -1] = S - 2
    kp = (torch.rand(B, N, generator=g) < keep).to(torch.uint8)
    L = S + 5 * N
    return dict(q=torch.randn(B, n_h, 5 * N, d_l + d_r, generator=g).to(dt),
                c=torch.randn(B, L, d_l, generator=g).to(dt), kr=torch.randn(B, L, d_r, generator=g).to(dt), an=an,
                kp=kp, dout=torch.randn(B, n_h, 5 * N, d_l, generator=g).to(dt))


def run(t, S, W, scale=capi.LATENT_SCALE, ws=None, bwd=True):
    d = {k: v.cuda() for k, v in t.items()}
    o, lse, ws = capi.latent_attn_fwd(d["q"], d["c"], d["kr"], d["an"], d["kp"], S, W, scale=scale, rope_base=BASE,
                                      workspace=ws)
    capi.get_error(ws)
    out = dict(o=o, lse=lse)
    if bwd:
        out["dq"], out["dc"], out["dkr"] = capi.latent_attn_bwd(
            d["q"], d["c"], d["kr"], d["an"], d["kp"], lse, d["dout"], S, W, scale=scale, rope_base=BASE, workspace=ws,
            flags=capi.FLAG_REUSE_DESCRIPTOR)
        capi.get_error(ws)
    return out


def compare(t, out, S, W, scale=capi.LATENT_SCALE):
    f = {k: v.double().numpy() for k, v in t.items() if k not in ("an", "kp")}
    bwd = "dq" in out
    val, err = lp.attn(f["q"], f["c"], f["kr"], t["an"].numpy(), t["kp"].numpy(), S, W, scale, BASE,
                       t["q"].dtype == torch.bfloat16, f["dout"] if bwd else None)
    for k in out:
        lp.check(k, out[k], val[k], err[k])


# name: B, S, N, W, n_h, d_l, d_r, keep
CASES = {
    "small": (2, 40, 4, 8, 3, 32, 16, 0.8),
    "odd_widths": (1, 33, 3, 9, 2, 37, 6, 1.0),
    "no_rope": (1, 30, 3, 9, 2, 24, 0, 1.0),
    "window_one": (1, 30, 4, 1, 2, 16, 8, 1.0),
    "window_wider_than_context": (2, 12, 3, 64, 2, 16, 8, 1.0),
    "shortest_context": (1, 2, 2, 4, 1, 8, 2, 1.0),
    "all_padding": (1, 30, 4, 8, 2, 16, 8, 0.0),
    # the page's widths
    "page_1_head": (1, 150, 3, 128, 1, 512, 64, 1.0),
    "page_16_heads": (1, 300, 9, 100, 16, 512, 64, 0.7),
    "page_20_heads_b2": (2, 200, 5, 128, 20, 512, 64, 0.9),
    "page_25_heads": (1, 140, 2, 24, 25, 512, 64, 1.0),
    "page_26_heads_window_one": (1, 64, 2, 1, 26, 512, 64, 1.0),
    "page_64_heads": (1, 260, 6, 128, 64, 512, 64, 1.0),
    "page_70_heads_window_two": (1, 90, 2, 2, 70, 512, 64, 1.0),
    "page_window_17": (3, 70, 5, 17, 6, 512, 64, 0.8),
    # more blocks than SMs: several blocks and tiles in turn on one SM
    "page_200_blocks": (1, 210, 200, 24, 30, 512, 64, 1.0),
    "page_window_129": (1, 300, 3, 129, 4, 512, 64, 1.0),
    "page_window_wider_than_context": (1, 40, 4, 128, 8, 512, 64, 1.0),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_against_oracle(name, dtype):
    B, S, N, W, n_h, d_l, d_r, keep = CASES[name]
    t = make(len(name) * 7 + N, B, S, N, n_h, d_l, d_r, dtype, keep)
    compare(t, run(t, S, W), S, W)


@pytest.mark.parametrize("n", ["N", "B"])
def test_nothing_to_attend(n):
    """N = 0: empty rows and zero key gradients. B = 0: nothing at all."""
    B, N = (1, 0) if n == "N" else (0, 3)
    t = make(3, B, 20, N, 2, 512, 64, "bf16")
    out = run(t, 20, 128)
    assert out["o"].numel() == 0 and out["dq"].numel() == 0
    assert torch.count_nonzero(out["dc"]) == 0 and torch.count_nonzero(out["dkr"]) == 0


@pytest.mark.parametrize("n_h", [4, 64])
def test_large_scores(n_h):
    """Scores of tens of units with a large spread: sums stay normalised, nothing overflows."""
    t = make(11, 1, 200, 4, n_h, 512, 64, "bf16")
    t["q"] = (t["q"].float() * 8).to(torch.bfloat16)
    compare(t, run(t, 200, 128), 200, 128)
    t["q"] = (t["q"].float() * 64).to(torch.bfloat16)  # nearly one-hot rows
    out = run(t, 200, 128)
    for v in out.values():
        assert torch.isfinite(v.float()).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values_outside_the_window_do_not_matter(dtype):
    """NaN and infinities in latents and rope keys that no kept block sees, and in the rows of padding blocks."""
    B, S, N, W, n_h = 1, 300, 6, 64, 5
    t = make(12, B, S, N, n_h, 512, 64, dtype)
    t["an"][0] = torch.tensor([3, 70, 71, 140, 200, 230], dtype=torch.int32)
    t["kp"][0] = torch.tensor([1, 1, 0, 1, 1, 0], dtype=torch.uint8)
    clean = run(t, S, W)
    seen = torch.zeros(S + 5 * N, dtype=torch.bool)
    for n in range(N):
        if t["kp"][0, n]:
            a = int(t["an"][0, n])
            seen[max(0, a - W + 1):a] = True
            seen[S + 5 * n:S + 5 * n + 5] = True
    bad = dict(t, c=t["c"].clone(), kr=t["kr"].clone(), q=t["q"].clone(), dout=t["dout"].clone())
    bad["c"][0, ~seen] = float("nan")
    bad["kr"][0, ~seen] = float("inf")
    for n in (2, 5):
        bad["q"][0, :, 5 * n:5 * n + 5] = float("nan")
        bad["dout"][0, :, 5 * n:5 * n + 5] = float("inf")
    out = run(bad, S, W)
    for k in out:
        if k in ("dc", "dkr"):  # sums whose order is free: compared with the oracle below
            assert torch.count_nonzero(out[k][0, ~seen]) == 0, k
        else:
            assert torch.equal(out[k], clean[k]), k
    compare(t, out, S, W)


def test_padding_rows_and_bad_anchors():
    t = make(13, 2, 100, 5, 6, 512, 64, "bf16", keep=1.0)
    t["kp"][0, 1] = 0
    t["an"][1, 2] = 99  # S - 1: no anchor
    d = {k: v.cuda() for k, v in t.items()}
    o, lse, ws = capi.latent_attn_fwd(d["q"], d["c"], d["kr"], d["an"], d["kp"], 100, 128)
    with pytest.raises(capi.DsparkError) as e:
        capi.get_error(ws)
    assert e.value.status == 4
    dq, dc, dkr = capi.latent_attn_bwd(d["q"], d["c"], d["kr"], d["an"], d["kp"], lse, d["dout"], 100, 128)
    for b, n in ((0, 1), (1, 2)):
        assert torch.count_nonzero(o[b, :, 5 * n:5 * n + 5]) == 0
        assert torch.isneginf(lse[b, :, 5 * n:5 * n + 5]).all()
        assert torch.count_nonzero(dq[b, :, 5 * n:5 * n + 5]) == 0
        assert torch.count_nonzero(dc[b, 100 + 5 * n:105 + 5 * n]) == 0
        assert torch.count_nonzero(dkr[b, 100 + 5 * n:105 + 5 * n]) == 0
    t["kp"][1, 2] = 0
    compare(t, dict(o=o, lse=lse, dq=dq, dc=dc, dkr=dkr), 100, 128)


def test_gradients_against_differences():
    """The library's own forward, differenced: f32 inputs, the loss summed in 64 bits."""
    S, N, W = 30, 3, 9
    t = make(14, 1, S, N, 2, 16, 8, "f32")
    out = run(t, S, W)
    g = torch.Generator().manual_seed(15)
    for k, gr in (("q", "dq"), ("c", "dc"), ("kr", "dkr")):
        u = torch.randn(t[k].shape, generator=g)
        f = []
        for e in (2.0 ** -6, -2.0 ** -6):
            o = run(dict(t, **{k: t[k] + e * u}), S, W, bwd=False)["o"]
            f.append((o.cpu().double() * t["dout"].double()).sum().item())
        want = (out[gr].cpu().double() * u.double()).sum().item()
        got = (f[0] - f[1]) * 2.0 ** 5
        # the difference's own errors: third order in the step (2^-12 times third derivatives of a few units times
        # the sums' size) and fp32 outputs (2^-24 times the sum of |o dout| ~ 500 over 2^-5)
        assert abs(got - want) <= 2.0 ** -9 * (abs(want) + 40), (k, got, want)


def test_strides_and_streams_and_capture():
    """Another stream, preallocated outputs, a captured and replayed call with new inputs, two workspaces."""
    S, N, W = 200, 5, 128
    t, t2 = make(16, 1, S, N, 8, 512, 64, "bf16"), make(17, 1, S, N, 8, 512, 64, "bf16")
    d = {k: v.cuda() for k, v in t.items()}
    prob = capi.latent_problem(1, 8, S, N, W)
    ws = capi.alloc_latent_workspace(prob, "cuda")
    o = torch.empty(1, 8, 5 * N, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, 8, 5 * N, device="cuda")
    grads = tuple(torch.empty_like(d[k]) for k in ("q", "c", "kr"))

    def call():
        capi.latent_attn_fwd(d["q"], d["c"], d["kr"], d["an"], d["kp"], S, W, workspace=ws, out=(o, lse))
        capi.latent_attn_bwd(d["q"], d["c"], d["kr"], d["an"], d["kp"], lse, d["dout"], S, W, workspace=ws, out=grads)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    compare(t, dict(o=o, lse=lse, dq=grads[0], dc=grads[1], dkr=grads[2]), S, W)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in d:
        d[k].copy_(t2[k])
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        compare(t2, dict(o=o, lse=lse, dq=grads[0], dc=grads[1], dkr=grads[2]), S, W)


def test_trained_shape_rows():
    """A workload-sized call (64 heads, 128 blocks of a 2048-token context): blocks picked at random against the
    oracle, and every element finite."""
    S, N, W, H = 2048, 128, 128, 64
    t = make(18, 1, S, N, H, 512, 64, "bf16", keep=0.9)
    out = run(t, S, W)
    for k in out:
        assert torch.isfinite(out[k].float())[torch.isfinite(out["lse"]) if k == "lse" else ...].all(), k
    pick = [0, 17, 64, N - 1]
    f = {k: t[k].double().numpy() for k in ("q", "c", "kr", "dout")}
    kp = np.zeros_like(t["kp"].numpy())
    kp[0, pick] = t["kp"].numpy()[0, pick]
    val, err = lp.attn(f["q"], f["c"], f["kr"], t["an"].numpy(), kp, S, W, capi.LATENT_SCALE, BASE, True, f["dout"])
    for n in pick:
        if not kp[0, n]:
            continue
        rows = slice(5 * n, 5 * n + 5)
        for k in ("o", "lse", "dq"):
            lp.check(k, out[k][0, :, rows], val[k][0, :, rows], err[k][0, :, rows])
        own = slice(S + 5 * n, S + 5 * n + 5)  # draft keys: only their own block's rows
        for k in ("dc", "dkr"):
            lp.check(k, out[k][0, own], val[k][0, own], err[k][0, own])
    # context keys: two positions with every block that sees them
    an, keep = t["an"].numpy()[0], t["kp"].numpy()[0]
    for pos in (int(an[pick[1]]) - 1, 1000):
        kp = np.zeros_like(t["kp"].numpy())
        kp[0] = keep * (an > pos) * (an - W + 1 <= pos)
        val, err = lp.attn(f["q"], f["c"], f["kr"], t["an"].numpy(), kp, S, W, capi.LATENT_SCALE, BASE, True,
                           f["dout"])
        for k in ("dc", "dkr"):
            lp.check(k, out[k][0, pos], val[k][0, pos], err[k][0, pos])
