"""The stream= argument of the binding: tensors that a call allocates belong to the stream that it runs on."""
import pytest
import torch

from speculative_draft_mla_b200 import build as dbuild
from speculative_draft_mla_b200 import capi, synth
from test_gpu_latent_attn import make
from test_gpu_latent_cache import filled

pytestmark = pytest.mark.gpu
S, W, N, N_H = 260, 100, 40, 16


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dbuild.build()
    return capi.load()


def calls():
    """name -> call(stream) of the latent operators without a workspace or results of the caller's."""
    d = {k: v.cuda() for k, v in make(3, 1, S, N, N_H, 512, 64, "bf16").items()}
    _, lse, _ = capi.latent_attn_fwd(d["q"], d["c"], d["kr"], d["an"], d["kp"], S, W)
    cache, _, _ = filled(4, "bf16", 20, 16, 512, 64)
    q = torch.randn(6, N_H, 576, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    table = torch.arange(20, dtype=torch.int32, device="cuda")[None]
    qs, kv = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, 6], [300]))
    slots = torch.arange(300).cuda()
    a = (d["q"], d["c"], d["kr"], d["an"], d["kp"])
    return {
        "fwd": lambda st: capi.latent_attn_fwd(*a, S, W, stream=st),
        "bwd": lambda st: capi.latent_attn_bwd(*a, lse, d["dout"], S, W, stream=st),
        "paged": lambda st: capi.latent_attn_paged(q, cache, table, qs, kv, stream=st),
        "read": lambda st: capi.latent_cache_read(cache, slots, stream=st),
    }


@pytest.mark.parametrize("name", ["fwd", "bwd", "paged", "read"])
def test_memory_of_a_call_on_another_stream_is_not_given_away(name, monkeypatch):
    """The caller drops the results at once and allocates: none of what the call was given may come back. (Nothing is
    launched: only whose memory it is matters, not whether the stream is still at work.)"""
    call = calls()[name]
    torch.cuda.synchronize()
    seen = []
    monkeypatch.setattr(capi, "_at", lambda t: (seen.append((t.data_ptr(), t.numel() * t.element_size())), 0)[1])
    monkeypatch.setattr(capi, "_call", lambda *a: None)
    st = torch.cuda.Stream()
    out = call(st)
    made = [p for p in seen if p[1]]
    del out
    mine = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in made for _ in range(2)]
    assert not {t.data_ptr() for t in mine} & {p for p, _ in made}
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["fwd", "bwd", "paged", "read"])
def test_results_on_another_stream(name):
    """Results, with memory of the current stream filled while the call's stream has not begun."""
    call = calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(100_000_000)
    got = call(st)
    junk = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for n in (1 << 10, 1 << 16, 1 << 20, 1 << 24)
            for _ in range(4)]
    torch.cuda.current_stream().wait_stream(st)
    for i, (a, b) in enumerate(zip(got, want)):
        if a.dtype == torch.uint8:
            continue  # a workspace
        if name == "bwd" and i:  # fp32 sums of tiles' contributions in any order, rounded to bf16
            a, b = a.float(), b.float()
            assert ((a - b).abs() <= torch.maximum(a.abs(), b.abs()) * 2.0 ** -7 + 1e-5).all()
        else:
            assert torch.equal(a, b)
    for t in junk:
        assert bool((t == 0x7f).all())


def older_calls():
    c = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in synth.random_case(7, 1, 300, 40, 64, 8, 192, 64, 256, "bf16").items()}
    a = (c["q"], c["kc"], c["kr"], c["v"], c["anchors"], c["keep"])
    o, lse, _ = capi.attn_fwd(*a, 300, 64)
    g = torch.Generator(device="cuda").manual_seed(9)
    logits = [torch.randn(30, 4096, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    y = torch.randint(0, 4096, (30,), generator=g, device="cuda", dtype=torch.int32)
    conf, m = torch.randn(30, generator=g, device="cuda"), torch.ones(30, dtype=torch.uint8, device="cuda")
    ids = torch.randint(0, 900, (2, 300), generator=g, device="cuda", dtype=torch.int32)
    lm = torch.ones(2, 300, dtype=torch.uint8, device="cuda")
    an, kp = capi.sample_anchors_gpu(lm, 20, 3)
    return {
        "attn_fwd": lambda st: capi.attn_fwd(*a, 300, 64, stream=st),
        "attn_bwd": lambda st: capi.attn_bwd(*a, o, lse, c["dout"], 300, 64, stream=st),
        "loss": lambda st: capi.dspark_loss(*logits, y, conf, m, stream=st),
        "anchors": lambda st: capi.sample_anchors_gpu(lm, 20, 3, stream=st),
        "draft_inputs": lambda st: tuple(capi.build_draft_inputs(ids, lm, an, kp, stream=st).values()),
    }


@pytest.mark.parametrize("name", ["attn_fwd", "attn_bwd", "loss", "anchors", "draft_inputs"])
def test_results_of_the_other_calls_are_not_given_away(name):
    call = older_calls()[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = call(st)
    made = {t.data_ptr(): t.numel() * t.element_size() for t in out}
    del out
    mine = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in made.values() for _ in range(2)]
    assert not {t.data_ptr() for t in mine} & set(made)
    got = call(st)
    torch.cuda.current_stream().wait_stream(st)
    for a, b in zip(got, want):
        if a.dtype == torch.uint8 and a.dim() == 1:
            continue  # a workspace
        if name == "attn_bwd":  # fp32 sums in any order, rounded to bf16
            a, b = a.float(), b.float()
            assert ((a - b).abs() <= torch.maximum(a.abs(), b.abs()) * 2.0 ** -7 + 1e-5).all()
        else:
            assert torch.equal(a, b)
