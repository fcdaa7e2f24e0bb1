"""Host-side checks of the latent-space entry points: statuses before any device work, sizes, and the binding's
own refusals. No kernel is launched."""
import ctypes

import pytest
import torch

from speculative_draft_mla_b200 import build as dbuild
from speculative_draft_mla_b200 import capi

OK, NULL, SHAPE, DTYPE, WS, ALIGN, UNSUP = 0, 1, 2, 3, 5, 8, 9
P = ctypes.c_void_p
FAKE, ODD = P(0x100000), P(0x100008)  # never dereferenced: every call below fails a check first


@pytest.fixture(scope="module")
def lib():
    dbuild.build()
    return capi.load()


def prob(**kw):
    d = dict(B=1, n_h=2, S=64, N=4, W=16, d_l=32, d_r=16)
    d.update(kw)
    return capi.latent_problem(**d)


def test_problem_checks(lib):
    assert capi.latent_workspace_size(prob()) % 256 == 0 and capi.latent_workspace_size(prob()) > 0
    for kw in (dict(n_h=0), dict(d_r=3), dict(d_r=-2), dict(dtype=7), dict(W=5000), dict(S=0), dict(N=-1), dict(W=0),
               dict(d_l=0), dict(d_l=513), dict(d_r=130), dict(N=8193), dict(rope_base=0.0), dict(scale=0.0),
               dict(scale=float("inf")), dict(rope_base=float("nan")), dict(B=-1), dict(B=65536),
               dict(S=2 ** 22, d_l=512), dict(n_h=2 ** 20, N=64, d_l=512)):
        assert capi.latent_workspace_size(prob(**kw)) == 0, kw
    p = prob()
    p.reserved[1] = 1
    assert capi.latent_workspace_size(p) == 0


def fwd(lib, p, ws=FAKE, nbytes=1 << 24, **kw):
    a = dict(q=FAKE, c=FAKE, kr=FAKE, an=FAKE, kp=FAKE, o=FAKE, lse=FAKE)
    a.update(kw)
    return lib.dspark_latent_attn_fwd(ctypes.byref(p) if p else None, a["q"], a["c"], a["kr"], a["an"], a["kp"],
                                      a["o"], a["lse"], ws, nbytes, 0, None)


def bwd(lib, p, ws=FAKE, nbytes=1 << 24, **kw):
    a = dict(q=FAKE, c=FAKE, kr=FAKE, an=FAKE, kp=FAKE, lse=FAKE, do=FAKE, dq=FAKE, dc=FAKE, dkr=FAKE)
    a.update(kw)
    return lib.dspark_latent_attn_bwd(ctypes.byref(p) if p else None, *[a[k] for k in (
        "q", "c", "kr", "an", "kp", "lse", "do", "dq", "dc", "dkr")], ws, nbytes, 0, None)


def test_draft_attention_statuses(lib):
    for f in (fwd, bwd):
        assert f(lib, None) == NULL
        assert f(lib, prob(dtype=4)) == DTYPE
        assert f(lib, prob(S=0)) == SHAPE
        assert f(lib, prob(d_l=600)) == UNSUP
        assert f(lib, prob(), ws=None) == WS
        assert f(lib, prob(), ws=P(0x100010)) == WS
        assert f(lib, prob(), nbytes=100) == WS
        for k in ("q", "c", "kr"):
            assert f(lib, prob(), **{k: None}) == NULL, k
            assert f(lib, prob(), **{k: ODD}) == ALIGN, k
        assert f(lib, prob(), an=None) == NULL
        assert f(lib, prob(), kp=None) == NULL
        assert f(lib, prob(), an=P(0x100002)) == ALIGN
        assert f(lib, prob(), lse=P(0x100002)) == ALIGN
    assert fwd(lib, prob(), o=None) == NULL
    for k in ("do", "dq", "dc", "dkr"):
        assert bwd(lib, prob(), **{k: None}) == NULL
        assert bwd(lib, prob(), **{k: ODD}) == ALIGN
    need = capi.latent_workspace_size(prob())
    assert bwd(lib, prob(), nbytes=need - 1) == WS


def test_row_bytes(lib):
    assert capi.latent_row_bytes(capi.CACHE_BF16, 512, 64) == 1152
    assert capi.latent_row_bytes(capi.CACHE_F32, 512, 64) == 2304
    assert capi.latent_row_bytes(capi.CACHE_FP8, 512, 64) == 656
    assert capi.latent_row_bytes(capi.CACHE_FP8, 128, 8) == 160  # 128 + 16 + 4, padded
    assert capi.latent_row_bytes(capi.CACHE_FP8, 256, 0) == 272
    for bad in ((3, 512, 64), (-1, 512, 64), (0, 0, 64), (0, 520, 64), (0, 12, 64), (2, 64, 64), (0, 512, 136),
                (0, 512, 4), (0, 512, -8)):
        assert capi.latent_row_bytes(*bad) == 0, bad


def cache_p(**kw):
    d = dict(T=4, d_l=512, d_r=64, kind=1, n_pages=2, page_size=16, dtype=1, reserved=0)
    d.update(kw)
    return capi.LatentCache(**d)


def test_cache_statuses(lib):
    def write(p, c=FAKE, kr=FAKE, w=None, eps=1e-5, base=1e4, pos=FAKE, slots=FAKE, cache=FAKE):
        return lib.dspark_latent_cache_write(ctypes.byref(p) if p else None, c, kr, w, eps, base, pos, slots, cache,
                                             None)

    def read(p, cache=FAKE, slots=FAKE, c=FAKE, kr=FAKE):
        return lib.dspark_latent_cache_read(ctypes.byref(p) if p else None, cache, slots, c, kr, None)

    for f in (write, read):
        assert f(None) == NULL
        assert f(cache_p(dtype=2)) == DTYPE and f(cache_p(kind=5)) == DTYPE
        assert f(cache_p(T=-1)) == SHAPE and f(cache_p(page_size=0)) == SHAPE and f(cache_p(reserved=1)) == SHAPE
        assert f(cache_p(d_l=500)) == UNSUP and f(cache_p(kind=2, d_l=192)) == UNSUP
        assert f(cache_p(), c=None) == NULL and f(cache_p(), c=ODD) == ALIGN
        assert f(cache_p(), slots=None) == NULL and f(cache_p(), slots=P(0x100004)) == ALIGN
        assert f(cache_p(), cache=None) == NULL and f(cache_p(), cache=ODD) == ALIGN
        assert f(cache_p(T=0), c=None, slots=None, cache=None) == OK
    assert write(cache_p(), eps=-1.0) == SHAPE and write(cache_p(), eps=float("nan")) == SHAPE
    assert write(cache_p(), base=0.0) == SHAPE
    assert write(cache_p(), w=ODD) == ALIGN and write(cache_p(), kr=None) == NULL
    assert write(cache_p(), pos=None) == NULL and write(cache_p(), pos=P(0x100002)) == ALIGN
    assert read(cache_p(), kr=ODD) == ALIGN


def paged_p(**kw):
    d = dict(n_seq=2, T=4, n_h=64, d_l=512, d_r=64, page_size=16, n_pages=9, max_pages=4, max_kv_len=64, window=0,
             causal=1, dtype=1, kind=1, reserved=0, q_token_stride=0, q_head_stride=0, o_token_stride=0,
             o_head_stride=0, rope_base=1e4, scale=0.1)
    d.update(kw)
    return capi.LatentPaged(**d)


def test_paged_statuses(lib):
    def call(p, q=FAKE, cache=FAKE, table=FAKE, qs=FAKE, kv=FAKE, o=FAKE, lse=FAKE, ws=FAKE, nbytes=1 << 30):
        return lib.dspark_latent_attn_paged(ctypes.byref(p) if p else None, q, cache, table, qs, kv, o, lse, ws,
                                            nbytes, None)

    assert call(None) == NULL
    assert capi.latent_paged_workspace_size(paged_p()) % 256 == 0
    assert capi.latent_paged_workspace_size(paged_p()) > 0
    for kw, want in ((dict(kind=7), DTYPE), (dict(dtype=0), DTYPE), (dict(kind=0, dtype=1), DTYPE),
                     (dict(n_seq=-1), SHAPE), (dict(T=-1), SHAPE), (dict(n_h=0), SHAPE), (dict(page_size=0), SHAPE),
                     (dict(window=-1), SHAPE), (dict(causal=2), SHAPE), (dict(scale=-1.0), SHAPE),
                     (dict(rope_base=0.0), SHAPE), (dict(reserved=1), SHAPE), (dict(max_kv_len=-1), SHAPE),
                     (dict(d_l=100), UNSUP), (dict(kind=2, d_l=64), UNSUP), (dict(d_r=12), UNSUP),
                     (dict(T=2 ** 26), UNSUP), (dict(max_pages=2 ** 28), UNSUP), (dict(n_seq=2 ** 24), UNSUP),
                     (dict(q_token_stride=577, q_head_stride=576), ALIGN), (dict(q_token_stride=-8, q_head_stride=8), SHAPE),
                     (dict(o_token_stride=1 << 41, o_head_stride=512), UNSUP),
                     (dict(o_token_stride=512, o_head_stride=512), SHAPE),   # tokens' rows overlap
                     (dict(o_token_stride=64 * 512, o_head_stride=8), SHAPE)):  # heads' rows overlap
        assert call(paged_p(**kw)) == want, kw
        assert capi.latent_paged_workspace_size(paged_p(**kw)) == 0
    assert call(paged_p(), ws=None) == WS and call(paged_p(), ws=P(0x100010)) == WS and call(paged_p(), nbytes=8) == WS
    for k in ("q", "cache", "table", "qs", "kv", "o", "lse"):
        assert call(paged_p(), **{k: None}) == NULL, k
        assert call(paged_p(), **{k: P(0x100002)}) == ALIGN, k
    # head-major outputs do not overlap either
    assert call(paged_p(o_token_stride=512, o_head_stride=4 * 512), nbytes=8) == WS


def test_binding_refusals():
    """Tensors on the CPU, wrong shapes and types raise before the library is called."""
    z = torch.zeros
    with pytest.raises((ValueError, TypeError)):
        capi.latent_attn_fwd(z(1, 2, 5, 40), z(1, 13, 32), z(1, 13, 8), z(1, 1, dtype=torch.int32),
                             z(1, 1, dtype=torch.uint8), 8, 4)
    with pytest.raises((ValueError, TypeError)):
        capi.latent_cache_write(z(2, 4, 40), z(1, 32), z(1, 8), z(1, dtype=torch.int32), z(1, dtype=torch.int64))
    with pytest.raises((ValueError, TypeError)):
        capi.latent_attn_paged(z(1, 2, 576), z(2, 4, 576), z(1, 2, dtype=torch.int32), z(2, dtype=torch.int32),
                               z(1, dtype=torch.int32))
    with pytest.raises(capi.DsparkError):
        capi.latent_cache(2, 4, d_l=500, device="cpu")


def test_paged_limits_of_sizes_and_strides(lib):
    for kw in (dict(n_pages=2 ** 27, page_size=16), dict(n_pages=2 ** 30, page_size=2, max_pages=0),
               dict(n_h=2 ** 29), dict(q_token_stride=1 << 40, q_head_stride=576)):
        assert capi.latent_paged_workspace_size(paged_p(**kw)) == 0, kw
    for kw in (dict(q_token_stride=0, q_head_stride=576), dict(q_token_stride=576 * 64, q_head_stride=0),
               dict(o_token_stride=0, o_head_stride=512), dict(o_token_stride=512 * 64, o_head_stride=0)):
        p = paged_p(**kw)
        assert capi.latent_paged_workspace_size(p) == 0, kw
        assert lib.dspark_latent_attn_paged(ctypes.byref(p), *[FAKE] * 8, 1 << 30, None) == SHAPE, kw
    # the stride of an extent of one is not used
    assert capi.latent_paged_workspace_size(paged_p(T=1, q_token_stride=0, q_head_stride=576)) > 0
