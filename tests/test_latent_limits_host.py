"""Limits of the latent-space entry points where 32-bit indices end: refused before any device work. No kernel is
launched (the calls that the limits allow are given a NULL tensor)."""
import ctypes

import pytest

from speculative_draft_mla_b200 import build as dbuild
from speculative_draft_mla_b200 import capi

NULL, UNSUP = 1, 9
FAKE = ctypes.c_void_p(0x100000)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    dbuild.build()
    return capi.load()


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("T,status", [(2 ** 31 - 1, UNSUP), (2 ** 31 - 4, UNSUP), (2 ** 31 - 63, UNSUP),
                                      (2 ** 31 - 64, NULL), (2 ** 20, NULL)])
def test_tokens_of_a_cache_call(lib, T, status, kind):
    p = capi.LatentCache(T, 128, 8, kind, 2, 16, 1, 0)
    assert lib.dspark_latent_cache_write(ctypes.byref(p), None, FAKE, None, 1e-5, 1e4, FAKE, FAKE, FAKE, None) == status
    assert lib.dspark_latent_cache_read(ctypes.byref(p), FAKE, FAKE, None, None, None) == status
