"""The codes that dsa_append_kv writes where its documentation fixes them exactly: blocks whose scale is 0, values
half way between two codes, and rows that need neither norm nor rotation."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
PAGE = 64


@pytest.fixture(scope="module")
def dsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dsa_sparse_attention_lightning_gb300 as m
    from dsa_sparse_attention_lightning_gb300 import _build
    _build.build()
    m.load()
    return m


def append(dsa, latent, latent_scale, nv, inv_freq=None, pos=None):
    """The rows of `latent` after the call, one page after the other."""
    T = latent.shape[0]
    pages = (T + PAGE - 1) // PAGE
    cache = torch.full((pages, PAGE, 352 if nv else 576), 0xA5, dtype=torch.uint8, device=DEV)
    at = torch.arange(T, dtype=torch.int32, device=DEV)
    dsa.dsa_append_kv(latent, None, 0.0, inv_freq, latent_scale, torch.arange(pages, dtype=torch.int32, device=DEV)[None],
                      torch.zeros_like(at), at, cache, nvfp4_latent=nv)
    return cache.view(-1, cache.shape[-1])[:T]


def nibbles(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def test_codes_of_a_block_whose_scale_is_zero(dsa):
    """Values of either sign too small for a scale: every code is 0, not the one of -0."""
    x = torch.zeros(3, 576, dtype=torch.bfloat16, device=DEV)
    x[0] = -1e-5
    x[1] = torch.where(torch.arange(576, device=DEV) % 2 == 0, -0.0, -2.0 ** -8).to(torch.bfloat16)   # / 6 < 2^-10
    x[2, ::3] = -1e-30
    row = append(dsa, x, 1.0, True)
    assert (row[:, :288] == 0).all()
