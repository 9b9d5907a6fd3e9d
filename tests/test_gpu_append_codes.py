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


def test_values_half_way_between_two_fp4_codes(dsa):
    """v / scale at every midpoint of E2M1, for every scale: the even code, whatever 1 / scale rounds to."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    even = torch.tensor([0, 2, 2, 4, 4, 6, 6], device=DEV)                     # codes of 0, 1, 1, 2, 2, 4, 4
    code = torch.arange(1, 0x7F, device=DEV, dtype=torch.uint8)                # all scales but 0 and NaN
    scale = code.view(torch.float8_e4m3fn).float()
    blocks = torch.zeros(128, 16, device=DEV)
    # 6, the midpoints, their negatives: exact in bf16 (a scale has 4 bits, a midpoint 3)
    blocks[:126, 0] = 6 * scale
    blocks[:126, 1:8] = mid * scale[:, None]
    blocks[:126, 8:15] = -mid * scale[:, None]
    x = torch.zeros(4, 576, dtype=torch.bfloat16, device=DEV)
    x[:, :512] = blocks.view(4, 512).to(torch.bfloat16)
    assert torch.equal(x[:, :512].float().view(128, 16), blocks)
    row = append(dsa, x, 1.0, True)
    assert torch.equal(row[:, 256:288].reshape(-1)[:126], code)
    el = nibbles(row[:, :256]).view(128, 16)[:126].long()
    assert (el[:, 0] == 7).all()
    assert (el[:, 1:8] == even).all() and (el[:, 8:15] == even + 8).all()


@pytest.mark.parametrize("scale", [1.0, 7.0, 3.0, 0.3, 0.15, 0.011, 1.1, 13 / 64, 448 / 13, 1 / 448])
def test_rows_without_norm_or_rotation_at_any_scale(dsa, scale):
    """Every bf16 value: the bytes of dsa_write_kv, of quotients by the scale, in rows of either format; a
    rotation at position 0 changes none of them."""
    bits = torch.arange(65536, device=DEV).to(torch.int16)
    x = torch.zeros(128, 576, dtype=torch.bfloat16, device=DEV)
    x.view(-1)[:65536] = bits.view(torch.bfloat16)
    x = x[torch.randperm(128, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)].contiguous()
    row = append(dsa, x, scale, False)
    kc = torch.zeros(2, 8448, dtype=torch.uint8, device=DEV)
    lc = torch.zeros(2, PAGE, 576, dtype=torch.uint8, device=DEV)
    pos = torch.arange(128, dtype=torch.int32, device=DEV)
    dsa.dsa_write_kv(torch.zeros(128, 128, dtype=torch.bfloat16, device=DEV), torch.ones(128, device=DEV),
                     torch.zeros(128, device=DEV), 1e-5, x, scale, torch.arange(2, dtype=torch.int32, device=DEV)[None],
                     torch.zeros_like(pos), pos, kc, lc)
    assert torch.equal(row, lc.view(-1, 576))
    assert torch.equal(append(dsa, x, scale, True)[:, 288:], row[:, 512:])
    finite = torch.nan_to_num(x, nan=1.0, posinf=1.0, neginf=-1.0)
    still = torch.zeros(32, dtype=torch.float64, device=DEV)                  # no turn at any position
    a, b = append(dsa, finite, scale, False)[:, 512:], append(dsa, finite, scale, False, still)[:, 512:]
    assert torch.equal(a.view(torch.float8_e4m3fn).float(), b.view(torch.float8_e4m3fn).float())
