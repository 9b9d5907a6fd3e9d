"""dsa_mla_decode where the softmax weights are far from even: maxima that move in every tile.

The logits are steered through the RoPE dims of the cached rows, which are no value dims: a token of
steering t has all 64 of them at t, and a head of strength w has q = w there.
"""
import math

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


def e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def steered(steer, values, strength, seed, B=1, rows=1, q_noise=0.0):
    """B requests of `rows` rows over one context (their block tables name the same pages): steer [n], values
    [n, 512], strength [H].  All rows see all n tokens."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n, H = steer.numel(), strength.numel()
    pages = (n + PAGE - 1) // PAGE
    flat = torch.full((pages * PAGE, 576), 0x7F, dtype=torch.uint8, device=DEV)
    flat[:n, :512] = e4m3(values)
    flat[:n, 512:] = e4m3(steer)[:, None]
    order = torch.randperm(pages, generator=g, device=DEV)
    cache = torch.empty(pages, PAGE, 576, dtype=torch.uint8, device=DEV)
    cache[order] = flat.view(pages, PAGE, 576)
    R = B * rows
    q = q_noise * torch.randn(R, H, 576, generator=g, device=DEV)
    q[..., 512:] = strength[None, :, None]
    return {"q": q.to(torch.bfloat16), "cache": cache, "bt": order.to(torch.int32).repeat(B, 1),
            "req": torch.arange(B, dtype=torch.int32, device=DEV).repeat_interleave(rows),
            "len": torch.full((R,), n, dtype=torch.int32, device=DEV)}


def call(dsa, s, **kw):
    return dsa.dsa_mla_decode(s["q"], s["cache"], 1.0, s["bt"], s["req"], s["len"], softmax_scale=1.0, **kw)


def truth(s, row):
    """One row in float64: out, lse, sum p |v|, largest p times largest |v|, logit error bound (2^-20 sum |q l|)."""
    n = int(s["len"][row])
    L = s["cache"][s["bt"][int(s["req"][row])].long()].view(-1, 576)[:n].view(torch.float8_e4m3fn).double()
    q = s["q"][row].double()
    x = q @ L.T
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    V = L[:, :512]
    lerr = 2.0 ** -20 * (q.abs() @ L.abs().T).amax(1)
    return p @ V, lse, p @ V.abs(), p.amax(1)[:, None] * V.abs().amax(0)[None, :], lerr


@pytest.mark.parametrize("octaves", [4, 40])
@pytest.mark.parametrize("B,rows", [(1, 1), (38, 1), (16, 4)])
def test_all_maxima_move_in_consecutive_tiles(dsa, octaves, B, rows):
    """Every column's maximum rises in each of 24 pages, so that every tile rescales all columns; the call is
    repeated, and repeats bit for bit.

    A page's weights are 2^-octaves of the next page's, and its tokens below 2^-15.5 of its largest weight may be
    dropped: 64 * 2^-15.5 * 16 / 15 < 2^-9 of the largest weight in all."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    n = 24 * PAGE
    page = torch.arange(n, device=DEV) // PAGE
    # multiples of 8 up to 128 are E4M3 values
    s = steered(8.0 * (page - 12), torch.randn(n, 512, generator=g, device=DEV),
                torch.full((64,), octaves * math.log(2) / (64 * 8), device=DEV), 4, B, rows, q_noise=0.02)
    out, lse = call(dsa, s)
    for _ in range(20):
        again = call(dsa, s)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    for row in {0, B * rows - 1}:
        o, z, absum, largest, lerr = truth(s, row)
        tol = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -11 + 2 * lerr[:, None]) * absum + 2.0 ** -9 * largest
        assert ((out[row].double() - o).abs() <= tol).all()
        assert ((lse[row].double() - z).abs() <= lerr + 2.0 ** -22 * z.abs() + 2.0 ** -20).all()
