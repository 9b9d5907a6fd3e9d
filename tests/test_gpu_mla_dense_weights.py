"""dsa_mla_decode where the softmax weights are far from even: maxima that move in every tile, and one token
with much of the mass over a long tail of small weights, which must neither vanish nor be biased.

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


def held(out, lse, s, row, tiles):
    """Holds a row to float64 with a bound that does not grow with the context but for fp32 sums.

    In a block of 32 tokens the kernel's largest weight is 2^7 to 2^8; a weight is rounded to f16 (2^-11 of it, or
    2^-25 absolute), then to two E4M3 terms: the first leaves 2^-4 of it, of which the second loses 2^-5 (2^-9 of the
    weight) or 2^-10 absolute, that is 2^-17 of the block's largest.  With p the exact weights the output is off by
    at most (2^-9 + 2^-11) sum p |v| + 2^-17 sum_blocks max(p) sum |v|, which is less than 2^-8 + 2^-12 of the
    largest |v| whatever the length.  The sum takes four fp32 products a page (2^-23 each where they are cut off), l one
    sum a page and a dozen within it (2^-24 each); exponentials are 2^-22 off.  The output rounds to bf16 (2^-8)."""
    n = int(s["len"][row])
    pages = (n + PAGE - 1) // PAGE
    codes = s["cache"][s["bt"][int(s["req"][row]), :pages].long()].view(-1, 576)
    codes[n:] = 0
    L = codes.view(torch.float8_e4m3fn).double()
    q = s["q"][row].double()
    x = q @ L.T
    x[:, n:] = -math.inf
    z = torch.logsumexp(x, 1)
    p = torch.exp(x - z[:, None])
    V = L[:, :512]
    lerr = (2.0 ** -20 * (q.abs() @ L.abs().T).amax(1))[:, None]
    o, absum = p @ V, p @ V.abs()
    del x
    block = p.view(p.shape[0], -1, 32).amax(2) @ V.abs().view(-1, 32, 512).sum(1)
    sums = tiles * (2.0 ** -21 + 2.0 ** -24) + 2.0 ** -19
    tol = 2.0 ** -8 * o.abs() + (2.0 ** -9 + 2.0 ** -11 + 2 * lerr + sums) * absum + 2.0 ** -17 * block + 2.0 ** -25
    e = (out[row].double() - o).abs()
    assert (e <= tol).all(), f"row {row}: out off by {(e / tol).max().item():.2f} x its bound, {e.max().item():.4f}"
    d, b = (lse[row].double() - z).abs(), lerr[:, 0] + 2.0 ** -22 * z.abs() + 2.0 ** -19 + tiles * 2.0 ** -24
    assert (d <= b).all(), f"row {row}: lse off by {(d / b).max().item():.2f} x its bound"


def longest_range(B, rows, H, n):
    """Pages that one CTA takes in a row at most: of all units, over the teams of CTAs that share them."""
    pages, units = (n + PAGE - 1) // PAGE, -(-rows * H // 64)
    return min(pages, -(-B * units * (pages + 8) // (152 // 4 * min(units, 4))) + 8)


# requests x rows of heads, tokens: a CTA takes whole contexts, 110,000 tokens of one, or a few pages
SHAPES = [(1, 1, 16, 4096), (128, 1, 64, 32768), (16, 4, 64, 262144), (16, 1, 16, 32768), (1, 1, 64, 1 << 20),
          (61, 3, 12, 20001), (3, 2, 100, 5000), (300, 1, 1, 3000)]


def strengths(H, lo, hi):
    """Head strengths for which a steering of 8 is lo to hi nats."""
    return (torch.linspace(lo, hi, H, device=DEV) if H > 1 else torch.tensor([hi], device=DEV)) / (64 * 8)


@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("shape", SHAPES)
def test_one_large_weight_over_an_even_tail(dsa, shape, where):
    """A token 8 to 13 nats above all others, which are equal: value 0 for it, 1 for them.  An output of 1 - its
    mass; the tail's equal weights leave no rounding to cancel."""
    B, rows, H, n = shape
    at = {"first": 0, "middle": n // 2 + 3, "last": n - 1}[where]
    steer, values = torch.zeros(n, device=DEV), torch.ones(n, 512, device=DEV)
    steer[at], values[at] = 8.0, 0.0
    s = steered(steer, values, strengths(H, 8.0, 13.0), 11, B, rows)
    out, lse = call(dsa, s)
    for row in {0, B * rows - 1}:
        held(out, lse, s, row, longest_range(B, rows, H, n))


@pytest.mark.parametrize("mass", [0.3, 0.5, 0.8])
@pytest.mark.parametrize("shape", SHAPES)
def test_one_large_weight_over_a_tail_within_two_nats(dsa, shape, mass):
    """Values with a common part of 1, and 0 for the large token."""
    B, rows, H, n = shape
    g = torch.Generator(device=DEV)
    g.manual_seed(12)
    # a tail of +-2 nats has a mean weight of sinh(2) / 2
    gap = math.log(mass / (1 - mass)) + math.log(n * math.sinh(2.0) / 2)
    steer = (torch.rand(n, generator=g, device=DEV) * 2 - 1) * (2.0 * 8 / gap)
    values = 1 + 0.5 * torch.randn(n, 512, generator=g, device=DEV)
    steer[5], values[5] = 8.0, 0.0
    s = steered(steer, values, strengths(H, gap, gap), 13, B, rows)
    out, lse = call(dsa, s)
    for row in {0, B * rows - 1}:
        held(out, lse, s, row, longest_range(B, rows, H, n))


@pytest.mark.parametrize("gap", [5.0, 9.0, 11.0])
def test_a_large_weight_in_every_block(dsa, gap):
    """Every 32nd token is `gap` nats above the others, which have the values."""
    n = 20000
    tok = torch.arange(n, device=DEV)
    steer = torch.where(tok % 32 == 7, 8.0, 0.0)
    values = torch.where(tok % 32 == 7, 0.0, 1.0)[:, None].repeat(1, 512)
    s = steered(steer, values, strengths(64, gap, gap), 14, 40, 1)
    out, lse = call(dsa, s)
    for row in (0, 39):
        held(out, lse, s, row, longest_range(40, 1, 64, n))


def test_large_weights_that_only_some_rows_see(dsa):
    """The last token of the longest row dominates it; the rows before it see only the even tail."""
    n, rows, H = 9000, 4, 30
    steer, values = torch.zeros(n, device=DEV), torch.ones(n, 512, device=DEV)
    steer[n - 1], values[n - 1] = 8.0, 0.0
    s = steered(steer, values, strengths(H, 8.0, 60.0), 15, 5, rows)
    s["len"] -= (rows - 1 - torch.arange(5 * rows, device=DEV) % rows).to(torch.int32)
    out, lse = call(dsa, s)
    for row in (0, 3, 10, 19):
        held(out, lse, s, row, longest_range(5, rows, H, n))


@pytest.mark.parametrize("steps", [(0, 30, 60), (60, 30, 0), (0, 90, 0, 90), (0, -90, 90), (20, 0, 44, 0, 25)])
def test_maxima_that_rise_and_fall_by_whole_pages(dsa, steps):
    """Runs of seven pages, each the given octaves from the first, beyond what one reference covers."""
    g = torch.Generator(device=DEV)
    g.manual_seed(16)
    n = 7 * PAGE * len(steps) - 9
    level = torch.tensor(steps, device=DEV, dtype=torch.float32)[torch.arange(n, device=DEV) // (7 * PAGE)]
    # a steering of one octave, in E4M3 the nearest to it
    s = steered(level, torch.randn(n, 512, generator=g, device=DEV), torch.full((40,), math.log(2) / 64, device=DEV),
                17, 3, 2, q_noise=0.02)
    out, lse = call(dsa, s)
    for row in (0, 5):
        held(out, lse, s, row, longest_range(3, 2, 40, n))


def test_a_row_is_the_same_beside_any_others(dsa):
    """How the call's rows cut the context moves an output by no more than the bound of each."""
    n = 32768
    steer, values = torch.zeros(n, device=DEV), torch.ones(n, 512, device=DEV)
    steer[0], values[0] = 8.0, 0.0
    s = steered(steer, values, strengths(16, 9.0, 12.0), 18, 200, 1)
    alone = {**s, "q": s["q"][:1], "bt": s["bt"][:1], "req": s["req"][:1], "len": s["len"][:1]}
    a, _ = call(dsa, alone)
    b, _ = call(dsa, s)
    # values 0 and 1: twice the bound of `held` is below 2 * (2^-8 + 2^-9 + 2^-11 + 2^-12 + 2^-13) < 2^-6
    assert ((a[0].double() - b[199].double()).abs() <= 2.0 ** -6).all()
    held(a, call(dsa, alone)[1], s, 0, longest_range(1, 1, 16, n))


@pytest.mark.parametrize("H", [5, 64])
def test_a_context_that_begins_with_pages_that_are_skipped(dsa, H):
    """Bad pages at the front of every context and at its end: no reference before the first visible token."""
    g = torch.Generator(device=DEV)
    g.manual_seed(19)
    n = 40 * PAGE
    steer = torch.rand(n, generator=g, device=DEV) * 4 + 30
    s = steered(steer, 1 + torch.randn(n, 512, generator=g, device=DEV), strengths(H, 8.0, 8.0), 20, 12, 2)
    good = {**s, "bt": s["bt"][:, 3:39].contiguous(), "len": s["len"] - 4 * PAGE}
    s["bt"][:, :3] = torch.tensor([-1, 40, 10 ** 6], dtype=torch.int32, device=DEV)
    s["bt"][:, 39] = -7
    ws = torch.empty(dsa.mla_decode_workspace_size(24, H), dtype=torch.uint8, device=DEV)
    out, lse = call(dsa, s, workspace=ws)
    assert dsa.check_device_status(ws) == 2
    for row in (0, 23):
        held(out, lse, good, row, longest_range(12, 2, H, n))
