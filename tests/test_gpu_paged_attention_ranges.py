"""Paged attention where scales, queries or weights are far apart: a row's result depends on what the row sees alone,
and to the accuracy that its own terms allow."""
import math

import pytest
import torch

from fp8_scaled_quantization_amax_b200 import fp8q, inputs
from tests import paged_bounds as bounds
from tests import paged_ref as ref
from tests.test_gpu_paged_attention import DEV, make_caches

pytestmark = pytest.mark.gpu


def slot(table, b, j, bs):
    return int(table[b, j // bs]), j % bs


def prefill(q, off, k, v, table, ln, *args, **kw):
    return fp8q.paged_attention_prefill(q, torch.as_tensor(off, device=DEV), k, v, table, ln, *args, **kw)


# --------------------------------------------------- values that are not finite, beside pages that are none ----

@pytest.mark.parametrize("Dh,fmt", [(64, 0), (128, 1), (256, 0)])
@pytest.mark.parametrize("what", ["code", "scale"])
def test_visible_nan_beside_a_page_that_is_none(Dh, fmt, what):
    """A tile that every row sees, one of its pages missing: a NaN code in V still reaches its element of every row, a
    scale that is infinite or NaN every element."""
    n, bs, new = 700, 16, 5
    k, v, table, ln = make_caches([n], 1, Dh, bs, fmt, seed=201)
    table[0, 2] = -1
    blk, at = slot(table, 0, 5, bs)
    if what == "code":
        v.cache[blk, at, 0, 3] = 0x7F
    else:
        v.scale_inv[blk, at, 0] = math.inf
    q = inputs.normal_bf16((new, 3, Dh), 1.0, seed=202).to(DEV)
    out, lse = prefill(q, [0, new], k, v, table, ln)
    one, _ = fp8q.paged_attention_decode(q[-1:], k, v, table, ln)
    assert torch.isfinite(lse).all()
    for x in (out, one):
        ok = torch.isfinite(x.float())
        want = torch.zeros_like(ok)
        if what == "code":
            want[..., 3] = True
        else:
            want[:] = True
        assert torch.equal(~ok, want)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("Dh,fmt,j", [(64, 0, 0), (128, 1, 150), (256, 0, 199), (64, 1, 199)])
def test_a_k_scale_that_is_not_finite(Dh, fmt, j, bad):
    """The elements of q . k are infinite with both signs, or NaN: every query that sees the token gets NaN, whichever
    sign the sum of its codes has, and no other query does."""
    n, bs = 200, 16
    k, v, table, ln = make_caches([n], 1, Dh, bs, fmt, seed=205)
    blk, at = slot(table, 0, j, bs)
    k.scale_inv[blk, at, 0] = bad
    q = inputs.normal_bf16((n, 4, Dh), 1.0, seed=206).to(DEV)
    for window, sinks in ((0, 0), (40, 2)):
        out, lse = prefill(q, [0, n], k, v, table, ln, window, sinks)
        one, l1 = fp8q.paged_attention_decode(q[-1:], k, v, table, ln, window, sinks)
        p = torch.arange(n, device=DEV)
        sees = (p >= j) & ((window == 0) | (j > p - window) | (j < sinks))
        for x, y in ((out, lse), (one, l1)):
            want = sees[-x.shape[0]:, None].expand(-1, 4)
            assert torch.equal(torch.isnan(y), want) and torch.equal(torch.isnan(x.float()).all(-1), want)
            assert torch.equal(torch.isnan(x.float()).any(-1), want)


# ------------------------------------------------------------------------- V scales that are far apart ----

@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("Dh", [64, 128, 256])
@pytest.mark.parametrize("up", [12, 22, 34, 90])
def test_hidden_scales_do_not_reach_a_row(Dh, fmt, up):
    """A later token, or one behind the window, whose V scale is 2^up times the others'."""
    n, new, bs = 150, 100, 16
    for j, window, sinks in ((140, 0, 0), (141, 60, 3), (20, 40, 2)):
        k, v, table, ln = make_caches([n], 1, Dh, bs, fmt, seed=211)
        blk, at = slot(table, 0, j, bs)
        v.scale_inv[blk, at] *= 2.0 ** up
        q = inputs.normal_bf16((new, 2, Dh), 1.0, seed=212).to(DEV)
        out, lse = prefill(q, [0, new], k, v, table, ln, window, sinks)
        rows = [(t, 0, n - new + t) for t in (0, 1, 8, 9, 10, 11, 50, 77, 89, 90, 91, 99)]
        bounds.check(out, lse, q, k, v, table, [n], rows, Dh ** -0.5, window, sinks)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("Dh,H,G,lens", [(128, 2, 3, [300]), (64, 4, 1, [150] * 60), (256, 1, 5, [200, 33]),
                                         (128, 1, 1, [3000])])
@pytest.mark.parametrize("bits", [10, 16, 40])
def test_prefill_scales_spread_at_random(Dh, H, G, lens, fmt, bits):
    """Scales over a range of 2^bits: units that one block covers and units that several do."""
    bs, new = 24, 40
    k, v, table, ln = make_caches(lens, H, Dh, bs, fmt, seed=221)
    g = torch.Generator().manual_seed(222)
    v.scale_inv.mul_(2.0 ** (bits * torch.rand(v.scale_inv.shape, generator=g)).floor().to(DEV))
    news = [min(n, new) for n in lens]
    off = torch.tensor([0] + news).cumsum(0)
    q = inputs.normal_bf16((int(off[-1]), H * G, Dh), 1.0, seed=223).to(DEV)
    out, lse = prefill(q, off, k, v, table, ln)
    some = range(len(lens)) if len(lens) < 5 else (0, 1, 30, len(lens) - 1)
    rows = [(int(off[b]) + i, b, lens[b] - news[b] + i) for b in some for i in (0, 17, news[b] - 1)]
    bounds.check(out, lse, q, k, v, table, lens, rows, Dh ** -0.5)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -12])
def test_padding_tokens_of_zeros(fmt, size):
    """V rows of zeros, whose scale is 1 whatever the others' are."""
    n, new, bs, Dh = 400, 30, 16, 128
    k, v, table, ln = make_caches([n], 2, Dh, bs, fmt, seed=231)
    x = inputs.normal_bf16((n, 2, Dh), size, seed=232)
    zero = torch.rand(n, generator=torch.Generator().manual_seed(233)) < 0.2
    zero[: 130] = False
    x[zero] = 0
    _, slots = inputs.paged_layout([n], bs, k.num_blocks, 231)
    v.write(x.to(DEV), slots.to(DEV))
    q = inputs.normal_bf16((new, 4, Dh), 1.0, seed=234).to(DEV)
    out, lse = prefill(q, [0, new], k, v, table, ln)
    rows = [(t, 0, n - new + t) for t in (0, 13, 29)]
    bounds.check(out, lse, q, k, v, table, [n], rows, Dh ** -0.5)
    one, l1 = fp8q.paged_attention_decode(q[-1:], k, v, table, ln)
    bounds.check(one, l1, q[-1:], k, v, table, [n], [(0, 0, n - 1)], Dh ** -0.5, prefill=False)


def steered(n, Dh, H, G, new, bs, fmt, seed, logits):
    """Caches whose token j has a logit near logits[j] (natural units, softmax scale 1) for every query."""
    k, v, table, ln = make_caches([n], H, Dh, bs, fmt, seed=seed)
    _, slots = inputs.paged_layout([n], bs, k.num_blocks, seed)
    u = torch.ones(Dh) / Dh ** 0.5
    k.write((logits[:, None, None] * u + inputs.normal_bf16((n, H, Dh), 0.05, seed=seed + 1).float()).bfloat16().to(DEV),
            slots.to(DEV))
    q = (u + inputs.normal_bf16((new, H * G, Dh), 0.02, seed=seed + 2).float()).bfloat16().to(DEV)
    return k, v, table, ln, q


def both(k, v, table, ln, q, n, scale=1.0, copies=1):
    """Prefill of q and decode of its last row, for as many sequences over the same pages: one is split over many
    thread blocks, of many each block takes whole ones."""
    new = q.shape[0]
    many, lens, off = table.repeat(copies, 1), ln.repeat(copies), torch.arange(copies + 1) * new
    out, lse = prefill(q.repeat(copies, 1, 1), off, k, v, many, lens, softmax_scale=scale)
    some = sorted({0, copies // 3, copies - 1})
    rows = [(c * new + t, c, n - new + t) for c in some for t in (0, new // 2, new - 1)]
    bounds.check(out, lse, q.repeat(copies, 1, 1), k, v, many, [n] * copies, rows, scale)
    last = q[-1:].repeat(copies, 1, 1)
    one, l1 = fp8q.paged_attention_decode(last, k, v, many, lens, softmax_scale=scale)
    bounds.check(one, l1, last, k, v, many, [n] * copies, [(c, c, n - 1) for c in some], scale, prefill=False)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("Dh", [64, 128, 256])
@pytest.mark.parametrize("j,copies", [(0, 1), (100, 1), (630, 1), (0, 160), (630, 160)])
def test_a_large_value_that_hardly_counts(Dh, fmt, j, copies):
    """A visible token with a V scale 2^40 times the others' and a weight of e^-60 or so."""
    n, bs = 700, 16
    logits = torch.zeros(n)
    logits[j] = -60.0
    k, v, table, ln, q = steered(n, Dh, 1, 3, 40, bs, fmt, 241, logits)
    blk, at = slot(table, 0, j, bs)
    v.scale_inv[blk, at] *= 2.0 ** 40
    both(k, v, table, ln, q, n, copies=copies)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("Dh", [64, 128, 256])
@pytest.mark.parametrize("n,slope", [(400, 0.25), (400, -0.25), (400, 0.05), (3000, 0.02), (3000, -0.02)])
@pytest.mark.parametrize("copies", [1, 160])
def test_weights_and_scales_that_cancel(Dh, fmt, n, slope, copies):
    """Logits that rise or fall by up to 100 along the sequence, in steps of a few per tile or fractions of one, while
    the V scales go the other way: every token counts."""
    bs = 16
    logits = slope * (torch.arange(n, dtype=torch.float32) - n / 2)
    k, v, table, ln, q = steered(n, Dh, 1, 2, 40, bs, fmt, 251, logits)
    at = inputs.paged_layout([n], bs, k.num_blocks, 251)[1].to(DEV)
    v.scale_inv.view(-1)[at] *= (2.0 ** (-logits / math.log(2)).round()).to(DEV)
    both(k, v, table, ln, q, n, copies=copies)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("e", [127, 126, 120, -110])
def test_scales_at_the_ends_of_their_type(fmt, e):
    """Every V scale 2^e, with codes so small that the values and their sums are finite."""
    n, bs, Dh = (60, 16, 64) if e > 0 else (300, 16, 64)
    k, v, table, ln = make_caches([n], 1, Dh, bs, fmt, seed=261)
    g = torch.Generator().manual_seed(262)
    lo, hi = (1, 8) if e > 0 else (0x10, 0x30)
    codes = torch.randint(lo, hi, v.cache.shape, generator=g, dtype=torch.uint8)
    codes |= torch.randint(0, 2, v.cache.shape, generator=g, dtype=torch.uint8) << 7
    v.cache.copy_(codes)
    v.scale_inv.fill_(2.0 ** e)
    q = inputs.normal_bf16((20, 2, Dh), 1.0, seed=263).to(DEV)
    both(k, v, table, ln, q, n, Dh ** -0.5)


# ------------------------------------------------------------------------------ logits out of the ordinary ----

@pytest.mark.parametrize("big", [1.0, 2.0 ** 20, 2.0 ** 24, 2.0 ** 33, 1e20, -1e20, 1e30])
@pytest.mark.parametrize("Dh", [64, 128, 256])
def test_logits_past_two_to_the_31(Dh, big):
    """Logits up to 8 |big| Dh, no two tokens' closer than 2^-9 of that: nothing but the largest visible one counts."""
    n, new, bs = 300, 140, 16
    k, v, table, ln = make_caches([n], 1, Dh, bs, 0, seed=281)
    _, slots = inputs.paged_layout([n], bs, k.num_blocks, 281)
    level = torch.linspace(-8, 8, n)[torch.randperm(n, generator=torch.Generator().manual_seed(282))]
    k.cache.view(-1, 1, Dh)[slots.to(DEV)] = 0x7E                      # 448
    k.scale_inv.view(-1, 1)[slots.to(DEV)] = (level / 448)[:, None].to(DEV)
    q = torch.full((new, 3, Dh), big, dtype=torch.bfloat16, device=DEV)
    scale = 32768.0 if abs(big) == 1.0 else 1.0                       # 8 Dh 2^15 is past 2^24 too
    host = ref.Cache(k, v)
    th, visible = table.cpu()[0].tolist(), torch.arange(n)
    for window, sinks in ((0, 0), (50, 2)):
        out, lse = prefill(q, [0, new], k, v, table, ln, window, sinks, softmax_scale=scale)
        one, l1 = fp8q.paged_attention_decode(q[-1:], k, v, table, ln, window, sinks, softmax_scale=scale)
        z = level.double() * float(q[0, 0, 0]) * Dh * scale
        for got, gl, p in [(out[t], lse[t], n - new + t) for t in (0, 1, 40, 100, new - 1)] + [(one[0], l1[0], n - 1)]:
            sees = (visible <= p) & ((window == 0) | (visible > p - window) | (visible < sinks))
            j = int(torch.where(sees, z, -math.inf).argmax())
            want = host.v[ref.slot_of(th, j, bs, k.num_blocks), 0]
            # V times its scale in fp16 (two roundings of 2^-11, weights and result one of 2^-11 and 2^-8)
            assert torch.all((got.float().cpu().double() - want).abs() <= (2.0 ** -8 + 2.0 ** -9) * want.abs()), (p, j)
            assert torch.all((gl.cpu().double() - z[j]).abs() <= Dh * 2.0 ** -23 * abs(float(z[j]))), (p, j)


# --------------------------------------------------------------------- queries that are far apart ----

@pytest.mark.parametrize("big", [1e20, 2.0 ** 100, 2.0 ** 14, 2.0 ** -60])
@pytest.mark.parametrize("Dh", [64, 128, 256])
def test_a_finite_query_row_leaves_the_others_their_bits(Dh, big):
    """One row 2^14 to 2^100 times the others in the same tile (or far below them), in the first or the second tile."""
    n, new, bs, G = 300, 100, 16, 4
    k, v, table, ln = make_caches([n], 2, Dh, bs, 0, seed=271)
    q = inputs.normal_bf16((new, 2 * G, Dh), 1.0, seed=272)
    for t in (17, 80):
        q[t, 1] = (q[t, 1].float() * big).bfloat16()
    q = q.to(DEV)
    for scale in (Dh ** -0.5, -0.1):
        out, lse = prefill(q, [0, new], k, v, table, ln, 150, 2, softmax_scale=scale)
        rows = [(t, 0, n - new + t) for t in (0, 16, 17, 18, 31, 63, 64, 80, 81, 99)]
        s = float(torch.tensor(scale))
        bounds.check(out, lse, q, k, v, table, [n], rows, s, 150, 2)


# ---------------------------------------------------------------------------------- workspace of a window ----

@pytest.mark.parametrize("window,sinks", [(100, 7), (1, 0), (64, 32), (97, 31)])
def test_weights_with_a_window_need_scratch_for_the_window_alone(window, sinks):
    """A long table, a short window: the scratch does not grow with the table, nothing is written behind it, and the
    results are those with more."""
    lens, H, G, Dh, bs = [5000, 300, 129], 4, 2, 64, 16
    k, v, table, ln = make_caches(lens, H, Dh, bs, 0, seed=291)
    q = inputs.normal_bf16((3, H * G, Dh), 1.0, seed=292).to(DEV)
    full = fp8q.paged_attention_workspace(3, H * G, H, Dh, table.shape[1] * bs, True)
    n = fp8q.paged_attention_workspace(3, H * G, H, Dh, window + sinks + 96, True).numel()
    parts = fp8q.paged_attention_workspace(3, H * G, H, Dh, 0, True).numel()
    assert n - parts < (full.numel() - parts) / 10
    memory = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    got = []
    for ws in (full, memory[:n], None):
        mass = torch.zeros((3, H, 5000), device=DEV)
        out, lse = fp8q.paged_attention_decode(q, k, v, table, ln, window, sinks, mass=mass, workspace=ws)
        got.append((out, lse, mass))
    assert torch.all(memory[n:] == 0xA5)
    for other in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got[0], other))
    with pytest.raises(fp8q.Fp8Error):
        fp8q.paged_attention_decode(q, k, v, table, ln, window, sinks, mass=torch.zeros((3, H, 5000), device=DEV),
                                    workspace=memory[:n - 256])
