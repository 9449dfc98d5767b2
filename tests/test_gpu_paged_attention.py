"""Attention over the paged FP8 cache (one new token per sequence; several) and eviction by attention weight,
against the 64-bit reference of tests/paged_ref.py."""
import math

import pytest
import torch

from fp8_scaled_quantization_amax_b200 import fp8q, inputs
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make_caches(lens, H, Dh, bs, fmt, seed, spare=2, stale=True):
    """K and V caches holding random tokens written by the library in shuffled pages; every other slot holds stale
    bytes (NaN codes among them) and NaN scales."""
    need = sum((n + bs - 1) // bs for n in lens)
    nb = need + spare
    table, slots = inputs.paged_layout(lens, bs, nb, seed)
    if table.shape[1] == 0:
        table = torch.full((len(lens), 1), -1, dtype=torch.int32)
    caches = []
    for i in range(2):
        c = fp8q.PagedKVCache(nb, bs, H, Dh, fmt, device=DEV)
        if stale:
            g = torch.Generator().manual_seed(seed + 10 + i)
            c.cache.copy_(torch.randint(0, 256, c.cache.shape, generator=g, dtype=torch.uint8))
            c.cache.view(-1)[::7] = 0x7F
            c.scale_inv.fill_(math.nan)
        if slots.numel():
            x = inputs.normal_bf16((slots.numel(), H, Dh), 1.0, seed=seed + 20 + i)
            c.write(x.to(DEV), slots.to(DEV))
        caches.append(c)
    return caches[0], caches[1], table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def check_rows(out, lse, q, k, v, table, lens, rows, scale, window, sinks, mass=None, mass0=None, decay=0.0,
               scaled_v=False):
    """rows: (t, b, p) of every query row; out / lse [T, Hq, ...]."""
    host = ref.Cache(k, v)
    H, G = k.H, q.shape[1] // k.H
    qh, oh, lh, th = q.cpu(), out.float().cpu().double(), lse.cpu().double(), table.cpu()
    cap = th.shape[1] * k.block_size
    for t, b, p in rows:
        n = min(max(int(lens[b]), 0), cap)
        for h in range(H):
            sl = slice(h * G, (h + 1) * G)
            r = ref.attend(host, th[b].tolist(), n, p, qh[t, sl], h, scale, window, sinks, scaled_v)
            err = (oh[t, sl] - r["out"]).abs()
            assert torch.all(err <= r["tol"]), (t, h, float((err / r["tol"]).max()))
            if not r["pos"]:
                assert torch.all(lh[t, sl] == -math.inf)
                assert torch.all(oh[t, sl] == 0)
            else:
                assert torch.all((lh[t, sl] - r["lse"]).abs() <= ref.lse_tol(r)), (t, h)
            if mass is not None:
                want = mass0[b, h].cpu().double().clone()
                tol = torch.zeros_like(want)
                for i, j in enumerate(r["pos"]):
                    if j < want.numel():
                        s = float(r["w"][:, i].sum())
                        old = float(want[j])
                        want[j] = s if decay == 0.0 else decay * old + s
                        tol[j] = (2 * float(r["ez"].max()) + 2.0 ** -19) * s + 2.0 ** -23 * abs(float(want[j])) + 1e-30
                got = mass[b, h].cpu().double()
                same = tol == 0
                assert torch.equal(got[same], want[same]), "a position that no query sees was written"
                assert torch.all((got - want).abs()[~same] <= tol[~same]), (b, h)


DECODE = [
    # lens, H, G, Dh, bs, fmt, window, sinks
    ([1], 1, 1, 16, 1, 0, 0, 0),
    ([37], 8, 4, 128, 16, 0, 0, 0),
    ([0, 1, 2, 15, 16, 17, 33], 2, 2, 64, 16, 0, 0, 0),
    ([129, 64, 511], 4, 1, 128, 64, 1, 0, 0),
    ([300, 5], 1, 7, 80, 24, 0, 0, 0),
    ([257], 3, 3, 96, 7, 1, 0, 0),
    ([200, 0, 190], 5, 8, 112, 100, 0, 0, 0),
    ([150], 1, 16, 128, 16, 0, 0, 0),
    ([150, 31], 2, 24, 48, 8, 1, 0, 0),
    ([140], 1, 71, 64, 16, 0, 0, 0),
    ([260, 77], 2, 5, 256, 32, 0, 0, 0),
    ([90], 6, 2, 192, 16, 1, 0, 0),
    ([700, 33, 5], 2, 4, 128, 16, 0, 64, 4),
    ([700, 33, 5], 2, 4, 128, 16, 0, 1, 0),
    ([300, 65], 4, 1, 64, 24, 1, 63, 37),
    ([1300], 2, 2, 128, 16, 0, 200, 300),
    ([40], 1, 4, 32, 16, 0, 1000, 5),
    ([2500, 1, 900, 40], 8, 1, 128, 16, 0, 0, 0),
    ([1025] * 9, 32, 1, 64, 128, 0, 0, 0),
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(str(x) for x in c[1:]) + f"-n{max(c[0])}x{len(c[0])}")
@pytest.mark.parametrize("weights", [False, True])
def test_decode(case, weights):
    lens, H, G, Dh, bs, fmt, window, sinks = case
    k, v, table, ln = make_caches(lens, H, Dh, bs, fmt, seed=3 * len(lens) + Dh)
    B = len(lens)
    q = inputs.normal_bf16((B, H * G, Dh), 1.0, seed=5).to(DEV)
    scale = Dh ** -0.5
    mass = mass0 = None
    if weights:
        mass0 = torch.rand((B, H, max(lens) + 3), generator=torch.Generator().manual_seed(1)).to(DEV)
        mass = mass0.clone()
    out, lse = fp8q.paged_attention_decode(q, k, v, table, ln, window, sinks, mass=mass, mass_decay=0.5)
    check_rows(out, lse, q, k, v, table, lens, [(b, b, n - 1) for b, n in enumerate(lens)], scale, window, sinks, mass,
               mass0, 0.5)


PREFILL = [
    # (length, new) of each sequence, H, G, Dh, bs, fmt, window, sinks
    ([(1, 1)], 1, 1, 16, 1, 0, 0, 0),
    ([(100, 100)], 2, 4, 128, 16, 0, 0, 0),
    ([(37, 37), (0, 0), (200, 5), (64, 1)], 2, 2, 64, 16, 0, 0, 0),
    ([(300, 129), (40, 17)], 1, 7, 80, 24, 1, 0, 0),
    ([(130, 130)], 3, 1, 96, 7, 0, 0, 0),
    ([(290, 257)], 1, 2, 128, 64, 0, 0, 0),
    ([(150, 70), (33, 2)], 1, 16, 128, 16, 0, 0, 0),
    ([(90, 40)], 2, 3, 256, 32, 0, 0, 0),
    ([(90, 33)], 1, 40, 48, 8, 1, 0, 0),
    ([(280, 200), (70, 70)], 2, 2, 128, 16, 0, 50, 4),
    ([(280, 90)], 1, 4, 64, 24, 1, 1, 0),
    ([(400, 300)], 1, 1, 128, 16, 0, 130, 140),
    ([(1000, 3), (5, 5), (900, 4)], 4, 4, 128, 16, 0, 0, 0),
]


@pytest.mark.parametrize("case", PREFILL, ids=lambda c: "-".join(str(x) for x in c[1:]) + f"-{c[0][0]}x{len(c[0])}")
def test_prefill(case):
    seqs, H, G, Dh, bs, fmt, window, sinks = case
    lens = [n for n, _ in seqs]
    k, v, table, ln = make_caches(lens, H, Dh, bs, fmt, seed=7 * len(lens) + Dh)
    off = torch.tensor([0] + [m for _, m in seqs]).cumsum(0)
    T = int(off[-1])
    q = inputs.normal_bf16((T, H * G, Dh), 1.0, seed=6).to(DEV)
    out, lse = fp8q.paged_attention_prefill(q, off.to(DEV), k, v, table, ln, window, sinks)
    rows = [(int(off[b]) + i, b, n - m + i) for b, (n, m) in enumerate(seqs) for i in range(m)]
    check_rows(out, lse, q, k, v, table, lens, rows, Dh ** -0.5, window, sinks, scaled_v=True)


def test_prefill_rows_of_no_sequence_are_left_alone_and_short_sequences_see_nothing():
    """Rows before the first and behind the last offset keep what they held; a sequence with more new rows than
    tokens has rows at negative positions, which see nothing."""
    lens = [4, 9]
    k, v, table, ln = make_caches(lens, 2, 64, 16, 0, seed=2)
    q = inputs.normal_bf16((20, 4, 64), 1.0, seed=6).to(DEV)
    off = torch.tensor([3, 9, 14], device=DEV)          # six rows over four tokens, five over nine
    out = torch.full_like(q, 7.0)
    lse = torch.full((20, 4), 5.0, device=DEV)
    fp8q.fp8_paged_attention_prefill(q, 256, 20, off, 2, 4, k.cache, k.scale_inv, v.cache, v.scale_inv, 2, 64, 16,
                                     k.num_blocks, 0, table, ln, table.shape[1], 0, 0, 0.125, out, lse,
                                     fp8q.paged_attention_workspace(2, 4, 2, 64, tokens=20))
    for t in (0, 1, 2, 14, 15, 19):
        assert torch.all(out[t] == 7.0) and torch.all(lse[t] == 5.0)
    rows = [(3 + i, 0, -2 + i) for i in range(6)] + [(9 + i, 1, 4 + i) for i in range(5)]
    check_rows(out, lse, q, k, v, table, lens, rows, 0.125, 0, 0, scaled_v=True)


@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 5)])
def test_prefill_with_many_tiles_and_units_per_cta(window, sinks):
    """Long sequences on many heads (every CTA goes through many units and tiles), checked on sampled rows, twice."""
    seqs = [(5000, 1025), (3001, 64), (700, 700), (4100, 513)]
    lens = [n for n, _ in seqs]
    H, G, Dh = 8, 4, 128
    k, v, table, ln = make_caches(lens, H, Dh, 32, 0, seed=77)
    off = torch.tensor([0] + [m for _, m in seqs]).cumsum(0)
    q = inputs.normal_bf16((int(off[-1]), H * G, Dh), 1.0, seed=6).to(DEV)
    out, lse = fp8q.paged_attention_prefill(q, off.to(DEV), k, v, table, ln, window, sinks)
    again, lse2 = fp8q.paged_attention_prefill(q, off.to(DEV), k, v, table, ln, window, sinks)
    torch.cuda.synchronize()
    assert fp8q.fp8_device_error() == 0
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    rows = [(int(off[b]) + i, b, n - m + i) for b, (n, m) in enumerate(seqs) for i in (0, 1, m // 3, m - 2, m - 1)]
    check_rows(out, lse, q, k, v, table, lens, rows, Dh ** -0.5, window, sinks, scaled_v=True)


def test_prefill_of_one_token_agrees_with_decode():
    lens = [300, 17]
    k, v, table, ln = make_caches(lens, 2, 128, 16, 0, seed=11)
    q = inputs.normal_bf16((2, 8, 128), 1.0, seed=12).to(DEV)
    a, la = fp8q.paged_attention_decode(q, k, v, table, ln)
    b, lb = fp8q.paged_attention_prefill(q, torch.tensor([0, 1, 2], device=DEV), k, v, table, ln)
    rows = [(i, i, n - 1) for i, n in enumerate(lens)]
    check_rows(a, la, q, k, v, table, lens, rows, 128 ** -0.5, 0, 0)
    check_rows(b, lb, q, k, v, table, lens, rows, 128 ** -0.5, 0, 0, scaled_v=True)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_bad_pages_are_not_visible_and_lengths_are_clamped(kind):
    """Page ids outside the pool hide their positions; lengths below 0 or past the table count as its ends."""
    lens = [70, 50, 33]
    k, v, table, _ = make_caches(lens, 2, 64, 16, 0, seed=4)
    table[0, 1] = -5
    table[0, 3] = k.num_blocks
    table[2, :] = -1                                     # nothing visible at all
    claimed = [70, -3, 33]
    claimed[1] = 10 ** 6                                 # past the table: its 5 columns count (one of them no page)
    ln = torch.tensor(claimed, dtype=torch.int32, device=DEV)
    q = inputs.normal_bf16((3, 4, 64), 1.0, seed=12).to(DEV)
    cap = table.shape[1] * 16
    # the last live page of sequence 1 ends inside its page: write the rest of it so that it holds no NaN
    for c in (k, v):
        c.scale_inv.nan_to_num_(0.5)
        c.cache[(c.cache & 0x7F) == 0x7F] = 1
    if kind == "decode":
        out, lse = fp8q.paged_attention_decode(q, k, v, table, ln)
    else:
        out, lse = fp8q.paged_attention_prefill(q, torch.tensor([0, 1, 2, 3], device=DEV), k, v, table, ln)
    eff = [70, cap, 33]
    check_rows(out, lse, q, k, v, table, eff, [(b, b, n - 1) for b, n in enumerate(eff)], 0.125, 0, 0,
               scaled_v=kind == "prefill")
    ln[1] = -3
    if kind == "decode":
        out, lse = fp8q.paged_attention_decode(q, k, v, table, ln)
    else:
        out, lse = fp8q.paged_attention_prefill(q, torch.tensor([0, 1, 2, 3], device=DEV), k, v, table, ln)
    assert torch.all(out[1] == 0) and torch.all(lse[1] == -math.inf)


def test_hidden_nan_stays_hidden_and_visible_nan_shows():
    """A NaN code in K or V at position j reaches exactly the queries that see j (V: only its own element)."""
    n, Dh, bs = 200, 64, 16
    for which in ("k", "v"):
        for j in (0, 100, 130, 199):
            k, v, table, ln = make_caches([n], 1, Dh, bs, 0, seed=9)
            c = k if which == "k" else v
            blk = int(table[0, j // bs])
            c.cache[blk, j % bs, 0, 5] = 0x7F
            q = inputs.normal_bf16((n, 2, Dh), 1.0, seed=12).to(DEV)
            for window, sinks in ((0, 0), (40, 2)):
                out, lse = fp8q.paged_attention_prefill(q, torch.tensor([0, n], device=DEV), k, v, table, ln, window,
                                                        sinks)
                p = torch.arange(n, device=DEV)
                sees = (p >= j) & ((window == 0) | (j > p - window) | (j < sinks))
                bad = torch.isnan(out.float())
                want = torch.zeros_like(bad)
                if which == "k":
                    want[sees] = True
                    assert torch.equal(torch.isnan(lse).all(-1), sees)
                else:
                    want[:, :, 5] = sees[:, None]
                    assert not torch.isnan(lse).any()
                assert torch.equal(bad, want), (which, j, window)
                o1, l1 = fp8q.paged_attention_decode(q[n - 1:], k, v, table, ln, window, sinks)
                assert torch.equal(torch.isnan(o1[0].float()), want[n - 1]), (which, j, window)


@pytest.mark.parametrize("spread", [1e-4, 1.0, 30.0])
def test_row_scales_of_very_different_size(spread):
    """Value rows a millionfold apart, and logits so large that one token holds all the weight."""
    lens = [260]
    k, v, table, ln = make_caches(lens, 2, 128, 16, 0, seed=21)
    g = torch.Generator().manual_seed(3)
    v.scale_inv.mul_(10.0 ** (torch.rand(v.scale_inv.shape, generator=g) * 6 - 3).to(DEV))
    k.scale_inv.mul_(spread)
    q = inputs.normal_bf16((1, 4, 128), 1.0, seed=12).to(DEV)
    out, lse = fp8q.paged_attention_decode(q, k, v, table, ln)
    check_rows(out, lse, q, k, v, table, lens, [(0, 0, 259)], 128 ** -0.5, 0, 0)
    o2, l2 = fp8q.paged_attention_prefill(q, torch.tensor([0, 1], device=DEV), k, v, table, ln)
    check_rows(o2, l2, q, k, v, table, lens, [(0, 0, 259)], 128 ** -0.5, 0, 0, scaled_v=True)


@pytest.mark.parametrize("qscale", [1e-30, 1e30])
def test_queries_of_extreme_size(qscale):
    lens = [90]
    k, v, table, ln = make_caches(lens, 1, 64, 16, 0, seed=23)
    q = (inputs.normal_bf16((1, 3, 64), 1.0, seed=12).float() * qscale).bfloat16().to(DEV)
    s = 0.125 / qscale
    out, lse = fp8q.paged_attention_decode(q, k, v, table, ln, softmax_scale=s)
    check_rows(out, lse, q, k, v, table, lens, [(0, 0, 89)], float(torch.tensor(s)), 0, 0)
    out, lse = fp8q.paged_attention_prefill(q, torch.tensor([0, 1], device=DEV), k, v, table, ln, softmax_scale=s)
    check_rows(out, lse, q, k, v, table, lens, [(0, 0, 89)], float(torch.tensor(s)), 0, 0, scaled_v=True)


def test_queries_inside_a_fused_projection_and_other_streams():
    """q as a strided slice; the calls on a side stream."""
    lens = [77, 130]
    k, v, table, ln = make_caches(lens, 2, 64, 16, 0, seed=31)
    fused = inputs.normal_bf16((2, 8 * 64), 1.0, seed=32).to(DEV)
    q = fused[:, :4 * 64].view(2, 4, 64)
    assert not q.is_contiguous()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = fp8q.paged_attention_decode(q, k, v, table, ln)
        o2, l2 = fp8q.paged_attention_prefill(q, torch.tensor([0, 1, 2], device=DEV), k, v, table, ln)
    torch.cuda.current_stream().wait_stream(s)
    rows = [(i, i, n - 1) for i, n in enumerate(lens)]
    check_rows(out, lse, q, k, v, table, lens, rows, 0.125, 0, 0)
    check_rows(o2, l2, q, k, v, table, lens, rows, 0.125, 0, 0, scaled_v=True)


def test_calls_repeat_bit_for_bit_and_replay_in_a_graph_with_new_lengths():
    lens = [900, 30, 411]
    k, v, table, ln = make_caches(lens, 4, 128, 16, 0, seed=41)
    q = inputs.normal_bf16((3, 16, 128), 1.0, seed=42).to(DEV)
    off = torch.arange(4, device=DEV)
    mass = torch.zeros((3, 4, 900), device=DEV)
    ws = fp8q.paged_attention_workspace(3, 16, 4, 128, table.shape[1] * 16, True)
    wp = fp8q.paged_attention_workspace(3, 16, 4, 128, tokens=3)

    def step():
        a = fp8q.paged_attention_decode(q, k, v, table, ln, 300, 4, mass=mass, mass_decay=0.0, workspace=ws)
        return a + fp8q.paged_attention_prefill(q, off, k, v, table, ln, workspace=wp)

    def bits(x):      # [899, 31, 255] below reads one stale slot (NaN): bit patterns are compared
        return x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)

    eager = [x.clone() for x in step()]
    again = step()
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(eager, again))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(g):
        got = step()
    for new in ([900, 30, 411], [16, 0, 1], [899, 31, 255]):
        ln.copy_(torch.tensor(new, dtype=torch.int32))
        mass.zero_()
        g.replay()
        torch.cuda.synchronize()
        graph = [x.clone() for x in got] + [mass.clone()]
        mass.zero_()
        want = [x.clone() for x in step()] + [mass.clone()]
        assert all(torch.equal(bits(x), bits(y)) for x, y in zip(graph, want)), new


def test_empty_calls():
    k, v, table, ln = make_caches([20], 2, 64, 16, 0, seed=1)
    z = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    out, lse = fp8q.paged_attention_decode(z, k, v, table[:0], ln[:0])
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = fp8q.paged_attention_prefill(z, torch.zeros(2, dtype=torch.int64, device=DEV), k, v, table, ln)
    assert out.shape == (0, 4, 64)
    # a cache without pages: nothing is visible
    e = fp8q.PagedKVCache(0, 16, 2, 64, device=DEV)
    q = inputs.normal_bf16((1, 4, 64), 1.0, seed=12).to(DEV)
    out, lse = fp8q.paged_attention_decode(q, e, e, table, ln)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)


EVICT = [
    # lens, H, Dh, bs, budget, sinks, recent
    ([1], 1, 8, 1, 1, 0, 0),
    ([2], 1, 16, 1, 1, 0, 0),
    ([2], 1, 16, 1, 1, 0, 1),
    ([0, 5, 64, 65, 66, 130], 2, 64, 16, 64, 4, 10),
    ([300, 20], 4, 128, 16, 100, 0, 0),
    ([300, 301], 2, 80, 24, 64, 30, 34),
    ([1000, 999], 3, 40, 7, 517, 3, 100),
    ([2100], 1, 128, 64, 33, 1, 0),
    ([5000, 700], 2, 16, 100, 600, 4, 50),
]


def run_evict(lens, H, Dh, bs, budget, sinks, recent, mass, seed=3):
    k, v, table, ln = make_caches(lens, H, Dh, bs, 0, seed=seed, stale=False)
    used = k.num_blocks
    need = [(min(n, budget) + bs - 1) // bs for n in lens]
    grow = sum(need) + 1
    for c in (k, v):
        c.cache = torch.cat([c.cache, torch.full((grow,) + c.cache.shape[1:], 0x55, dtype=torch.uint8, device=DEV)])
        c.scale_inv = torch.cat([c.scale_inv, torch.full((grow,) + c.scale_inv.shape[1:], 3.0, device=DEV)])
        c.num_blocks += grow
    perm = torch.randperm(grow, generator=torch.Generator().manual_seed(seed)) + used
    dst = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        dst[b, :m] = perm[at:at + m].int()
        at += m
    before = [x.clone() for x in (k.cache, k.scale_inv, v.cache, v.scale_inv)]
    kept, mo, lo = fp8q.paged_kv_evict(k, v, table, ln, mass, dst.to(DEV), budget, sinks, recent)
    return k, v, table, ln, dst, before, kept, mo, lo


@pytest.mark.parametrize("case", EVICT, ids=lambda c: "-".join(str(x) for x in c[1:]) + f"-n{max(c[0])}")
@pytest.mark.parametrize("values", ["random", "ties", "strange"])
def test_evict(case, values):
    lens, H, Dh, bs, budget, sinks, recent = case
    B, ld = len(lens), max(max(lens), 1)
    g = torch.Generator().manual_seed(5)
    mass = torch.rand((B, H, ld), generator=g)
    if values == "ties":
        mass = (mass * 4).floor()
        mass[torch.rand(mass.shape, generator=g) < 0.2] = -0.0
    elif values == "strange":
        mass -= 0.5
        for i, x in enumerate((math.nan, math.inf, -math.inf, 1e-44, -1e-44)):
            mass[torch.rand(mass.shape, generator=g) < 0.1] = x
        mass = mass[..., :max(1, ld - 20)].contiguous()      # later positions have no mass recorded
    mass = mass.to(DEV)
    k, v, table, ln, dst, before, kept, mo, lo = run_evict(lens, H, Dh, bs, budget, sinks, recent, mass)
    kc, ks, vc, vs = (x.clone().flatten(0, 1).cpu() for x in before)
    mh, th = mass.cpu(), table.cpu()
    ld = mass.shape[2]
    want_mass = torch.zeros_like(mh)
    for b, n in enumerate(lens):
        assert int(lo[b]) == min(n, budget)
        for h in range(H):
            want = ref.evict(mh[b, h].tolist(), n, budget, sinks, recent)
            assert kept[b, h].tolist() == want + [-1] * (budget - len(want)), (b, h)
            for r, j in enumerate(want):
                if r < ld:
                    want_mass[b, h, r] = mh[b, h, j] if j < ld else 0.0
                s = ref.slot_of(th[b].tolist(), j, bs, k.num_blocks)
                d = int(dst[b, r // bs]) * bs + r % bs
                for x, y in ((kc, before[0]), (ks, before[1]), (vc, before[2]), (vs, before[3])):
                    x[d, h] = y.flatten(0, 1)[s, h].cpu()
    assert torch.equal(mo.cpu().view(torch.int32), want_mass.view(torch.int32))
    for x, y in ((kc, k.cache), (ks, k.scale_inv), (vc, v.cache), (vs, v.scale_inv)):
        assert torch.equal(x, y.flatten(0, 1).cpu())          # every other slot is as it was


def test_evict_bad_pages_and_lengths_in_place():
    """A source page that is none is copied as zeros, a destination page that is none is skipped; lens_out may be
    seq_lens itself."""
    k, v, table, ln = make_caches([64], 2, 64, 16, 0, seed=8, stale=False, spare=6)
    used = sorted(int(x) for x in table[0])
    free = [x for x in range(k.num_blocks) if x not in used]
    dst = torch.tensor([[free[0], k.num_blocks + 3, free[1]]], dtype=torch.int32, device=DEV)
    table[0, 1] = -7
    mass = torch.arange(64, dtype=torch.float32, device=DEV).repeat(1, 2, 1)
    kept = torch.empty((1, 2, 40), dtype=torch.int32, device=DEV)
    mo = torch.empty((1, 2, 10), device=DEV)
    b0 = k.cache.clone()
    fp8q.fp8_paged_kv_evict(k.cache, k.scale_inv, v.cache, v.scale_inv, 2, 64, 16, k.num_blocks, table, ln, 1, 4, mass,
                            64, dst, 3, 40, 12, 0, kept, mo, 10, ln)
    assert int(ln[0]) == 40
    want = list(range(12)) + list(range(36, 64))
    assert kept[0, 0].tolist() == want and mo[0, 1].tolist() == [float(x) for x in want[:10]]
    old = torch.zeros((40, 2, 64), dtype=torch.uint8)
    for r, j in enumerate(want):
        blk = int(table[0, j // 16])
        if blk >= 0:
            old[r] = b0[blk, j % 16].cpu()
    assert torch.equal(k.cache[free[0]].cpu(), old[:16])
    assert torch.equal(k.cache[free[1]][:8].cpu(), old[32:])
    assert torch.equal(k.cache[free[1]][8:], b0[free[1]][8:])


def test_a_sequence_lives_through_prefill_decode_eviction_and_decode():
    """The calls as a server makes them: prompt written and attended, tokens generated while their weights add up, the
    sequence cut to a budget, generation going on over the pages that remain."""
    H, G, Dh, bs, n0, steps, budget, sinks, recent = 2, 4, 64, 16, 90, 12, 48, 4, 16
    nb = 24
    k, v = (fp8q.PagedKVCache(nb, bs, H, Dh, device=DEV) for _ in range(2))
    pages = torch.randperm(nb, generator=torch.Generator().manual_seed(1))
    table = pages[None, :8].int().to(DEV)
    fresh = pages[None, 8:12].int().to(DEV)
    scale = Dh ** -0.5

    def write(table, first, count, seed):
        j = torch.arange(first, first + count, device=DEV)
        slots = table[0, j // bs].long() * bs + j % bs
        for i, c in enumerate((k, v)):
            c.write(inputs.normal_bf16((count, H, Dh), 1.0, seed=seed + i).to(DEV), slots)

    write(table, 0, n0, 100)
    ln = torch.tensor([n0], dtype=torch.int32, device=DEV)
    q = inputs.normal_bf16((n0, H * G, Dh), 1.0, seed=7).to(DEV)
    out, lse = fp8q.paged_attention_prefill(q, torch.tensor([0, n0], device=DEV), k, v, table, ln)
    check_rows(out, lse, q, k, v, table, [n0], [(t, 0, t) for t in range(n0)], scale, 0, 0, scaled_v=True)
    mass = torch.zeros((1, H, 128), device=DEV)
    n = n0
    total = torch.zeros((H, 128), dtype=torch.float64)
    bound = torch.zeros((H, 128), dtype=torch.float64)
    for s in range(steps):
        write(table, n, 1, 200 + 2 * s)
        n += 1
        ln.fill_(n)
        q = inputs.normal_bf16((1, H * G, Dh), 1.0, seed=300 + s).to(DEV)
        out, lse = fp8q.paged_attention_decode(q, k, v, table, ln, mass=mass)
        check_rows(out, lse, q, k, v, table, [n], [(0, 0, n - 1)], scale, 0, 0)
        host = ref.Cache(k, v)
        for h in range(H):
            r = ref.attend(host, table[0].tolist(), n, n - 1, q[0, h * G:(h + 1) * G].cpu(), h, scale)
            w = r["w"].sum(0)
            total[h, :n] += w
            bound[h, :n] += (2 * r["ez"].max() + 2.0 ** -19) * w + steps * 2.0 ** -24 * total[h, :n]
    assert torch.all((mass[0].cpu().double() - total).abs() <= bound + 1e-30)
    kept, mass2, ln2 = fp8q.paged_kv_evict(k, v, table, ln, mass, fresh, budget, sinks, recent)
    for h in range(H):
        assert kept[0, h].tolist() == ref.evict(mass[0, h].tolist(), n, budget, sinks, recent)
    q = inputs.normal_bf16((1, H * G, Dh), 1.0, seed=400).to(DEV)
    out, lse = fp8q.paged_attention_decode(q, k, v, fresh, ln2, mass=mass2)
    check_rows(out, lse, q, k, v, fresh, [budget], [(0, 0, budget - 1)], scale, 0, 0)
    # the same rows attended where they came from, through a table that names the kept positions one by one
    host = ref.Cache(k, v)
    for h in range(H):
        r = ref.attend(host, table[0].tolist(), n, n - 1, q[0, h * G:(h + 1) * G].cpu(), h, scale)
        idx = [r["pos"].index(j) for j in kept[0, h].tolist()]
        ss = [ref.slot_of(table[0].tolist(), j, bs, nb) for j in kept[0, h].tolist()]
        w = r["w"][:, idx]
        w = w / w.sum(-1, keepdim=True)
        want = w @ host.v[ss, h]
        tol = 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * (2.0 ** -11 + 2.0 ** -18 + 2 * r["ez"][:, None]) * (
            w @ host.v[ss, h].abs())
        assert torch.all((out[0, h * G:(h + 1) * G].float().cpu().double() - want).abs() <= tol)


def test_a_token_leaves_the_batch_unchanged_for_the_others():
    """A padded batch: an empty slot's table row may hold anything."""
    lens = [50, 0, 20]
    k, v, table, ln = make_caches(lens, 2, 64, 16, 0, seed=51)
    table[1] = 10 ** 9
    q = inputs.normal_bf16((3, 4, 64), 1.0, seed=52).to(DEV)
    out, lse = fp8q.paged_attention_decode(q, k, v, table, ln)
    check_rows(out, lse, q, k, v, table, lens, [(b, b, n - 1) for b, n in enumerate(lens)], 0.125, 0, 0)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_more_sequences_than_threads(kind):
    """1300 sequences of 0 to 40 tokens, one or two of them new (more row blocks than one pass of the planning
    kernels takes), checked at the ends of the passes and in between."""
    B, H, G, Dh, bs = 1300, 2, 2, 32, 8
    lens = [(7 * b) % 41 for b in range(B)]
    k, v, table, ln = make_caches(lens, H, Dh, bs, 0, seed=61)
    new = [1] * B if kind == "decode" else [min(n, 1 + b % 2) for b, n in enumerate(lens)]
    off = torch.tensor([0] + new).cumsum(0)
    q = inputs.normal_bf16((int(off[-1]), H * G, Dh), 1.0, seed=62).to(DEV)
    if kind == "decode":
        out, lse = fp8q.paged_attention_decode(q, k, v, table, ln)
    else:
        out, lse = fp8q.paged_attention_prefill(q, off.to(DEV), k, v, table, ln)
    some = sorted(set(range(0, B, 37)) | {511, 512, 513, 1022, 1023, 1024, 1025, B - 2, B - 1})
    rows = [(int(off[b]) + i, b, lens[b] - new[b] + i) for b in some for i in range(new[b])]
    check_rows(out, lse, q, k, v, table, lens, rows, Dh ** -0.5, 0, 0, scaled_v=kind == "prefill")


@pytest.mark.parametrize("slope", [0.4, -0.4, 8.0])
@pytest.mark.parametrize("Dh", [64, 256])
def test_logits_that_rise_or_fall_along_the_sequence(slope, Dh):
    """Every tile moves the softmax reference, by up to a thousand powers of two (or none after the first does)."""
    n, bs = 700, 16
    k, v, table, ln = make_caches([n], 1, Dh, bs, 0, seed=71)
    _, slots = inputs.paged_layout([n], bs, k.num_blocks, 71)
    u = torch.ones(Dh) / Dh ** 0.5
    ramp = slope * (torch.arange(n, dtype=torch.float32) - n / 2)
    noise = inputs.normal_bf16((n, 1, Dh), 0.5, seed=72).float()
    k.write((ramp[:, None, None] * u + noise).bfloat16().to(DEV), slots.to(DEV))
    new = 150
    q = (u + inputs.normal_bf16((new, 3, Dh), 0.05, seed=73).float()).bfloat16().to(DEV)
    out, lse = fp8q.paged_attention_prefill(q, torch.tensor([0, new], device=DEV), k, v, table, ln, softmax_scale=1.0)
    rows = [(i, 0, n - new + i) for i in (0, 1, 31, 77, 127, 128, new - 1)]
    check_rows(out, lse, q, k, v, table, [n], rows, 1.0, 0, 0, scaled_v=True)
    out, lse = fp8q.paged_attention_decode(q[-1:], k, v, table, ln, softmax_scale=1.0)
    check_rows(out, lse, q[-1:], k, v, table, [n], [(0, 0, n - 1)], 1.0, 0, 0)


def test_two_calls_at_once():
    """Decode and prefill side by side on two streams, each with its own workspace, give what they give alone; the
    sequences share pages."""
    lens = [3000, 2000, 2500]
    H, G, Dh = 4, 2, 128
    k, v, table, ln = make_caches(lens, H, Dh, 16, 0, seed=81)
    table[1, :40] = table[0, :40]                        # a prefix in common
    q = inputs.normal_bf16((3, H * G, Dh), 1.0, seed=82).to(DEV)
    q2 = inputs.normal_bf16((600, H * G, Dh), 1.0, seed=83).to(DEV)
    off = torch.tensor([0, 200, 400, 600], device=DEV)
    ws = fp8q.paged_attention_workspace(3, H * G, H, Dh, table.shape[1] * 16)
    wp = fp8q.paged_attention_workspace(3, H * G, H, Dh, tokens=600)
    alone = [x.clone() for x in fp8q.paged_attention_decode(q, k, v, table, ln, workspace=ws)]
    alone2 = [x.clone() for x in fp8q.paged_attention_prefill(q2, off, k, v, table, ln, workspace=wp)]
    check_rows(*alone, q, k, v, table, lens, [(b, b, n - 1) for b, n in enumerate(lens)], Dh ** -0.5, 0, 0)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got, got2 = [], []
    for _ in range(10):
        with torch.cuda.stream(s1):
            got.append(fp8q.paged_attention_decode(q, k, v, table, ln, workspace=ws))
        with torch.cuda.stream(s2):
            got2.append(fp8q.paged_attention_prefill(q2, off, k, v, table, ln, workspace=wp))
    torch.cuda.synchronize()
    for r, r2 in zip(got, got2):
        assert torch.equal(r[0], alone[0]) and torch.equal(r[1], alone[1])
        assert torch.equal(r2[0], alone2[0]) and torch.equal(r2[1], alone2[1])
    assert fp8q.fp8_device_error() == 0


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_softmax_scales_of_zero_and_below(scale):
    """Zero weighs all visible tokens alike; a negative scale turns the order round."""
    lens, new, Dh = [333, 20], [40, 20], 128
    k, v, table, ln = make_caches(lens, 2, Dh, 16, 0, seed=91)
    off = torch.tensor([0, 40, 60])
    q = inputs.normal_bf16((60, 6, Dh), 1.0, seed=92).to(DEV)
    s = float(torch.tensor(scale))                       # as the call takes it: fp32
    out, lse = fp8q.paged_attention_prefill(q, off.to(DEV), k, v, table, ln, 100, 3, softmax_scale=scale)
    rows = [(int(off[b]) + i, b, lens[b] - new[b] + i) for b in range(2) for i in (0, 7, new[b] - 1)]
    check_rows(out, lse, q, k, v, table, lens, rows, s, 100, 3, scaled_v=True)
    out, lse = fp8q.paged_attention_decode(q[:2], k, v, table, ln, 100, 3, softmax_scale=scale)
    check_rows(out, lse, q, k, v, table, lens, [(b, b, n - 1) for b, n in enumerate(lens)], s, 100, 3)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_query_that_is_not_finite_stays_in_its_row(bad):
    lens, new = [200, 150], 100
    k, v, table, ln = make_caches(lens, 2, 64, 16, 0, seed=95)
    off = torch.tensor([0, new, 2 * new], device=DEV)
    q = inputs.normal_bf16((2 * new, 4, 64), 1.0, seed=96).to(DEV)
    q2 = q.clone()
    q2[17, 1, 5] = bad
    out, lse = fp8q.paged_attention_prefill(q, off, k, v, table, ln)
    o2, l2 = fp8q.paged_attention_prefill(q2, off, k, v, table, ln)
    assert not torch.isfinite(l2[17, 1]) and not torch.isfinite(o2[17, 1].float()).all()
    hit = torch.zeros(2 * new, 4, dtype=torch.bool, device=DEV)
    hit[17, 1] = True
    assert torch.equal(o2[~hit], out[~hit]) and torch.equal(l2[~hit], lse[~hit])
    out, lse = fp8q.paged_attention_decode(q[16:18], k, v, table, ln)
    o2, l2 = fp8q.paged_attention_decode(q2[16:18], k, v, table, ln)
    assert not torch.isfinite(l2[1, 1]) and not torch.isfinite(o2[1, 1].float()).all()
    assert torch.equal(o2[~hit[16:18]], out[~hit[16:18]]) and torch.equal(l2[~hit[16:18]], lse[~hit[16:18]])


@pytest.mark.parametrize("bs", [64, 7])
def test_a_pool_past_four_gigabytes(bs):
    """Pages whose bytes lie behind 2^32 give what the same pages give in a small pool, bit for bit."""
    lens, H, Dh = [200, 91], 8, 256
    k, v, table, ln = make_caches(lens, H, Dh, bs, 0, seed=97, spare=40)
    nb = 2200000 // bs
    assert nb * bs * H * Dh > 1 << 32
    K, V = (fp8q.PagedKVCache(nb, bs, H, Dh, 0, device=DEV) for _ in range(2))
    shift = nb - k.num_blocks
    for big, small in ((K, k), (V, v)):
        big.cache[shift:] = small.cache
        big.scale_inv[shift:] = small.scale_inv
    far = torch.where(table >= 0, table + shift, table)
    q = inputs.normal_bf16((60, 16, Dh), 1.0, seed=98).to(DEV)
    off = torch.tensor([0, 40, 60], device=DEV)
    mass, mass2 = (torch.zeros((2, H, 200), device=DEV) for _ in range(2))
    got = [fp8q.paged_attention_decode(q[:2], *c, t, ln, mass=m) + fp8q.paged_attention_prefill(q, off, *c, t, ln)
           for c, t, m in (((k, v), table, mass), ((K, V), far, mass2))]
    assert all(torch.equal(x, y) for x, y in zip(*got)) and torch.equal(mass, mass2)
    used = {int(x) for x in table.flatten()}
    free = [x for x in range(k.num_blocks) if x not in used]
    n = (50 + bs - 1) // bs
    dst = torch.tensor([free[:n], free[n:2 * n]], dtype=torch.int32, device=DEV)
    a = fp8q.paged_kv_evict(k, v, table, ln, mass, dst, 50, 2, 10)
    b = fp8q.paged_kv_evict(K, V, far, ln, mass2, dst + shift, 50, 2, 10)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    for big, small in ((K, k), (V, v)):
        assert torch.equal(big.cache[shift:], small.cache)
        assert torch.equal(big.scale_inv[shift:].nan_to_num(7.0), small.scale_inv.nan_to_num(7.0))
        assert not big.cache[:1000].any()
