"""Arguments that the paged attention and eviction calls refuse, before any device access (no GPU needed)."""
import ctypes

import pytest
import torch

from fp8_scaled_quantization_amax_b200 import fp8q
from tests import paged_ref as ref

OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, CUDA = range(6)
P = ctypes.c_void_p
FAKE, ODD, N = P(0x10000), P(0x10002), P(0)
BIG = 1 << 40


def decode(**kw):
    a = dict(q=FAKE, ld_q=512, B=2, Hq=8, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, H=2, Dh=64, bs=16, nb=10, fmt=0, table=FAKE,
             lens=FAKE, mb=4, window=0, sinks=0, scale=0.125, out=FAKE, lse=None, mass=None, ld_mass=0, decay=1.0,
             ws=FAKE, ws_bytes=1 << 40, stream=N)
    a.update(kw)
    return fp8q.lib().fp8_paged_attention_decode(*a.values())


def prefill(**kw):
    a = dict(q=FAKE, ld_q=512, T=9, off=FAKE, B=2, Hq=8, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, H=2, Dh=64, bs=16, nb=10,
             fmt=0, table=FAKE, lens=FAKE, mb=4, window=0, sinks=0, scale=0.125, out=FAKE, lse=None, ws=FAKE,
             ws_bytes=1 << 40, stream=N)
    a.update(kw)
    return fp8q.lib().fp8_paged_attention_prefill(*a.values())


def evict(**kw):
    a = dict(kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, H=2, Dh=64, bs=16, nb=10, table=FAKE, lens=FAKE, B=2, mb=4, mass=FAKE,
             ld_mass=64, dst=FAKE, dmb=4, budget=32, sinks=4, recent=8, kept=FAKE, mo=FAKE, ld_out=64, lo=FAKE, stream=N)
    a.update(kw)
    return fp8q.lib().fp8_paged_kv_evict(*a.values())


SHARED = [
    (dict(fmt=2), INVALID), (dict(fmt=-1), INVALID),
    (dict(Dh=24, ld_q=512), SHAPE), (dict(Dh=272, ld_q=4096), SHAPE), (dict(Dh=0), SHAPE), (dict(Dh=8), SHAPE),
    (dict(H=0), SHAPE), (dict(H=-1), SHAPE), (dict(H=256, Hq=256, ld_q=BIG), SHAPE), (dict(Hq=7), SHAPE),
    (dict(Hq=0), SHAPE), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(bs=0), SHAPE), (dict(nb=-1), SHAPE),
    (dict(nb=1 << 30), SHAPE), (dict(bs=1 << 31, nb=0), SHAPE), (dict(mb=-1), SHAPE), (dict(mb=1 << 27), SHAPE), (dict(window=-1), SHAPE),
    (dict(sinks=-1), SHAPE), (dict(ld_q=504), SHAPE), (dict(ld_q=516), ALIGN),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(lens=None), INVALID), (dict(table=None), INVALID),
    (dict(kc=None), INVALID), (dict(ks=None), INVALID), (dict(vc=None), INVALID), (dict(vs=None), INVALID),
    (dict(q=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(kc=ODD), ALIGN), (dict(vc=ODD), ALIGN), (dict(ws=ODD), ALIGN),
]


@pytest.mark.parametrize("call", [decode, prefill])
@pytest.mark.parametrize("kw,status", SHARED, ids=lambda x: str(x))
def test_attention_refuses(call, kw, status):
    assert call(**kw) == status


def test_attention_refuses_what_is_its_own():
    assert prefill(T=-1) == SHAPE
    assert prefill(T=1 << 30) == SHAPE               # T * Hq past 2^31
    assert prefill(off=None) == INVALID
    assert decode(mass=FAKE, ld_mass=-1) == SHAPE
    assert decode(mass=FAKE, ld_mass=64, decay=float("nan")) == INVALID
    assert decode(B=0) == OK and prefill(B=0) == OK and prefill(T=0) == OK


def test_attention_refuses_more_rows_than_it_can_number():
    """Row blocks of 256 rows have to end below 2^31, and decode's join takes a block per 32 elements of a row."""
    assert prefill(T=(1 << 28) - 1) == SHAPE and prefill(T=1, Hq=(1 << 31) - 2, ld_q=BIG) == SHAPE
    for Dh, Hq in ((64, 1 << 20), (80, 1 << 19), (128, 1 << 19), (256, 1 << 18)):
        assert decode(B=1 << 10, Hq=Hq, Dh=Dh, ld_q=BIG) == SHAPE       # 2^31 blocks
        assert decode(B=1 << 10, Hq=Hq - 2, Dh=Dh, ld_q=BIG, q=None) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(H=0), SHAPE), (dict(Dh=12), SHAPE), (dict(H=256), SHAPE), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE),
    (dict(bs=0), SHAPE), (dict(nb=1 << 30), SHAPE), (dict(mb=-1), SHAPE), (dict(dmb=-1), SHAPE), (dict(mb=1 << 27), SHAPE), (dict(dmb=1 << 27), SHAPE),
    (dict(ld_mass=-1), SHAPE), (dict(ld_out=-1), SHAPE), (dict(budget=0), SHAPE), (dict(budget=1 << 31), SHAPE),
    (dict(sinks=-1), SHAPE), (dict(recent=-1), SHAPE), (dict(sinks=20, recent=13), SHAPE), (dict(sinks=BIG), SHAPE),
    (dict(recent=BIG), SHAPE), (dict(lens=None), INVALID), (dict(kept=None), INVALID), (dict(mo=None), INVALID),
    (dict(lo=None), INVALID), (dict(mass=None), INVALID), (dict(table=None), INVALID), (dict(dst=None), INVALID),
    (dict(kc=None), INVALID), (dict(vs=None), INVALID), (dict(kc=ODD), ALIGN), (dict(vc=ODD), ALIGN), (dict(B=0), OK),
], ids=lambda x: str(x))
def test_evict_refuses(kw, status):
    assert evict(**kw) == status


def test_without_a_device_nothing_runs():
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert decode() in (UNSUPPORTED, CUDA)
    assert prefill() in (UNSUPPORTED, CUDA)
    assert evict() in (UNSUPPORTED, CUDA)


def test_wrappers_refuse_host_tensors_and_unlike_caches():
    c = fp8q.PagedKVCache(2, 4, 1, 16, device="cpu")
    d = fp8q.PagedKVCache(2, 4, 1, 16, fp8q.E5M2, device="cpu")
    q = torch.zeros((1, 1, 16), dtype=torch.bfloat16)
    t, n = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fp8q.paged_attention_decode(q, c, c, t, n)
    with pytest.raises(ValueError):
        fp8q.paged_attention_prefill(q, torch.tensor([0, 1]), c, c, t, n)
    with pytest.raises(ValueError):
        fp8q.paged_kv_evict(c, d, t, n, torch.zeros((1, 1, 8)), t, 4)
    with pytest.raises(ValueError):
        fp8q.PagedKVCache.from_tensors(c.cache, c.scale_inv)


def test_reference_against_closed_forms():
    """The 64-bit reference itself: uniform attention is the mean, a window of one is the token itself."""
    c = fp8q.PagedKVCache(3, 4, 1, 16, device="cpu")
    codes = torch.randint(0, 126, c.cache.shape, generator=torch.Generator().manual_seed(0), dtype=torch.uint8)
    c.cache.copy_(codes)
    c.scale_inv.fill_(0.25)
    host = ref.Cache(c, c)
    vals = codes.view(torch.float8_e4m3fn).double() * 0.25
    q = torch.zeros((2, 16), dtype=torch.bfloat16)
    r = ref.attend(host, [2, 0, -1], 10, 9, q, 0, 1.0)
    rows = torch.cat([vals[2, :, 0], vals[0, :, 0]])           # page 2, page 0; the third page is none
    assert torch.allclose(r["out"][0], rows.mean(0), rtol=1e-14) and r["pos"] == list(range(8))
    assert abs(float(r["lse"][0]) - 2.0794415416798357) < 1e-14
    r = ref.attend(host, [2, 0, 1], 10, 9, q + 1, 0, 1.0, window=1)
    assert torch.allclose(r["out"][1], vals[1, 1, 0], rtol=1e-14) and r["pos"] == [9]
    r = ref.attend(host, [2, 0, 1], 10, 9, q + 1, 0, 1.0, window=2, sinks=3)
    assert r["pos"] == [0, 1, 2, 8, 9]
    assert ref.evict([0.0, 5.0, 5.0, 1.0, 5.0, 0.0], 6, 4, 1, 1) == [0, 1, 2, 5]
    assert ref.evict([0.0, 5.0], 2, 4, 1, 1) == [0, 1]
