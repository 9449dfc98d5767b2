"""Paged attention where scales, queries or weights are far apart: a row's result depends on what the row sees alone,
and to the accuracy that its own terms allow."""
import math

import pytest
import torch

from fp8_scaled_quantization_amax_b200 import fp8q, inputs
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
