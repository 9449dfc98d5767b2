"""Error bounds of the paged attention kernels that take only what a query sees into account: no scale, code or query
of another row enters them.  Beside tests/paged_ref.py, whose bounds are wider."""
import torch

from tests import paged_ref as ref


def out_tol(cache, table_row, r, h, prefill):
    """Bound [G, Dh] on the output of ref.attend's r: w_j the weights, d_j the scales' and c_j the codes' magnitudes.

    Both kernels: bf16 result 2^-8 (2^-134 in its subnormals); weights from logits off by ez (numerator and sum), exp
      2^-18, fp16 2^-11.  A weight is an fp32 number, 2^(z - r) for a reference r that is at most the row's largest
      logit (or ends there, by factors that are such numbers too), and zero below 2^-126: a position whose weight is
      less than 2^-125 of the largest (a bit for the logits' error) may be missing altogether.
    One new token: the products p_j d_j are held in fp16 under a power of two that brings the largest so far to 2^6 or
      more (2^5 after a reference that moved by no whole power of two): below 2^-14 off by 2^-25, so 2^-30 of the
      largest w_j d_j, for each code.
    Several: either V holds the scales (the factor and the product rounded to fp16, 2^-11 each; weights reach 2^7, so
      theirs lose 2^-32 d_j c_j at most; E5M2 products below 2^-14 lose 2^-16 d_j; only scales within 2^12 of each
      other, the exponents' 2^11 and the fractions, are held so), or the weights do: p_j d_j reaches 2^12 and is off by
      2^-25 at most, 2^-37 of the largest w_j d_j for each code."""
    ss = [ref.slot_of(table_row, j, cache.bs, cache.nb) for j in r["pos"]]
    if not ss:
        return torch.zeros_like(r["out"])
    w, d, c = r["w"], cache.vscale[ss, h].double().abs(), cache.vcode[ss, h].abs()
    wv = w @ (c * d[:, None])
    tol = 2.0 ** -8 * r["out"].abs() + (1 + 2.0 ** -7) * (2.0 ** -11 + 2.0 ** -18 + 2 * r["ez"][:, None]) * wv
    tol = tol + (w * (w < 2.0 ** -125 * w.amax(-1, keepdim=True))) @ (c * d[:, None])
    most = (w * d).amax(-1)[:, None] * c.sum(0)
    if not prefill:
        return tol + 2.0 ** -30 * most + 2.0 ** -133
    tol = tol + (1 + 2.0 ** -7) * 2.0 ** -10 * wv + 2.0 ** -37 * most
    least = d[d > 0].min() if (d > 0).any() else 0.0
    tol = tol + 2.0 ** -32 * (d.clamp(max=2.0 ** 12 * least) @ c)
    if cache.fmt == 1:
        tol = tol + 2.0 ** -16 * (w @ d)[:, None]
    return tol + 2.0 ** -133


def check(out, lse, q, k, v, table, lens, rows, scale, window=0, sinks=0, prefill=True):
    """rows: (t, b, p) of the query rows to compare with 64 bits; out, lse [T, Hq, ...]."""
    host, H, G = ref.Cache(k, v), k.H, q.shape[1] // k.H
    qh, oh, lh, th = q.cpu(), out.float().cpu().double(), lse.cpu().double(), table.cpu()
    for t, b, p in rows:
        for h in range(H):
            sl = slice(h * G, (h + 1) * G)
            r = ref.attend(host, th[b].tolist(), int(lens[b]), p, qh[t, sl], h, scale, window, sinks)
            tol = out_tol(host, th[b].tolist(), r, h, prefill)
            err = (oh[t, sl] - r["out"]).abs()
            assert torch.all(err <= tol), (t, h, float((err / tol).max()))
            assert torch.all((lh[t, sl] - r["lse"]).abs() <= ref.lse_tol(r)), (t, h)
