"""64-bit reference of attention over a paged FP8 cache and of eviction from it, from the formulas, on the CPU
(plain loops over sequences and heads; no library code), and the error bounds the kernels are held to."""
import math

import torch


def value_table(fmt):
    """The 256 code values of E4M3 (0) or E5M2 (1)."""
    man, bias = (3, 7) if fmt == 0 else (2, 15)
    out = []
    for c in range(256):
        e, f = (c & 127) >> man, c & ((1 << man) - 1)
        v = f * 2.0 ** (1 - bias - man) if e == 0 else (1 + f / (1 << man)) * 2.0 ** (e - bias)
        if fmt == 0 and (c & 127) == 127:
            v = math.nan
        if fmt == 1 and e == 31:
            v = math.nan if f else math.inf
        out.append(-v if c & 128 else v)
    return torch.tensor(out, dtype=torch.float64)


def slot_of(table_row, j, bs, num_blocks):
    """Slot of position j, None where the table holds no page."""
    if j // bs >= len(table_row):
        return None
    blk = int(table_row[j // bs])
    return blk * bs + j % bs if 0 <= blk < num_blocks else None


class Cache:
    """Host copy of a K and a V cache."""

    def __init__(self, k, v):
        self.fmt, self.bs, self.H, self.Dh, self.nb = k.fmt, k.block_size, k.H, k.Dh, k.num_blocks
        vals = value_table(k.fmt)
        self.vcode, self.vscale = vals[v.cache.cpu().reshape(-1, v.H, v.Dh).long()], v.scale_inv.cpu().reshape(-1, v.H)
        self.k = vals[k.cache.cpu().reshape(-1, k.H, k.Dh).long()] * k.scale_inv.cpu().reshape(-1, k.H, 1).double()
        self.v = vals[v.cache.cpu().reshape(-1, k.H, k.Dh).long()] * v.scale_inv.cpu().reshape(-1, k.H, 1).double()


def attend(cache, table_row, n, p, q, h, scale, window=0, sinks=0, scaled_v=False):
    """q [G, Dh] at position p of a sequence of n tokens, KV head h -> dict of out [G, Dh], lse [G], positions,
    weights [G, visible], and the bounds: ez [G] on a logit, tol [G, Dh] on out (scaled_v: of the kernel for several
    tokens, whose fp16 V holds the rows' scales)."""
    G, Dh = q.shape
    js, ss = [], []
    for j in range(0, min(n, p + 1)):
        if window > 0 and j <= p - window and j >= sinks:
            continue
        s = slot_of(table_row, j, cache.bs, cache.nb)
        if s is not None:
            js.append(j)
            ss.append(s)
    q = q.double()
    if not js:
        z = torch.zeros(G, dtype=torch.float64)
        return dict(out=torch.zeros(G, Dh, dtype=torch.float64), lse=torch.full((G,), -math.inf, dtype=torch.float64),
                    pos=js, w=torch.zeros(G, 0, dtype=torch.float64), ez=z, tol=torch.zeros(G, Dh, dtype=torch.float64))
    k, v = cache.k[ss, h], cache.v[ss, h]
    z = scale * (q @ k.T)
    lse = torch.logsumexp(z, -1)
    w = torch.exp(z - lse[:, None])
    out = w @ v
    # A logit: Dh exact products summed in fp32 (each addition off by at most one step, 2^-23, of a partial sum that
    # sum |q k| bounds), one rounded scale and the factors that turn it into a power of two (4 half steps).
    ez = (Dh * 2.0 ** -23 * abs(scale) * (q.abs() @ k.abs().T) + 2.0 ** -22 * z.abs()).amax(-1)
    # The weights: exp (2 ulp and the logit's error, in numerator and sum), rounded once to fp16 (2^-11) for the
    # product with V; fp32 sums; bf16 result (2^-8).
    tol = 2.0 ** -8 * out.abs() + (1 + 2.0 ** -8) * (2.0 ** -11 + 2.0 ** -18 + 2 * ez[:, None]) * (w @ v.abs())
    # What fp16's subnormals lose.  The product with V takes p_j d_j f, where d_j is the row's scale, f a power of two
    # with f max(d) >= 2^8, and p_j = exp(z_j - r) for a reference r that is at most the largest logit, so that
    # l = sum p >= 1.  Rounding below 2^-14 is off by at most 2^-25 for each j, which reaches the result divided by f l:
    # 2^-25 sum |code_j| / (f l) <= 2^-33 max(d) sum |code_j|.
    dmax, codes = cache.vscale[ss, h].double().abs().max(), cache.vcode[ss, h].abs().sum(0)
    if scaled_v:
        # fp16 V = code_j d_j f: the factor d_j f and the product are rounded once each (2^-11 more, twice), and below
        # 2^-14 the product is off by at most 2^-25, that is 2^-25 / f in the result, a weighted mean.  f is a power
        # of two with f max(d) >= 2^6 (E4M3) or 2^-1 (E5M2), the maximum over every live position of the sequence.
        # The weights reach at least 2^7 (l >= 2^7), so that theirs loses at most 2^-32 max(d) sum |code_j|.
        live = [x for x in (slot_of(table_row, j, cache.bs, cache.nb) for j in range(n)) if x is not None]
        dall = cache.vscale[live, h].double().abs().max()
        tol = tol + (1 + 2.0 ** -7) * 2.0 ** -10 * (w @ v.abs()) + 2.0 ** (-31 if cache.fmt == 0 else -24) * dall
        tol = tol + 2.0 ** -32 * dmax * codes
    else:
        tol = tol + 2.0 ** -33 * dmax * codes
    return dict(out=out, lse=lse, pos=js, w=w, ez=ez, tol=tol + 1e-30)


def lse_tol(r):
    return 2 * r["ez"] + 2.0 ** -20 * (1 + r["lse"].abs())


def evict(mass_row, n, budget, sinks, recent):
    """Kept positions (ascending) of one (sequence, head); mass_row: list of floats."""
    if n <= budget:
        return list(range(n))
    m = [float(mass_row[j]) if j < len(mass_row) else 0.0 for j in range(n)]
    m = [-math.inf if math.isnan(x) else x for x in m]
    middle = sorted(range(sinks, n - recent), key=lambda j: (-m[j], j))[:budget - sinks - recent]
    return sorted(list(range(sinks)) + middle + list(range(n - recent, n)))
