"""Cases of the paged FP8 cache's attention and eviction operators, for timing and comparison.

``run`` computes one pass of an operator: in plain torch operations (32-bit arithmetic on the dequantized cache)
while ``own`` is false, through the library's public calls while it is true.  ``exact`` gives the same results in
64 bits, written apart from the plain form.

Kinds of case
  decode   one new token per sequence attends over its pages (optionally a sliding window plus a few first tokens
           that stay visible, optionally returning the attention weight each cached token received)
  prefill  several new tokens per sequence (a prompt, a chunk of one, a few drafted tokens) attend causally
  evict    sequences are cut to a budget of tokens by accumulated attention weight, copied into new pages
"""
import math
import random

import torch

own = False

E4M3, E5M2 = 0, 1


def listed():
    return [
        # one user's chat turn: latency of the smallest call
        dict(name="decode_one_short", kind="decode", B=1, H=8, G=4, Dh=128, bs=16, len=37, ragged=False, fmt=E4M3,
             window=0, sinks=0, weights=False),
        # a serving batch of ragged sequences, no shared heads (the sizes of the paged cache benchmark)
        dict(name="decode_batch_mha", kind="decode", B=32, H=32, G=1, Dh=128, bs=16, len=8192, ragged=True, fmt=E4M3,
             window=0, sinks=0, weights=False),
        # one very long document with grouped heads: all parallelism has to come from the length
        dict(name="decode_long_gqa", kind="decode", B=1, H=8, G=8, Dh=128, bs=64, len=131072, ragged=False, fmt=E4M3,
             window=0, sinks=0, weights=False),
        # streaming generation: window and first tokens, E5M2, small heads, an odd page size
        dict(name="decode_window_sinks", kind="decode", B=48, H=4, G=7, Dh=64, bs=24, len=30000, ragged=True, fmt=E5M2,
             window=1500, sinks=4, weights=False),
        # decode that feeds an eviction policy: the weights come back too
        dict(name="decode_weights", kind="decode", B=8, H=8, G=4, Dh=128, bs=16, len=16384, ragged=True, fmt=E4M3,
             window=0, sinks=0, weights=True),
        # a short prompt: latency
        dict(name="prefill_short", kind="prefill", B=1, H=8, G=4, Dh=128, bs=16, len=100, new=100, ragged=False,
             fmt=E4M3, window=0, sinks=0),
        # drafted tokens checked against a long context: few rows, long axis
        dict(name="prefill_drafts", kind="prefill", B=4, H=8, G=4, Dh=128, bs=16, len=20000, new=5, ragged=True,
             fmt=E4M3, window=0, sinks=0),
        # chunks of long prompts with a window and first tokens, ragged
        dict(name="prefill_chunk_window", kind="prefill", B=6, H=8, G=4, Dh=128, bs=32, len=7000, new=1025, ragged=True,
             fmt=E4M3, window=2048, sinks=4),
        # a whole long prompt, causal
        dict(name="prefill_full", kind="prefill", B=1, H=8, G=4, Dh=128, bs=16, len=8192, new=8192, ragged=False,
             fmt=E4M3, window=0, sinks=0),
        # one sequence a little over its budget
        dict(name="evict_one", kind="evict", B=1, H=8, G=1, Dh=128, bs=16, len=1100, ragged=False, fmt=E4M3,
             budget=1024, sinks=4, recent=128),
        # a ragged batch with an odd head size and budget
        dict(name="evict_ragged", kind="evict", B=24, H=4, G=1, Dh=80, bs=24, len=9001, ragged=True, fmt=E5M2,
             budget=1777, sinks=4, recent=333),
        # every sequence of a full cache halved
        dict(name="evict_batch", kind="evict", B=16, H=32, G=1, Dh=128, bs=16, len=8192, ragged=False, fmt=E4M3,
             budget=4096, sinks=4, recent=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {c["name"]: work(c) for c in listed()}
    while True:
        kind = rng.choice(["decode", "decode", "prefill", "evict"])
        c = dict(kind=kind, B=_log(rng, 1, 48), H=rng.choice([1, 2, 3, 4, 5, 8, 16, 32]),
                 G=rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), Dh=rng.choice([64, 80, 96, 112, 128, 128, 192, 256]),
                 bs=rng.choice([8, 16, 16, 24, 32, 64, 100, 128]), ragged=rng.random() < 0.7,
                 fmt=rng.choice([E4M3, E4M3, E5M2]))
        if c["H"] * c["Dh"] > 8192 or c["H"] * c["G"] > 128:
            continue
        sinks = rng.choice([0, 1, 4, 4, 16, 37])
        if kind == "decode":
            c.update(len=_log(rng, 1, 131072), window=rng.choice([0, 0, _log(rng, 1, 8192)]), sinks=sinks,
                     weights=rng.random() < 0.4)
            cap = most["decode_batch_mha"]
        elif kind == "prefill":
            c.update(len=_log(rng, 1, 20000), window=rng.choice([0, 0, _log(rng, 1, 4096)]), sinks=sinks)
            c.update(new=min(c["len"], _log(rng, 1, 8192)))
            cap = most["prefill_full"]
        else:
            budget = _log(rng, 64, 8192)
            c.update(G=1, len=max(1, int(budget * rng.uniform(0.5, 8.0))), budget=budget, sinks=min(sinks, budget // 4),
                     recent=rng.randint(0, budget // 2))
            cap = most["evict_batch"]
        w = work(c)
        # the plain form works on padded batches: bound what it pads to as well
        padded = c["B"] * c["len"] * c["H"] * c["Dh"]
        scores = c["B"] * c["len"] * c["H"] * c["G"] * c.get("new", 1)
        if (w["bytes"] <= cap["bytes"] and w["flops"] <= cap["flops"] and padded <= 32 * 8192 * 32 * 128
                and scores <= 32 * 8192 * 8192):
            return c


def _lens(c):
    """Sequence lengths: equal, or ragged (the first is the longest, and the last of a batch of 8 or more is an
    empty slot, as in a padded batch)."""
    B, n = c["B"], c["len"]
    if not c["ragged"]:
        return [n] * B
    r = random.Random(B * 1000003 + n)
    out = [n] + [max(1, int(n * r.uniform(0.05, 1.0))) for _ in range(B - 1)]
    if B >= 8:
        out[-1] = 0
    return out


def _news(c):
    """New tokens of each sequence (prefill), at most its length."""
    r = random.Random(c["len"] * 7919 + c["new"])
    lens = _lens(c)
    if not c["ragged"]:
        return [min(c["new"], n) for n in lens]
    return [min(n, c["new"] if i == 0 else max(1, int(c["new"] * r.uniform(0.2, 1.0)))) for i, n in enumerate(lens)]


def _visible(p, window, sinks):
    """How many positions the query at position p sees."""
    if window <= 0:
        return p + 1
    lo = max(0, p - window + 1)
    return p + 1 - lo + min(sinks, lo)


def work(c):
    H, G, Dh = c["H"], c["G"], c["Dh"]
    lens = _lens(c)
    row = Dh + 4                        # one head's codes and scale
    if c["kind"] == "decode":
        vis = sum(_visible(n - 1, c["window"], c["sinks"]) for n in lens if n)
        return {"bytes": vis * H * 2 * row + c["B"] * H * G * (4 * Dh + 4) + (4 * vis * H if c["weights"] else 0),
                "flops": 4 * vis * H * G * Dh}
    if c["kind"] == "prefill":
        pairs = union = 0
        for n, q in zip(lens, _news(c)):
            pairs += sum(_visible(p, c["window"], c["sinks"]) for p in range(n - q, n))
            lo = max(0, n - q - c["window"] + 1) if c["window"] > 0 else 0
            union += n - lo + min(c["sinks"], lo) if q else 0
        return {"bytes": union * H * 2 * row + sum(_news(c)) * H * G * (4 * Dh + 4), "flops": 4 * pairs * H * G * Dh}
    keep = sum(min(n, c["budget"]) for n in lens)
    return {"bytes": 4 * sum(lens) * H + keep * H * (2 * 2 * row + 8), "flops": sum(lens) * H}


def _pages(c, lens, gen, dev):
    """A block table [B, max_blocks] int32 of shuffled pages (-1 = unused) over a pool of that many pages."""
    need = [(n + c["bs"] - 1) // c["bs"] for n in lens]
    mb, total = max(1, max(need)), max(1, sum(need))
    perm = torch.randperm(total, generator=gen, device=dev, dtype=torch.int32)
    count = torch.tensor(need, device=dev)
    at = torch.arange(mb, device=dev)
    index = (torch.cumsum(count, 0) - count)[:, None] + at[None]
    return torch.where(at[None] < count[:, None], perm[index.clamp(max=total - 1)], -1), total


def _slots(table, bs, length):
    """Slot of every position [B, length] (0 where the table has no page: callers mask it)."""
    j = torch.arange(length, device=table.device)
    return (table[:, j // bs].long() * bs + j % bs).clamp(min=0)


def _fill(c, pool, used, lens, gen, dev, sink_dir):
    """One cache tensor: codes of random rows in the used pages' live slots, stale bytes everywhere else."""
    H, Dh, bs = c["H"], c["Dh"], c["bs"]
    slots = pool * bs
    dtype, fmax = (torch.float8_e4m3fn, 448.0) if c["fmt"] == E4M3 else (torch.float8_e5m2, 57344.0)
    codes = torch.randint(0, 256, (slots, H, Dh), generator=gen, device=dev, dtype=torch.uint8)
    scale = torch.rand((slots, H), generator=gen, device=dev)
    L = max(max(lens), 1)
    idx = _slots(used, bs, L)
    pos = torch.arange(L, device=dev)[None].expand(len(lens), L)
    live = pos < torch.tensor(lens, device=dev)[:, None]
    idx, pos = idx[live], pos[live]
    x = torch.randn((idx.numel(), H, Dh), generator=gen, device=dev)
    if sink_dir is not None:            # the first tokens draw extra attention, as they do in trained models
        x += (pos < 4).float()[:, None, None] * sink_dir[None]
    x = x.to(torch.bfloat16).float()
    s = fmax / x.abs().amax(-1)
    codes[idx] = (x * s[..., None]).clamp(-fmax, fmax).to(dtype).view(torch.uint8)
    scale[idx] = 1.0 / s
    return codes.view(pool, bs, H, Dh), scale.view(pool, bs, H)


def prepare(c, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    H, G, Dh, B = c["H"], c["G"], c["Dh"], c["B"]
    lens = _lens(c)
    st = {"case": c, "softmax_scale": Dh ** -0.5}
    if c["kind"] == "evict":
        src, used = _pages(c, lens, gen, dev)
        dst, more = _pages(c, [min(n, c["budget"]) for n in lens], gen, dev)
        st["first_dst"] = used
        st["dst_table"] = torch.where(dst >= 0, dst + used, dst)
        st["table"], pool = src, used + more
    else:
        st["table"], pool = _pages(c, lens, gen, dev)
    direction = torch.randn((H, Dh), generator=gen, device=dev)
    st["kc"], st["ks"] = _fill(c, pool, st["table"], lens, gen, dev, direction)
    st["vc"], st["vs"] = _fill(c, pool, st["table"], lens, gen, dev, None)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if c["kind"] == "evict":
        # accumulated weights: heavy-tailed, many equal (tokens that were never attended to hold an exact zero)
        ld = max(lens)
        m = torch.rand((B, H, ld), generator=gen, device=dev).pow(8) * 4
        st["mass"] = torch.where(torch.rand((B, H, ld), generator=gen, device=dev) < 0.3, torch.zeros_like(m), m)
        st["first_dst_slot"] = st["first_dst"] * c["bs"]
        # the destination pages start out as zeros so that both forms return the same bytes behind the last row
        for x in ("kc", "ks", "vc", "vs"):
            st[x][st["first_dst"]:] = 0
    else:
        T = B if c["kind"] == "decode" else sum(_news(c))
        q = torch.randn((T, H, G, Dh), generator=gen, device=dev) + 0.5 * direction[None, :, None]
        st["q"] = q.view(T, H * G, Dh).to(torch.bfloat16)
    if c["kind"] == "prefill":
        st["offsets"] = torch.tensor([0] + _news(c), device=dev).cumsum(0)
    if own:
        from fp8_scaled_quantization_amax_b200 import fp8q
        st["k_cache"] = fp8q.PagedKVCache.from_tensors(st["kc"], st["ks"], c["fmt"])
        st["v_cache"] = fp8q.PagedKVCache.from_tensors(st["vc"], st["vs"], c["fmt"])
        if c["kind"] == "decode":
            st["workspace"] = fp8q.paged_attention_workspace(
                B, H * G, H, Dh, max_context=st["table"].shape[1] * c["bs"], weights=c["weights"])
            if c["weights"]:
                st["mass"] = torch.empty((B, H, max(lens)), device=dev)
        elif c["kind"] == "prefill":
            st["workspace"] = fp8q.paged_attention_workspace(B, H * G, H, Dh, tokens=st["q"].shape[0])
    return st


def _rows(codes, scale, slots, live, fmt):
    """Dequantized rows [B, L, H, Dh] in 32 bits; zero where not live (stale slots may hold NaN codes)."""
    dtype = torch.float8_e4m3fn if fmt == E4M3 else torch.float8_e5m2
    x = codes.flatten(0, 1)[slots].view(dtype).float() * scale.flatten(0, 1)[slots][..., None]
    return torch.where(live[..., None, None], x, 0.0)


def _attend(z, see, v):
    """Masked softmax of z [B, H, G, Q, L] and its product with v [B, L, H, Dh]; (out, lse, weights)."""
    z = torch.where(see, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    w = torch.exp(z - m)
    total = w.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    p = w / torch.where(total == 0, 1.0, total)
    return torch.einsum("bhgql,blhd->bqhgd", p, v), lse, p


def _plain_attention(st):
    c = st["case"]
    B, H, G, Dh = c["B"], c["H"], c["G"], c["Dh"]
    L = max(1, c["len"])
    slots = _slots(st["table"], c["bs"], L)
    j = torch.arange(L, device="cuda")
    live = j[None] < st["lens"][:, None]
    k = _rows(st["kc"], st["ks"], slots, live, c["fmt"])
    v = _rows(st["vc"], st["vs"], slots, live, c["fmt"])
    if c["kind"] == "decode":
        q = st["q"].float().view(B, 1, H, G, Dh)
        pos = st["lens"].long()[:, None] - 1
    else:
        first, count = st["offsets"][:-1], st["offsets"].diff()
        i = torch.arange(c["new"], device="cuda")
        there = i[None] < count[:, None]
        row = (first[:, None] + i[None]).clamp(max=st["q"].shape[0] - 1)
        q = torch.where(there[..., None, None], st["q"][row].float(), 0.0).view(B, c["new"], H, G, Dh)
        pos = torch.where(there, (st["lens"].long() - count)[:, None] + i[None], -1)
    see = live[:, None] & (j[None, None] <= pos[..., None])
    if c["window"] > 0:
        see &= (j[None, None] > pos[..., None] - c["window"]) | (j < c["sinks"])[None, None]
    z = torch.einsum("bqhgd,blhd->bhgql", q, k) * st["softmax_scale"]
    out, lse, p = _attend(z, see[:, None, None], v)
    lse = lse.permute(0, 3, 1, 2)
    if c["kind"] == "decode":
        res = {"out": out.reshape(B, H * G, Dh).to(torch.bfloat16), "lse": lse.reshape(B, H * G)}
        if c["weights"]:
            # of the positions a query cannot see nothing is said: zeros here
            res["weights"] = p[:, :, :, 0].sum(2)
        return res
    return {"out": out[there].reshape(-1, H * G, Dh).to(torch.bfloat16), "lse": lse[there].reshape(-1, H * G)}


def _plain_evict(st):
    c = st["case"]
    B, H, bs, budget = c["B"], c["H"], c["bs"], c["budget"]
    mass, n = st["mass"], st["lens"].long()[:, None, None]
    L = mass.shape[2]
    j = torch.arange(L, device="cuda")
    forced = (j < c["sinks"]) | (j >= n - c["recent"])
    key = torch.where(torch.isnan(mass), -math.inf, mass)
    key = torch.where(forced, math.inf, key)
    key = torch.where(j < n, key, -math.inf).expand(B, H, L)
    # live positions before dead ones at equal keys: a stable sort keeps the lower index first
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    keep = min(L, budget)
    count = n.clamp(max=budget)
    at = torch.arange(keep, device="cuda")
    kept = torch.where(at < count, order, L).sort(-1).values
    there = at < count
    kept_out = torch.full((B, H, budget), -1, dtype=torch.int32, device="cuda")
    kept_out[..., :keep] = torch.where(there, kept, -1).int()
    safe = kept.clamp(max=L - 1)
    mass_out = torch.zeros((B, H, L), device="cuda")
    mass_out[..., :keep] = torch.where(there, mass.gather(2, safe), 0.0)
    src = torch.gather(_slots(st["table"], bs, L)[:, None].expand(B, H, L), 2, safe)
    dst = _slots(st["dst_table"], bs, keep)[:, None].expand(B, H, keep)
    h = torch.arange(H, device="cuda")[None, :, None].expand(B, H, keep)
    there = there.expand(B, H, keep)
    src, dst, h = src[there], dst[there], h[there]
    for x in ("kc", "ks", "vc", "vs"):
        flat = st[x].flatten(0, 1)
        flat[dst, h] = flat[src, h]
    return kept_out, mass_out, n.view(-1).clamp(max=budget).int()


def run(st):
    c = st["case"]
    if own:
        from fp8_scaled_quantization_amax_b200 import fp8q
        if c["kind"] == "decode":
            if c["weights"]:
                # the weights of this step alone (decay 0); unseen positions are left as they were
                st["mass"].zero_()
            out, lse = fp8q.paged_attention_decode(
                st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"], window=c["window"], sinks=c["sinks"],
                softmax_scale=st["softmax_scale"], mass=st["mass"] if c["weights"] else None, mass_decay=0.0,
                workspace=st["workspace"])
            res = {"out": out, "lse": lse}
            if c["weights"]:
                res["weights"] = st["mass"]
            return res
        if c["kind"] == "prefill":
            out, lse = fp8q.paged_attention_prefill(
                st["q"], st["offsets"], st["k_cache"], st["v_cache"], st["table"], st["lens"], window=c["window"],
                sinks=c["sinks"], softmax_scale=st["softmax_scale"], workspace=st["workspace"])
            return {"out": out, "lse": lse}
        kept, mass, lens = fp8q.paged_kv_evict(
            st["k_cache"], st["v_cache"], st["table"], st["lens"], st["mass"], st["dst_table"], c["budget"],
            sinks=c["sinks"], recent=c["recent"])
    elif c["kind"] == "evict":
        kept, mass, lens = _plain_evict(st)
    else:
        return _plain_attention(st)
    dtype = torch.float8_e4m3fn if c["fmt"] == E4M3 else torch.float8_e5m2
    f = st["first_dst"]
    return {"kept": kept, "mass": mass, "lens": lens, "k": st["kc"][f:].view(dtype), "k_scale": st["ks"][f:],
            "v": st["vc"][f:].view(dtype), "v_scale": st["vs"][f:]}


def _value_table(fmt):
    """The 256 values of the format, from its definition."""
    man = 3 if fmt == E4M3 else 2
    bias = 7 if fmt == E4M3 else 15
    vals = []
    for code in range(256):
        e, f = (code & 127) >> man, code & ((1 << man) - 1)
        v = f * 2.0 ** (1 - bias - man) if e == 0 else (1 + f / (1 << man)) * 2.0 ** (e - bias)
        if fmt == E4M3 and (code & 127) == 127:
            v = math.nan
        if fmt == E5M2 and e == 31:
            v = math.nan if f else math.inf
        vals.append(-v if code & 128 else v)
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def exact(c, seed):
    st = prepare(c, seed)
    lens, H, G, Dh, bs = _lens(c), c["H"], c["G"], c["Dh"], c["bs"]
    table = st["table"].cpu().tolist()

    def slots_of(row, n):
        pages = torch.tensor(row, device="cuda", dtype=torch.int64)
        return (pages[:, None] * bs + torch.arange(bs, device="cuda")).reshape(-1)[:n]

    if c["kind"] == "evict":
        kept = torch.full((c["B"], H, c["budget"]), -1, dtype=torch.int32, device="cuda")
        mass = torch.zeros_like(st["mass"], dtype=torch.float64)
        outs = {x: st[x].clone().flatten(0, 1) for x in ("kc", "ks", "vc", "vs")}
        dst_rows = st["dst_table"].cpu().tolist()
        for b, n in enumerate(lens):
            m = st["mass"][b].double().cpu()
            src = slots_of(table[b], n)
            n_keep = min(n, c["budget"])
            dst = slots_of(dst_rows[b], n_keep)
            for h in range(H):
                if n <= c["budget"]:
                    chosen = torch.arange(n)
                else:
                    first, last = min(c["sinks"], n), n - c["recent"]
                    middle = m[h, first:last]
                    take = c["budget"] - first - c["recent"]
                    best = torch.sort(-middle, stable=True).indices[:take] + first
                    chosen = torch.cat([torch.arange(first), best.sort().values, torch.arange(last, n)])
                kept[b, h, :n_keep] = chosen.int().cuda()
                mass[b, h, :n_keep] = m[h, chosen].cuda()
                for x in outs:
                    outs[x][dst, h] = outs[x][src[chosen.cuda()], h]
        dtype = torch.float8_e4m3fn if c["fmt"] == E4M3 else torch.float8_e5m2
        f = st["first_dst_slot"]
        shape = (-1, bs, H)
        return {"kept": kept, "mass": mass, "lens": torch.tensor([min(n, c["budget"]) for n in lens], dtype=torch.int32),
                "k": outs["kc"][f:].view(dtype).view(*shape, Dh), "k_scale": outs["ks"][f:].view(shape),
                "v": outs["vc"][f:].view(dtype).view(*shape, Dh), "v_scale": outs["vs"][f:].view(shape)}

    values = _value_table(c["fmt"])
    news = [min(1, n) for n in lens] if c["kind"] == "decode" else _news(c)
    T = st["q"].shape[0]
    out = torch.zeros((T, H * G, Dh), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H * G), -math.inf, dtype=torch.float64, device="cuda")
    weights = torch.zeros((c["B"], H, max(lens)), dtype=torch.float64, device="cuda")
    t = 0
    for b, (n, new) in enumerate(zip(lens, news)):
        if n:
            s = slots_of(table[b], n)
            for h in range(H):
                k = values[st["kc"].flatten(0, 1)[s, h].long()] * st["ks"].flatten(0, 1)[s, h].double()[:, None]
                v = values[st["vc"].flatten(0, 1)[s, h].long()] * st["vs"].flatten(0, 1)[s, h].double()[:, None]
                for r0 in range(0, new, 1024):
                    rows = torch.arange(r0, min(new, r0 + 1024), device="cuda")
                    p = n - new + rows
                    j = torch.arange(n, device="cuda")
                    hidden = j[None] > p[:, None]
                    if c["window"] > 0:
                        hidden |= (j[None] <= p[:, None] - c["window"]) & (j[None] >= c["sinks"])
                    qs = st["q"][t + rows][:, h * G:(h + 1) * G].double()
                    z = (qs @ k.T) * st["softmax_scale"]
                    z.masked_fill_(hidden[:, None], -math.inf)
                    norm = torch.logsumexp(z, -1)
                    a = torch.exp(z - norm[..., None])
                    out[t + rows, h * G:(h + 1) * G] = a @ v
                    lse[t + rows, h * G:(h + 1) * G] = norm
                    if c["kind"] == "decode":
                        weights[b, h, :n] = a[0].sum(0)
        t += 1 if c["kind"] == "decode" else new
    res = {"out": out, "lse": lse}
    if c["kind"] == "decode" and c["weights"]:
        res["weights"] = weights
    return res
