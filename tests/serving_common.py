"""Plain references of the operators around the prompt pass, written from
their definitions (NumPy / float64, loops), and helpers for their tests."""
import numpy as np
import torch


def plan_oracle(new, length, table, free, count, P, max_tokens):
    """One step of the paged cache's bookkeeping, request by request."""
    new, length = [int(x) for x in new], [int(x) for x in length]
    table, free = table.copy(), free.copy()
    R, width = table.shape
    num, cap = free.size, width * P
    count = min(max(int(count), 0), num)
    length = [min(max(x, 0), cap) for x in length]
    pages = lambda tokens: -(-tokens // P)
    for r in range(R):
        if new[r] < 0:
            for j in range(pages(length[r])):
                if count < num:
                    free[count] = table[r, j]
                    count += 1
    cu, total = [], 0
    for r in range(R):
        cu.append(total)
        total += max(new[r], 0)
    cu.append(total)
    slots = np.full(max_tokens, -1, np.int64)
    admitted, out = np.ones(R, np.int64), list(length)
    avail, asked, top = count, 0, count
    for r in range(R):
        if new[r] < 0:
            out[r] = 0
        if new[r] <= 0:
            continue
        after = length[r] + new[r]
        admitted[r] = 0
        if after > cap or cu[r + 1] > max_tokens:
            continue
        need = pages(after) - pages(length[r])
        asked += need
        if need > 0 and asked > avail:
            continue
        admitted[r], out[r] = 1, after
        for j in range(need):
            top -= 1
            table[r, pages(length[r]) + j] = free[top]
        for i in range(new[r]):
            q = length[r] + i
            slots[cu[r] + i] = table[r, q // P] * P + q % P
    return dict(table=table, free=free, length=np.array(out, np.int64).reshape(R), count=top,
                cu=np.minimum(np.array(cu, np.int64), 2 ** 31 - 1), slots=slots, admitted=admitted)


class PlanState:
    """Device tensors of one planning step and the call on them."""

    def __init__(self, new, length, table, free, count, P, max_tokens, device, in_place=False):
        t = lambda a: torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).to(device)
        R = len(new)
        self.P, self.new, self.length = P, t(new), t(length)
        self.table, self.free, self.count = t(table), t(free), t([count])
        full = lambda n: torch.full((n,), -77, dtype=torch.int32, device=device)
        self.length_out = self.length if in_place else full(R)
        self.count_out = self.count if in_place else full(1)
        self.cu, self.slots, self.admitted = full(R + 1), full(max_tokens), full(R)

    def call(self, fb, stream=None):
        fb.sparge_kv_plan(self.new, self.length, self.table, self.free, self.count, self.P,
                          self.length_out, self.count_out, self.cu, self.slots, self.admitted,
                          stream=stream)

    def outputs(self):
        n = lambda x: x.cpu().numpy().astype(np.int64)
        return dict(table=n(self.table), free=n(self.free), length=n(self.length_out),
                    count=int(self.count_out), cu=n(self.cu), slots=n(self.slots),
                    admitted=n(self.admitted))


def same(a, b):
    for k in b:
        assert np.array_equal(a[k], b[k]), (k, a[k], b[k])


def random_plan(rng, R, P, width, new_max, ended=0.2, spare=1.0, idle=0.1):
    """A consistent state: distinct pages in the rows and on the free stack."""
    length = rng.integers(0, width * P + 1, R)
    new = rng.integers(1, new_max + 1, R)
    new[rng.random(R) < ended] = -1
    new[rng.random(R) < idle] = 0
    have = -(-length // P)
    need = int(sum(max(0, -(-(l + max(n, 0)) // P) - -(-l // P)) for l, n in zip(length, new)))
    count = int(need * spare)
    num = int(have.sum()) + need + 5
    ids = rng.permutation(num)
    table = np.full((R, width), -1)
    at = 0
    for r in range(R):
        table[r, :have[r]] = ids[at:at + have[r]]
        at += have[r]
    free = np.full(num, -1)
    free[:count] = ids[at:at + count]
    return new, length, table, free, count, P


# ----------------------------------------------------------------------------
# the 4-bit cache
# ----------------------------------------------------------------------------

MAX_SCALE = np.float16(16376.0)


def kv4_quantise(x, group):
    """(codes int [.., d], scales fp16 [.., d/group]) of float32 rows, and whether any scale
    was saturated."""
    x = np.asarray(x, np.float32)
    y = x.reshape(*x.shape[:-1], -1, group)
    with np.errstate(all="ignore"):
        s = np.abs(y).max(-1) / np.float32(7)                   # a NaN stays one
        high = s > np.float32(MAX_SCALE)
        s = np.where(high, MAX_SCALE, s.astype(np.float16))
        q = y / s.astype(np.float32)[..., None]
        c = np.where(s[..., None] > 0, np.clip(np.rint(q), -7, 7), 0)
    return c.astype(np.int64).reshape(x.shape), s, bool(high.any())


def kv4_values(c, s):
    """What codes and scales stand for, float32 (exact: 4 by 11 bits)."""
    with np.errstate(all="ignore"):
        y = c.reshape(*s.shape, -1).astype(np.float32) * s.astype(np.float32)[..., None]
    return y.reshape(c.shape)


def kv4_write(cache, slot, page_size, kc, ks, vc, vs):
    """One token's codes [Hkv, d] and scales [Hkv, ng] into the cache's bytes
    [pages, Hkv, page/16, tile], by the documented layout."""
    page, tok = divmod(slot, page_size)
    tile, k = divmod(tok, 16)
    Hkv, d = kc.shape
    ng = ks.shape[1]
    for h in range(Hkv):
        b = cache[page, h, tile]
        for j in range(d // 32):
            for t in range(4):
                for n, (lo, hi) in enumerate(((0, 2), (4, 6), (1, 3), (5, 7))):
                    at = 32 * j + 8 * t
                    b[k * (d // 2) + (t * (d // 32) + j) * 4 + n] = \
                        (kc[h, at + lo] + 8) | (kc[h, at + hi] + 8) << 4
        p = 4 * ((k % 8) // 2) + 2 * (k // 8) + k % 2
        for w in range(d // 64):
            for g in range(8):
                for i in range(4):
                    at = 64 * w + 16 * i + 2 * g
                    b[8 * d + ((w * 8 + g) * 16 + p) * 4 + i] = (vc[h, at] + 8) | (vc[h, at + 1] + 8) << 4
        sc = np.concatenate([ks[h], vs[h]]).astype(np.float16).view(np.uint8)
        b[16 * d + k * ng * 4:16 * d + (k + 1) * ng * 4] = sc


# ----------------------------------------------------------------------------
# attention over the cache
# ----------------------------------------------------------------------------

class AttnCase:
    """A filled cache, its tables and queries on the device, and the exact answer.

    lens: tokens of each request (its new ones included); news: new tokens.  The cache is
    written by the library's append; what it then holds is read back once in float32 and is
    what the definition works on, in float64."""

    def __init__(self, fb, device, lens, news, Hq, Hkv, d, group, page, dtype, seed=0, q_scale=2.0,
                 stale=True, kscale=1.0, vscale=1.0, pad=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.fb, self.lens, self.news, self.pad = fb, list(lens), list(news), pad
        R, P = len(lens), page
        counts = [-(-max(n, 0) // P) for n in lens]
        pages = sum(counts) + 2
        self.c = fb.make_kv4(Hkv, d, group, P, pages)
        self.cache = fb.kv4_cache(self.c, device)
        # unwritten memory: any bytes, among them scales that are NaN or infinite
        self.cache.copy_(torch.randint(0, 256, self.cache.shape, dtype=torch.uint8, device=device)
                         if stale else torch.full_like(self.cache, 255))
        ids = torch.randperm(pages, generator=g, device=device).int()
        self.table = torch.full((R, max([1] + counts)), -1, dtype=torch.int32, device=device)
        at = 0
        for r, n in enumerate(counts):
            self.table[r, :n] = ids[at:at + n]
            at += n
        self.slots = []
        for r, n in enumerate(lens):
            i = torch.arange(max(n, 0), device=device)
            self.slots.append((self.table[r, i // P] * P + i % P).int())
        flat = torch.cat(self.slots) if self.slots else torch.zeros(0, dtype=torch.int32, device=device)
        rnd = lambda *s: torch.randn(*s, generator=g, device=device)
        n = flat.numel()
        k = (kscale * (rnd(n, Hkv, d) * (0.3 + torch.rand(d, generator=g, device=device)) + 0.3 * rnd(d))).to(dtype)
        v = (vscale * rnd(n, Hkv, d)).to(dtype)
        fb.sparge_kv4_append(self.c, k, v, flat, self.cache)
        self.k, self.v = (torch.zeros(n, Hkv, d, device=device) for _ in "kv")
        fb.sparge_kv4_read(self.c, self.cache, flat, self.k, self.v)
        T = sum(news) + pad
        self.q = (q_scale * rnd(T, Hq + 1, d)).to(dtype)[:, :Hq]
        self.lens_t = torch.tensor(self.lens, dtype=torch.int32, device=device)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device=device)
        self.T, self.max_q, self.P = T, max([0] + list(news)), P

    def run(self, causal=True, scale=None, lse=True, stream=None, ws=None, max_q=None, **kw):
        fb, q = self.fb, self.q
        o = torch.full(q.shape, 7.0, dtype=q.dtype, device=q.device)
        out = torch.full(q.shape[:2], 5.0, device=q.device) if lse else None
        max_q = self.max_q if max_q is None else max_q
        if ws is None:
            ws = fb.kv4_workspace(self.c, q.shape[1], self.T, len(self.lens), max_q,
                                  kw.get("max_len") or self.table.shape[1] * self.P, q.device)
        self.ws = ws
        fb.sparge_kv4_attn(self.c, q, self.cache, self.table, self.lens_t, self.cu, max_q, o, ws,
                           scale=scale, causal=causal, lse=out, stream=stream, **kw)
        return o, out

    def exact(self, causal=True, scale=None):
        """(o, lse, size, err, keys, round, many): float64; per row sum_n p_n |v_n|, the E of its
        scores (see check_attn), the number of its keys, scale max_n sum |q||k_n| where K is
        rounded, and whether its request has more than 64 rows for a KV head."""
        T, Hq, d = self.q.shape
        Hkv = self.c.Hkv
        scale = d ** -0.5 if scale is None else scale
        o = torch.zeros(T, Hq, d, dtype=torch.float64, device=self.q.device)
        lse = torch.full((T, Hq), -np.inf, dtype=torch.float64, device=self.q.device)
        size, err, keys, sums = (torch.zeros_like(x) for x in (o, lse, lse, lse))
        many = torch.zeros_like(lse, dtype=torch.bool)
        at = row = 0
        for n, m in zip(self.lens, self.news):
            k, v = (x[at:at + n].double().repeat_interleave(Hq // Hkv, 1) for x in (self.k, self.v))
            q = self.q[row:row + m].double()
            s = torch.einsum("ihd,nhd->ihn", q, k) * scale
            if causal:
                see = torch.arange(n, device=q.device)[None] <= (n - m + torch.arange(m, device=q.device))[:, None]
            else:
                see = torch.ones(m, n, dtype=torch.bool, device=q.device)
            s = s.masked_fill(~see[:, None], -np.inf)
            lse[row:row + m] = torch.logsumexp(s, -1) if n else -np.inf
            p = torch.exp(s - lse[row:row + m, :, None].clamp(min=-1e300)) if n else s
            p = torch.where(see[:, None], p, torch.zeros_like(p))
            o[row:row + m] = torch.einsum("ihn,nhd->ihd", p, v)
            size[row:row + m] = torch.einsum("ihn,nhd->ihd", p, v.abs())
            keys[row:row + m] = see.sum(-1)[:, None].double()
            if n and m:
                step = k.view(n, Hq, d // self.c.group, self.c.group).abs().amax(-1) * (16 / 7)
                mass = q.abs().view(m, Hq, d // self.c.group, self.c.group).sum(-1)
                big = torch.einsum("ihg,nhg->ihn", mass, step) * scale
                err[row:row + m] = torch.where(see[:, None], big, torch.zeros_like(big)).amax(-1)
                mass = torch.einsum("ihd,nhd->ihn", q.abs(), k.abs()) * scale
                sums[row:row + m] = torch.where(see[:, None], mass, torch.zeros_like(mass)).amax(-1)
            many[row:row + m] = m * (Hq // Hkv) > 64
            at, row = at + n, row + m
        return o, lse, size, err, keys, sums * many * (self.q.dtype is torch.bfloat16), many


def check_attn(case, got, want):
    """Tolerance.  Codes and scales enter exactly; so does Q, up to 2^-37 of a row's largest.
    Scores: products of up to 7 s |q| in float32 accumulators, at most eight instructions a
    group, each off by at most 2^-22 of the running size: 2^-19 E with E = scale sum_g 16 s_g
    sum |q_g| and s_g = max|k_g| / 7; with the group sums and the exponent's own argument below
    2^-17 E.  exp2 and the (at most some twenty) rescalings and joins, 2^-22 each: 2^-17.  So a
    weight and the sum of weights are each off by w = 2^-17 (E + 1), relatively, and lse by as
    much.  p is rounded to fp16 and p s again: 2^-10 sum p |v|, and below fp16's normal range
    2^-25 (1 + s) a key, s up to max |v| / 7, times a code of up to 7 (the sum of weights is at least 1):
    6 standard deviations of n independent ones.  Sums of up to max |v| in n/64 (at most 512) steps a warp, each off by
    2^-22 of them.  Then the output's rounding.

    Requests with more than 64 rows for a KV head: sums of n/64 steps (any number), and in
    bf16 the values of K and V are rounded to fp16 first: 2^-11 of each, so scores are off by up
    to 2^-11 scale max_n sum |q||k_n| more and o by 2^-11 sum p |v|; P up to 2^8 is rounded
    once.  In fp16 K and V are sums of exact parts."""
    (o, lse), (wo, wl, size, err, keys, rounded, many) = got, want
    n = case.T - case.pad
    w = 2.0 ** -17 * (err + 1) + 2.0 ** -11 * rounded
    vmax = float(case.v.abs().nan_to_num(0, 0, 0).max()) if case.v.numel() else 0.0
    steps = keys / 64 + 2
    steps = torch.where(many, 8 * steps, steps.clamp(max=514))    # eight products a step, or one
    tol = (2.0 ** -10 + 2 * w)[..., None] * size + \
        (6 * (7 + vmax) * 2.0 ** -25 * keys.sqrt() + steps * 2.0 ** -22 * vmax)[..., None]
    tol = tol * (1 + 2.0 ** -8) + torch.finfo(o.dtype).eps / 2 * wo.abs() + 2.0 ** -25
    # an exact value beyond the type's largest is an infinity there; next to it either may come
    big = torch.finfo(o.dtype).max
    beyond = wo.abs() > big + tol
    assert bool(torch.isinf(o[:n][beyond[:n]]).all())
    near = (wo.abs() >= big - tol)[:n] & torch.isinf(o[:n])
    d = torch.where(near, torch.zeros_like(wo[:n]), (o[:n].double() - wo[:n]).abs())
    assert bool((d <= tol[:n]).all()), (float((d - tol[:n]).max()), float(d.max()))
    if lse is not None:
        fin = torch.isfinite(wl[:n])
        assert torch.equal(torch.isfinite(lse[:n]), fin)
        assert bool((lse[:n][~fin] == -np.inf).all())
        dl = (lse[:n].double() - wl[:n])[fin].abs()
        tl = (w + 2.0 ** -22 * wl.abs())[:n][fin]
        assert bool((dl <= tl).all()), float((dl - tl).max())
        assert bool((lse[n:] == 5).all())
    assert bool((o[n:] == 7).all())
