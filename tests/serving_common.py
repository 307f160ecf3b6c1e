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
