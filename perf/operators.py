"""Serving operators around the sparse prompt pass, as cases to measure: rotary positions with several
axes, block tables and slot maps, the 4-bit key/value cache and the attention that reads it.

Every case runs in two forms on the same inputs: a plain one of elementary torch operations, and
(``own``) the library's kernels through the public binding.

Layout of the 4-bit cache, shared by both forms: uint8 [pages, Hkv, page/16, tile], one tile for 16
tokens of one head, d = 64 or 128 channels in ng = d/group groups:
  8d bytes   codes of K: token rows of d/2 bytes; byte b of word (t, j), t < 4, j < d/32, holds channels
             32j + 8t + e of e = (0,2), (4,6), (1,3), (5,7) for b = 0..3, low half first
  8d bytes   codes of V: [d/64][8 g][16 pos][4 i]; a byte holds channels 64w + 16i + 2g, low half, and
             the next one, high half; token k stands at pos 4((k%8)/2) + 2(k/8) + k%2
  64ng bytes scales, fp16: [16 tokens][ng of K, ng of V]
A code c = rint(x/s), |c| <= 7, of s = fp16(max|x| of the group / 7) is held as c + 8.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 sequences: the query and key heads of a packed projection, turned in one call
        dict(name="rope_step", op="rope", B=1, H=40, N=64, d=128, rot=128, axes=3, interleaved=False, dtype="bf16",
             layout="packed", order="", inverse=False, far=200000),
        # the video grid's queries, from the projection's [B, N, H, d] straight into Hilbert order
        dict(name="rope_video", op="rope", B=1, H=24, N=17776, d=64, rot=64, axes=3, interleaved=True, dtype="f16",
             layout="bnhd", order="shuffled", inverse=False, far=64),
        # gradient of the queries of a 128K prompt: the inverse rotation, half of the channels unturned
        dict(name="rope_128k_inverse", op="rope", B=1, H=32, N=131072, d=128, rot=64, axes=1, interleaved=False,
             dtype="bf16", layout="bhnd", order="", inverse=True, far=131072),
        # a decode step of 256 sequences: one token each, a few end, a few need a page
        dict(name="plan_step", op="plan", R=256, page=64, max_len=32768, new=1, ended=9),
        # 500 prompts at once into small pages, about a million tokens
        dict(name="plan_prompts", op="plan", R=500, page=16, max_len=8192, new=4096, ended=20),
        # one new token of each of 60 sequences into the smallest pages, four rows of padding behind them, and back
        dict(name="cache_step", op="cache", R=60, max_len=4000, last=1, pad=4, Hkv=12, d=64, group=64, page=16, dtype="f16"),
        # three prompts of the 8 key/value heads into the cache, and back in 16 bits
        dict(name="cache_prompts", op="cache", R=3, max_len=16383, last=16383, pad=0, Hkv=8, d=128, group=32, page=64, dtype="bf16"),
        # the shortest answer to a single request: latency
        dict(name="attn_one", op="attn", R=1, max_len=1009, min_len=1009, q=1, Hq=32, Hkv=8, d=128, group=32, page=64,
             dtype="bf16"),
        # an ordinary decode step of a ragged batch
        dict(name="attn_step", op="attn", R=48, max_len=8192, min_len=700, q=1, Hq=32, Hkv=8, d=128, group=64, page=64,
             dtype="bf16"),
        # single tokens at the end of 128K contexts: the cache's bytes are all that counts
        dict(name="attn_128k", op="attn", R=3, max_len=131072, min_len=98303, q=1, Hq=32, Hkv=8, d=128, group=32, page=64,
             dtype="bf16"),
        # a few guessed tokens checked at once, every head with keys of its own, one scale a token and head
        dict(name="attn_guess", op="attn", R=9, max_len=4001, min_len=1, q=5, Hq=12, Hkv=12, d=64, group=64, page=16,
             dtype="f16"),
        # pieces of two prompts against the context that the cache holds already
        dict(name="attn_piece", op="attn", R=2, max_len=32768, min_len=20001, q=512, Hq=32, Hkv=8, d=128, group=128, page=64,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "plan", "cache", "attn", "attn", "attn"])
    if op == "rope":
        d, dtype = rng.choice([64, 128]), rng.choice(["f16", "bf16", "f32"])
        H, B = _log(rng, 1, 40), rng.choice([1, 1, 2])
        N = _log(rng, 1, max(1, min(131072, (1 << 28) // (B * H * d))))
        return dict(op=op, B=B, H=H, N=N, d=d, rot=rng.choice([d, d, d // 2]), axes=rng.choice([1, 2, 3]),
                    interleaved=rng.random() < 0.5, dtype=dtype, layout=rng.choice(["bhnd", "bnhd", "packed"]),
                    order=rng.choice(["", "shuffled"]), inverse=rng.random() < 0.4, far=_log(rng, 64, 1000000))
    if op == "plan":
        R = _log(rng, 1, 1000)
        new = _log(rng, 1, max(1, min(4096, 1000000 // R)))
        return dict(op=op, R=R, page=rng.choice([16, 32, 64, 128]), max_len=_log(rng, 256, 32768), new=new, ended=rng.randint(0, R // 4))
    d, dtype, page = rng.choice([64, 128]), rng.choice(["f16", "bf16"]), rng.choice([16, 32, 64, 128])
    group = rng.choice([g for g in (32, 64, 128) if g <= d])
    if op == "cache":
        R, Hkv = _log(rng, 1, 12), rng.choice([1, 2, 4, 8, 16])
        max_len = _log(rng, 1, max(1, 400000 // (R * Hkv)))
        return dict(op=op, R=R, max_len=max_len, last=rng.choice([1, max_len]), pad=rng.randint(0, 9), Hkv=Hkv, d=d, group=group, page=page,
                    dtype=dtype)
    Hkv = rng.choice([1, 2, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 4, 6, 8])
    q = rng.choice([1, 1, 1, 1, 2, 3, 5, _log(rng, 2, 256)])
    R = _log(rng, 1, 64 if q < 8 else 4)
    top = min(131072, (1 << 28) // (R * Hkv * d), (1 << 28) // (R * Hq * q))
    max_len = max(q, _log(rng, 1, max(1, top)))
    return dict(op=op, R=R, max_len=max_len, min_len=min(max_len, rng.choice([q, max(q, max_len // 2), max_len])), q=q,
                Hq=Hq, Hkv=Hkv, d=d, group=group, page=page, dtype=dtype)


def _lens(case):
    """Ragged lengths, the longest first, down to min_len."""
    R, hi, lo = case["R"], case["max_len"], case.get("min_len", max(1, case["max_len"] // 3))
    return [hi - (r * (hi - lo)) // max(R - 1, 1) for r in range(R)]


def _news(case):
    """New tokens of each request: q, fewer for some."""
    return [max(1, min(n, case["q"] - (5 * r) % ((case["q"] + 1) // 2))) for r, n in enumerate(_lens(case))]


def _asked(case):
    """Tokens that each request of a plan brings, spread over 1..new; -1 for those that end."""
    n = case["R"] - case["ended"]
    return [-1] * case["ended"] + [1 + i * case["new"] // n for i in range(n)]


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _keys(g, shape):
    """Keys with channels of unlike spread and a constant part, as projections give them."""
    d = shape[-1]
    return _randn(g, *shape) * (0.4 + 1.2 * torch.rand(d, generator=g, device="cuda")) + 0.5 * _randn(g, d)


def _tables(g, lens, page):
    """A block table of shuffled pages (-1 behind each row's end) and the number of pages."""
    counts = [-(-n // page) for n in lens]
    pages = torch.randperm(sum(counts) + 3, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(1, max(counts))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(counts):
        table[r, :n] = pages[at:at + n]
        at += n
    return table, sum(counts) + 3


def _pack(k, v, group):
    """Codes and scales of k, v [pages, P, Hkv, d] (float32) in the cache's layout."""
    n, P, Hkv, d = k.shape
    out = []
    scales = []
    for x in (k, v):
        x = x.view(n, P // 16, 16, Hkv, d // group, group)
        s = (x.abs().amax(-1, keepdim=True) / torch.full((), 7.0, device=x.device)).half().float()
        c = torch.where(s > 0, x / s, torch.zeros_like(x)).round().clamp(-7, 7) + 8
        out.append(c.to(torch.uint8).permute(0, 3, 1, 2, 4, 5).reshape(n, Hkv, P // 16, 16, d))
        scales.append(s.half().permute(0, 3, 1, 2, 4, 5).reshape(n, Hkv, P // 16, 16, d // group))
    u = out[0].view(n, Hkv, P // 16, 16, d // 32, 4, 4, 2)                 # [.., j, t, e/2, e%2]
    kb = torch.stack([u[..., 0, 0] | u[..., 1, 0] << 4, u[..., 2, 0] | u[..., 3, 0] << 4,
                      u[..., 0, 1] | u[..., 1, 1] << 4, u[..., 2, 1] | u[..., 3, 1] << 4], -1)
    kb = kb.transpose(4, 5).reshape(n, Hkv, P // 16, 8 * d)
    u = out[1].view(n, Hkv, P // 16, 2, 4, 2, d // 64, 4, 8, 2)            # [.., k/8, k%8/2, k%2, w, i, g, h]
    vb = (u[..., 0] | u[..., 1] << 4).permute(0, 1, 2, 6, 8, 4, 3, 5, 7).reshape(n, Hkv, P // 16, 8 * d)
    sb = torch.cat(scales, -1).view(torch.uint8).reshape(n, Hkv, P // 16, -1)
    return torch.cat([kb, vb, sb], -1).contiguous()


def _prepare_rope(case, seed):
    g = _gen(seed)
    B, H, N, d, dt = case["B"], case["H"], case["N"], case["d"], DTYPES[case["dtype"]]
    if case["layout"] == "bhnd":
        x = torch.empty(B, H, N, d, dtype=dt, device="cuda").normal_(generator=g)
    elif case["layout"] == "bnhd":
        x = torch.empty(B, N, H, d, dtype=dt, device="cuda").normal_(generator=g).transpose(1, 2)
    else:                                                                  # queries and keys in front of the values
        x = torch.empty(B, N, H + 8, d, dtype=dt, device="cuda").normal_(generator=g)[:, :, :H].transpose(1, 2)
    pairs, axes = case["rot"] // 2, case["axes"]
    axis = torch.arange(pairs, device="cuda") * axes // pairs              # neighbouring pairs share an axis
    return dict(x=x, axis=axis.int(), inv_freq=1e4 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs),
                pos=torch.randint(0, case["far"], (axes, N), generator=g, device="cuda").int(),
                perm=torch.randperm(N, generator=g, device="cuda").int() if case["order"] else None)


def _prepare_plan(case, seed):
    g = _gen(seed)
    R, P = case["R"], case["page"]
    length = torch.randint(0, case["max_len"] + 1, (R,), generator=g, device="cuda")
    new = torch.tensor(_asked(case), device="cuda")[torch.randperm(R, generator=g, device="cuda")]
    width = -(-(case["max_len"] + case["new"]) // P)
    have, after = (length + P - 1) // P, (length + new.clamp(min=0) + P - 1) // P
    used, spare = int(have.sum()), int((after - have).sum())
    spare = spare - spare // 50 + 1                                        # now and then one request finds no page left
    pages = torch.randperm(R * width, generator=g, device="cuda").int()   # the rest are others' pages
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda") < have[:, None]] = pages[:used]
    free = torch.full((R * width,), -1, dtype=torch.int32, device="cuda")
    free[:spare] = pages[used:used + spare]
    T = sum(n for n in _asked(case) if n > 0)
    return dict(new=new.int(), length=length.int(), table=table, free=free, count=_ints([spare]), page=P, tokens=T + T // 16 + 1)


def _prepare_cache(case, seed):
    g = _gen(seed)
    lens, Hkv, d, dt, P = _lens(case), case["Hkv"], case["d"], DTYPES[case["dtype"]], case["page"]
    table, pages = _tables(g, lens, P)
    lasts = [min(n, case["last"]) for n in lens]
    at = torch.cat([torch.arange(n - m, n, device="cuda") for n, m in zip(lens, lasts)])
    row = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(lasts, device="cuda"))
    slots = torch.cat([table[row, at // P] * P + at % P, torch.full((case["pad"],), -1, device="cuda")])
    T = slots.numel()
    kv = torch.cat([_keys(g, (T, Hkv, d)), _randn(g, T, Hkv, d)], 1).to(dt)    # [T, 2 Hkv, d], as a projection leaves it
    tile = 16 * (d + 4 * (d // case["group"]))
    return dict(k=kv[:, :Hkv], v=kv[:, Hkv:], slots=slots.int(), group=case["group"], page=P,
                out=[torch.zeros(T, Hkv, d, dtype=dt, device="cuda") for _ in "kv"],
                cache=torch.zeros(pages, Hkv, P // 16, tile, dtype=torch.uint8, device="cuda"))


def _prepare_attn(case, seed):
    g = _gen(seed)
    lens, news, P, Hq, Hkv, d = _lens(case), _news(case), case["page"], case["Hq"], case["Hkv"], case["d"]
    table, pages = _tables(g, lens, P)
    cache = _pack(_keys(g, (pages, P, Hkv, d)), _randn(g, pages, P, Hkv, d), case["group"])
    T = sum(news)
    qkv = (2 * _randn(g, T, Hq + 2 * Hkv, d)).to(DTYPES[case["dtype"]])     # as a projection leaves it
    cu = _ints([sum(news[:r]) for r in range(len(news) + 1)])
    return dict(q=qkv[:, :Hq], cache=cache, table=table, lens=_ints(lens), cu=cu, max_q=max(news), group=case["group"], page=P)


def prepare(case, seed):
    op = case["op"]
    state = (_prepare_rope if op == "rope" else _prepare_plan if op == "plan" else _prepare_cache if op == "cache" else _prepare_attn)(case, seed)
    return dict(state, case=case)


# ------------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------------

def _plain_rope(s):
    case, x = s["case"], s["x"].float()
    rot, half = case["rot"], case["rot"] // 2
    a = s["pos"].double()[s["axis"].long()] * s["inv_freq"][:, None]       # far positions: 64 bits
    cos, sin = a.cos().float().t(), a.sin().float().t()                    # [N, pairs]
    if case["inverse"]:
        sin = -sin
    src = None if s["perm"] is None else s["perm"].long()
    if src is not None:
        cos, sin = cos[src], sin[src]
        if not case["inverse"]:
            x = x[:, :, src]
    if case["interleaved"]:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
    else:
        u, v = x[..., :half], x[..., half:rot]
        turned = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
    y = torch.cat([turned, x[..., rot:]], -1).to(s["x"].dtype)
    if src is not None and case["inverse"]:
        y = torch.empty_like(y).index_copy_(2, src, y)
    return y


def _plain_plan(s):
    P, table, new, length = s["page"], s["table"].long(), s["new"].long(), s["length"].long()
    R, width = table.shape
    cols, count = torch.arange(width, device=table.device), s["count"].long()
    have = (length + P - 1) // P
    back = torch.where(new < 0, have, 0)                                   # pages that ended requests give back
    at = count + back.cumsum(0) - back
    free, held = s["free"].long().clone(), cols < back[:, None]
    free[(at[:, None] + cols)[held]] = table[held]
    avail = count + back.sum()
    add = new.clamp(min=0)
    cu = torch.cat([add.new_zeros(1), add.cumsum(0)])
    fits = (new > 0) & (length + add <= width * P) & (cu[1:] <= s["tokens"])
    need = torch.where(fits, (length + add + P - 1) // P - have, 0)
    upto = need.cumsum(0)
    ok = fits & ((need == 0) | (upto <= avail))
    rank = cols - have[:, None]
    gets = ok[:, None] & (rank >= 0) & (rank < need[:, None])
    table = torch.where(gets, free[(avail - 1 - (upto - need)[:, None] - rank).clamp(0, free.numel() - 1)], table)
    t = torch.arange(s["tokens"], device=table.device)
    row = torch.searchsorted(cu, t, right=True).sub(1).clamp(max=R - 1)
    pos = length[row] + t - cu[row]
    there = (t < cu[R]) & ok[row]
    slots = torch.where(there, table[row, (pos // P).clamp(0, width - 1)] * P + pos % P, -1)
    i32 = torch.int32
    return dict(table=table.to(i32), free=free.to(i32), count=(avail - torch.where(ok, need, 0).sum()).to(i32).view(1),
                length=torch.where(new < 0, 0, torch.where(ok, length + add, length)).to(i32), cu=cu.to(i32),
                slots=slots.to(i32), admitted=(ok | (new <= 0)).to(i32))


def _plain_values(x, group):
    """What the 4-bit codes of x [.., d] stand for."""
    y = x.float().unflatten(-1, (-1, group))
    scale = (y.abs().amax(-1, keepdim=True) / torch.full((), 7.0, device=x.device)).half().float()
    return (torch.where(scale > 0, y / scale, torch.zeros_like(y)).round().clamp(-7, 7) * scale).flatten(-2)


def _plain_unpack(tiles, group):
    """K and V in float32, [R, Hkv, L, d], of tiles [R, pages, Hkv, page/16, bytes]."""
    R, n, Hkv, nt, nbytes = tiles.shape
    d = nbytes * group // (16 * (group + 4))
    ng = d // group
    k = torch.stack([tiles[..., :8 * d] & 15, tiles[..., :8 * d] >> 4], -1).view(R, n, Hkv, nt, 16, 4, d // 32, 2, 4)
    v = torch.stack([tiles[..., 8 * d:16 * d] & 15, tiles[..., 8 * d:16 * d] >> 4], -1).view(R, n, Hkv, nt, d // 64, 8, 4, 2, 2, 4, 2)
    s = tiles[..., 16 * d:].contiguous().view(torch.float16).view(R, n, Hkv, nt, 16, 2, ng, 1).permute(5, 0, 2, 1, 3, 4, 6, 7).float()
    k = k.permute(0, 2, 1, 3, 4, 6, 5, 8, 7)                               # [.., token, j, t, e/2, e%2]
    v = v.permute(0, 2, 1, 3, 7, 6, 8, 4, 9, 5, 10)                        # [.., k/8, k%8/2, k%2, w, i, g, h]
    out = [((c.reshape(R, Hkv, n, nt, 16, ng, group).float() - 8) * s[i]).reshape(R, Hkv, n * nt * 16, d) for i, c in enumerate((k, v))]
    return out


def _plain_cache(s):
    there = (s["slots"] >= 0)[:, None, None]                               # padding keeps what it held
    return {n: torch.where(there, _plain_values(s[n], s["group"]).to(o.dtype), o) for n, o in zip("kv", s["out"])}


def _plain_attn(s):
    q = s["q"].float()
    T, Hq, d = q.shape
    k, v = _plain_unpack(s["cache"][s["table"].long().clamp(min=0)], s["group"])
    R, Hkv, L, _ = k.shape
    cu, lens, Q, G = s["cu"].long(), s["lens"].long(), s["max_q"], Hq // Hkv
    step = torch.arange(Q, device=q.device)
    mine = q[(cu[:-1, None] + step).clamp(max=T - 1)].view(R, Q, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(R, Hkv, Q * G, d)
    p = mine @ k.transpose(-1, -2) / math.sqrt(d)
    last = lens[:, None] - (cu[1:] - cu[:-1])[:, None] + step              # the position of each query
    sees = torch.arange(L, device=q.device) <= torch.minimum(last, lens[:, None] - 1)[..., None]
    p = p.view(R, Hkv, Q, G, L).masked_fill_(~sees[:, None, :, None], -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    o = (p / p.sum(-1, keepdim=True)).view(R, Hkv, Q * G, L) @ v
    o = o.view(R, Hkv, Q, G, d).permute(0, 2, 1, 3, 4).reshape(R, Q, Hq, d)
    t = torch.arange(T, device=q.device)
    row = torch.searchsorted(cu, t, right=True) - 1
    return o[row, t - cu[row]].to(s["q"].dtype)


# ------------------------------------------------------------------------------------------------
# the library's operators
# ------------------------------------------------------------------------------------------------

def _own_rope(s):
    import free_block_sparse_predict_b200 as fb
    case, x = s["case"], s["x"]
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    turn = fb.sparge_rope_inverse if case["inverse"] else fb.sparge_rope_apply
    turn(x, y, s["pos"], s["inv_freq"], s["axis"], perm=s["perm"], interleaved=case["interleaved"])
    return y


def _own_plan(s):
    import free_block_sparse_predict_b200 as fb
    if "plan" not in s:                                                    # the buffers that a serving loop keeps
        R = s["new"].numel()
        s["plan"] = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (R, 1, R + 1, s["tokens"], R)]
    length, count, cu, slots, admitted = s["plan"]
    fb.sparge_kv_plan(s["new"], s["length"], s["table"], s["free"], s["count"], s["page"], length, count, cu, slots, admitted)
    return dict(table=s["table"], free=s["free"], count=count, length=length, cu=cu, slots=slots, admitted=admitted)


def _cache_of(s, fb):
    if "kv4" not in s:
        case = s["case"]
        s["kv4"] = fb.make_kv4(case["Hkv"], case["d"], case["group"], s["page"], s["cache"].shape[0])
    return s["kv4"]


def _own_cache(s):
    import free_block_sparse_predict_b200 as fb
    c = _cache_of(s, fb)
    fb.sparge_kv4_append(c, s["k"], s["v"], s["slots"], s["cache"])
    fb.sparge_kv4_read(c, s["cache"], s["slots"], *s["out"])
    return dict(k=s["out"][0], v=s["out"][1])


def _own_attn(s):
    import free_block_sparse_predict_b200 as fb
    c, q = _cache_of(s, fb), s["q"]
    if "ws" not in s:
        s["ws"] = fb.kv4_workspace(c, q.shape[1], q.shape[0], s["lens"].numel(), s["max_q"], s["table"].shape[1] * s["page"])
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    fb.sparge_kv4_attn(c, q, s["cache"], s["table"], s["lens"], s["cu"], s["max_q"], o, s["ws"])
    return o


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_rope(state) if op == "rope" else _own_plan(state) if op == "plan" else _own_cache(state) if op == "cache" else _own_attn(state)
    return _plain_rope(state) if op == "rope" else _plain_plan(state) if op == "plan" else _plain_cache(state) if op == "cache" else _plain_attn(state)


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "rope":
        n, es = case["B"] * case["H"] * case["N"] * case["d"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * n * es + 4 * case["N"] * case["axes"], "flops": 3 * n * case["rot"] // case["d"]}
    if op == "plan":                                                       # lengths, counts and flags; a slot a token; the pages that change hands
        T, R = sum(n for n in _asked(case) if n > 0), case["R"]
        moved = T / case["page"] + case["ended"] * case["max_len"] / 2 / case["page"]
        return {"bytes": 20 * R + 4 * T + 8 * moved, "flops": 0}
    Hkv, d, ng = case["Hkv"], case["d"], case["d"] // case["group"]
    lens = _lens(case)
    if op == "cache":                                                      # values in, codes out, codes in, values out
        T = sum(min(n, case["last"]) for n in lens)
        return {"bytes": T * Hkv * (2 * 2 * 2 * d + 2 * (d + 4 * ng)), "flops": T * Hkv * 2 * d * 4}
    news, Hq = _news(case), case["Hq"]
    pairs = sum(m * n - m * (m - 1) // 2 for n, m in zip(lens, news))
    return {"bytes": sum(lens) * Hkv * (d + 4 * ng) + 4 * sum(news) * Hq * d, "flops": 4 * pairs * Hq * d}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------

def _exact_rope(case, s):
    x, rot = s["x"].double(), case["rot"]
    n = rot // 2
    first = torch.arange(n, device="cuda") * 2 if case["interleaved"] else torch.arange(n, device="cuda")
    second = first + (1 if case["interleaved"] else n)
    y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    order = torch.arange(case["N"], device="cuda") if s["perm"] is None else s["perm"].long()
    for h in range(case["H"]):
        src = x[:, h] if case["inverse"] else x[:, h][:, order]
        out = src.clone()
        z = torch.complex(src[..., first], src[..., second])
        a = s["pos"][:, order].double()[s["axis"].long()].t() * s["inv_freq"] * (-1 if case["inverse"] else 1)
        z = z * torch.polar(torch.ones_like(a), a)
        out[..., first], out[..., second] = z.real, z.imag
        if case["inverse"]:
            y[:, h, order] = out
        else:
            y[:, h] = out
    return y


def _exact_values(x, group):
    """The definition: the code is the nearest whole number to the quotient in float32, ties to even."""
    y = x.float().reshape(-1, group)
    s = (y.abs().max(1).values.double() / 7).float().half().float()
    c = torch.div(y, s[:, None].clamp(min=2.0 ** -24)).round().clamp(-7, 7)
    return (c.double() * s.double()[:, None]).reshape(x.shape)


def _exact_cache(case, s):
    out = dict(k=_exact_values(s["k"].contiguous(), case["group"]), v=_exact_values(s["v"].contiguous(), case["group"]))
    for x in out.values():
        x[s["slots"] < 0] = 0
    return out


def _exact_attn(case, s):
    P, d, G, group = case["page"], case["d"], case["Hq"] // case["Hkv"], case["group"]
    ng = d // group
    tok, ch = torch.arange(16, device="cuda")[:, None], torch.arange(d, device="cuda")[None]
    e = ch % 8
    kbyte = tok * (d // 2) + (ch // 8 % 4) * (d // 8) + (ch // 32) * 4 + 2 * (e % 2) + e // 4
    kshift = 4 * (e // 2 % 2) + 0 * tok
    pos = 4 * (tok % 8 // 2) + 2 * (tok // 8) + tok % 2
    vbyte = 8 * d + ((ch // 64 * 8 + ch % 16 // 2) * 16 + pos) * 4 + ch // 16 % 4
    vshift = 4 * (ch % 2) + 0 * tok
    scales = s["cache"][..., 16 * d:].contiguous().view(torch.float16).view(*s["cache"].shape[:3], 16, 2, ng)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for r, (n, m) in enumerate(zip(_lens(case), _news(case))):
        pages = s["table"][r, :-(-n // P)].long()
        for h in range(case["Hkv"]):
            kv = []
            for i, (byte, shift) in enumerate(((kbyte, kshift), (vbyte, vshift))):
                c = (s["cache"][pages, h][:, :, byte].int() >> shift & 15).double() - 8           # [pages, tiles, 16, d]
                x = (c * scales[pages, h][:, :, :, i].double().repeat_interleave(group, -1)).reshape(-1, d)[:n]
                kv.append(x)
            for j in range(0, m, 64):
                top = min(m, j + 64)
                q = s["q"][at + j:at + top, h * G:h * G + G].double()
                a = torch.einsum("qgd,kd->qgk", q, kv[0]) * d ** -0.5
                hide = torch.arange(n, device="cuda")[None] > torch.arange(n - m + j, n - m + top, device="cuda")[:, None]
                a = torch.softmax(a.masked_fill(hide[:, None], -math.inf), -1)
                out[at + j:at + top, h * G:h * G + G] = torch.einsum("qgk,kd->qgd", a, kv[1])
        at += m
    return out


def exact(case, seed):
    op = case["op"]
    if op == "plan":                                                       # whole numbers
        return None
    s = prepare(case, seed)
    return _exact_rope(case, s) if op == "rope" else _exact_cache(case, s) if op == "cache" else _exact_attn(case, s)
