"""The operators around the prompt pass together, as a serving program runs
them: rotary positions, pages, the 4-bit cache, the sparse prompt pass, then
single tokens, eagerly and as one captured graph."""
import numpy as np
import pytest
import torch

import free_block_sparse_predict_b200 as fb

from gpu_common import dev
from serving_common import kv4_quantise, kv4_values

pytestmark = pytest.mark.gpu

HQ, HKV, D, GROUP, PAGE = 8, 2, 128, 32, 32


class Server:
    """What a serving loop keeps: cache, tables, lengths, free pages, static step buffers."""

    def __init__(self, R, width, pages, tokens):
        i32 = dict(dtype=torch.int32, device=dev())
        self.c = fb.make_kv4(HKV, D, GROUP, PAGE, pages)
        self.cache = fb.kv4_cache(self.c, dev())
        self.table = torch.full((R, width), -1, **i32)
        self.length, self.new = torch.zeros(R, **i32), torch.zeros(R, **i32)
        self.free = torch.randperm(pages, device=dev()).int()
        self.count = torch.tensor([pages], **i32)
        self.cu, self.ok = torch.zeros(R + 1, **i32), torch.zeros(R, **i32)
        self.slots = torch.zeros(tokens, **i32)
        self.inv_freq, self.axis = fb.rope_frequencies((16, 24, 24), joint=True, device=dev())
        self.qkv = torch.zeros(tokens, HQ + 2 * HKV, D, dtype=torch.bfloat16, device=dev())
        self.pos = torch.zeros(3, tokens, **i32)
        self.o = torch.zeros(tokens, HQ, D, dtype=torch.bfloat16, device=dev())
        self.ws = fb.kv4_workspace(self.c, HQ, tokens, R, tokens, width * PAGE, dev())
        self.R, self.tokens = R, tokens

    def step(self, max_q):
        """Projection's output in, attention's out: nothing here waits for the GPU."""
        qk = self.qkv[None, :, :HQ + HKV].transpose(1, 2)
        fb.sparge_rope_apply(qk, qk, self.pos, self.inv_freq, self.axis)
        fb.sparge_kv_plan(self.new, self.length, self.table, self.free, self.count, PAGE,
                          self.length, self.count, self.cu, self.slots, self.ok)
        fb.sparge_kv4_append(self.c, self.qkv[:, HQ:HQ + HKV], self.qkv[:, HQ + HKV:], self.slots,
                             self.cache, self.ws)
        fb.sparge_kv4_attn(self.c, self.qkv[:, :HQ], self.cache, self.table, self.length, self.cu,
                           max_q, self.o, self.ws)


class Model:
    """The same in float64, request by request."""

    def __init__(self, R, inv_freq, axis):
        self.k = [[] for _ in range(R)]
        self.v = [[] for _ in range(R)]
        self.f, self.a = inv_freq.cpu().numpy(), axis.cpu().numpy()

    def turn(self, x, pos):
        ang = pos[self.a].astype(np.float64) * self.f
        u, v = x[..., :D // 2], x[..., D // 2:]
        return np.concatenate([u * np.cos(ang) - v * np.sin(ang), u * np.sin(ang) + v * np.cos(ang)], -1)

    def token(self, r, k, v):
        """k and v as the cache is given them: turned keys in bf16."""
        for store, x in ((self.k, k), (self.v, v)):
            store[r].append(kv4_values(*kv4_quantise(x, GROUP)[:2]).astype(np.float64))

    def attend(self, r, q, upto):
        k, v = (np.repeat(np.stack(x[r][:upto]), HQ // HKV, 1) for x in (self.k, self.v))
        s = np.einsum("hd,nhd->hn", q, k) / np.sqrt(D)
        p = np.exp(s - s.max(1, keepdims=True))
        return np.einsum("hn,nhd->hd", p / p.sum(1, keepdims=True), v)


def feed(s, g, news, positions):
    """Random projections and positions of one step into the static buffers."""
    s.new.copy_(torch.tensor(news, dtype=torch.int32))
    s.qkv.copy_((1.5 * torch.randn(s.qkv.shape, generator=g, device=dev())).bfloat16())
    n = sum(max(x, 0) for x in news)
    s.pos[:, :n] = torch.from_numpy(positions).to(dev())
    return s.qkv.float().cpu().numpy().astype(np.float64)[:n]


def settle(s, m, news, raw, positions):
    """Checks one step's outputs against the float64 model and moves the model on."""
    torch.cuda.synchronize()
    assert fb.sparge_device_status(s.ws) == 0
    now = s.qkv.float().cpu().numpy()                        # q and k turned, rounded to bf16
    o = s.o.float().cpu().numpy()
    t = 0
    for r, n in enumerate(news):
        if n < 0:
            m.k[r], m.v[r] = [], []
        for _ in range(max(n, 0)):
            turned = m.turn(raw[t, :HQ + HKV], positions[:, t])
            # bf16 rounds by 2^-9 of the value; the float32 turning is far below (2^-20)
            mix = np.hypot(raw[t, :HQ + HKV, :D // 2], raw[t, :HQ + HKV, D // 2:])
            tol = 2.0 ** -8 * np.abs(turned) + 2.0 ** -19 * np.concatenate([mix, mix], -1)
            assert np.all(np.abs(now[t, :HQ + HKV] - turned) <= tol)
            m.token(r, now[t, HQ:HQ + HKV], now[t, HQ + HKV:])
            t += 1
    t = 0
    for r, n in enumerate(news):
        for i in range(max(n, 0)):
            want = m.attend(r, now[t, :HQ].astype(np.float64), len(m.k[r]) - n + i + 1)
            vmax = max(np.abs(x).max() for x in m.v[r])
            # weights 2^-11 (rounded once) and 2^-10 (scores of up to E = 400: 2^-17 E, twice
            # over numerator and sum, below 2^-7), values up to vmax; the output's own 2^-9
            assert np.all(np.abs(o[t] - want) <= (2.0 ** -11 + 2.0 ** -7) * vmax + 2.0 ** -8 * np.abs(want))
            t += 1


def positions_of(news, lengths):
    """Text counts up on all axes; every third token of a prompt is an image patch."""
    out = []
    for n, length in zip(news, lengths):
        for i in range(max(n, 0)):
            p = length + i
            out.append((p, p, p) if p % 3 else (p, p // 7, p % 7))
    return np.array(out, np.int32).reshape(-1, 3).T.copy()


@pytest.mark.parametrize("captured", [False, True])
def test_prompts_then_single_tokens(captured):
    R, g = 3, torch.Generator(device=dev()).manual_seed(11)
    s = Server(R, 6, 14, 150)
    m = Model(R, s.inv_freq, s.axis)
    lengths = [0] * R
    graph = None
    # prompts, then tokens; request 1 ends and a new prompt takes its pages
    plan = [[70, 33, 40]] + [[1, 1, 1]] * 4 + [[1, -1, 1], [1, 90, 1]] + [[1, 1, 1]] * 3
    for news in plan:
        pos = positions_of(news, lengths)
        raw = feed(s, g, news, pos)
        if captured and max(news) == 1:
            if graph is None:
                graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
                torch.cuda.synchronize()
                with torch.cuda.graph(graph, stream=side, capture_error_mode="relaxed"):
                    s.step(1)
            graph.replay()
        else:
            s.step(max(max(news), 1))
        settle(s, m, news, raw, pos)
        lengths = [0 if n < 0 else x + n for n, x in zip(news, lengths)]
        assert s.length.tolist() == lengths and s.ok.tolist() == [1] * R


def test_prompt_by_the_sparse_pass_and_by_the_cache():
    """sparge_forward over a prompt with every block kept, and the cache's attention over the same
    tokens: the same rows up to what 4 bits take from K and V.  Both against the float64 answer
    on what each of them sees."""
    N, g = 333, torch.Generator(device=dev()).manual_seed(3)
    s = Server(1, 12, 12, N)
    pos = positions_of([N], [0])
    raw = feed(s, g, [N], pos)
    rope = fb.Rope(s.pos, s.inv_freq, s.axis)
    q, k, v = (s.qkv[None, :, a:b].transpose(1, 2) for a, b in
               ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
    p = fb.make_params(1, HQ, HKV, N, D, 1.0, 2.0, -float("inf"), causal=True, io_dtype=torch.bfloat16)
    o, mask, _, cnt = fb.sparge_forward(p, q, k, v.contiguous(), rope=rope)
    before = s.qkv.clone()
    s.step(N)
    m = Model(1, s.inv_freq, s.axis)
    settle(s, m, [N], raw, pos)
    now = s.qkv.float().cpu().numpy().astype(np.float64)
    assert torch.equal(before[:, HQ + HKV:], s.qkv[:, HQ + HKV:])
    exact = Model(1, s.inv_freq, s.axis)
    exact.k, exact.v = [list(now[:, HQ:HQ + HKV])], [list(now[:, HQ + HKV:])]
    got = o[0].transpose(0, 1).float().cpu().numpy()
    for t in range(0, N, 7):
        want = exact.attend(0, now[t, :HQ], t + 1)
        # fp16 weights and values (2^-11 each) of up to |v| < 8, and the output's rounding
        assert np.all(np.abs(got[t] - want) <= 2.0 ** -9 * 8 + 2.0 ** -8 * np.abs(want))


@pytest.mark.parametrize("captured", [False, True])
def test_calls_in_a_row_wait_for_one_another(captured):
    """Launches begin before the one ahead of them has ended: steps that follow one another without
    a pause, each reading what the calls before it wrote (tables, cache, its own output as the next
    queries), give the bits of the same steps with a wait after every call."""
    def run(pause):
        torch.manual_seed(5)
        R, tokens = 40, 3000
        s = Server(R, 40, 1400, tokens)
        s.free.copy_(torch.arange(1400, dtype=torch.int32))
        s.pos.random_(0, 1000)
        s.qkv.normal_()
        names = ["sparge_rope_apply", "sparge_kv_plan", "sparge_kv4_append", "sparge_kv4_read",
                 "sparge_kv4_attn"]
        kept = {n: getattr(fb, n) for n in names}

        def waiting(f):
            def call(*a, **kw):
                f(*a, **kw)
                torch.cuda.synchronize()
            return call

        def steps():
            for max_q, n in ((70, 1), (1, 50)):
                s.new.fill_(max_q)
                for _ in range(n):
                    s.step(max_q)
                    fb.sparge_kv4_read(s.c, s.cache, s.slots, s.qkv[:, HQ:HQ + HKV],
                                       s.qkv[:, HQ + HKV:])
                    s.qkv[:, :HQ].copy_(s.o)

        if pause:
            for n in names:
                setattr(fb, n, waiting(kept[n]))
        try:
            torch.cuda.synchronize()
            if captured and not pause:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=torch.cuda.Stream(), capture_error_mode="relaxed"):
                    steps()
                graph.replay()
            else:
                steps()
        finally:
            for n in names:
                setattr(fb, n, kept[n])
        torch.cuda.synchronize()
        assert fb.sparge_device_status(s.ws) == 0
        return s.o, s.qkv, s.table, s.length, s.count, s.slots

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)
