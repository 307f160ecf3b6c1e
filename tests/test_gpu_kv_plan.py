"""Block tables, slots and the free stack of a paged cache, against the
request-by-request definition: whole numbers, equal everywhere (entries that
are not named stay as they were)."""
import numpy as np
import pytest
import torch

import free_block_sparse_predict_b200 as fb

from gpu_common import dev
from serving_common import PlanState, plan_oracle, random_plan, same

pytestmark = pytest.mark.gpu


def run(args, tokens, in_place=False):
    s = PlanState(*args, tokens, dev(), in_place)
    s.call(fb)
    same(s.outputs(), plan_oracle(*args, tokens))
    return s


@pytest.mark.parametrize("R,P,width,new_max", [
    (1, 16, 3, 5), (7, 16, 40, 200), (33, 64, 9, 1), (200, 1, 50, 30), (500, 48, 20, 700),
    (1024, 16, 8, 20), (1025, 32, 5, 1), (4096, 16, 4, 9), (3, 128, 400, 40000),
    (4000, 16, 9, 100), (300, 7, 90, 600)])
@pytest.mark.parametrize("spare", [1.0, 0.6, 0.0])
def test_matches_the_definition(R, P, width, new_max, spare):
    rng = np.random.default_rng(R + int(10 * spare))
    args = random_plan(rng, R, P, width, new_max, spare=spare)
    total = int(np.maximum(args[0], 0).sum())
    run(args, total + 13)
    run(args, total, in_place=True)
    run(args, max(0, total // 2))                 # slots for half of the tokens only
    run(args, 0)


def test_many_padding_slots():
    """More slots than a whole grid of threads writes at once, nearly all of them padding."""
    rng = np.random.default_rng(9)
    run(random_plan(rng, 5, 16, 30, 300), 700_001, in_place=True)


def test_ends_only_and_idle_only():
    rng = np.random.default_rng(3)
    args = random_plan(rng, 60, 16, 11, 5, ended=1.0, idle=0.0)
    s = run(args, 40)
    assert int(s.count_out) == args[4] + int((-(-args[1] // 16)).sum())
    args = random_plan(rng, 60, 16, 11, 5, ended=0.0, idle=1.0)
    s = run(args, 40)
    assert torch.equal(s.length_out, s.length) and bool((s.slots == -1).all())


def test_pages_of_the_ended_are_handed_on():
    """Nothing is free at first: what two requests give back is all there is, top first."""
    table = np.array([[4, 9, -1, -1], [-1] * 4, [7, -1, -1, -1], [-1] * 4])
    args = (np.array([-1, 20, -5, 16]), np.array([17, 0, 16, 0]), table, np.full(10, -3), 0, 16)
    s = run(args, 36)
    assert s.table[1, :2].tolist() == [7, 9] and s.table[3, 0].item() == 4
    assert int(s.count_out) == 0 and s.admitted.tolist() == [1, 1, 1, 1]


def test_refused_requests_hold_later_ones_back_but_not_those_without_need():
    table = np.full((5, 4), -1)
    table[3, 0] = 2
    args = (np.array([16, 64, 1, 3, 16]), np.array([0, 0, 0, 5, 0]), table, np.arange(10), 3, 16)
    s = run(args, 200)
    # 1 page, then 4 of the 2 left: refused; its need counts on, so 2 and 4 are refused too
    assert s.admitted.tolist() == [1, 0, 0, 1, 0]


def test_inconsistent_numbers_stay_in_bounds():
    table = np.arange(12).reshape(3, 4)
    for length, new, count in [([-5, 1000, 64], [3, -1, -1], 2), ([64, 64, 64], [-1, -1, -1], 9),
                               ([0, 10, 20], [2 ** 31 - 1, 5, 2 ** 31 - 1], 99),
                               ([63, 64, 0], [1, 1, -2 ** 31], -4)]:
        run((np.array(new), np.array(length), table, np.arange(9) + 50, count, 16), 30)


def test_nothing():
    z = np.zeros(0, np.int64)
    s = run((z, z, np.zeros((0, 4), np.int64), np.arange(6), 4, 16), 5)
    assert s.cu.tolist() == [0] and s.slots.tolist() == [-1] * 5
    run((np.array([1, -1]), np.array([0, 0]), np.zeros((2, 0), np.int64), z, 0, 16), 3)


@pytest.mark.parametrize("slots", [50, 40_000])   # one cluster of CTAs, a whole grid
def test_replayed_graph_advances_its_state(slots):
    """Captured in place, the step decodes by itself: each replay is the definition's next step."""
    rng = np.random.default_rng(5)
    new, length, table, free, count, P = random_plan(rng, 40, 16, 12, 1, ended=0.0, idle=0.2)
    length = length // 2
    args = (new, length, table, free, count, P)
    s = PlanState(*args, slots, dev(), in_place=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side, capture_error_mode="relaxed"):
        s.call(fb)
    for _ in range(20):
        g.replay()
        want = plan_oracle(new, length, table, free, count, P, slots)
        torch.cuda.synchronize()
        same(s.outputs(), want)
        length, table, free, count = want["length"], want["table"], want["free"], want["count"]


def test_binding_refusals():
    rng = np.random.default_rng(0)
    base = PlanState(*random_plan(rng, 5, 16, 6, 9), 50, dev())
    for name, bad in [("new", base.new[:4]), ("new", base.new.long()), ("new", base.new.cpu()),
                      ("length", base.length[::2]), ("table", base.table[0]), ("cu", base.cu[:5]),
                      ("admitted", base.admitted[:3]), ("count", base.count[:0]),
                      ("table", base.table.t()), ("length_out", base.admitted),
                      ("slots", base.table.view(-1)), ("length_out", base.new)]:
        s = PlanState.__new__(PlanState)
        s.__dict__.update(base.__dict__)
        setattr(s, name, bad)
        with pytest.raises(fb.SpargeError):
            s.call(fb)
    base.P = 0
    with pytest.raises(fb.SpargeError):
        base.call(fb)
