"""A serving call that the CUDA runtime refuses reports that itself and leaves nothing behind for the
next call to report.  The refusal here is the host's: a launch into a stream whose capture has
already been given up."""
import ctypes

import numpy as np
import pytest
import torch

import free_block_sparse_predict_b200 as fb

from gpu_common import dev
from serving_common import AttnCase, PlanState, random_plan

pytestmark = pytest.mark.gpu


def calls():
    plan = random_plan(np.random.default_rng(0), 20, 16, 12, 9)
    few, many = PlanState(*plan, 200, dev()), PlanState(*plan, 40_000, dev())
    case = AttnCase(fb, dev(), [100], [40], 4, 2, 64, 64, 16, torch.float16)
    case.run()
    o = torch.empty(case.q.shape, dtype=case.q.dtype, device=dev())
    args = (case.c, case.q, case.cache, case.table, case.lens_t, case.cu, 40, o, case.ws)
    slots = case.slots[0]
    rows = torch.zeros(100, 2, 64, dtype=torch.float16, device=dev())
    x = torch.zeros(1, 2, 9, 64, device=dev())
    pos = torch.zeros(1, 9, dtype=torch.int32, device=dev())
    rope = fb.rope_frequencies((32,), device=dev())
    return dict(plan_step=lambda s: few.call(fb, s), plan_prompts=lambda s: many.call(fb, s),
                attn=lambda s: fb.sparge_kv4_attn(*args, stream=s),
                append=lambda s: fb.sparge_kv4_append(case.c, rows, rows, slots, case.cache, stream=s),
                read=lambda s: fb.sparge_kv4_read(case.c, case.cache, slots, rows, rows, stream=s),
                rope=lambda s: fb.sparge_rope_apply(x, x, pos, *rope, stream=s))


@pytest.mark.parametrize("name", ["plan_step", "plan_prompts", "attn", "append", "read", "rope"])
def test_a_refused_launch_is_reported_once(name):
    call, rt, side = calls()[name], ctypes.CDLL("libcudart.so.12"), torch.cuda.Stream()
    perm = torch.empty(64, dtype=torch.int32, device=dev())
    ws = torch.zeros(fb.sparge_hilbert_workspace_bytes(1, 8, 8), dtype=torch.uint8, device=dev())
    call(None)
    torch.cuda.synchronize()
    s, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    assert rt.cudaStreamBeginCapture(s, 2) == 0          # relaxed
    try:
        assert rt.cudaStreamSynchronize(s) == 900        # not allowed: the capture is given up
        with pytest.raises(fb.SpargeError) as e:
            call(side)
        assert e.value.code == 3
    finally:
        rt.cudaStreamEndCapture(s, ctypes.byref(graph))
        rt.cudaGetLastError()
    fb.sparge_hilbert_index(64, 0, 1, 8, 8, perm, ws)    # asks the runtime for the last error
    call(None)
    torch.cuda.synchronize()
    assert sorted(perm.tolist()) == list(range(64))
