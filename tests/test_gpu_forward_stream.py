"""sparge_forward on a stream that is not the current one: its temporaries belong to that stream, so
what the current stream allocates afterwards is other memory."""
import numpy as np
import pytest
import torch

import free_block_sparse_predict_b200 as fb
from oracle import sparge_oracle as orc

from gpu_common import dev, params_for, to_dev, workload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_rope", [False, True])
@pytest.mark.parametrize("kind", ["stream", "address"])
def test_memory_of_a_call_on_another_stream_is_not_handed_on(kind, with_rope):
    """The other stream is kept waiting while the current one fills all the memory that it is given."""
    w, t = workload("image_dit", Hq=2, Hkv=2)
    p = params_for(w, o_dtype={"f16": torch.float16, "bf16": torch.bfloat16}[w.dtype])
    q, k, v = (to_dev(t[x], w.dtype) for x in ("q", "k", "v"))
    perm = torch.from_numpy(orc.hilbert_permutation(w.N, w.prefix_len, *w.grid).astype(np.int32)).to(dev())
    rope = fb.Rope(fb.grid_positions(w.N, w.prefix_len, *w.grid), *fb.rope_frequencies((16, 24, 24))) \
        if with_rope else None
    want = fb.sparge_forward(p, q, k, v, perm=perm, rope=rope)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    waits = torch.cuda.Event()
    call = lambda: fb.sparge_forward(p, q, k, v, perm=perm, rope=rope,
                                     stream=side if kind == "stream" else side.cuda_stream)
    call()                                            # the other stream's memory is there
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(500_000_000)                # a quarter of a second
        waits.record()
    got = call()
    assert not waits.query()
    fills = [torch.full((n,), 255, dtype=torch.uint8, device=dev())
             for n in (q.numel() * 2, k.numel() * 2, v.numel() * 2, fb.sparge_workspace_bytes(p)) for _ in range(4)]
    torch.cuda.current_stream().synchronize()
    assert not waits.query()
    torch.cuda.synchronize()
    assert all(bool((x == 255).all()) for x in fills)
    for a, b in zip(got, want):
        assert a.shape == b.shape
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[3], want[3])
