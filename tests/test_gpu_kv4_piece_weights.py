"""Requests with more than 64 rows for a KV head where light keys carry the answer: weights keep their
bits down to 2^-20 of the row's largest, whatever the size of V."""
import pytest
import torch

from test_gpu_kv4_light_keys import heavy_case
from test_gpu_kv4_small_scales import check_pieces

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("vscale", [1.0, 0.02, 0.002])
@pytest.mark.parametrize("nats", [0.0, 12.0, 16.5])
def test_light_keys_of_pieces_of_prompts(nats, vscale, dtype):
    """A heavy key in every 32, its values zero or small; units of one CTA and of several."""
    check_pieces(heavy_case(700, 80, 2, 2, 64, 32, dtype, nats, vscale), least=2.0 ** -20)
    check_pieces(heavy_case(6000, 40, 8, 2, 128, 128, dtype, nats, vscale, left=1e-3), least=2.0 ** -20)
