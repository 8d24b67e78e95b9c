"""Edges of the cache calls on the GPU: waits that run out, odd offsets, no rows,
windows without an end, NaN, steps that were overtaken, graphs and threads."""
import threading

import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests.helpers import require_gpu, to_np_f32
from tests.test_gpu_kv4 import DEV, F32, I32, attn_case, dev, same, state
from tests.test_gpu_kv_cache import LAYERS, bytes_of, cache, inputs, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    import mixture_experts_layer_fwd_gb300 as m
    m.moe_sync_status()
    yield
    assert m.moe_sync_status() == 0


def moe():
    import mixture_experts_layer_fwd_gb300 as m
    return m


def attn_args(c):
    return (c["q"].to(DEV), dev(c["pool"]), dev(c["gk"]), dev(c["gv"]), dev(c["starts"]), dev(c["lens"]), dev(c["table"]))


# heads, new tokens of each sequence: the 16-row kernel, the decode kernel that
# makes its own schedule, the one with a schedule in front, the 256-row kernel
KERNELS = [(64, [1, 2]), (128, [1, 2]), (128, [1] * 40), (64, [300, 90]), (128, [300, 90])]


# ------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("lazy", [False, True])
@pytest.mark.parametrize("limit_us", [1000, 20000])
def test_attention_waits_give_up_near_their_limit(lazy, limit_us):
    """They count tests of about 4 us (5 % more where they sleep in between): within a factor of two of the limit."""
    m = moe()
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    t[0].record()
    m.moe_selftest_attention_wait_timeout(1000 * limit_us, lazy)
    t[1].record()
    assert m.moe_sync_status() == 5 and m.moe_sync_status() == 0
    assert limit_us / 2 <= 1000 * t[0].elapsed_time(t[1]) <= 2 * limit_us
