"""GPU tests of the key/value cache calls at the edges of what their documentation allows:
capacities whose keys nearly fill the default shared memory, rollbacks that add nothing, counts
and indexes out of range, infinities and NaN where nothing looks, and handles whose tensors moved."""

import math
import os
import subprocess
import sys
import threading

import pytest
import torch

import block_sparse_attention_ab_b200 as ab
from cache_reference import F64, HostCache, attn, keep, mass, score

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_attention_ab_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ab.lib()


def _flag():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_keep_refuses_sizes_outside_32_bits():
    g = HostCache([40], 1, 64, 16, BF, seed=17).to_gpu()
    for budget in (0, -1, 5 - 2 ** 32, -2 ** 31 - 1, 2 ** 32 + 5, 2 ** 62):
        with pytest.raises((ValueError, ab.AbError)):
            ab.cache_keep(g, budget)
    for recent in (-1, 5 - 2 ** 32, 2 ** 32 + 5):
        with pytest.raises((ValueError, ab.AbError)):
            ab.cache_keep(g, 8, recent=recent, next_pos=_i32(40))
