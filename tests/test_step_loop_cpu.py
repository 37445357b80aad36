"""Buffers of a loop of steps: what a step leaves is what the next one starts from."""
import torch

from mla_split_kv_gb300 import runtime as rt


def test_a_steps_buffers_share_the_pools_count():
    pool = rt.alloc_pool(10, 32, device="cpu")
    step = rt.alloc_step(3, 64, pool=pool)
    assert step.free_count is pool.count and pool.count.item() == 10
    assert step.context_lens.tolist() == [0, 0, 0] and step.slots.shape == (64,) and step.slots.device == pool.count.device


def test_without_a_pool_the_count_is_the_steps_own():
    step = rt.alloc_step(3, 64, device="cpu")
    assert step.free_count.tolist() == [0] and step.q_indptr.dtype is torch.int32
