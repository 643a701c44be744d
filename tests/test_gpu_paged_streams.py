"""The workspace that a prepared attention call allocates, on other streams
than the one it was allocated on: neither work queued there before nor work
queued after the call is dropped may meet the call's kernels in that memory."""
import numpy as np
import pytest
import torch

from quantized_kv_cache_03_gb300 import kvq

from kvq_cases import SM_SCALE, dev
from paged_cases import Batch, i32, to_dev

pytestmark = pytest.mark.gpu
CYCLES = 40_000_000   # of a device sleep: some 20 ms, bounded


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


class Work:
    def __init__(self):
        self.b = Batch([3000, 40], [3, 1], H=2, Hq=8, page=16, seed=9)     # cut tiles: the workspace is used
        self.want = self.b.attn()[0]
        b = self.b
        self.out = torch.zeros((b.T, b.Hq, 128), device=dev())
        self.args = (b.pool, to_dev(b.q), i32(b.q_start), 3, i32(b.lens), to_dev(b.table), True, SM_SCALE, self.out)
        probe = kvq.PagedAttnCall(*self.args)
        self.size = probe.workspace_size()
        assert self.size > 1 << 20
        del probe
        torch.cuda.synchronize()
        torch.cuda.empty_cache()

    def right(self):
        torch.cuda.synchronize()
        return np.array_equal(self.out.cpu().numpy().astype(np.float64), self.want)


@pytest.mark.parametrize("how", ["prepared", "function", "handle"])
def test_memory_still_in_use_where_the_workspace_was_allocated(how):
    w, side = Work(), torch.cuda.Stream()
    x = torch.full((w.size,), 7, dtype=torch.uint8, device=dev())
    torch.cuda.synchronize()
    at = x.data_ptr()
    torch.cuda._sleep(CYCLES)
    y = x.clone()            # queued: reads x in 20 ms
    del x                    # the block is free for this stream's next tensor
    if how == "prepared":
        call = kvq.PagedAttnCall(*w.args)
        assert call._own.data_ptr() == at, "the allocator gave the call other memory: the test shows nothing"
        call(side)
    else:
        kvq.kvq_paged_attn(*w.args, stream=side if how == "function" else side.cuda_stream)
    assert w.right()
    assert (y == 7).all()


@pytest.mark.parametrize("how", ["prepared", "function", "handle"])
def test_memory_given_away_when_the_call_is_dropped(how):
    w, side = Work(), torch.cuda.Stream()
    call = kvq.PagedAttnCall(*w.args)
    at = call._own.data_ptr()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    if how == "prepared":
        call(side)
    else:
        del call
        kvq.kvq_paged_attn(*w.args, stream=side if how == "function" else side.cuda_stream)
        call = None
    del call
    z = torch.full((w.size,), 7, dtype=torch.uint8, device=dev())   # on this stream, at once
    assert w.right()
    assert (z == 7).all(), "the call's kernels wrote into memory that torch had given away (%s)" % (z.data_ptr() == at)


def test_a_call_first_made_in_a_capture():
    w = Work()
    call = kvq.PagedAttnCall(*w.args)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        w.out.zero_()
        g.replay()
        assert w.right()
    w.out.zero_()
    call(torch.cuda.Stream())
    assert w.right()
