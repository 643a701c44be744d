"""The paged attention kernels' bounded copy waits, driven to run out on purpose.

kvq_debug_paged_lose_copy runs the call on test flavours of the kernels whose
first CTA arms one copy's barrier without issuing the copy.  The wait for it,
given a short limit, gives up; the roles leave, having waited for every copy
they did issue; the CTA's rows come out as NaN, in pieces that it had not come
to as well, and the wait counter grows by one.  No kernel faults or waits
without a limit.  out, lse and the workspace are filled with finite numbers
first, so a row that nobody wrote shows."""
import numpy as np
import pytest
import torch

from quantized_kv_cache_03_gb300 import kvq

from kvq_cases import SM_SCALE, dev
from paged_cases import Batch, i32, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _lose(b, copy):
    """NaN mask [rows][q heads] after a lost copy; every other row is checked."""
    o = torch.full((b.T, b.Hq, 128), 777.0, device=dev())
    ls = torch.full((b.T, b.Hq), 777.0, device=dev())
    call = kvq.PagedAttnCall(b.pool, to_dev(b.q), i32(b.q_start), b.max_q, i32(b.lens), to_dev(b.table), True, SM_SCALE, o, ls)
    call._keep[-1].zero_()
    torch.cuda.synchronize()
    kvq.kvq_reset_wait_timeouts()
    try:
        kvq.kvq_debug_paged_lose_copy(call, copy)
        torch.cuda.synchronize()
        assert kvq.kvq_wait_timeouts() == 1
    finally:
        torch.cuda.synchronize()
        kvq.kvq_reset_wait_timeouts()
    o, ls = o.cpu().numpy().astype(np.float64), ls.cpu().numpy().astype(np.float64)
    lost = np.isnan(ls)
    assert np.array_equal(np.isnan(o).all(-1), lost) and np.array_equal(np.isnan(o).any(-1), lost)
    a, _, el = b.bounds()
    for s in range(len(b.lens)):
        t0, n = b.q_start[s], b.new[s]
        ok = ~lost[t0:t0 + n]
        if ok.any():
            ro, rl = b.reference(s, True)
            assert (np.abs(o[t0:t0 + n] - ro)[ok] <= a).all() and (np.abs(ls[t0:t0 + n] - rl)[ok] <= el).all()
    b.check()     # the device stays usable, and nothing gives up
    return lost


@pytest.mark.parametrize("copy", [0, 2, 3])
def test_row_tiles_that_lose_a_stage(copy):
    """Sequences of three stages: the first warp takes one stage of every piece,
    a piece per kv head; the last piece of the CTA's share is cut.  The piece
    that lost its stage is NaN, and so are the later ones of the CTA."""
    B, H, group = 300, 8, 4
    b = Batch([70] * B, [1] * B, H=H, Hq=H * group, page=32, seed=copy)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lost = _lose(b, copy).reshape(B * H, group)     # in the order of the line of work
    assert np.array_equal(lost.all(1), lost.any(1))
    at = np.flatnonzero(lost.any(1))
    assert at[0] == copy and np.array_equal(at, np.arange(copy, at[-1] + 1)) and at[-1] > copy
    # three stages each: the CTA's share, cut in the last one it begins
    shares = [-(-B * H * 3 // (sms * k)) for k in (1, 2, 3, 4)]
    assert at[-1] in [-(-n // 3) - 1 for n in shares], (at, shares)


@pytest.mark.parametrize("copy", [0, 1, 7, 8, 13, 14])
def test_chunks_that_lose_a_copy(copy):
    """160 rows per kv head over 300 positions: two row tiles of three KV tiles
    per head; a CTA's share is several pieces, the last of them cut.  All rows of
    the first CTA are NaN, whichever K or V part of which piece is lost."""
    B, H, group, new = 100, 2, 4, 40
    b = Batch([300] * B, [new] * B, H=H, Hq=H * group, page=64, seed=copy)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    share = max(3, -(-B * H * 6 // sms))
    lost = _lose(b, copy)
    want = np.zeros_like(lost)
    for k in range(-(-share // 3)):      # the k-th row tile of the line
        s, h, rt = k // 4, k // 2 % 2, k % 2
        rows = np.arange(128 * rt, min(128 * rt + 128, new * group))
        want[s * new + rows // group, h * group + rows % group] = True
    assert np.array_equal(lost, want)
    assert share > 6 and share % 3


def test_a_long_sequence_over_many_ctas_loses_a_copy():
    """Cut tiles: the first CTA's piece is one of many, and every row of the tile is NaN."""
    for new, copy in ((2, 0), (40, 5), (40, 4)):
        b = Batch([20000, 64], [new, 1], H=1, Hq=4, page=64, seed=new)
        lost = _lose(b, copy)
        assert lost[:min(new, 32)].all()
