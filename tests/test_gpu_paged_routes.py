"""The paged attention's routes and bounds: every kernel a batch can be sent to
by the documented knobs, and row ranges that lie outside the arrays."""
import numpy as np
import pytest
import torch

from quantized_kv_cache_03_gb300 import kvq

from kvq_cases import SM_SCALE, dev
from paged_cases import Batch, i32, to_dev

pytestmark = pytest.mark.gpu

Q4, Q8 = kvq.V_Q4_0, kvq.V_Q8_0


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("knob", [("KVQ_PREFILL", "0"), ("KVQ_PREFILL", "1"), ("KVQ_TC_ROWS", "1"), ("KVQ_TC_ROWS", "5"), ("KVQ_TC_ROWS", "9"),
                                  ("KVQ_TC_ROWS", "20"), ("KVQ_TC_ROWS", "100"), ("KVQ_TC_ROWS", "100000"), ("KVQ_TC_ROWS", "0")])
@pytest.mark.parametrize("v_type", [Q4, Q8])
def test_kernels_by_rows(knob, v_type, monkeypatch):
    """Chunks on the row tiles, and short sequences on the chunk kernel."""
    monkeypatch.setenv(*knob)
    ragged = Batch([300, 37, 64, 129, 5, 0, 511, 40, 1], [7, 37, 1, 64, 5, 0, 100, 33, 1], H=2, Hq=8, page=32, v_type=v_type, seed=3, pad_rows=2)
    cut = Batch([5000], [40], H=1, Hq=4, page=64, v_type=v_type, seed=4)
    alike = [Batch([200, 300, 1], [n, n, 1], H=2, Hq=8, page=16, v_type=v_type, seed=n, pad_rows=2 * n - n - 1 if n > 1 else 0) for n in (1, 2, 6, 40)]
    single = [Batch([2000], [n], H=2, Hq=8, page=16, v_type=v_type, seed=n) for n in (1, 6)]
    for out in (torch.float32, torch.float16):
        for b in [ragged, cut] + alike + single:
            b.check(out=out, what="%s=%s" % knob)


@pytest.mark.parametrize("lens,T,qs", [
    (lens, T, qs) for lens, T in (([50, 60, 70], 6), ([3000, 2500, 2000], 6), ([400, 2500, 3000], 150))
    for qs in ([0, 1 / 3, 1 << 20, 1 << 20], [-5, -1, 2 / 3, 1.0], [0, 2 / 3, 1 / 3, 1.0], [9 << 20] * 4, [0, 2 ** 31 - 1, -2 ** 31, 1 / 2],
               [1 / 2, 1 / 2, 1.0, -1])])
def test_row_ranges_outside_the_arrays(lens, T, qs):
    """q_start past the rows, decreasing or negative: held to [0, n_tokens].
    Rows that one sequence owns are right, rows of none and the memory before
    and behind out and lse keep what they held.  (Fractions are of the rows.)"""
    b = Batch(lens, [1] * 3, H=2, Hq=8, page=32, seed=T, pad_rows=T - 3)
    qs = [int(x * T) if isinstance(x, float) else x for x in qs]
    b.q_start = np.array(qs, np.int32)
    o, ls = (torch.full((T + 8, 8) + d, 777.0, device=dev()) for d in ((128,), ()))
    kvq.kvq_paged_attn(b.pool, to_dev(b.q), i32(b.q_start), T, i32(b.lens), to_dev(b.table), True, SM_SCALE, o[4:4 + T], ls[4:4 + T])
    torch.cuda.synchronize()
    assert kvq.kvq_wait_timeouts() == 0
    o, ls = o.cpu().numpy().astype(np.float64), ls.cpu().numpy().astype(np.float64)
    for x in (o, ls):
        assert (x[:4] == 777).all() and (x[4 + T:] == 777).all()
    o, ls = o[4:4 + T], ls[4:4 + T]
    at = [min(max(x, 0), T) for x in qs]
    owners = np.zeros(T, int)
    for s in range(3):
        owners[at[s]:max(at[s], at[s + 1])] += 1
    assert (o[owners == 0] == 777).all() and (ls[owners == 0] == 777).all()
    a, _, el = b.bounds()
    for s in range(3):
        n = at[s + 1] - at[s]
        if n <= 0:
            continue
        b.q_start, b.new = np.array(at, np.int32), [n] * 3
        ro, rl = b.reference(s, True)
        one = owners[at[s]:at[s] + n] == 1
        assert (np.abs(o[at[s]:at[s] + n] - ro)[one] <= a).all() and (np.abs(ls[at[s]:at[s] + n] - rl)[one] <= el).all()
