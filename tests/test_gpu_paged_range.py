"""The paged cache on a GPU where numbers are small, large or not numbers:
attention over blocks whose fp16 scales are subnormal or at the top of their
range, against the fp64 oracle block by block."""
import numpy as np
import pytest
import torch

import oracle
from quantized_kv_cache_03_gb300 import kvq

from kvq_cases import SM_SCALE
from paged_cases import Batch, values

pytestmark = pytest.mark.gpu

I8, F16 = kvq.K_I8, kvq.K_F16
Q4, Q8 = kvq.V_Q4_0, kvq.V_Q8_0


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _check_by_block(b, out, causal=True):
    """b.attn against the oracle, each 32-block of the output held to the size
    of that block's own stored V.  A weight is off by es (Batch.bounds); p * d
    keeps 2^-21 of itself and the sums sqrt(L) * 2^-23.  The row tiles hold p * d
    in fp16 parts, whose least step is 2^-25 where the stage's largest p * d is
    2^9 at least: n * 2^-34 of the largest V for n positions of any weight.
    fp16 output rounds p * d (2^-11) and the result (2^-11, and 2^-25 at least)."""
    o, ls = b.attn(causal=causal, out=out)
    assert kvq.kvq_wait_timeouts() == 0
    for s, (L, n) in enumerate(zip(b.lens, b.new)):
        t0 = b.q_start[s]
        k, v = values(oracle.quantize_kv(*b.kv[s], b.v_type, k_type=b.k_type), b.v_type)   # [H][L][128]
        kn = np.linalg.norm(k, axis=-1).max()
        qn = np.linalg.norm(b.q[t0:t0 + n].astype(np.float64), axis=-1).max()
        es = 32 * 2.0 ** -24 * kn * qn * SM_SCALE * 1.03 + 2.0 ** -20
        vb = np.abs(v).reshape(-1, 4, 32).max((0, 2))                                      # each block's largest
        a = vb * (2 * es + 2.0 ** -21 + np.sqrt(L) * 2.0 ** -23) + vb.max() * L * 2.0 ** -34
        rel = 0.0
        if out == torch.float16:
            a, rel = a + vb * 2.0 ** -11 + 2.0 ** -25, 2.0 ** -11
        ro, rl = b.reference(s, causal)
        d = np.abs(o[t0:t0 + n] - ro).reshape(n, b.Hq, 4, 32)
        lim = a[:, None] + rel * np.abs(ro).reshape(d.shape)
        worst = (d / lim).max((0, 1, 3))
        assert (d <= lim).all(), "seq %d (L %d, n %d): error over bound by block %s, over the block's largest V %s" % (
            s, L, n, worst.round(2), (d.max((0, 1, 3)) / vb))
        assert (np.abs(ls[t0:t0 + n] - rl) <= es + 2.0 ** -22 * (kn * qn * SM_SCALE + 20)).all()


AMPS = {"1e-2": 1e-2, "1e-3": 1e-3, "1e-4": 1e-4, "blocks": (1.0, 1e-2, 1e-3, 1e-4), "rising": "rising", "falling": "falling"}


@pytest.mark.parametrize("amp", AMPS)
@pytest.mark.parametrize("new", [1, 6, 40])
@pytest.mark.parametrize("k_type,v_type", [(I8, Q4), (I8, Q8), (F16, Q8)])
def test_small_values(new, k_type, v_type, amp):
    """V down to fp16's subnormal scales, over the whole cache, block by block
    of a row, or along the sequence (by 4 decades, up or down)."""
    def shape(kv):
        f = AMPS[amp]
        if isinstance(f, str):
            n = kv.shape[1]
            f = 10.0 ** (np.linspace(-4, 0, n) if f == "rising" else np.linspace(0, -4, n))[:, None, None]
        elif isinstance(f, tuple):
            f = np.repeat(f, 32)
        kv[1] *= f
        return kv
    b = Batch([700, 150], [new, new], H=2, Hq=8, page=16, k_type=k_type, v_type=v_type, seed=new, shape=shape)
    b.q = (b.q * 0.25).astype(np.float16)
    for out in (torch.float32, torch.float16):
        _check_by_block(b, out)


@pytest.mark.parametrize("amp", [1e-2, 1e-3, 1e-4])
@pytest.mark.parametrize("new", [1, 6, 40])
def test_small_keys_under_large_queries(new, amp):
    def shape(kv):
        kv[0] *= amp
        return kv
    b = Batch([700, 150], [new, new], H=2, Hq=8, page=32, v_type=Q8, seed=new, shape=shape)
    b.q = (b.q * (0.25 / amp)).astype(np.float16)
    _check_by_block(b, torch.float32)


@pytest.mark.parametrize("new", [1, 6, 40])
@pytest.mark.parametrize("v_type", [Q4, Q8])
def test_largest_values(new, v_type):
    """Blocks that hold fp16's largest numbers: 127 times their scale rounds
    past fp16's range."""
    def shape(kv):
        kv[1][:, :, 5] = 65504
        kv[1][:, :, 40] = -65504
        kv[1][:, :, 70] = 65472
        return kv
    b = Batch([700, 150], [new, new], H=2, Hq=8, page=64, v_type=v_type, seed=new, shape=shape)
    b.q = (b.q * 0.25).astype(np.float16)
    _check_by_block(b, torch.float32)
    keys = Batch([300], [new], H=2, Hq=8, page=64, v_type=v_type, seed=new, shape=lambda kv: np.stack([kv[0] * 0 + 65504 * np.sign(kv[0]), kv[1]]))
    keys.q = (keys.q * 2e-5).astype(np.float16)
    _check_by_block(keys, torch.float32)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("L", [90, 3000])   # whole row tiles, and tiles cut over CTAs
@pytest.mark.parametrize("new", [1, 6, 40])
@pytest.mark.parametrize("k_type", [I8, F16])
def test_a_query_that_is_not_finite_gives_nan(k_type, new, L, bad):
    """Rows whose query holds one value that is not finite: NaN in out and lse,
    every other row what it is without them; a row that sees nothing stays empty."""
    for at in (0, 77, 127):
        b = Batch([L, new - 1], [new, new], H=2, Hq=8, page=32, k_type=k_type, v_type=Q8, seed=new)
        want = b.attn()
        a, _, el = b.bounds()
        hit = np.zeros((b.T, b.Hq), bool)
        hit[[0, new // 2, new, b.T - 1], [0, 3, 1, 5]] = True
        b.q[hit, at] = bad
        o, ls = b.attn()
        seen = np.ones(b.T, bool)
        seen[new] = False          # the first of new rows over new - 1 positions
        assert np.isnan(o[hit & seen[:, None]]).all() and np.isnan(ls[hit & seen[:, None]]).all()
        assert (o[new] == 0).all() and np.isneginf(ls[new]).all()
        # the rows of a tile move their zero points together, so the others need not keep their bits: each run
        # is within the bounds of the exact values
        fin = ~hit & seen[:, None]
        assert (np.abs(o[fin] - want[0][fin]) <= 2 * a).all() and (np.abs(ls[fin] - want[1][fin]) <= 2 * el).all()


@pytest.mark.parametrize("L", [90, 3000])
@pytest.mark.parametrize("new", [1, 6, 40])
@pytest.mark.parametrize("k_type", [I8, F16])
def test_an_infinite_score_gives_nan(k_type, new, L):
    """The newest key holds infinities that the query turns into scores of
    +inf (an int8 key's infinity has code -127): the last row is NaN."""
    def shape(kv):
        kv[0][-1, :, 7::32] = np.inf
        return kv
    b = Batch([L], [new], H=2, Hq=8, page=32, k_type=k_type, v_type=Q4, seed=new, shape=shape)
    b.q[:, :, 7::32] = np.abs(b.q[:, :, 7::32]) + np.float16(0.5)
    if k_type == I8:
        b.q[:, :, 7::32] *= -1
    o, ls = b.attn()
    assert np.isnan(o[-1]).all() and np.isnan(ls[-1]).all()
    assert np.isfinite(o[:-1]).all() and np.isfinite(ls[:-1]).all()


@pytest.mark.parametrize("max_q", [1, 5, 33])
@pytest.mark.parametrize("k_type", [I8, F16])
def test_rows_past_max_q_do_not_move_the_others(k_type, max_q):
    """The first max_q rows of a longer sequence see what they see without the
    bound; the rest is left alone."""
    b = Batch([90, 700, 17, 60], [3, 60, 17, 60], H=2, Hq=8, page=16, k_type=k_type, seed=max_q, pad_rows=1)
    for causal in (True, False):
        o, ls = b.attn(causal=causal, max_q=max_q)
        a, _, el = b.bounds()
        for s, n in enumerate(b.new):
            t0, m = b.q_start[s], min(n, max_q)
            ro, rl = b.reference(s, causal)
            assert (np.abs(o[t0:t0 + m] - ro[:m]) <= a).all() and (np.abs(ls[t0:t0 + m] - rl[:m]) <= el).all()
            assert (o[t0 + m:t0 + n] == 777).all() and (ls[t0 + m:t0 + n] == 777).all()
        assert (o[-1] == 777).all()
