"""Long query chunks over segments whose V is small or at the top of fp16's
range, against the fp64 oracle, each 32-block of the output held to the size
of that block's own V."""
import numpy as np
import pytest
import torch

import oracle
from quantized_kv_cache_03_gb300 import kvq

from kvq_cases import SM_SCALE, dev, to_dev
from paged_cases import values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("amp", [1.0, 1e-2, 1e-3, 1e-4, (1.0, 1e-2, 1e-3, 1e-4), "largest"])
@pytest.mark.parametrize("v_type", [kvq.V_Q4_0, kvq.V_Q8_0])
def test_chunks_over_values_of_any_size(v_type, amp):
    L, t_q, H, Hq = 700, 40, 2, 8
    r = np.random.default_rng(5)
    kv = r.standard_normal((2, L, H, 128)).astype(np.float32)
    if amp == "largest":
        kv[1][:, :, [5, 40, 70]] = 65504, -65504, 65472
    else:
        kv[1] *= np.repeat(amp, 32) if isinstance(amp, tuple) else amp
    kv = kv.astype(np.float16)
    q = (r.standard_normal((1, t_q, Hq, 128)) * 0.25).astype(np.float16)
    cache = kvq.Cache(1, H, v_type, max_segs=1)
    cache.add_segment(0, L)
    kvq.kvq_append(cache, [0], [L], to_dev(kv[0]), to_dev(kv[1]))
    call = dict(cache=cache, n_q_heads=Hq, t_q=t_q, causal_tail=True, max_len=L, head_map=None, sm_scale=SM_SCALE)
    assert {x["kernel"] for x in kvq.kvq_debug_plan([call], 152)[0]} == {"prefill"}
    out = torch.empty((1, t_q, Hq, 128), device=dev())
    lse = torch.empty((1, t_q, Hq), device=dev())
    n = kvq.kvq_decode_workspace_size(cache, Hq, t_q, L)
    kvq.kvq_decode_attn(cache, to_dev(q), Hq, t_q, True, torch.tensor([L], dtype=torch.int32, device=dev()), L, None, SM_SCALE,
                        out, lse, torch.empty(n, dtype=torch.uint8, device=dev()) if n else None)
    torch.cuda.synchronize()
    stored = oracle.quantize_kv(kv[0], kv[1], v_type)
    ref = oracle.decode_seq(stored, q[0], oracle.default_head_map(Hq, H), True, SM_SCALE, v_type, n_threads=8)
    k, v = values(stored, v_type)
    # a score: 32 fp32 roundings of |q||k| at most; a weight that and 2^-20 for ex2, lg2, the reciprocal and the
    # sums; P.V 2^-21 of each product and 2^-23 of the running sum per root of its length
    es = 32 * 2.0 ** -24 * np.linalg.norm(k, axis=-1).max() * np.linalg.norm(q.astype(np.float64), axis=-1).max() * SM_SCALE * 1.03 + 2.0 ** -20
    vb = np.abs(v).reshape(-1, 4, 32).max((0, 2))
    lim = vb * (2 * es + 2.0 ** -21 + np.sqrt(L) * 2.0 ** -23)
    d = np.abs(out[0].cpu().numpy() - ref["out"]).reshape(t_q, Hq, 4, 32)
    assert (d <= lim[:, None]).all(), "error over the block's largest V: %s, allowed %s" % (d.max((0, 1, 3)) / vb, lim / vb)
