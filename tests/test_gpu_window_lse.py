"""Log-sum-exp of window attention where a row sees a NaN: the row is not empty, so it is NaN as O is."""
import pytest
import torch

import sparse_attention_long_head_b200 as vs
from vs_testutil import bf16_to_dev
from vs_workloads import gen_qkv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,Hq,Hkv,d,bad", [(600, 2, 1, 64, 100), (300, 4, 2, 128, 299), (129, 1, 1, 64, 128),
                                            (700, 4, 1, 128, 0), (1, 2, 2, 128, 0)])
def test_lse_of_rows_that_see_a_nan_key(N, Hq, Hkv, d, bad, cuda_device):
    window, sinks = 50, 2
    Q, K, V = (bf16_to_dev(x) for x in gen_qkv(N + bad, N, Hq, Hkv, d, 10000.0))
    ref, lref = vs.window_attention(Q, K, V, window, sinks)
    K[bad] = float("nan")
    seen = torch.zeros(N, dtype=torch.bool, device="cuda")
    seen[bad:N if bad < sinks else bad + window] = True
    O, lse = vs.window_attention(Q, K, V, window, sinks)
    # the same rows in a packed batch, behind another sequence
    cu = torch.tensor([0, N, 2 * N], dtype=torch.int32, device="cuda")
    Q2, K2, V2 = (torch.cat([x, x]) for x in (Q, K, V))
    K2[bad] = K2[bad + 1 if bad + 1 < N else 0] if N > 1 else 1.0  # the first sequence has no NaN
    O2, lse2 = torch.empty_like(Q2), torch.empty((Hq, 2 * N), device="cuda")
    vs.vs_window_attn_fwd_varlen(Q2, K2, V2, cu, N, window, sinks, O2, lse2, vs.workspace(256))
    assert torch.isfinite(lse2[:, :N]).all()
    for o, l in ((O, lse), (O2[N:], lse2[:, N:])):
        assert o[seen].isnan().all() and l[:, seen].isnan().all()
        assert torch.equal(o[~seen], ref[~seen]) and torch.equal(l[:, ~seen], lref[:, ~seen])
