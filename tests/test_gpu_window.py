"""Sliding-window attention with visible first keys vs the fp64 oracle (the window as the slash
offsets below it, the first keys as vertical columns), single sequences and packed batches.

Tolerance of O: P is rounded to bf16 before the product with V (half a step, finfo(bfloat16).eps / 2 =
2^-8 of each weight) and O once at the end (2^-8 of the value), so |err| <= 2^-8 max|V| + 2^-8 max|V|;
the fp32 sums, the exponential and the log-sum-exp are off by less than 1e-4 at these sizes (scores below 32, at most
128 fp32 additions per score)."""
import numpy as np
import pytest
import torch

import oracle
import sparse_attention_long_head_b200 as vs
from vs_testutil import bf16_to_dev, dev_to_f64, sets_to_rows
from vs_workloads import bf16_bits_to_f32, gen_qkv

pytestmark = pytest.mark.gpu


def _check(O, lse, Qb, Kb, Vb, window, sinks, what=""):
    """Every row of one sequence, some heads: O [N, Hq, d], lse [Hq, N] as float64."""
    N, Hq, _ = Qb.shape
    vi, vc = sets_to_rows([np.arange(min(sinks, N))])
    si, sc = sets_to_rows([np.arange(min(window, N))])
    tol = 2.0 ** -7 * np.abs(bf16_bits_to_f32(Vb)).max() + 1e-4
    for h in sorted({0, Hq // 2, Hq - 1}):
        Or, lr = oracle.attn_rows(Qb, Kb, Vb, h, np.arange(N), vi, vc, si, sc)
        err = np.abs(O[:, h] - Or).max()
        assert err <= tol, (what, h, err, tol)
        assert np.abs(lse[h] - lr).max() <= 1e-4, (what, h)


@pytest.mark.parametrize("N", [1, 2, 127, 128, 129, 256, 257, 700, 1153])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (128, 0), (129, 130), (300, 257), (1 << 30, 0),
                                          (5, 1 << 30)])
def test_window_against_oracle(N, window, sinks, cuda_device):
    d, Hq, Hkv = (64, 2, 2) if N % 2 else (128, 4, 1)
    Qb, Kb, Vb = gen_qkv(N + window % 1000, N, Hq, Hkv, d, 10000.0)
    Q, K, V = (bf16_to_dev(x) for x in (Qb, Kb, Vb))
    ws = vs.workspace(256)
    O, lse = vs.window_attention(Q, K, V, window, sinks, ws=ws)
    assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)
    _check(dev_to_f64(O), lse.cpu().numpy().astype(np.float64), Qb, Kb, Vb, window, sinks)


def test_whole_window_is_dense(cuda_device):
    Q, K, V = (bf16_to_dev(x) for x in gen_qkv(3, 900, 4, 2, 128, 10000.0))
    O, lse = vs.window_attention(Q, K, V, 900)
    Od, lsed = vs.dense_attention(Q, K, V)
    assert torch.equal(O, Od) and torch.equal(lse, lsed)


@pytest.mark.parametrize("lengths,d,Hq,Hkv,window,sinks", [
    ([1, 300, 1000, 129, 0, 2048], 128, 4, 2, 200, 5),
    ([640, 1, 777], 64, 7, 1, 64, 129),
    ([5, 3, 1, 2], 64, 2, 2, 2, 1),
])
def test_varlen_against_oracle(lengths, d, Hq, Hkv, window, sinks, cuda_device):
    parts = [gen_qkv(11 + i, n, Hq, Hkv, d, 10000.0) if n else None for i, n in enumerate(lengths)]
    Qb, Kb, Vb = (np.concatenate([p[t] for p in parts if p is not None]) for t in range(3))
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    T = cu[-1] + 70  # rows behind the last sequence: filled with NaN, never read into a result
    pad = np.full((70,) + Kb.shape[1:], 0x7FC0, np.uint16)
    Q, K, V = (bf16_to_dev(np.concatenate([x, p])) for x, p in
               ((Qb, np.full((70, Hq, d), 0x7FC0, np.uint16)), (Kb, pad), (Vb, pad)))
    O = torch.full_like(Q, 7.0)
    lse = torch.full((Hq, T), 7.0, device="cuda")
    ws = vs.workspace(256)
    vs.vs_window_attn_fwd_varlen(Q, K, V, torch.from_numpy(cu).cuda(), max(lengths), window, sinks, O, lse, ws)
    assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)
    assert (O[cu[-1]:] == 7).all() and (lse[:, cu[-1]:] == 7).all()
    Od, ld = dev_to_f64(O), lse.cpu().numpy().astype(np.float64)
    for b, n in enumerate(lengths):
        sl = slice(cu[b], cu[b + 1])
        if n:
            _check(Od[sl], ld[:, sl], Qb[sl], Kb[sl], Vb[sl], window, sinks, f"sequence {b}")


def test_neighbours_never_reach_a_sequence(cuda_device):
    """A sequence between others full of infinities and NaN gives the bits it gives alone."""
    n, d = 333, 128
    Q, K, V = (bf16_to_dev(x) for x in gen_qkv(5, n, 2, 1, d, 10000.0))
    O1, lse1 = vs.window_attention(Q, K, V, 100, 3)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38], device="cuda").bfloat16()
    big = lambda x: torch.cat([bad.repeat(x[0].numel() * 50).view(200, *x.shape[1:]), x,
                               bad.repeat(x[0].numel() * 50).view(200, *x.shape[1:])])  # noqa: E731
    cu = torch.tensor([0, 200, 200 + n, 400 + n], dtype=torch.int32, device="cuda")
    Qp, Kp, Vp = big(Q), big(K), big(V)
    O = torch.empty_like(Qp)
    lse = torch.empty((2, 400 + n), device="cuda")
    ws = vs.workspace(256)
    vs.vs_window_attn_fwd_varlen(Qp, Kp, Vp, cu, n, 100, 3, O, lse, ws)
    assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)
    assert torch.equal(O[200:200 + n], O1) and torch.equal(lse[:, 200:200 + n], lse1)


def test_infinite_keys_out_of_sight(cuda_device):
    """K may hold anything where no query of interest sees it: rows past the window of an infinite key."""
    N = 600
    Q, K, V = (bf16_to_dev(x) for x in gen_qkv(6, N, 2, 1, 64, 10000.0))
    ref, lref = vs.window_attention(Q, K, V, 50, 2)
    K[100] = float("nan")
    O, lse = vs.window_attention(Q, K, V, 50, 2)
    seen = torch.zeros(N, dtype=torch.bool, device="cuda")
    seen[100:150] = True
    assert torch.equal(O[~seen], ref[~seen]) and torch.equal(lse[:, ~seen], lref[:, ~seen])
    assert O[seen].isnan().all()


def test_strided_rows_and_scale(cuda_device):
    N, Hq, Hkv, d = 500, 4, 2, 64
    Qb, Kb, Vb = gen_qkv(8, N, Hq, Hkv, d, 10000.0)
    wide = [torch.zeros((N, h + 3, d), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv)]
    Q, K, V = (w[:, :x.shape[1]] for w, x in zip(wide, (Qb, Kb, Vb)))
    for t, x in ((Q, Qb), (K, Kb), (V, Vb)):
        t.copy_(bf16_to_dev(x))
    out = torch.full((N, Hq + 3, d), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = vs.workspace(256)
    vs.vs_window_attn_fwd(Q, K, V, 77, 9, out[:, :Hq], None, ws, softmax_scale=0.25)
    # the scale folded into Q: 0.25 = 2 / sqrt(64), an exact power of two
    O, _ = vs.window_attention(bf16_to_dev(Qb) * 2, bf16_to_dev(Kb), bf16_to_dev(Vb), 77, 9)
    assert torch.equal(out[:, :Hq], O) and (out[:, Hq:] == 5).all()


def test_malformed_offsets_are_flagged_and_contained(cuda_device):
    lengths = [300, 500, 300]
    Q, K, V = (bf16_to_dev(x) for x in gen_qkv(9, 1100, 2, 1, 128, 10000.0))
    cu = torch.tensor([0, 300, 800, 1100], dtype=torch.int32, device="cuda")
    O = torch.full_like(Q, 7.0)
    ws = vs.workspace(256)
    vs.vs_window_attn_fwd_varlen(Q, K, V, cu, 400, 64, 4, O, None, ws)
    rc, flags = vs.vs_read_device_status(ws)
    assert rc == vs.VS_ERR_DEVICE_BOUNDS and flags & vs.VS_DEVFLAG_BOUNDS
    assert (O[300:800] == 7).all()
    for a, n in ((0, lengths[0]), (800, lengths[2])):
        sl = slice(a, a + n)
        O1, _ = vs.window_attention(Q[sl].clone(), K[sl].clone(), V[sl].clone(), 64, 4)
        assert torch.equal(O[sl], O1)
