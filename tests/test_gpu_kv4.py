"""The 4-bit paged cache on the GPU vs the 64-bit reference: what append writes is compared byte for
byte, decode within derived bounds, eviction byte for byte.

Bounds of decode.  A bf16 has 8 significant bits, so rounding to it is off by at most half a step,
finfo(bfloat16).eps / 2 = 2^-8 of the value.  The only roundings below fp32 are that of p s, which acts
on n - 8 (at most 8 in size), and O's own: |err| <= 2^-8 (8 max s + max |v|) + 4e-4 max |v|.
The last term is fp32: a score is 64 products a group of |q| <= 5 and codes below 2, each of 64
additions off by at most 2^-24 of a sum below 64, times 16 s / sqrt(d): below 4e-4 for s <= 0.5; a
weight is off by that share of itself."""
import numpy as np
import pytest
import torch

import sparse_attention_long_head_b200 as vs
import vs_kv4_ref as ref
from vs_testutil import dev_to_f64

pytestmark = pytest.mark.gpu


def _dev(x):
    """float64 (bf16 values) -> bf16 on the GPU."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().bfloat16()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lengths):
    return _ints(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32))


def _table(rng, slots, extra=0):
    """Pages in random order (one spare page between sequences) -> numpy [B, width], pages."""
    need = [-(-max(n, 0) // 64) for n in slots]
    width, total = max(1, max(need)) + extra, sum(need) + 1
    order = rng.permutation(total)
    t = np.full((len(slots), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t, total


def _random_pool(rng, pages, Hkv, d):
    """Quantised N(0, 1) values in the cache's format (uint8 numpy)."""
    g = d // 64
    pool = np.empty((pages, Hkv, g * 4608), np.uint8)
    pool[..., :g * 4096] = rng.integers(0, 256, (pages, Hkv, g * 4096), dtype=np.uint8)
    s = rng.uniform(0.15, 0.4, (pages, Hkv, 2 * g * 64))
    pair = np.stack([s, -7.5 * s + rng.normal(0, 0.2, s.shape)], -1)
    pool[..., g * 4096:] = ref.bf16_bits(ref.bf16_round(pair)).view(np.uint8).reshape(pages, Hkv, g * 512)
    return pool


# ------------------------------------------------------------------------------ append and read


def _append_case(rng, start, new, Hkv, d, x=None):
    T = sum(new)
    K = ref.bf16_round(rng.standard_normal((T, Hkv, d)) if x is None else x[0])
    V = ref.bf16_round(rng.standard_normal((T, Hkv, d)) * 3 if x is None else x[1])
    end = [a + b for a, b in zip(start, new)]
    table, pages = _table(rng, end)
    return K, V, end, table, np.full((pages, Hkv, d // 64 * 4608), 0xAB, np.uint8)


def _expect(pool, K, V, start, new, table):
    want = pool.copy()
    at = 0
    for b, n in enumerate(new):
        for i in range(n):
            for h in range(K.shape[1]):
                for kv, x in enumerate((K, V)):
                    q = ref.quantize(x[at + i, h].reshape(-1, 64))
                    ref.pool_write(want, table[b], h, start[b] + i, kv, *q)
        at += n
    return want


@pytest.mark.parametrize("start,new,Hkv,d", [
    ([0], [1], 1, 64), ([63], [2], 2, 128), ([0, 5, 64, 100], [1, 130, 0, 64], 2, 128),
    ([7, 0, 0], [1, 1, 1], 3, 64), ([0], [200], 8, 64),
])
def test_append_bytes_and_read(start, new, Hkv, d, cuda_device):
    rng = np.random.default_rng(sum(start) + d)
    K, V, end, table, pool = _append_case(rng, start, new, Hkv, d)
    pd, td, cu = torch.from_numpy(pool).cuda(), torch.from_numpy(table).cuda(), _cu(new)
    ws = vs.workspace(256)
    B, ld = len(new), max(end) + 3
    G = 2
    A_v = rng.uniform(0, 4, (Hkv * G, sum(new))).astype(np.float32)
    acc = torch.full((B, Hkv, ld), -1.0, device="cuda")
    pos = torch.full((B, Hkv, ld), -1, dtype=torch.int32, device="cuda")
    seen = [e + 11 * b for b, e in enumerate(end)]
    vs.vs_kv4_append(_dev(K), _dev(V), cu, max(new), pd, td, _ints(end), ws, n_tokens=_ints(seen),
                     A_v=torch.from_numpy(A_v).cuda(), acc=acc, pos=pos)
    assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)
    want = _expect(pool, K, V, start, new, table)
    assert np.array_equal(pd.cpu().numpy(), want)
    wa, wp = np.full((B, Hkv, ld), -1.0), np.full((B, Hkv, ld), -1)
    at = 0
    for b, n in enumerate(new):
        wa[b, :, start[b]:end[b]] = A_v[:, at:at + n].astype(np.float64).reshape(Hkv, G, n).sum(1)
        wp[b, :, start[b]:end[b]] = np.arange(seen[b] - n, seen[b])
        at += n
    assert np.array_equal(pos.cpu().numpy(), wp)
    assert np.abs(acc.cpu().numpy() - wa).max() <= 8 * 2.0 ** -24 * 2  # two fp32 additions of values up to 8
    # read back: s n + m rounded once, exactly
    out = [torch.full((sum(new) + 2, Hkv + 1, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    Ko, Vo = (o[:, :Hkv] for o in out)
    vs.vs_kv4_read(pd, td, _ints(end), _ints(start), cu, max(new), Ko, Vo, ws)
    assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)
    c = ref.Cache(want)
    for o, kv in ((out[0], 0), (out[1], 1)):
        o = dev_to_f64(o)
        assert (o[:, Hkv:] == 9).all() and (o[sum(new):] == 9).all()
        at = 0
        for b, n in enumerate(new):
            for h in range(Hkv):
                if n:
                    v = c.rows(table[b], h, np.arange(start[b], end[b]), kv)
                    assert np.array_equal(o[at:at + n, h], ref.bf16_round(v))
            at += n


def test_append_extreme_groups(cuda_device):
    """Constant, tiny, huge, infinite and NaN groups, signed zeros, and values at the codes' borders."""
    rng = np.random.default_rng(3)
    n, d = 24, 64
    x = np.zeros((2, n, 1, d))
    x[:, 0] = 0.0
    x[:, 1] = -3.25
    x[:, 2, 0, 0] = np.inf
    x[:, 3, 0, 63] = np.nan
    x[:, 4, 0, :2] = [-np.inf, np.inf]
    x[:, 5] = np.where(np.arange(64) % 2, 3.38e38, -3.38e38)
    x[:, 6] = rng.standard_normal(64) * 1e-39      # subnormal
    x[:, 7] = rng.standard_normal(64) * 1e38
    x[:, 8] = (np.arange(64) % 31) * 0.5           # halves: ties everywhere
    x[:, 9] = (np.arange(64) % 31) * 0.5 - 7.5
    x[:, 10] = np.where(np.arange(64) % 2, 0.0, -0.0)
    x[:, 11] = 1 + np.arange(64) * 2.0 ** -7       # one bf16 step apart
    x[:, 12] = np.where(np.arange(64) == 3, 1e4, rng.standard_normal(64) * 1e-4)
    x[:, 13] = np.where(np.arange(64) == 3, 9.2e-41, 0.0)   # one subnormal step: s rounds to 0
    for i in range(14, n):
        x[:, i] = rng.integers(-60, 61, (2, 1, 64)) * 2.0 ** (i - 20)  # many borders
    K, V, end, table, pool = _append_case(rng, [3], [n], 1, d, x)
    pd = torch.from_numpy(pool).cuda()
    ws = vs.workspace(256)
    # bits are uploaded as they are: a float32 copy would keep every value here
    Kd, Vd = (torch.from_numpy(ref.bf16_bits(t).view(np.int16)).cuda().view(torch.bfloat16) for t in (K, V))
    vs.vs_kv4_append(Kd, Vd, _cu([n]), n, pd, torch.from_numpy(table).cuda(), _ints(end), ws)
    want = _expect(pool, K, V, [3], [n], table)
    got, wc = ref.Cache(pd.cpu().numpy()), ref.Cache(want)
    assert np.array_equal(got.codes, wc.codes)
    assert np.array_equal(got.s, wc.s, equal_nan=True) and np.array_equal(got.m, wc.m, equal_nan=True)


def test_append_many_borders(cuda_device):
    """Coarse bf16 values, where quotients often fall on or next to a half."""
    rng = np.random.default_rng(17)
    n, d, H = 600, 128, 2
    x = rng.integers(-255, 256, (2, n, H, d)) * 2.0 ** rng.integers(-6, 3, (2, n, H, 1))
    x += rng.integers(-255, 256, (2, n, H, 1)) * 1.0
    K, V, end, table, pool = _append_case(rng, [0], [n], H, d, x)
    pd = torch.from_numpy(pool).cuda()
    ws = vs.workspace(256)
    vs.vs_kv4_append(_dev(K), _dev(V), _cu([n]), n, pd, torch.from_numpy(table).cuda(), _ints(end), ws)
    c = ref.Cache(pd.cpu().numpy())
    t = np.arange(n)
    pg = table[0][t // 64]
    for kv, x in ((0, K), (1, V)):
        for h in range(H):
            nq, s, m = ref.quantize(x[:, h].reshape(n, 2, 64))
            assert np.array_equal(c.codes[pg, h, kv, :, t % 64], nq)
            assert np.array_equal(c.s[pg, h, kv, :, t % 64], s)


def test_append_strided_and_without_extras(cuda_device):
    rng = np.random.default_rng(5)
    K, V, end, table, pool = _append_case(rng, [10, 0], [70, 9], 2, 64)
    wide = [torch.zeros((79, 5, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for w, x in zip(wide, (K, V)):
        w[:, 1:3] = _dev(x)
    pd = torch.from_numpy(pool).cuda()
    ws = vs.workspace(256)
    vs.vs_kv4_append(wide[0][:, 1:3], wide[1][:, 1:3], _cu([70, 9]), 70, pd, torch.from_numpy(table).cuda(),
                     _ints(end), ws)
    assert np.array_equal(pd.cpu().numpy(), _expect(pool, K, V, [10, 0], [70, 9], table))


def test_append_refuses_what_does_not_fit(cuda_device):
    rng = np.random.default_rng(6)
    new = [3, 4, 5, 2]
    K, V, end, table, pool = _append_case(rng, [0, 0, 0, 0], new, 1, 64)
    pd, td = torch.from_numpy(pool).cuda(), torch.from_numpy(table).cuda()
    ws = vs.workspace(256)
    acc = torch.full((4, 1, 64), -1.0, device="cuda")
    # sequence 0 claims fewer slots than new tokens, 1 more than the table holds, 2 is fine, 3 has a bad page
    td[3, 0] = pool.shape[0]
    vs.vs_kv4_append(_dev(K), _dev(V), _cu(new), 5, pd, td, _ints([2, 65, 5, 2]), ws, acc=acc)
    rc, flags = vs.vs_read_device_status(ws)
    assert rc == vs.VS_ERR_DEVICE_BOUNDS and flags == vs.VS_DEVFLAG_BOUNDS
    want = _expect(pool, K[7:12], V[7:12], [0], [5], table[2:3])
    assert np.array_equal(pd.cpu().numpy(), want)
    a = acc.cpu().numpy()
    assert (a[:2] == -1).all() and (a[2, 0, :5] == 0).all() and (a[2, 0, 5:] == -1).all()
    # rows of acc too short for a sequence
    acc = torch.full((1, 1, 4), -1.0, device="cuda")
    vs.vs_kv4_append(_dev(K[7:12]), _dev(V[7:12]), _cu([5]), 5, pd, torch.from_numpy(table[2:3]).cuda(), _ints([5]),
                     ws, acc=acc)
    assert vs.vs_read_device_status(ws)[0] == vs.VS_ERR_DEVICE_BOUNDS and (acc == -1).all()
    # read of slots that are not in use
    out = torch.full((5, 1, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    for start, lens in ((1, 5), (-1, 5), (0, 4)):
        vs.vs_kv4_read(pd, torch.from_numpy(table[2:3]).cuda(), _ints([lens]), _ints([start]), _cu([5]), 5, out, out,
                       ws)
        assert vs.vs_read_device_status(ws)[0] == vs.VS_ERR_DEVICE_BOUNDS and (out == 9).all()


# ---------------------------------------------------------------------------------------- decode


def _decode_case(rng, lens, Hq, Hkv, d, extra=1):
    table, pages = _table(rng, lens, extra)
    pool = _random_pool(rng, pages, Hkv, d)
    q = ref.bf16_round(rng.standard_normal((len(lens), Hq, d)))
    return q, table, pool


def _check_decode(O, lse, q, pool, table, lens, window, sinks, acc=None, acc0=None, scale=None):
    c = ref.Cache(pool)
    O, lse = dev_to_f64(O), lse.cpu().numpy().astype(np.float64)
    for b, n in enumerate(lens):
        Or, lr, w = ref.decode(q[b], c, table[b], n, window, sinks, scale)
        if n == 0:
            assert (O[b] == 0).all() and np.isneginf(lse[:, b]).all()
            continue
        t = np.arange(n)  # the steps and values of the slots in use; what lies behind them may be anything
        smax = max(c.s[table[b][t // 64], h, 1, :, t % 64].max() for h in range(pool.shape[1]))
        vmax = max(np.abs(c.rows(table[b], h, t, 1)).max() for h in range(pool.shape[1]))
        tol = 2.0 ** -8 * (8 * smax + vmax) + 4e-4 * vmax
        assert np.abs(O[b] - Or).max() <= tol, (b, n, np.abs(O[b] - Or).max(), tol)
        assert np.abs(lse[:, b] - lr).max() <= 4e-4, (b, n)
        if acc is not None:
            got = acc[b, :, :n] - acc0[b, :, :n]
            assert (np.abs(got - w) <= 4e-4 * w + 2.0 ** -23 * (1 + np.abs(acc0[b, :, :n]))).all(), (b, n)
            assert np.array_equal(acc[b, :, n:], acc0[b, :, n:])


@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 64), (4, 2, 128), (8, 1, 128), (7, 1, 64), (6, 2, 128), (9, 1, 64),
                                      (16, 1, 128), (34, 2, 64), (20, 1, 128), (8, 8, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 3), (64, 64), (700, 130)])
def test_decode_against_reference(Hq, Hkv, d, window, sinks, cuda_device):
    rng = np.random.default_rng(Hq * 100 + d + window)
    lens = [1, 63, 64, 65, 0, 700, 1500, 2]
    q, table, pool = _decode_case(rng, lens, Hq, Hkv, d)
    Q, pd, td, ln = _dev(q), torch.from_numpy(pool).cuda(), torch.from_numpy(table).cuda(), _ints(lens)
    B, ld = len(lens), 1600
    ws = vs.workspace(vs.vs_kv4_decode_workspace_size(B, Hq, Hkv, d, 1500, True))
    acc0 = rng.uniform(0, 1, (B, Hkv, ld)).astype(np.float32)
    acc = torch.from_numpy(acc0).cuda()
    O, lse = torch.full_like(Q, 7.0), torch.full((Hq, B), 7.0, device="cuda")
    vs.vs_kv4_decode_attn_fwd(Q, pd, td, ln, 1500, O, lse, ws, window, sinks, acc_in=acc, acc_out=acc)
    assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)
    _check_decode(O, lse, q, pool, table, lens, window, sinks, acc.cpu().numpy().astype(np.float64), acc0)
    # without weights: the same bits
    O2, lse2 = vs.kv4_decode_attention(Q, pd, td, ln, 1500, window, sinks)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lens,Hq,Hkv,d,window", [([40001], 4, 1, 128, 0), ([9000, 3, 20000, 64], 2, 2, 64, 0),
                                                  ([30000] * 3, 16, 1, 128, 20000)])
def test_decode_split_rows(lens, Hq, Hkv, d, window, cuda_device):
    """Rows that many CTAs share, and the same bits every time."""
    rng = np.random.default_rng(len(lens) + d)
    q, table, pool = _decode_case(rng, lens, Hq, Hkv, d)
    Q, pd, td, ln = _dev(q), torch.from_numpy(pool).cuda(), torch.from_numpy(table).cuda(), _ints(lens)
    ws = vs.workspace(vs.vs_kv4_decode_workspace_size(len(lens), Hq, Hkv, d, max(lens), True))
    acc = torch.zeros((len(lens), Hkv, max(lens)), device="cuda")
    O, lse = torch.empty_like(Q), torch.empty((Hq, len(lens)), device="cuda")
    vs.vs_kv4_decode_attn_fwd(Q, pd, td, ln, max(lens), O, lse, ws, window, 5 if window else 0, acc_out=acc)
    assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)
    _check_decode(O, lse, q, pool, table, lens, window, 5, acc.cpu().numpy().astype(np.float64),
                  np.zeros(acc.shape, np.float32))
    for _ in range(3):
        O2, lse2, acc2 = torch.empty_like(O), torch.empty_like(lse), torch.zeros_like(acc)
        vs.vs_kv4_decode_attn_fwd(Q, pd, td, ln, max(lens), O2, lse2, ws, window, 5 if window else 0, acc_out=acc2)
        assert torch.equal(O, O2) and torch.equal(lse, lse2) and torch.equal(acc, acc2)


@pytest.mark.parametrize("Hq,d,weights", [(4, 128, False), (4, 128, True), (8, 128, False), (4, 64, False), (16, 128, False)])
def test_decode_same_bits_from_cold_and_warm_caches(Hq, d, weights, cuda_device):
    """Pages that come from memory arrive late and out of order; the result does not depend on it."""
    n = 60000
    gen = torch.Generator("cuda").manual_seed(Hq + d)
    pages = 4 * (n // 64 + 1)
    pool = torch.randint(0, 256, (pages, 2, d // 64 * 4608), dtype=torch.uint8, device="cuda", generator=gen)
    pool[..., d // 64 * 4096:].view(torch.bfloat16).copy_(
        torch.tensor([0.25, -2.0], device="cuda").repeat(d // 64 * 128))
    table = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32).view(4, -1)
    lens = _ints([n, n - 777, n // 2, n - 64])
    Q = torch.randn((4, Hq * 2, d), device="cuda", generator=gen).bfloat16()
    acc = torch.zeros((4, 2, n), device="cuda") if weights else None
    ws = vs.workspace(vs.vs_kv4_decode_workspace_size(4, Hq * 2, 2, d, n, weights))
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    first = None
    for i in range(60):
        O, lse = torch.empty_like(Q), torch.empty((Hq * 2, 4), device="cuda")
        if i % 4:
            flush.fill_(i)
        vs.vs_kv4_decode_attn_fwd(Q, pool, table, lens, n, O, lse, ws, acc_out=acc)
        now = [O, lse] + ([acc.clone()] if weights else [])
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(now, first)), i
    assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)


@pytest.mark.parametrize("Hq,window,sinks", [(131, 0, 0), (260, 150, 70), (130, 0, 0)])
def test_decode_weights_of_many_heads_per_kv_head(Hq, window, sinks, cuda_device):
    rng = np.random.default_rng(Hq)
    lens, Hkv, d = [1300, 1, 700], 2 if Hq == 260 else 1, 64
    q, table, pool = _decode_case(rng, lens, Hq, Hkv, d)
    Q, pd, td, ln = _dev(q), torch.from_numpy(pool).cuda(), torch.from_numpy(table).cuda(), _ints(lens)
    ws = vs.workspace(vs.vs_kv4_decode_workspace_size(3, Hq, Hkv, d, 1300, True))
    acc0 = rng.uniform(0, 1, (3, Hkv, 1301)).astype(np.float32)
    acc = torch.from_numpy(acc0).cuda()
    O, lse = torch.empty_like(Q), torch.empty((Hq, 3), device="cuda")
    vs.vs_kv4_decode_attn_fwd(Q, pd, td, ln, 1300, O, lse, ws, window, sinks, acc_in=acc, acc_out=acc)
    assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)
    # the weights' sums have Hq / Hkv terms, so their rounding is counted per unit of the sum
    w0 = acc.cpu().numpy().astype(np.float64) - acc0
    assert np.abs(w0.sum(-1) - Hq // Hkv).max() <= 4e-4 * Hq // Hkv + 1301 * 2.0 ** -20
    _check_decode(O, lse, q, pool, table, lens, window, sinks)
    c = ref.Cache(pool)
    for b, n in enumerate(lens):
        w = ref.decode(q[b], c, table[b], n, window, sinks)[2]
        # fp32 sums of up to 130 terms, then onto a sum of at most 131: half a unit in the last place each
        assert (np.abs(w0[b, :, :n] - w) <= (4e-4 + 131 * 2.0 ** -24) * w + 2.0 ** -16).all(), b


def test_tensors_of_another_device_are_refused(cuda_device):
    pool, table, lens = vs.kv4_pool(2, 1, 64), torch.zeros((1, 2), dtype=torch.int32, device="cuda"), _ints([3])
    Q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    ws = vs.workspace(vs.vs_kv4_decode_workspace_size(1, 2, 1, 64, 128))
    for bad in range(4):
        args = [x.cpu() if i == bad else x for i, x in enumerate((Q, pool, table, lens))]
        with pytest.raises(ValueError):
            vs.vs_kv4_decode_attn_fwd(*args, 128, torch.empty_like(Q), None, ws)
    K = Q[:, :1].contiguous()
    with pytest.raises(ValueError):
        vs.vs_kv4_append(K.cpu(), K.cpu(), _cu([1]), 1, pool, table, lens, ws)
    with pytest.raises(ValueError):
        vs.vs_window_attn_fwd(Q, K.cpu(), K.cpu(), 4, 1, torch.empty_like(Q), None, ws)


def test_decode_many_short_sequences(cuda_device):
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 130, 700)]
    q, table, pool = _decode_case(rng, lens, 2, 1, 64)
    O, lse = vs.kv4_decode_attention(_dev(q), torch.from_numpy(pool).cuda(), torch.from_numpy(table).cuda(),
                                     _ints(lens), 192)
    _check_decode(O, lse, q, pool, table, lens, 0, 0)


def test_decode_never_reads_what_is_not_in_use(cuda_device):
    """Slots behind the length hold NaN, infinities; pages out of sight are not in the pool at all."""
    rng = np.random.default_rng(9)
    lens, d = [70, 1000, 1], 128
    q, table, pool = _decode_case(rng, lens, 8, 2, d)
    args = _dev(q), torch.from_numpy(table).cuda(), _ints(lens)
    clean = vs.kv4_decode_attention(args[0], torch.from_numpy(pool).cuda(), args[1], args[2], 1000, 300, 10)
    dirty, t2 = pool.copy(), table.copy()
    words = dirty.view(np.uint32)
    for b, n in enumerate(lens):
        for t in range(n, -(-n // 64) * 64):
            pg = table[b, t // 64]
            for kv in range(2):
                for g in range(2):
                    words[pg, :, (2 * 2 * 2048 + (kv * 2 + g) * 256) // 4 + t % 64] = \
                        rng.choice([0x7FC07FC0, 0x7F807F80, 0xFF80FF80, 0xFFFFFFFF])
    t2[1, 1:(1000 - 300) // 64] = 1 << 30
    t2[:, -1] = -7
    ws = vs.workspace(vs.vs_kv4_decode_workspace_size(3, 8, 2, d, 1000, True))
    O, lse, acc = torch.empty_like(args[0]), torch.empty((8, 3), device="cuda"), torch.zeros((3, 2, 1000), device="cuda")
    vs.vs_kv4_decode_attn_fwd(args[0], torch.from_numpy(dirty).cuda(), torch.from_numpy(t2).cuda(), args[2], 1000, O,
                              lse, ws, 300, 10, acc_out=acc)
    assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)
    assert torch.equal(O, clean[0]) and torch.equal(lse, clean[1])
    assert torch.isfinite(acc).all() and abs(acc.sum().item() - 24) < 1e-3


def test_decode_nan_in_sight_reaches_its_heads_only(cuda_device):
    rng = np.random.default_rng(10)
    q, table, pool = _decode_case(rng, [200, 90], 4, 2, 64)
    pool.view(np.uint32)[table[0, 1], 1, (4096 + 0) // 4 + 5] = 0x7FC07FC0  # key pair of slot 69, head 1
    O, lse = vs.kv4_decode_attention(_dev(q), torch.from_numpy(pool).cuda(), torch.from_numpy(table).cuda(),
                                     _ints([200, 90]), 200)
    assert O[0, 2:].isnan().all() and lse[2:, 0].isnan().all()
    assert torch.isfinite(O[0, :2]).all() and torch.isfinite(O[1]).all() and torch.isfinite(lse[:, 1]).all()


def test_decode_bad_pages_and_lengths_are_flagged(cuda_device):
    rng = np.random.default_rng(11)
    lens = [300, 200, 100]
    q, table, pool = _decode_case(rng, lens, 4, 1, 128)
    Q, pd = _dev(q), torch.from_numpy(pool).cuda()
    bad = table.copy()
    bad[0, 2] = pool.shape[0]
    bad[0, 4] = -1
    ws = vs.workspace(vs.vs_kv4_decode_workspace_size(3, 4, 1, 128, 300, True))
    O, lse = torch.empty_like(Q), torch.empty((4, 3), device="cuda")
    acc = torch.zeros((3, 1, 300), device="cuda")
    # sequence 1 is longer than max_len says: it counts as empty
    vs.vs_kv4_decode_attn_fwd(Q, pd, torch.from_numpy(bad).cuda(), _ints([300, 301, 100]), 300, O, lse, ws, acc_out=acc)
    rc, flags = vs.vs_read_device_status(ws)
    assert rc == vs.VS_ERR_DEVICE_BOUNDS and flags == vs.VS_DEVFLAG_BOUNDS
    assert (O[1] == 0).all() and torch.isinf(lse[:, 1]).all()
    # sequence 0: the slots of the bad pages are invisible
    c = ref.Cache(pool)
    t = np.array([t for t in range(300) if t // 64 not in (2, 4)])
    k, v = c.rows(table[0], 0, t, 0), c.rows(table[0], 0, t, 1)
    z = q[0] @ k.T / np.sqrt(128)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    assert np.abs(dev_to_f64(O)[0] - p @ v).max() <= 2.0 ** -8 * (8 * c.s.max() + np.abs(v).max()) + 2e-3
    a = acc.cpu().numpy()
    assert (a[0, 0, 128:192] == 0).all() and (a[0, 0, 256:] == 0).all() and abs(a[0].sum() - 4) < 1e-3
    assert (a[1] == 0).all() and abs(a[2].sum() - 4) < 1e-3


def test_decode_scale_strides_and_offsets(cuda_device):
    rng = np.random.default_rng(12)
    lens = [129, 5]
    q, table, pool = _decode_case(rng, lens, 4, 2, 64)
    wide = torch.full((2, 7, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:6] = _dev(q)
    out = torch.full((2, 7, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((4, 2), device="cuda")
    big = torch.zeros((2, 9), dtype=torch.int32, device="cuda")
    big[:, 3:3 + table.shape[1]] = torch.from_numpy(table).cuda()
    ws = vs.workspace(vs.vs_kv4_decode_workspace_size(2, 4, 2, 64, 129))
    vs.vs_kv4_decode_attn_fwd(wide[:, 2:6], torch.from_numpy(pool).cuda(), big[:, 3:3 + table.shape[1]], _ints(lens),
                              129, out[:, 2:6], lse, ws, softmax_scale=0.3)
    assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)
    assert (out[:, :2] == 3).all() and (out[:, 6:] == 3).all()
    _check_decode(out[:, 2:6], lse, q, pool, table, lens, 0, 0, scale=0.3)


def test_decode_captured_follows_lengths(cuda_device):
    """One graph of append and decode, replayed while the lengths grow; on a stream of its own."""
    rng = np.random.default_rng(13)
    B, Hq, Hkv, d, top = 3, 4, 2, 64, 140
    table, pages = _table(rng, [top] * B)
    td, pd = torch.from_numpy(table).cuda(), torch.zeros((pages, Hkv, 4608), dtype=torch.uint8, device="cuda")
    lens, cu = _ints([62, 0, 100]), _cu([1] * B)
    K, V, Q = (torch.zeros((B, h, d), dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, Hq))
    O, lse = torch.empty_like(Q), torch.empty((Hq, B), device="cuda")
    ws, ws2 = vs.workspace(vs.vs_kv4_decode_workspace_size(B, Hq, Hkv, d, top)), vs.workspace(256)
    fill = torch.randn((100, Hkv, d), device="cuda").bfloat16()
    vs.vs_kv4_append(torch.cat([fill[:62], fill]), torch.cat([fill[:62], fill]), _cu([62, 0, 100]), 100, pd, td, lens, ws2)

    def step():
        lens.add_(1)
        vs.vs_kv4_append(K, V, cu, 1, pd, td, lens, ws2)
        vs.vs_kv4_decode_attn_fwd(Q, pd, td, lens, top, O, lse, ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lens.sub_(1)
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.synchronize()
    for i in range(5):
        k, v, q = (ref.bf16_round(rng.standard_normal(t.shape)) for t in (K, V, Q))
        for t, x in ((K, k), (V, v), (Q, q)):
            t.copy_(_dev(x))
        graph.replay()
        torch.cuda.synchronize()
        now = lens.tolist()
        assert now == [63 + i, 1 + i, 101 + i]
        _check_decode(O, lse, q, pd.cpu().numpy(), table, now, 0, 0)
    assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)


# ----------------------------------------------------------------------------------------- evict


def _evict(pool, table, lens, seen, acc, pos, keep, sinks, recent, ld_out=None):
    pd = torch.from_numpy(pool).cuda()
    B, Hkv, _ = acc.shape
    ld_out = ld_out or min(keep, acc.shape[2]) + 2
    ws = vs.workspace(vs.vs_kv4_evict_workspace_size(B, Hkv, acc.shape[2], keep))
    lo = torch.full((B,), -5, dtype=torch.int32, device="cuda")
    ao = torch.full((B, Hkv, ld_out), -9.0, device="cuda")
    po = torch.full((B, Hkv, ld_out), -9, dtype=torch.int32, device="cuda")
    vs.vs_kv4_evict(pd, torch.from_numpy(table).cuda(), _ints(lens), _ints(seen), acc.shape[2],
                    torch.from_numpy(acc).cuda(), torch.from_numpy(pos).cuda(), keep, sinks, recent, lo, ao, po, ws)
    return pd.cpu().numpy(), lo.tolist(), ao.cpu().numpy(), po.cpu().numpy(), vs.vs_read_device_status(ws)


def _check_evict(pool, table, lens, seen, acc, pos, keep, sinks, recent):
    got, lo, ao, po, status = _evict(pool, table, lens, seen, acc, pos, keep, sinks, recent)
    assert status == (vs.VS_OK, 0)
    want = pool.copy()
    g = pool.shape[2] // 4608
    spans = [(i * 2048, 32) for i in range(2 * g)] + [(4096 * g + i * 256, 4) for i in range(2 * g)]
    for b, n in enumerate(lens):
        k = min(n, keep)
        assert lo[b] == k
        for h in range(acc.shape[1]):
            src = ref.evict_order(acc[b, h, :n], pos[b, h, :n], seen[b], keep, sinks, recent)
            assert np.array_equal(po[b, h, :k], pos[b, h, src]), (b, h)
            assert np.array_equal(ao[b, h, :k], acc[b, h, src], equal_nan=True)
            assert (po[b, h, k:] == -9).all() and (ao[b, h, k:] == -9).all()
            dst = np.nonzero(src != np.arange(k))[0]
            for d, s in zip(dst, src[dst]):
                pd_, ps = table[b, d // 64], table[b, s // 64]
                for off, size in spans:
                    a, e = off + size * (d % 64), off + size * (s % 64)
                    want[pd_, h, a:a + size] = pool[ps, h, e:e + size]
    assert np.array_equal(got, want)


@pytest.mark.parametrize("lens,Hkv,d,keep,sinks,recent", [
    ([1], 1, 64, 1, 0, 1), ([100, 0, 64, 65], 2, 128, 64, 4, 20), ([500, 33], 1, 64, 1, 0, 0),
    ([5000, 4500], 2, 64, 4096, 4, 512), ([300], 3, 128, 299, 0, 0), ([20000, 70], 1, 64, 1000, 7, 100),
    ([40003], 1, 64, 39000, 0, 3), ([200, 150], 2, 64, 500, 1, 1), ([128], 1, 64, 5, 5, 0),
])
def test_evict_against_reference(lens, Hkv, d, keep, sinks, recent, cuda_device):
    rng = np.random.default_rng(sum(lens) + keep)
    table, pages = _table(rng, lens)
    pool = rng.integers(0, 256, (pages, Hkv, d // 64 * 4608), dtype=np.uint8)
    shape = (len(lens), Hkv, max(max(lens), 1))
    acc = np.exp(rng.standard_normal(shape) * 2).astype(np.float32)
    pos = np.cumsum(rng.integers(1, 3, shape), -1).astype(np.int32) - 1
    seen = [int(pos[b, :, max(n, 1) - 1].max()) + 1 for b, n in enumerate(lens)]
    _check_evict(pool, table, lens, seen, acc, pos, keep, sinks, recent)


def test_evict_ties_nan_infinities_and_any_order_of_positions(cuda_device):
    rng = np.random.default_rng(2)
    lens, Hkv = [700, 9000], 2
    table, pages = _table(rng, lens)
    pool = rng.integers(0, 256, (pages, Hkv, 4608), dtype=np.uint8)
    acc = rng.choice(np.array([0, -0.0, 1, 2, np.nan, np.inf, -np.inf, 1e-40, -3], np.float32), (2, Hkv, 9000))
    pos = np.stack([[rng.permutation(9000) for _ in range(Hkv)] for _ in range(2)]).astype(np.int32)
    for keep in (100, 350, 650):
        _check_evict(pool, table, lens, [9000, 9000], acc, pos, keep, 11, 30)
    acc[:] = 0  # all the same: the lowest slots stay
    _check_evict(pool, table, lens, [9000, 9000], acc, pos, 333, 0, 0)


def test_evict_flags_bad_lengths_and_pages(cuda_device):
    rng = np.random.default_rng(4)
    table, pages = _table(rng, [200, 200])
    pool = rng.integers(0, 256, (pages, 1, 4608), dtype=np.uint8)
    acc = rng.uniform(0, 1, (2, 1, 200)).astype(np.float32)
    pos = np.tile(np.arange(200, dtype=np.int32), (2, 1, 1))
    got, lo, ao, po, status = _evict(pool, table, [201, 200], [200, 200], acc, pos, 100, 0, 0)
    assert status[0] == vs.VS_ERR_DEVICE_BOUNDS and lo == [0, 100]
    assert (ao[0] == -9).all() and (po[1, 0, :100] >= 0).all()
    bad = table.copy()
    bad[1, 3] = 1 << 20  # slots 192.. cannot be moved; the lists are still as defined
    got, lo, ao, po, status = _evict(pool, bad, [200, 200], [200, 200], acc, pos, 100, 0, 8)
    assert status[0] == vs.VS_ERR_DEVICE_BOUNDS and lo == [100, 100]
    src = ref.evict_order(acc[1, 0], pos[1, 0], 200, 100, 0, 8)
    assert np.array_equal(po[1, 0, :100], src)


def test_pool_beyond_32_bit_offsets(cuda_device):
    """Pages behind the first 4 GiB of a pool: the same bytes and bits as in a small pool."""
    rng = np.random.default_rng(31)
    Hkv, d, n = 8, 128, 300
    far = (5 << 30) // (Hkv * 9216)
    big, small = vs.kv4_pool(far + 8, Hkv, d), vs.kv4_pool(8, Hkv, d)
    K, V, Q = (_dev(ref.bf16_round(rng.standard_normal((m, h, d)))) for m, h in ((n, Hkv), (n, Hkv), (1, 32)))
    acc = torch.rand((1, Hkv, n), device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda").expand(1, Hkv, n).contiguous()
    ws = vs.workspace(1 << 24)
    got = []
    for pool, first in ((big, far), (small, 0)):
        pool[first:].zero_()
        table = torch.arange(5, dtype=torch.int32, device="cuda").view(1, 5) + first
        vs.vs_kv4_append(K, V, _cu([n]), n, pool, table, _ints([n]), ws)
        O, lse = vs.kv4_decode_attention(Q, pool, table, _ints([n]), n)
        out = [_ints([0]), torch.zeros((1, Hkv, 100), device="cuda"),
               torch.zeros((1, Hkv, 100), dtype=torch.int32, device="cuda")]
        vs.vs_kv4_evict(pool, table, _ints([n]), _ints([n]), n, acc, pos, 100, 2, 9, *out, ws)
        Kr, Vr = torch.zeros((100, Hkv, d), dtype=torch.bfloat16, device="cuda"), torch.zeros((100, Hkv, d), dtype=torch.bfloat16, device="cuda")
        vs.vs_kv4_read(pool, table, out[0], None, _cu([100]), 100, Kr, Vr, ws)
        assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)
        got.append([O, lse, Kr, Vr, pool[first:].clone()] + out)
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_captured_weights_and_eviction_replay_like_eager_calls(cuda_device):
    """Decode with weights and evict (two kernels each) in one graph, replayed on a stream of its own while
    another stream runs the same calls with a workspace and a cache of its own."""
    rng = np.random.default_rng(33)
    lens, Hq, Hkv, d, keep = [900, 64, 3000], 8, 2, 64, 800
    B, top = len(lens), 3000
    q, table, pool0 = _decode_case(rng, lens, Hq, Hkv, d)
    Q, td, ln = _dev(q), torch.from_numpy(table).cuda(), _ints(lens)
    pos = torch.arange(top, dtype=torch.int32, device="cuda").expand(B, Hkv, top).contiguous()
    acc0 = torch.rand((B, Hkv, top), device="cuda")

    class Side:
        def __init__(self):
            self.pool, self.acc = torch.from_numpy(pool0).cuda(), torch.zeros_like(acc0)
            self.O, self.lse = torch.empty_like(Q), torch.empty((Hq, B), device="cuda")
            self.out = [torch.zeros_like(ln), torch.zeros((B, Hkv, keep), device="cuda"),
                        torch.zeros((B, Hkv, keep), dtype=torch.int32, device="cuda")]
            self.ws = vs.workspace(max(vs.vs_kv4_decode_workspace_size(B, Hq, Hkv, d, top, True),
                                       vs.vs_kv4_evict_workspace_size(B, Hkv, top, keep)))

        def step(self):
            vs.vs_kv4_decode_attn_fwd(Q, self.pool, td, ln, top, self.O, self.lse, self.ws, acc_in=acc0,
                                      acc_out=self.acc)
            vs.vs_kv4_evict(self.pool, td, ln, ln, top, self.acc, pos, keep, 4, 100, *self.out, self.ws)

        def results(self):
            return [self.O, self.lse, self.acc, self.pool] + self.out

    a, b, eager = Side(), Side(), Side()
    eager.pool.copy_(torch.from_numpy(pool0).cuda())
    eager.step()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s1):
            a.step()
    torch.cuda.synchronize()
    for _ in range(5):
        for side in (a, b):
            side.pool.copy_(torch.from_numpy(pool0).cuda())
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graph.replay()
        with torch.cuda.stream(s2):
            b.step()
        torch.cuda.synchronize()
        for side in (a, b):
            assert all(torch.equal(x, y) for x, y in zip(side.results(), eager.results()))
            assert vs.vs_read_device_status(side.ws) == (vs.VS_OK, 0)


# -------------------------------------------------------------------------------------- together


def test_prefill_cache_decode_evict_together(cuda_device):
    """Window prefill, column sums, append, eviction to a budget, then decode steps that accumulate
    weight, append and evict again -- every step against the reference on the state before it."""
    rng = np.random.default_rng(21)
    lens, Hq, Hkv, d, keep = [300, 150], 4, 2, 64, 128
    T, B, G = sum(lens), len(lens), Hq // Hkv
    Q, K, V = (_dev(ref.bf16_round(rng.standard_normal((T, h, d)))) for h in (Hq, Hkv, Hkv))
    cu = _cu(lens)
    ws = vs.workspace(1 << 24)
    O, lse = torch.empty_like(Q), torch.empty((Hq, T), device="cuda")
    vs.vs_window_attn_fwd_varlen(Q, K, V, cu, max(lens), 100, 4, O, lse, ws)
    A_v, _ = vs.aggregate_varlen(Q, K, V, cu, max(lens))
    table, pages = _table(rng, [512] * B)
    td, pool = torch.from_numpy(table).cuda(), vs.kv4_pool(pages, Hkv, d)
    pool.random_(0, 256)
    ld = 512
    acc = [torch.zeros((B, Hkv, ld), device="cuda") for _ in range(2)]
    pos = [torch.zeros((B, Hkv, ld), dtype=torch.int32, device="cuda") for _ in range(2)]
    ln, seen = [_ints(lens), _ints([0, 0])], _ints(lens)
    vs.vs_kv4_append(K, V, cu, max(lens), pool, td, ln[0], ws, n_tokens=seen, A_v=A_v, acc=acc[0], pos=pos[0])
    one = _cu([1] * B)

    def evict():
        before, n = pool.cpu().numpy(), ln[0].tolist()
        a, p = acc[0].cpu().numpy(), pos[0].cpu().numpy()
        vs.vs_kv4_evict(pool, td, ln[0], seen, ld, acc[0], pos[0], keep, 4, 16, ln[1], acc[1], pos[1], ws)
        for b in range(B):
            k = min(n[b], keep)
            cb, ca = ref.Cache(before), ref.Cache(pool.cpu().numpy())
            for h in range(Hkv):
                src = ref.evict_order(a[b, h, :n[b]], p[b, h, :n[b]], int(seen[b]), keep, 4, 16)
                assert np.array_equal(pos[1][b, h, :k].cpu().numpy(), p[b, h, src])
                for kv in range(2):
                    assert np.array_equal(ca.rows(table[b], h, np.arange(k), kv), cb.rows(table[b], h, src, kv))
        for x in (ln, acc, pos):
            x.reverse()

    evict()
    assert ln[0].tolist() == [128, 128]
    for step in range(4):
        q, k, v = (ref.bf16_round(rng.standard_normal((B, h, d))) for h in (Hq, Hkv, Hkv))
        ln[0].add_(1)
        seen.add_(1)
        vs.vs_kv4_append(_dev(k), _dev(v), one, 1, pool, td, ln[0], ws, n_tokens=seen, acc=acc[0], pos=pos[0])
        a0 = acc[0].cpu().numpy()
        o, l = torch.empty((B, Hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty((Hq, B), device="cuda")
        vs.vs_kv4_decode_attn_fwd(_dev(q), pool, td, ln[0], ld, o, l, ws, acc_in=acc[0], acc_out=acc[0])
        assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)
        _check_decode(o, l, q, pool.cpu().numpy(), table, ln[0].tolist(), 0, 0,
                      acc[0].cpu().numpy().astype(np.float64), a0)
        if step % 2:
            evict()
    assert ln[0].tolist() == [128, 128] and seen.tolist() == [304, 154]
