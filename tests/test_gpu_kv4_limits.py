"""The cache's calls at the ends of what they accept: eviction of rows that one CTA, clusters of every size
and every key count take, decode at the ends of its numeric range, and the values of long rows."""
import numpy as np
import pytest
import torch

import sparse_attention_long_head_b200 as vs
import vs_kv4_ref as ref
from test_gpu_kv4 import _decode_case, _dev, _ints, _random_pool, _table
from vs_testutil import dev_to_f64

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------------------- evict


def _evict_sources(acc, pos, seen, keep, sinks, recent):
    """vs_kv4_ref.evict_order without a loop over the slots."""
    n = len(acc)
    k = min(n, keep)
    fixed = (pos < sinks) | (pos >= seen - recent)
    nan = np.isnan(acc)
    rank = np.where(fixed, 0, np.where(nan, 2, 1))
    value = np.where(fixed | nan, 0.0, -acc.astype(np.float64))
    stay = np.zeros(n, bool)
    stay[np.lexsort((np.arange(n), value, rank))[:k]] = True
    src = np.arange(k)
    src[~stay[:k]] = k + np.nonzero(stay[k:])[0]
    return src


# (rows, longest row): with 148 SMs, rows of up to 8192 slots take one CTA, longer ones clusters of
# 1 to 8 CTAs: as many as 16384 slots a CTA need, more while two clusters a row would not fill the device
@pytest.mark.parametrize("B,Hkv,top,keep", [
    (3, 1, 8192, 5000), (40, 2, 8193, 8000), (40, 2, 16384, 700), (24, 2, 9000, 8500), (24, 2, 30001, 12000),
    (24, 1, 9001, 4097), (24, 1, 20000, 19000), (20, 1, 65536, 3000), (1, 1, 32768, 9000), (2, 1, 131072, 60000),
    (1, 1, 131073, 100000), (1, 2, 200001, 8192), (1, 1, 262144, 261000),
])
def test_evict_rows_of_every_cluster_size(B, Hkv, top, keep, cuda_device):
    rng = np.random.default_rng(B * 1000 + top)
    lens = [top] + [int(x) for x in rng.integers(top // 2, top + 1, B - 1)]
    if B > 3:
        lens[1:4] = [0, 1, keep]
    table, pages = _table(rng, lens)
    pool = rng.integers(0, 256, (pages, Hkv, 4608), dtype=np.uint8)
    # few different weights: the boundary's ties lie in every part of a row
    acc = rng.choice(np.array([0, 0.5, 0.5, 1, 2, np.nan, -1], np.float32), (B, Hkv, top))
    pos = np.cumsum(rng.integers(1, 3, (B, Hkv, top)), -1).astype(np.int32) - 1
    seen = [int(pos[b, :, max(n, 1) - 1].max()) + 1 for b, n in enumerate(lens)]
    sinks, recent = 5, min(keep - 5, 300)
    pd, td, ad, od = (torch.from_numpy(x).cuda() for x in (pool, table, acc, pos))
    lo, ao = _ints([-5] * B), torch.full((B, Hkv, keep), -9.0, device="cuda")
    po = torch.full((B, Hkv, keep), -9, dtype=torch.int32, device="cuda")
    ws = vs.workspace(vs.vs_kv4_evict_workspace_size(B, Hkv, top, keep))
    vs.vs_kv4_evict(pd, td, _ints(lens), _ints(seen), top, ad, od, keep, sinks, recent, lo, ao, po, ws)
    assert vs.vs_read_device_status(ws) == (vs.VS_OK, 0)
    assert lo.tolist() == [min(n, keep) for n in lens]
    ao, po = ao.cpu().numpy(), po.cpu().numpy()
    want = pool.copy()
    views = [(x[..., :4096].reshape(pages, Hkv, 2, 64, 32), x[..., 4096:].reshape(pages, Hkv, 2, 64, 4))
             for x in (want, pool)]
    codes, pairs = (np.zeros_like(v) for v in views[1])
    codes[:], pairs[:] = views[1]
    for b, n in enumerate(lens):
        k = min(n, keep)
        for h in range(Hkv):
            src = _evict_sources(acc[b, h, :n], pos[b, h, :n], seen[b], keep, sinks, recent)
            assert np.array_equal(po[b, h, :k], pos[b, h, src]), (b, h)
            assert np.array_equal(ao[b, h, :k], acc[b, h, src], equal_nan=True), (b, h)
            assert (po[b, h, k:] == -9).all() and (ao[b, h, k:] == -9).all()
            dst = np.nonzero(src != np.arange(k))[0]
            src = src[dst]
            codes[table[b, dst // 64], h, :, dst % 64] = views[1][0][table[b, src // 64], h, :, src % 64]
            pairs[table[b, dst // 64], h, :, dst % 64] = views[1][1][table[b, src // 64], h, :, src % 64]
    got = pd.cpu().numpy()
    assert np.array_equal(got[..., :4096].reshape(codes.shape), codes)
    assert np.array_equal(got[..., 4096:].reshape(pairs.shape), pairs)


# ---------------------------------------------------------------------------------------- decode


def _set_pairs(pool, kv, change):
    """Replaces the (s, m) pairs of keys (kv 0) or values (1) by change(s, m), in float64."""
    g = pool.shape[2] // 4608
    raw = pool[..., g * 4096:].reshape(*pool.shape[:2], 2, g, 64, 4)
    bits = np.ascontiguousarray(raw[:, :, kv]).view(np.uint16).astype(np.uint32) << 16
    val = bits.view(np.float32).astype(np.float64)
    pair = np.stack(change(val[..., 0], val[..., 1]), -1)
    raw[:, :, kv] = ref.bf16_bits(ref.bf16_round(pair)).view(np.uint8).reshape(raw[:, :, kv].shape)


@pytest.mark.parametrize("Hq,d", [(4, 128), (3, 64), (8, 64), (16, 128)])
@pytest.mark.parametrize("v_exp", [-40, 0, 40])
@pytest.mark.parametrize("q", ["one", "small", "zero", "large", "apart", "constant keys"])
def test_decode_at_the_ends_of_its_range(Hq, d, v_exp, q, cuda_device):
    """Q from 0 to 2^113 (keys scaled back, by exact powers of two, so that the scores stay as they are),
    heads 2^60 apart, constant groups (s = 0), value steps of 2^-40 and up to 2^40.

    Bounds: the weights' and the output's roundings, as in test_gpu_kv4: 2^-8 (8 max s + max |v|) and
    4e-4 max |v| for the scores.  At steps of 2^-40 a product of a weight and a code is a multiple of
    2^-149, where the heaviest slot's is 2^-125: 2^-24 of s for each of 700 slots, in the 4e-4."""
    rng = np.random.default_rng(Hq + d + v_exp + len(q))
    lens = [1, 70, 700]
    qv, table, pool = _decode_case(rng, lens, Hq, 1, d)
    raw = pool[..., d // 64 * 4096:].reshape(len(pool), 1, 2, d // 64, 64, 4)
    flat = rng.random(raw.shape[:-1]) < 0.3  # a third of the groups, keys and values

    def scaled(e, kv):
        def change(s, m):
            if kv:  # values: steps of [1/4, 1], or of [1/2, 1] at the lower end
                s, m = s / s.max(), m / s.max()
                s = np.maximum(s, 0.5) if v_exp < 0 else s
            s = np.where(flat[:, :, kv], 0.0, s) if kv or q == "constant keys" else s
            return s * 2.0 ** e, m * 2.0 ** e
        return change

    # the largest step is 2^40, the smallest 2^-40
    _set_pairs(pool, 1, scaled(v_exp + (1 if v_exp < 0 else 0), 1))
    k_exp = 0
    if q == "small":
        qv *= 2.0 ** -30
    elif q == "zero":
        qv[:] = 0
    elif q == "large":  # up to 1.95 2^112, and the keys 2^-111 of what they were
        qv = ref.bf16_round(np.clip(qv, -3.9, 3.9)) * 2.0 ** 111
        k_exp = -111
    elif q == "apart":
        qv[:, ::2] *= 2.0 ** -60
    _set_pairs(pool, 0, scaled(k_exp, 0))
    O, lse = vs.kv4_decode_attention(_dev(qv), torch.from_numpy(pool).cuda(), torch.from_numpy(table).cuda(),
                                     _ints(lens), 700)
    O, lse = dev_to_f64(O), lse.cpu().numpy().astype(np.float64)
    c = ref.Cache(pool)
    for b, n in enumerate(lens):
        Or, lr, _ = ref.decode(qv[b], c, table[b], n)
        t = np.arange(n)
        smax = c.s[table[b][t // 64], 0, 1, :, t % 64].max()
        vmax = np.abs(c.rows(table[b], 0, t, 1)).max()
        tol = 2.0 ** -8 * (8 * smax + vmax) + 4e-4 * vmax
        assert np.abs(O[b] - Or).max() <= tol, (b, np.abs(O[b] - Or).max(), tol)
        assert np.abs(lse[:, b] - lr).max() <= 4e-4, (b, n)


@pytest.mark.parametrize("lens,Hq,Hkv,d,window", [([40001], 4, 1, 128, 0), ([20000, 9000], 8, 1, 64, 0),
                                                  ([30000] * 2, 16, 1, 128, 20000), ([50000], 2, 2, 64, 0)])
def test_values_of_long_rows(lens, Hq, Hkv, d, window, cuda_device):
    """Over many slots the values average out (O of 0.02 here), far below the largest value that bounds the
    single slot's error, so the error is held to what the roundings of n weights w leave on average.  The
    rounding of p s to bf16 is off by up to 2^-8 w s |n - 8| in slot t, the fp32 score by up to 4e-4 w |v|,
    with signs that do not follow the slots: the rms over the channels is at most the root of the sum of
    squares.  O's own rounding adds 2^-8 of O, the fp32 sums less than 2^-20 max |v|."""
    rng = np.random.default_rng(len(lens) * 7 + d)
    q, table, pool = _decode_case(rng, lens, Hq, Hkv, d)
    sinks = 5 if window else 0
    O, _ = vs.kv4_decode_attention(_dev(q), torch.from_numpy(pool).cuda(), torch.from_numpy(table).cuda(), _ints(lens),
                                   max(lens), window, sinks)
    O, c = dev_to_f64(O), ref.Cache(pool)
    rms = lambda x: np.sqrt((x ** 2).mean())  # noqa: E731
    for b, n in enumerate(lens):
        Or, lr, _ = ref.decode(q[b], c, table[b], n, window, sinks)
        t = ref.visible(n, window, sinks)
        pg, r = table[b][t // 64], t % 64
        for h in range(Hq):
            g = h // (Hq // Hkv)
            k, v = (c.rows(table[b], g, t, kv) for kv in (0, 1))
            w = np.exp(k @ q[b, h] * d ** -0.5 - lr[h])
            code = (c.s[pg, g, 1, :, r][..., None] * (c.codes[pg, g, 1, :, r].astype(np.float64) - 8)).reshape(len(t), d)
            slot = (2.0 ** -8 * code) ** 2 + (4e-4 * v) ** 2
            bound = np.sqrt((w ** 2 @ slot).mean()) + 2.0 ** -8 * rms(Or[h]) + 2.0 ** -20 * np.abs(v).max()
            assert bound <= 0.1 * rms(Or[h])  # the bound sees an error of a tenth of O
            assert rms(O[b, h] - Or[h]) <= bound, (b, h, rms(O[b, h] - Or[h]), bound)
