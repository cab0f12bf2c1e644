"""The cache's host-side reference against small worked cases (no GPU)."""
import numpy as np

import vs_kv4_ref as ref


def test_quantize_known_groups():
    x = np.zeros((3, 64))
    x[0] = np.arange(64) % 16                      # 0..15: s = 1, m = 0, exact
    x[1] = -2.5                                    # constant
    x[2, 5] = np.inf
    n, s, m = ref.quantize(x)
    assert np.array_equal(n[0], np.arange(64) % 16) and s[0] == 1 and m[0] == 0
    assert (n[1] == 0).all() and s[1] == 0 and m[1] == -2.5
    assert np.isnan(s[2]) and np.isnan(m[2])


def test_ties_go_to_even_codes():
    x = np.zeros((1, 64))
    x[0, :6] = [15, 0.5, 1.5, 2.5, 13.5, 14.5]
    n, s, _ = ref.quantize(x)
    assert s[0] == 1 and list(n[0, :6]) == [15, 0, 2, 2, 14, 14]


def test_write_and_rows_agree():
    rng = np.random.default_rng(0)
    pool = np.full((3, 2, 2 * 4608), 0xAB, np.uint8)
    table = np.array([2, 0])
    x = ref.bf16_round(rng.standard_normal((70, 2, 2, 128)))  # slot, head, K/V
    for t in range(70):
        for h in range(2):
            for kv in range(2):
                n, s, m = ref.quantize(x[t, h, kv].reshape(2, 64))
                ref.pool_write(pool, table, h, t, kv, n, s, m)
    c = ref.Cache(pool)
    for h in range(2):
        for kv in range(2):
            got = c.rows(table, h, np.arange(70), kv)
            step = np.repeat(ref.quantize(x[:, h, kv].reshape(70, 2, 64))[1], 64, 1)
            # half a step, and at the top what 15 s falls short of the range (2^-9 of 15 steps)
            assert (np.abs(got - x[:, h, kv]) <= step * (0.5 + 15 * 2.0 ** -9)).all()


def test_evict_order_small():
    acc = np.array([5, 1, 9, 1, 7, 1, 3.0])
    pos = np.arange(7)
    # keep 4: sink 0, newest 6, then 9 (slot 2) and 7 (slot 4); slots 1 and 3 go
    assert list(ref.evict_order(acc, pos, 7, 4, 1, 1)) == [0, 4, 2, 6]
    assert list(ref.evict_order(acc, pos, 7, 9, 1, 1)) == list(range(7))
    # ties to the lower slot, NaN after -inf
    assert list(ref.evict_order(np.array([np.nan, -np.inf, 2, 2, 2]), pos[:5], 5, 2, 0, 0)) == [2, 3]
    assert list(ref.evict_order(np.array([np.nan, -np.inf, 2, 2, 2]), pos[:5], 5, 4, 0, 0)) == [4, 1, 2, 3]
