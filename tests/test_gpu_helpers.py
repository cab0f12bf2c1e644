"""The allocation helpers on the GPU: queries sliced out of a fused projection, calls on another stream."""
import functools

import pytest
import torch

import sparse_attention_long_head_b200 as vs

pytestmark = pytest.mark.gpu

N, HQ, HKV, D = 700, 8, 2, 64


def _fused(n):
    gen = torch.Generator("cuda").manual_seed(n)
    x = torch.randn((n, HQ + 2 * HKV, D), device="cuda", generator=gen).bfloat16()
    return x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]


@functools.cache  # kept: a call on another stream needs its inputs until it has run
def _ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@functools.cache
def _rows(n, step):
    idx = torch.arange(0, n, step, dtype=torch.int32, device="cuda").view(1, -1)
    return idx, _ints(idx.shape[1])


@functools.cache
def _cache():
    gen = torch.Generator("cuda").manual_seed(3)
    pool = torch.randint(0, 256, (40, HKV, 4608), dtype=torch.uint8, device="cuda", generator=gen)
    pool[..., 4096:].view(torch.bfloat16).copy_(torch.tensor([0.25, -2.0], device="cuda").repeat(128))
    table = torch.randperm(40, device="cuda", generator=gen).to(torch.int32).view(4, 10)
    return pool, table, _ints(640, 3, 100, 77)


HELPERS = {
    "window_attention": lambda Q, K, V, **kw: vs.window_attention(Q, K, V, 90, 4, **kw),
    "kv4_decode_attention": lambda Q, K, V, **kw: vs.kv4_decode_attention(Q[:4], *_cache(), 640, **kw),
    "dense_attention": lambda Q, K, V, **kw: vs.dense_attention(Q, K, V, **kw),
    "sparse_attention": lambda Q, K, V, **kw: vs.sparse_attention(Q, K, V, *_rows(N, 50), *_rows(N, 40), **kw),
    "block_prefill": lambda Q, K, V, **kw: vs.block_prefill(Q, K, V, 0.1, **kw),
    "block_prefill_varlen": lambda Q, K, V, **kw: vs.block_prefill_varlen(Q, K, V, _ints(0, 300, N), 400, 0.1, **kw),
    "aggregate": lambda Q, K, V, **kw: vs.aggregate(Q, K, V, **kw),
    "aggregate_varlen": lambda Q, K, V, **kw: vs.aggregate_varlen(Q, K, V, _ints(0, 300, N), 400, **kw),
}


def _close(name, a, b):
    if name.startswith("aggregate"):  # sums by atomics
        return torch.allclose(a, b, rtol=1e-4, atol=1e-4)
    return torch.equal(a, b)


@pytest.mark.parametrize("name", HELPERS)
def test_sliced_queries_give_what_packed_ones_give(name, cuda_device):
    Q, K, V = _fused(N)
    want = HELPERS[name](*(x.contiguous() for x in (Q, K, V)))
    got = HELPERS[name](Q, K, V)
    for a, b in zip(got, want):
        assert _close(name, a, b)


@pytest.mark.parametrize("name", HELPERS)
def test_calls_on_a_busy_stream_keep_their_memory(name, cuda_device):
    """The call waits on its own stream while the current one allocates and fills what is free there."""
    Q, K, V = _fused(N)
    want = HELPERS[name](Q, K, V)
    sizes = [256, 4096, 1 << 20, 2 << 20, 8 << 20] + [t.untyped_storage().nbytes() for t in want]
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # some 10 ms
        got = HELPERS[name](Q, K, V, stream=side)
        for n in 3 * sizes:
            torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(got, want):
            assert _close(name, a, b)
        del got
