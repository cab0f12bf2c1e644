"""What the window and cache calls check of their tensors before the library is reached.  The library is
replaced, so no test here launches anything: a call that passes every check ends in Reached."""
import pytest
import torch

import sparse_attention_long_head_b200 as vs

B, HQ, HKV, D, T, N = 2, 4, 2, 64, 5, 256


class Reached(Exception):
    pass


class _Library:
    def __getattr__(self, name):
        def call(*args):
            raise Reached(name)
        return call


class _OnDevice(torch.Tensor):
    """A CPU tensor that says it is on device 0."""

    def get_device(self):
        return 0


@pytest.fixture
def no_library(monkeypatch):
    monkeypatch.setattr(vs, "lib", lambda: _Library())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(vs, "_raw_stream", lambda device: 0)


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _cache():
    return dict(pool=torch.zeros((3, HKV, 4608), dtype=torch.uint8), table=_ints(B, 4), lens=_ints(B))


def _bytes():
    return torch.zeros(1 << 12, dtype=torch.uint8)


def _window_args():
    return dict(Q=_bf16(T, HQ, D), K=_bf16(T, HKV, D), V=_bf16(T, HKV, D), O=_bf16(T, HQ, D),
                lse=torch.zeros((HQ, T)), ws=_bytes())


CALLS = {
    "window": (lambda **a: vs.vs_window_attn_fwd(window=3, sinks=1, **a), _window_args),
    "window, packed": (lambda **a: vs.vs_window_attn_fwd_varlen(max_seqlen=3, window=3, sinks=1, **a),
                       lambda: dict(cu_seqlens=_ints(B + 1), **_window_args())),
    "append": (lambda **a: vs.vs_kv4_append(max_new=3, **a),
               lambda: dict(K=_bf16(T, HKV, D), V=_bf16(T, HKV, D), cu_seqlens=_ints(B + 1), ws=_bytes(),
                            n_tokens=_ints(B), A_v=torch.zeros((HQ, T)), acc=torch.zeros((B, HKV, N)),
                            pos=_ints(B, HKV, N), **_cache())),
    "read": (lambda **a: vs.vs_kv4_read(max_read=3, **a),
             lambda: dict(start=_ints(B), cu_seqlens=_ints(B + 1), K=_bf16(T, HKV, D), V=_bf16(T, HKV, D),
                          ws=_bytes(), **_cache())),
    "decode": (lambda **a: vs.vs_kv4_decode_attn_fwd(max_len=N, **a),
               lambda: dict(Q=_bf16(B, HQ, D), O=_bf16(B, HQ, D), lse=torch.zeros((HQ, B)), ws=_bytes(),
                            acc_in=torch.zeros((B, HKV, N)), acc_out=torch.zeros((B, HKV, N)), **_cache())),
    "evict": (lambda **a: vs.vs_kv4_evict(max_len=N, keep=9, sinks=1, recent=2, **a),
              lambda: dict(n_tokens=_ints(B), acc=torch.zeros((B, HKV, N)), pos=_ints(B, HKV, N), lens_out=_ints(B),
                           acc_out=torch.zeros((B, HKV, 9)), pos_out=_ints(B, HKV, 9), ws=_bytes(), **_cache())),
}
TENSORS = [(name, key) for name, (_, make) in CALLS.items() for key in make()]


@pytest.mark.parametrize("name,elsewhere", TENSORS, ids=[f"{a}-{b}" for a, b in TENSORS])
def test_every_tensor_must_be_on_the_current_device(name, elsewhere, no_library):
    call, make = CALLS[name]
    here = {k: t.as_subclass(_OnDevice) for k, t in make().items()}
    with pytest.raises(Reached):
        call(**here)
    with pytest.raises(ValueError, match="current device"):
        call(**here | {elsewhere: make()[elsewhere]})


@pytest.mark.parametrize("name", ["window", "window, packed"])
@pytest.mark.parametrize("other", ["K", "V", "O", "KV"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32, torch.uint8])
def test_window_tensors_are_of_one_type(name, other, dtype, no_library):
    """Keys of another type would be read as the queries' (bytes: out of their range)."""
    call, make = CALLS[name]
    args = {k: t.as_subclass(_OnDevice) for k, t in make().items()}
    with pytest.raises(Reached):
        call(**args)
    with pytest.raises(AssertionError):
        call(**args | {k: args[k].to(dtype) for k in other})


# ------------------------------------------------------------------------------ allocation helpers


class _Accepting:
    """A library whose calls succeed without doing anything."""

    def __getattr__(self, name):
        return lambda *args: 4096 if name.endswith(("_size", "_size_ld", "_size_varlen")) else 0


@pytest.fixture
def accepting_library(monkeypatch):
    monkeypatch.setattr(vs, "lib", lambda: _Accepting())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # what CPU tensors report
    monkeypatch.setattr(vs, "_raw_stream", lambda device: 0)


def _index():
    return _ints(1, 8), _ints(1), _ints(1, 8), _ints(1)


HELPERS = {
    "window_attention": lambda Q, K, V, **kw: vs.window_attention(Q, K, V, 3, 1, **kw),
    "kv4_decode_attention": lambda Q, K, V, **kw: vs.kv4_decode_attention(
        Q, torch.zeros((3, HKV, 4608), dtype=torch.uint8), _ints(T, 4), _ints(T), N, **kw),
    "dense_attention": lambda Q, K, V, **kw: vs.dense_attention(Q, K, V, **kw),
    "sparse_attention": lambda Q, K, V, **kw: vs.sparse_attention(Q, K, V, *_index(), **kw),
    "block_prefill": lambda Q, K, V, **kw: vs.block_prefill(Q, K, V, 0.1, **kw),
    "block_prefill_varlen": lambda Q, K, V, **kw: vs.block_prefill_varlen(Q, K, V, _ints(B + 1), T, 0.1, **kw),
    "aggregate": lambda Q, K, V, **kw: vs.aggregate(Q, K, V, **kw),
    "aggregate_varlen": lambda Q, K, V, **kw: vs.aggregate_varlen(Q, K, V, _ints(B + 1), T, **kw),
}


@pytest.mark.parametrize("name", HELPERS)
def test_helpers_give_the_output_the_rows_of_a_sliced_query(name, accepting_library, monkeypatch):
    """Q as a slice of a fused projection: the calls have one row stride for Q and O, so an O with packed
    rows would be refused, or written behind its end."""
    fused = _bf16(T, HQ + 2 * HKV, D)
    Q, K, V = fused[:, :HQ], fused[:, HQ:HQ + HKV], fused[:, HQ + HKV:]
    outputs = []
    for call in ("vs_dense_attn_fwd", "vs_dense_attn_fwd_varlen"):
        def fwd(*args, _call=getattr(vs, call), **kw):
            outputs.append(args[3 if _call.__name__ == "vs_dense_attn_fwd" else 5])
            return _call(*args, **kw)
        monkeypatch.setattr(vs, call, fwd)
    out = HELPERS[name](Q, K, V)
    for O in outputs or out[:1]:
        assert O.shape == Q.shape and O.stride() == Q.stride() and O.dtype is Q.dtype


@pytest.mark.parametrize("name,positional", [(n, False) for n in (*HELPERS, "select", "select_varlen")] +
                         [("window_attention", True), ("select", True)])
def test_helpers_allocate_on_the_stream_of_the_call(name, positional, accepting_library, monkeypatch):
    """What a helper allocates for another stream's call comes from that stream's memory: the current
    stream's may still be written by its earlier kernels, and is handed out again when the helper
    returns, before the other stream has run."""
    current, side = object(), type("Stream", (), {"cuda_stream": 77, "device_index": -1})()
    state = {"now": current}
    allocated, recorded = [], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            self.before, state["now"] = state["now"], self.stream

        def __exit__(self, *exc):
            state["now"] = self.before

    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *device: state["now"])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    for alloc in ("empty", "empty_strided", "full"):
        def make(*args, _make=getattr(torch, alloc), **kw):
            allocated.append(state["now"])
            return _make(*args, **kw)
        monkeypatch.setattr(torch, alloc, make)
    q, k = torch.zeros((T, HQ, D), dtype=torch.bfloat16), torch.zeros((T, HKV, D), dtype=torch.bfloat16)
    scores = torch.zeros((HQ, T))
    select = {"select": lambda **kw: vs.select(scores, 0, 3, **kw),
              "select_varlen": lambda **kw: vs.select_varlen(scores, _ints(B + 1), T, 0, _ints(B), 3, **kw)}
    if positional:
        run = {"window_attention": lambda: vs.window_attention(q, k, k, 3, 1, None, True, side),
               "select": lambda: vs.select(scores, 0, 3, 1.0, None, side)}[name]
    else:
        run = (lambda: select[name](stream=side)) if name in select else lambda: HELPERS[name](q, k, k, stream=side)
    out = run()
    assert allocated and all(s is side for s in allocated)
    # the caller's stream reads the results, so their memory waits for it too
    assert {p for p, s in recorded if s is current} >= {t.data_ptr() for t in out}
    assert state["now"] is current
    del allocated[:], recorded[:]
    if not positional:
        select[name]() if name in select else HELPERS[name](q, k, k)
        assert allocated and all(s is current for s in allocated) and not recorded


@pytest.mark.parametrize("name", HELPERS)
def test_helpers_refuse_a_stream_of_another_device(name, accepting_library, monkeypatch):
    """Taking over the stream's device would run kernels there on this device's tensors."""
    elsewhere = type("Stream", (), {"cuda_stream": 77, "device_index": 1})()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *device: object())
    monkeypatch.setattr(torch.cuda, "stream", lambda s: pytest.fail("the stream was entered"))
    with pytest.raises(ValueError, match="current device"):
        HELPERS[name](_bf16(T, HQ, D), _bf16(T, HKV, D), _bf16(T, HKV, D), stream=elsewhere)


def test_rows_of_one_kv_head_may_be_slices_of_longer_ones():
    """Of a size of 1 the stride says nothing: the row length is that of the other dimension."""
    wide = torch.zeros((3, 40))
    one_head, one_sequence = wide[:, :30].unsqueeze(1), wide[:, :30].unsqueeze(0)
    assert vs._kv4_rows(one_head, torch.float32, 3, 1, 30) == 40
    assert vs._kv4_rows(one_sequence, torch.float32, 1, 3, 30) == 40
    assert vs._kv4_rows(wide[:1, :30].unsqueeze(0), torch.float32, 1, 1, 30) == 30
    assert vs._kv4_rows(torch.zeros((3, 2, 40))[..., :30], torch.float32, 3, 2, 30) == 40
    for bad in (wide[:, :30].t()[:3].unsqueeze(1),                   # entries of a row apart
                wide[:1].expand(3, 40)[:, :30].unsqueeze(1),         # rows that are one row
                torch.zeros((3, 5, 40))[:, ::2, :30]):               # heads and sequences of different steps
        with pytest.raises(AssertionError):
            vs._kv4_rows(bad, torch.float32, *bad.shape[:2], bad.shape[2])
    assert vs._kv4_rows(torch.zeros((3, 4, 40))[:, :1, :30], torch.float32, 3, 1, 30) == 160
