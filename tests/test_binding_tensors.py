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
