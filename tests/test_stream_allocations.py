"""A call that is given a stream allocates on that stream: its memory comes from what that stream
has freed and goes back to it, so no other stream's work touches it while the call runs.  On the
CPU, with the library, the allocator and the stream contexts replaced by records of their use."""
import contextlib

import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv

BF16, F32, U8, I8 = torch.bfloat16, torch.float32, torch.uint8, torch.int8


class FakeStream:
    cuda_stream = 77


class FakeLibrary:
    """Every entry point succeeds; the sizes are 4096 bytes."""

    def __getattr__(self, name):
        return lambda *args: 4096 if name.endswith("bytes") else 0


@pytest.fixture
def allocations(monkeypatch):
    """[(function, stream that was current)] of every allocation."""
    record, current = [], [None]

    @contextlib.contextmanager
    def on_stream(s):
        before, current[0] = current[0], s
        yield
        current[0] = before

    def wrap(name):
        real = getattr(torch, name)

        def call(*args, **kw):
            kw.pop("device", None)
            record.append((name, current[0]))
            return real(*args, **kw)
        monkeypatch.setattr(torch, name, call)

    for name in ("empty", "empty_like", "tensor", "zeros"):
        wrap(name)
    monkeypatch.setattr(torch.cuda, "stream", on_stream)
    monkeypatch.setattr(nv, "lib", FakeLibrary)
    monkeypatch.setattr(nv, "_calls", FakeLibrary)
    monkeypatch.setattr(nv, "_bf16_2d", lambda x, name: x)
    monkeypatch.setattr(nv, "_stream", lambda stream=None: 0 if stream is None else stream.cuda_stream)
    scalar = nv._scalar
    monkeypatch.setattr(nv, "_scalar", lambda t, *a, **kw:
                        t if isinstance(t, torch.Tensor) or t is None else scalar_of(scalar, t, *a, **kw))
    return record


def scalar_of(scalar, t, *a, **kw):
    try:
        return scalar(t, *a, **kw)
    except TypeError:                  # made, and refused for not being on a GPU
        return None


X = torch.zeros(4, 64, dtype=BF16)
P, SF, ONE = torch.zeros(4, 32, dtype=U8), torch.zeros(512, dtype=U8), torch.ones(1)
Q, S = torch.zeros(4, 64, dtype=I8), torch.ones(4)
CALLS = {
    "hadamard_rotate": lambda s: nv.hadamard_rotate(X, 16, stream=s),
    "nvfp4_quantize": lambda s: nv.nvfp4_quantize(X, stream=s),
    "nvfp4_quantize_static": lambda s: nv.nvfp4_quantize(X, 0, 3.0, stream=s),
    "pack_weight": lambda s: nv.pack_weight(X, 16, stream=s),
    "nvfp4_gemm": lambda s: nv.nvfp4_gemm(P, SF, P, SF, ONE, None, 4, 4, 64, stream=s),
    "nvfp4_gemm_float": lambda s: nv.nvfp4_gemm(P, SF, P, SF, 0.5, None, 4, 4, 64, stream=s),
    "nvfp4_debug_gemm_f32": lambda s: nv.nvfp4_debug_gemm_f32(P, SF, P, SF, ONE, None, 4, 4, 64, stream=s),
    "prepare_weight_scales": lambda s: nv.prepare_weight_scales(SF, 4, 64, stream=s),
    "nvfp4_gemm_prepared": lambda s: nv.nvfp4_gemm_prepared(P, SF, P, SF, ONE, None, 4, 4, 64, stream=s),
    "nvfp4_linear": lambda s: nv.nvfp4_linear(X, P, SF, ONE, 4, gsf_x=2.0, stream=s),
    "nvfp4_gemm_quantize_out": lambda s: nv.nvfp4_gemm_quantize_out(P, SF, P, SF, ONE, 4, 64, 64, 2.0, stream=s),
    "int8_quantize_rows": lambda s: nv.int8_quantize_rows(X, stream=s),
    "int8_gemm": lambda s: nv.int8_gemm(Q, S, Q, S, stream=s),
    "int8_linear": lambda s: nv.int8_linear(X, Q, S, stream=s),
    "int8_rmsnorm_quantize": lambda s: nv.int8_rmsnorm_quantize(X, None, 1e-6, residual=X, stream=s),
    "nvfp4_rmsnorm_quantize": lambda s: nv.nvfp4_rmsnorm_quantize(X, None, ONE, 1e-6, residual=X, stream=s),
    "nvfp4_gemm_act": lambda s: nv.nvfp4_gemm_act(P, SF, P, SF, ONE, None, 4, 4, 64, stream=s),
    "int8_gemm_act": lambda s: nv.int8_gemm_act(Q, S, Q, S, stream=s),
    "nvfp4_linear_act": lambda s: nv.nvfp4_linear_act(X, P, SF, ONE, 4, stream=s),
    "int8_linear_act": lambda s: nv.int8_linear_act(X, Q, S, stream=s),
    "nvfp4_dequantize": lambda s: nv.nvfp4_dequantize(P, SF, 2.0, 64, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_allocations_are_on_the_stream_given(allocations, name):
    side = FakeStream()
    CALLS[name](side)
    assert allocations                                   # each of these calls allocates
    assert [a for a in allocations if a[1] is not side] == []


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_no_context_is_entered(allocations, name):
    CALLS[name](None)
    assert allocations and all(s is None for _, s in allocations)
