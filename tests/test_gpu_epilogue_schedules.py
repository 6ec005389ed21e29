"""The products with an epilogue on each of their four schedules, for both kinds of operands: odd
widths, residuals in place, rows behind the last, tails, streams, and weights written just
before the call.  Which kernel a shape runs is looked up, not assumed."""
import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv
from nvfp4_block_scaled_17_b200 import workloads as W
import plain_ops as P
from test_gpu_epilogue import extras, one, operands, product, run

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16

# schedule -> its kernel, and shapes (M, N, K) that run on it: the first even, the others odd
KERNELS = {"stream": "gemm_stream_kernel", "cluster": "gemm_small_kernel", "split_k": "gemm_kernel",
           "pair": "gemm_pair_kernel"}
SHAPES = {"stream": [(1, 19456, 512), (3, 19203, 192), (20, 25601, 64), (50, 19459, 5184)],
          "cluster": [(4, 1024, 2048), (3, 519, 192), (31, 2049, 64), (32, 513, 4160)],
          "split_k": [(100, 520, 2624), (33, 519, 2624), (130, 517, 5184), (64, 1031, 5120)],
          "pair": [(300, 520, 576), (300, 519, 192), (129, 2061, 64), (2500, 1033, 192)]}
ALL = [(s, *shape) for s, shapes in SHAPES.items() for shape in shapes]
EVEN = [(s, *shapes[0]) for s, shapes in SHAPES.items()]
KINDS = ["int8", "nvfp4"]


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("schedule", KERNELS)
def test_the_shapes_run_on_their_schedule(kind, schedule):
    from torch.profiler import ProfilerActivity, profile
    for M, N, K in SHAPES[schedule]:
        ops = operands(kind, M, N, K)
        torch.cuda.synchronize()
        with profile(activities=[ProfilerActivity.CUDA]) as prof:
            run(kind, ops, M, N, K, None, "gelu", False, None)
            torch.cuda.synchronize()
        names = [e.key for e in prof.key_averages() if "gemm" in e.key]
        if not names:
            pytest.skip("no kernel records here")
        assert len(names) == 1 and f"::{KERNELS[schedule]}<" in names[0], (M, N, K, names)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("schedule,M,N,K", ALL)
def test_odd_widths(kind, schedule, M, N, K):
    one(kind, M, N, K, "silu", False, True, True)
    one(kind, M, N, K, "gelu", False, False, True, prepared=True)
    one(kind, M, N, K, "none", False, True, False, seed=2)
    gated = N // 2 * 2
    one(kind, M, gated, K, "gelu_tanh", True, True, True)
    one(kind, M, gated, K, "relu", True, False, True, prepared=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("schedule,M,N,K", ALL)
@pytest.mark.parametrize("gated", [False, True])
def test_in_place_and_what_stands_around(kind, schedule, M, N, K, gated):
    """The residual is the output; values before it and behind its last row stay."""
    N = N // 2 * 2 if gated else N
    cols = N // 2 if gated else N
    ops = operands(kind, M, N, K)
    bias, res = extras(M, N, gated, True, True)
    want = run(kind, ops, M, N, K, bias, "silu", gated, res)
    pad = 256
    whole = torch.full((pad + M * cols + pad,), 7.0, dtype=BF16, device=DEV)
    live = whole[pad:pad + M * cols].view(M, cols)
    for prepared in (False, True):
        live.copy_(res)
        got = run(kind, ops, M, N, K, bias, "silu", gated, live, prepared, out=live)
        torch.cuda.synchronize()
        assert got is live and nv.last_device_status() == nv.OK
        assert same(live, want)
        assert (whole[:pad] == 7.0).all() and (whole[pad + M * cols:] == 7.0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("schedule,M,N,K", EVEN)
def test_large_values(kind, schedule, M, N, K):
    ops = operands(kind, M, N, K)
    big = torch.linspace(-300.0, 300.0, N, device=DEV).to(BF16)
    v, dv = product(kind, ops, M, N, K, big)
    for act in P.ACTS:
        for gated in (False, True):
            y = run(kind, ops, M, N, K, big, act, gated, None)
            P.check(y, *P.epilogue_64(v, dv, act, gated, None), f"{kind} {schedule} {act} {gated}")


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_at_once(kind):
    jobs = []
    for _, M, N, K in ALL:
        ops = operands(kind, M, N, K)
        b, r = extras(M, N, False, True, True)
        want = run(kind, ops, M, N, K, b, "silu", False, r)
        jobs.append((ops, M, N, K, b, r, want, [torch.empty_like(want) for _ in range(2)]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for ops, M, N, K, b, r, _, outs in jobs:
            for s, out in zip(streams, outs):
                run(kind, ops, M, N, K, b, "silu", False, r, out=out, stream=s)
    torch.cuda.synchronize()
    assert nv.last_device_status() == nv.OK
    assert all(same(out, want) for *_, want, outs in jobs for out in outs)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("schedule,M,N,K", EVEN)
@pytest.mark.parametrize("prepared", [False, True])
def test_linear_weights_written_just_before(kind, schedule, M, N, K, prepared):
    """The linears load the first stages of their weight before the quantizer has ended."""
    if prepared and kind == "int8":
        pytest.skip("int8 weights have no prepared form")
    g = W._gen(M + N, DEV)
    x = W.normal((M, K), 1.0, g, DEV).to(BF16)
    ws = [W.normal((N, K), 0.05, g, DEV).to(BF16) for _ in range(3)]
    packs = [nv.int8_quantize_rows(w) if kind == "int8" else nv.pack_weight(w) for w in ws]
    if prepared:
        packs = [(p, nv.prepare_weight_scales(sf, N, K), s) for p, sf, s in packs]

    def call(w, **kw):
        if kind == "int8":
            return nv.int8_linear_act(x, *w, activation="gelu", **kw)
        return nv.nvfp4_linear_act(x, *w, N, activation="gelu", prepared=prepared, **kw)

    live = tuple(t.clone() for t in packs[0])
    want = [call(w) for w in packs]
    torch.cuda.synchronize()
    for _ in range(3):
        for k in (1, 2, 0):
            for t, s in zip(live, packs[k]):
                t.copy_(s)
            y = call(live)
            torch.cuda.synchronize()
            assert same(y, want[k])
