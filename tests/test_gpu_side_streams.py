"""Calls on a stream that is not the current one, with memory they allocate themselves: what the
current stream allocates, writes or still has to write meanwhile does not reach them."""
import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv
from nvfp4_block_scaled_17_b200 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, U8, I8 = torch.bfloat16, torch.float32, torch.uint8, torch.int8
M, N, K = 96, 768, 1024
HOLD = 20_000_000                      # cycles that a stream is kept busy: about 10 ms


@pytest.fixture(scope="module")
def calls():
    """name -> f(x, stream), everything else given and ready."""
    g = W._gen(1, DEV)
    w = W.normal((N, K), 0.05, g, DEV).to(BF16)
    wq, sw = nv.int8_quantize_rows(w)
    wp, wsf, gw = nv.pack_weight(w)
    weight = (1 + W.normal((K,), 0.2, g, DEV)).to(BF16)
    gsf = torch.tensor([100.0], device=DEV)
    residual = W.normal((M, K), 1.0, g, DEV).to(BF16)
    torch.cuda.synchronize()
    return {
        "int8_linear": lambda x, s: nv.int8_linear(x, wq, sw, stream=s),
        "nvfp4_linear": lambda x, s: nv.nvfp4_linear(x, wp, wsf, gw, N, stream=s),
        "nvfp4_linear_float_scale": lambda x, s: nv.nvfp4_linear(x, wp, wsf, gw, N, gsf_x=100.0, stream=s),
        "int8_linear_act": lambda x, s: nv.int8_linear_act(x, wq, sw, activation="gelu", stream=s),
        "nvfp4_linear_act": lambda x, s: nv.nvfp4_linear_act(x, wp, wsf, gw, N, activation="silu", stream=s),
        "nvfp4_quantize": lambda x, s: nv.nvfp4_quantize(x, 64, stream=s),
        "int8_rmsnorm_quantize": lambda x, s: nv.int8_rmsnorm_quantize(
            x, weight, 1e-6, residual=residual, stream=s),
        "nvfp4_rmsnorm_quantize": lambda x, s: nv.nvfp4_rmsnorm_quantize(
            x, weight, gsf, 1e-6, residual=residual, stream=s),
    }


NAMES = ["int8_linear", "nvfp4_linear", "nvfp4_linear_float_scale", "int8_linear_act",
         "nvfp4_linear_act", "nvfp4_quantize", "int8_rmsnorm_quantize", "nvfp4_rmsnorm_quantize"]


def parts(out):
    return [t.clone() for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def sizes():
    """Bytes of what the calls allocate."""
    return [nv.nvfp4_linear_workspace_bytes(M, K), int(nv.lib().int8_linear_workspace_bytes(M, K)),
            nv.nvfp4_quantize_workspace_bytes(), 2 * M * N, M * K // 2, M * K, 2 * M * K,
            nv.nvfp4_scale_bytes(M, K), 4 * M, 4]


def scribble():
    """On the current stream: blocks of these sizes, several of each, written and freed."""
    blocks = [torch.full((n,), 0xFF, dtype=U8, device=DEV) for n in sizes() for _ in range(4)]
    del blocks


def rows(seed):
    x = W.normal((M, K), 1.0, W._gen(seed, DEV), DEV).to(BF16)
    torch.cuda.synchronize()
    return x


@pytest.mark.parametrize("name", NAMES)
def test_allocations_behind_the_call(calls, name):
    """The current stream allocates and writes while the call still waits on its stream."""
    f, x, side = calls[name], rows(2), torch.cuda.Stream()
    want = parts(f(x, None))
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(HOLD)
        out = f(x, side)
        scribble()
        torch.cuda.synchronize()
        assert same(parts(out), want)
    assert nv.last_device_status() == nv.OK


@pytest.mark.parametrize("name", NAMES)
def test_writes_that_the_current_stream_still_has_to_make(calls, name):
    """Blocks that were freed while the current stream's writes to them are waiting."""
    f, x, side = calls[name], rows(3), torch.cuda.Stream()
    want = parts(f(x, None))
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(HOLD)
        scribble()
        out = f(x, side)
        torch.cuda.synchronize()
        assert same(parts(out), want)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_freed_while_the_current_stream_reads_them(calls, name):
    f, side = calls[name], torch.cuda.Stream()
    x, other = rows(4), rows(5)
    want = parts(f(x, None))
    torch.cuda.synchronize()
    for _ in range(3):
        out = f(x, side)
        side.synchronize()
        torch.cuda._sleep(HOLD)
        got = parts(out)                                 # copies that wait
        del out
        f(other, side)
        torch.cuda.synchronize()
        assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_a_branch_of_a_captured_graph(calls, name):
    """The stream joins a capture of the current one; outputs are used on the current stream."""
    f, side, x = calls[name], torch.cuda.Stream(), rows(6)
    inputs = [rows(7), rows(8)]
    wants = [parts(f(t, None)) for t in inputs]
    f(x, side)                                           # the stream's first call, outside
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        first = f(x, side)
        second = f(x, side)
        main.wait_stream(side)
        got = parts(first) + parts(second)
        del first, second
    for t, want in list(zip(inputs, wants)) * 2:
        x.copy_(t)
        scribble()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want + want)
