"""nvfp4_gemm_act, int8_gemm_act and their linears on the GPU against 64-bit forms of the
same product and epilogue (tests/plain_ops.py derives the bounds), over every schedule of
the GEMMs, odd sizes, in-place residuals, streams and graphs."""
import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv
from nvfp4_block_scaled_17_b200 import workloads as W
import plain_ops as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16

# M, N, K: the swapped-operand kernel (M <= 32), split-K, persistent tiles, a full wave with
# a split tail, widths that no wide store takes
FP4_SHAPES = [(1, 256, 64), (1, 5120, 5120), (7, 1030, 576), (32, 514, 1024), (33, 250, 64),
              (100, 520, 2048), (300, 520, 576), (128, 256, 256), (2500, 2064, 192),
              (1024, 5120, 5120), (257, 10, 128)]
INT8_SHAPES = [(1, 256, 32), (1, 5120, 5120), (7, 1030, 608), (32, 514, 1024), (33, 250, 32),
               (100, 520, 2048), (300, 520, 544), (128, 256, 256), (2500, 2064, 96),
               (1024, 5120, 5120), (257, 10, 160)]


def operands(kind, M, N, K, seed=0):
    g = W._gen(seed + M + 3 * N + 7 * K, DEV)
    x = W.with_outliers((M, K), 0.01, 20.0, g, DEV)
    w = W.normal((N, K), 1.5 * K ** -0.5, g, DEV).to(BF16)
    if kind == "int8":
        return nv.int8_quantize_rows(x) + nv.int8_quantize_rows(w)
    a, sfa, ga = nv.nvfp4_quantize(x)
    b, sfb, gb = nv.pack_weight(w)
    return a, sfa, b, sfb, 1.0 / (ga * gb)


def extras(M, N, gated, bias, residual, seed=0):
    g = W._gen(seed + M + N, DEV)
    b = W.normal((N,), 0.5, g, DEV).to(BF16) if bias else None
    r = W.normal((M, N // 2 if gated else N), 2.0, g, DEV).to(BF16) if residual else None
    return b, r


def run(kind, ops, M, N, K, bias, act, gated, residual, prepared=False, **kw):
    if kind == "int8":
        a, sa, b, sb = ops
        return nv.int8_gemm_act(a, sa[:M], b, sb[:N], bias, act, gated, residual, **kw)
    a, sfa, b, sfb, alpha = ops
    if prepared:
        sfb = nv.prepare_weight_scales(sfb, N, K)
    return nv.nvfp4_gemm_act(a, sfa, b, sfb, alpha, bias, M, N, K, act, gated, residual, prepared,
                             **kw)


def product(kind, ops, M, N, K, bias):
    if kind == "int8":
        a, sa, b, sb = ops
        return P.int8_product_64(a, sa[:M], b, sb[:N], bias)
    a, sfa, b, sfb, alpha = ops
    return P.fp4_product_64(a, sfa, b, sfb, alpha, bias, M, N, K)


def one(kind, M, N, K, act, gated, bias, residual, prepared=False, seed=0):
    ops = operands(kind, M, N, K, seed)
    b, r = extras(M, N, gated, bias, residual, seed)
    y = run(kind, ops, M, N, K, b, act, gated, r, prepared)
    torch.cuda.synchronize()
    assert nv.last_device_status() == nv.OK
    v, dv = product(kind, ops, M, N, K, b)
    y64, bound = P.epilogue_64(v, dv, act, gated, r)
    P.check(y, y64, bound, f"{kind} {M}x{N}x{K} {act} gated={gated} bias={bias} residual={residual}")
    return y


CASES = [("int8",) + s for s in INT8_SHAPES] + [("nvfp4",) + s for s in FP4_SHAPES]


@pytest.mark.parametrize("kind,M,N,K", CASES)
@pytest.mark.parametrize("gated", [False, True])
def test_shapes(kind, M, N, K, gated):
    one(kind, M, N, K, "silu", gated, True, True)
    one(kind, M, N, K, "gelu", gated, False, True, prepared=True)
    one(kind, M, N, K, "none", gated, True, False)


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
@pytest.mark.parametrize("act", P.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [3, 90, 1300])
def test_activations(kind, act, gated, M):
    for bias, residual in ((True, True), (False, False)):
        one(kind, M, 2048, 256, act, gated, bias, residual, seed=1)


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
@pytest.mark.parametrize("M", [2, 70, 3000])
def test_large_values(kind, M):
    """Biases that push the activations into both tails."""
    N, K = 512, 128
    ops = operands(kind, M, N, K)
    big = torch.linspace(-300.0, 300.0, N, device=DEV).to(BF16)
    for act in P.ACTS:
        for gated in (False, True):
            y = run(kind, ops, M, N, K, big, act, gated, None)
            v, dv = product(kind, ops, M, N, K, big)
            y64, bound = P.epilogue_64(v, dv, act, gated, None)
            P.check(y, y64, bound, f"{kind} {act} {gated}")


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(5, 264, 256), (200, 264, 1024), (3000, 1024, 256)])
def test_none_equals_the_plain_product(kind, M, N, K):
    """Without activation and residual the result is the existing product's, bit for bit."""
    ops = operands(kind, M, N, K)
    b, _ = extras(M, N, False, True, False)
    y = run(kind, ops, M, N, K, b, "none", False, None)
    if kind == "int8":
        ref = nv.int8_gemm(ops[0], ops[1], ops[2], ops[3], b)
    else:
        ref = nv.nvfp4_gemm(*ops, b, M, N, K)
    assert torch.equal(y.view(torch.int16), ref.view(torch.int16))


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
@pytest.mark.parametrize("M,N,K,gated", [(4, 512, 256, False), (150, 520, 512, False),
                                         (2600, 2064, 192, False), (2600, 2064, 192, True),
                                         (150, 260, 64, True), (150, 261, 64, False)])
def test_residual_in_place(kind, M, N, K, gated):
    ops = operands(kind, M, N, K)
    b, r = extras(M, N, gated, True, True)
    want = run(kind, ops, M, N, K, b, "gelu_tanh", gated, r)
    stream = r.clone()
    got = run(kind, ops, M, N, K, b, "gelu_tanh", gated, stream, out=stream)
    assert got is stream
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    for _ in range(3):                                    # the same bits every time
        again = run(kind, ops, M, N, K, b, "gelu_tanh", gated, r)
        assert torch.equal(again.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
def test_rows_behind_the_last_are_left(kind):
    for M, N in ((3, 256), (130, 520), (130, 260)):
        ops = operands(kind, M, N, 256)
        y = torch.full((M + 130, N), 5.0, dtype=BF16, device=DEV)
        _, r = extras(M, N, False, False, True)
        run(kind, ops, M, N, 256, None, "relu", False, r, out=y[:M])
        torch.cuda.synchronize()
        assert (y[M:] == 5.0).all()


def test_empty():
    a = torch.empty(0, 64, dtype=torch.int8, device=DEV)
    b = torch.zeros(8, 64, dtype=torch.int8, device=DEV)
    s0, s8 = torch.empty(0, device=DEV), torch.ones(8, device=DEV)
    assert nv.int8_gemm_act(a, s0, b, s8, activation="silu").shape == (0, 8)
    assert nv.int8_gemm_act(b, s8, a, s0).shape == (8, 0)


@pytest.mark.parametrize("rows", [1, 40, 700])
def test_linear_act(rows):
    """The linears with an epilogue equal their own two steps, bit for bit."""
    N, K = 768, 512
    g = W._gen(rows, DEV)
    x = W.with_outliers((rows, K), 0.01, 20.0, g, DEV)
    w = W.normal((N, K), 0.05, g, DEV).to(BF16)
    bias, r = extras(rows, N, True, True, True)
    wp, wsf, gw = nv.pack_weight(w, 64)
    y = nv.nvfp4_linear_act(x, wp, wsf, gw, N, bias, "silu", True, r, rotate_group=64)
    alpha = torch.empty(1, device=DEV)
    xp, xsf, _ = nv.nvfp4_quantize(x, 64, None, gsf_w=gw, alpha_out=alpha)
    ref = nv.nvfp4_gemm_act(xp, xsf, wp, wsf, alpha, bias, rows, N, K, "silu", True, r)
    assert torch.equal(y.view(torch.int16), ref.view(torch.int16))
    prep = nv.prepare_weight_scales(wsf, N, K)
    y = nv.nvfp4_linear_act(x, wp, prep, gw, N, bias, "silu", True, r, rotate_group=64,
                            prepared=True)
    assert torch.equal(y.view(torch.int16), ref.view(torch.int16))
    wq, sw = nv.int8_quantize_rows(w)
    y = nv.int8_linear_act(x, wq, sw, bias, "gelu", True, r)
    ref = nv.int8_gemm_act(*nv.int8_quantize_rows(x), wq, sw, bias, "gelu", True, r)
    assert torch.equal(y.view(torch.int16), ref.view(torch.int16))


# --- the operators together: the feed-forward half of a pre-norm block -------------------

def block(kind, st, x, stream):
    """stream += down(silu(gate) * up)(norm(stream + x)), everything in place on stream."""
    M, D = x.shape
    if kind == "int8":
        q, s, _ = nv.int8_rmsnorm_quantize(x, st["w"], 1e-6, residual=stream, residual_out=stream)
        f = nv.int8_gemm_act(q, s, st["gu"][0], st["gu"][1], None, "silu", True)
        fq, fs = nv.int8_quantize_rows(f)
        return (q, s, f, fq, fs,
                nv.int8_gemm_act(fq, fs, st["dn"][0], st["dn"][1], None, residual=stream, out=stream))
    p, sf, _ = nv.nvfp4_rmsnorm_quantize(x, st["w"], st["gsf"], 1e-6, residual=stream,
                                         residual_out=stream, gsf_w=st["gu"][2],
                                         alpha_out=st["alpha"])
    F = st["F"]
    f = nv.nvfp4_gemm_act(p, sf, st["gu"][0], st["gu"][1], st["alpha"], None, M, 2 * F, D, "silu", True)
    return (p, sf, f, nv.nvfp4_linear_act(f, *st["dn"], D, residual=stream, out=stream))


def block_state(kind, D, F):
    g = W._gen(D + F, DEV)
    gate, up = (W.normal((F, D), 0.05, g, DEV).to(BF16) for _ in range(2))
    down = W.normal((D, F), 0.03, g, DEV).to(BF16)
    gu = nv.interleave_gate_up(gate, up)
    st = {"F": F, "w": (1 + W.normal((D,), 0.2, g, DEV)).to(BF16)}
    if kind == "int8":
        st["gu"], st["dn"] = nv.int8_quantize_rows(gu), nv.int8_quantize_rows(down)
    else:
        st["gu"], st["dn"] = nv.pack_weight(gu), nv.pack_weight(down)
        st["gsf"] = torch.tensor([2688.0 / 20.3], device=DEV)
        st["alpha"] = torch.empty(1, device=DEV)
    return st


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
@pytest.mark.parametrize("M", [1, 77, 900])
def test_block(kind, M):
    D, F = 512, 1280
    st = block_state(kind, D, F)
    g = W._gen(M, DEV)
    x = W.normal((M, D), 1.0, g, DEV).to(BF16)
    stream0 = W.normal((M, D), 2.0, g, DEV).to(BF16)
    stream = stream0.clone()
    res = block(kind, st, x, stream)
    torch.cuda.synchronize()
    assert nv.last_device_status() == nv.OK
    h, n = P.norm_rows(x, stream0, st["w"], 1e-6)
    # each step against 64 bits on the codes that the step before it wrote
    if kind == "int8":
        q, s, f, fq, fs, y = res
        q2, s2 = nv.int8_quantize_rows(n)
        assert torch.equal(q, q2) and torch.equal(s, s2)
        v, dv = P.int8_product_64(q, s, *st["gu"], None)
        v2, dv2 = P.int8_product_64(fq, fs, *st["dn"], None)
    else:
        p, sf, f, y = res
        p2, sf2, _ = nv.nvfp4_quantize(n, 0, st["gsf"])
        assert torch.equal(p, p2) and torch.equal(sf, sf2)
        v, dv = P.fp4_product_64(p, sf, st["gu"][0], st["gu"][1], st["alpha"], None, M, 2 * F, D)
        a2 = torch.empty(1, device=DEV)
        fp, fsf, _ = nv.nvfp4_quantize(f, 0, None, gsf_w=st["dn"][2], alpha_out=a2)
        v2, dv2 = P.fp4_product_64(fp, fsf, st["dn"][0], st["dn"][1], a2, None, M, D, F)
    P.check(f, *P.epilogue_64(v, dv, "silu", True, None), "gate and up")
    P.check(y, *P.epilogue_64(v2, dv2, "none", False, h), "down")
    assert y is stream


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
@pytest.mark.parametrize("M", [1, 300])
def test_block_in_a_graph(kind, M):
    """Captured once and replayed on new inputs; a second graph of its own replayed between."""
    D, F = 512, 1280
    st = block_state(kind, D, F)
    g = W._gen(M + 1, DEV)
    xs = [W.normal((M, D), 1.0, g, DEV).to(BF16) for _ in range(3)]
    rs = [W.normal((M, D), 2.0, g, DEV).to(BF16) for _ in range(3)]
    want = []
    for x, r in zip(xs, rs):
        r = r.clone()
        block(kind, st, x, r)
        want.append(r)
    side = torch.cuda.Stream()
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        x, r = xs[0].clone(), rs[0].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            keep = block(kind, st, x, r)
        graphs.append((graph, x, r, keep))
    for i in (2, 0, 1):
        for graph, x, r, _ in graphs:
            x.copy_(xs[i])
            r.copy_(rs[i])
            graph.replay()
        torch.cuda.synchronize()
        for _, _, r, _ in graphs:
            assert torch.equal(r.view(torch.int16), want[i].view(torch.int16))


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
@pytest.mark.parametrize("M", [1, 16, 17, 32, 64, 128])
@pytest.mark.parametrize("N,K", [(19200, 320), (38038, 64), (25602, 1152), (19202, 5184)])
def test_long_weights(kind, M, N, K):
    """Few rows against a weight with more row blocks than SMs."""
    one(kind, M, N, K, "silu", True, True, True, prepared=True)
    one(kind, M, N, K, "gelu", False, False, True)
    one(kind, M, N, K, "none", True, True, False)


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
def test_linear_act_weights_written_just_before(kind):
    """The linears may load their weight before the activation quantizer has ended; weights
    that the stream wrote just before the call have to be seen."""
    for rows, N, K in ((1, 19456, 512), (200, 19456, 512), (1, 512, 2048), (100, 512, 2048)):
        g = W._gen(rows + N, DEV)
        x = W.normal((rows, K), 1.0, g, DEV).to(BF16)
        ws = [W.normal((N, K), 0.05, g, DEV).to(BF16) for _ in range(3)]
        if kind == "int8":
            packs = [nv.int8_quantize_rows(w) for w in ws]
        else:
            packs = [nv.pack_weight(w) for w in ws]
        live = tuple(t.clone() for t in packs[0])

        def call():
            if kind == "int8":
                return nv.int8_linear_act(x, *live, activation="gelu")
            return nv.nvfp4_linear_act(x, *live, N, activation="gelu")

        for k in (1, 2, 0):
            for t, s in zip(live, packs[k]):
                t.copy_(s)
            y = call()
            torch.cuda.synchronize()
            ref = (nv.int8_linear_act(x, *packs[k], activation="gelu") if kind == "int8"
                   else nv.nvfp4_linear_act(x, *packs[k], N, activation="gelu"))
            assert torch.equal(y.view(torch.int16), ref.view(torch.int16))


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(64, 1030, 2560), (512, 1024, 5120), (130, 260, 1280),
                                   (300, 520, 2624)])
@pytest.mark.parametrize("gated", [False, True])
def test_split_k(kind, M, N, K, gated):
    """Few tiles of a long K: clusters that share it."""
    one(kind, M, N, K, "silu", gated, True, True, prepared=True)
    one(kind, M, N, K, "gelu", gated, False, False)


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
def test_two_streams_at_once(kind):
    """Calls of every schedule on two streams, none waiting for the other."""
    shapes = [(1, 19456, 512), (4, 1024, 2048), (100, 520, 2048), (2500, 1024, 512)]
    jobs = []
    for M, N, K in shapes:
        ops = operands(kind, M, N, K)
        b, r = extras(M, N, False, True, True)
        want = run(kind, ops, M, N, K, b, "silu", False, r)
        outs = [torch.empty_like(want) for _ in range(2)]
        jobs.append((ops, M, N, K, b, r, want, outs))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for ops, M, N, K, b, r, _, outs in jobs:
            for s, out in zip(streams, outs):
                run(kind, ops, M, N, K, b, "silu", False, r, out=out, stream=s)
    torch.cuda.synchronize()
    assert nv.last_device_status() == nv.OK
    for *_, want, outs in jobs:
        for out in outs:
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_refusals_with_cuda_tensors():
    ops = operands("int8", 4, 16, 64)
    with pytest.raises(TypeError, match="must be on"):
        nv.int8_gemm_act(ops[0], ops[1].cpu(), ops[2], ops[3])
    y = torch.empty(4 * 16 + 1, dtype=BF16, device=DEV)[1:].view(4, 16)
    with pytest.raises(nv.NVFP4Error) as e:
        nv.int8_gemm_act(ops[0], ops[1], ops[2], ops[3], out=y)
    assert e.value.status == nv.ERR_ALIGN
    with pytest.raises(nv.NVFP4Error) as e:
        nv.int8_linear_act(torch.zeros(4, 64, dtype=BF16, device=DEV), ops[2], ops[3],
                           workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    assert e.value.status == nv.ERR_WORKSPACE
