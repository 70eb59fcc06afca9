"""Every kernel of the 4-bit linear layer, at sizes that a CPU test holds to it (mx4_kernels.py): depths,
activations, scales that are NaN, outputs in place, streams and graphs.

The products are exact in fp32 where codes and scales are those of exact_operands(); else
bounds are mx4_util's.  The 64-bit products are torch's, on the GPU.
"""
import threading

import pytest
import torch

import activation_epilogue_amd as fl
from gpu_util import say
from moe_util import DT, U32, act64, act_bound, worst
from mx4_kernels import KERNELS, depth, plan_of
from mx4_util import MAGNITUDES

pytestmark = pytest.mark.gpu
FF = 255


def values_of(q):
    """(rows, K) in 64 bits, on the device."""
    rows, blocks = q.scales.shape
    c = torch.stack([q.codes & 15, q.codes >> 4], 2).view(rows, blocks, 32).int()
    v = MAGNITUDES.cuda()[c & 7] * (1 - 2 * (c >> 3)).double()
    v = v * torch.exp2(q.scales.double() - 127)[..., None]
    v = torch.where((q.scales == FF)[..., None], torch.full_like(v, float("nan")), v)
    return v.view(rows, blocks * 32)[:, :q.K].contiguous()


def product(a, b):
    return a @ b.t().contiguous()


def operand(rows, K, g, spread=2):
    """Any codes, scales of 2^0 to 2^(spread-1): sums of products are multiples of 1/4 below 2^22, exact in fp32 in
    any order.  The arrays lie among bytes of 255 (NaN scales), the scales at an odd address."""
    blocks = (K + 31) // 32
    cbuf = torch.full((rows * blocks * 16 + 4096,), FF, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((rows * blocks + 4096,), FF, dtype=torch.uint8, device="cuda")
    codes, scales = cbuf[1024:1024 + rows * blocks * 16].view(rows, blocks * 16), sbuf[1025:1025 + rows * blocks].view(rows, blocks)
    codes.copy_(torch.randint(0, 256, codes.shape, generator=g, device="cuda", dtype=torch.uint8))
    if K % 32:  # what fills the last block up is zero
        live = (torch.arange(blocks * 32) < K).view(-1, 2).long()
        codes &= (live * torch.tensor([15, 240])).sum(1).to(torch.uint8).cuda()
    scales.copy_(127 + torch.randint(0, spread, scales.shape, generator=g, device="cuda", dtype=torch.uint8))
    return fl.Mx4(codes, scales, K)


def exact_operands(k, blocks, g):
    return operand(k.M, depth(blocks), g), operand(k.N, depth(blocks), g)


def guarded(M, N, dtype):
    buf = torch.full((M * N + 128,), float("nan"), dtype=dtype, device="cuda")
    return buf[33:33 + M * N].view(M, N), buf


def untouched(buf, n):
    return bool(torch.isnan(buf[:33]).all()) and bool(torch.isnan(buf[33 + n:]).all())


def reached(k, blocks, values, dtype):
    p = fl.mx4_plan(k.M, k.N, depth(blocks), values, dtype)
    assert plan_of(p) == k.plan and p.quantize == (0 if not values else 2 if k.inside else 1)


@pytest.mark.parametrize("name", KERNELS)
def test_depths(name):
    """Every count of blocks in the last stage and the last scales, with the arrays' ends at every place."""
    k = KERNELS[name]
    g = torch.Generator(device="cuda").manual_seed(k.M)
    for blocks in k.sweep:
        say("depth", name, blocks)
        A, B = exact_operands(k, blocks, g)
        a, b = values_of(A), values_of(B)
        want = product(a, b)
        reached(k, blocks, False, torch.float32)
        out, buf = guarded(k.M, k.N, torch.float32)
        fl.fused_linear_mx4(A, B, act="none", out=out, dtype=torch.float32)
        assert torch.equal(out.double(), want) and untouched(buf, out.numel())
        # the same values given as such, whose scales are theirs
        reached(k, blocks, True, torch.float32)
        out.fill_(float("nan"))
        fl.fused_linear_mx4(a.float(), B, act="none", out=out)
        assert torch.equal(out.double(), product(values_of(fl.quantize_mx4(a.float())), b)) and untouched(buf, out.numel())


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "glu"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("name", KERNELS)
def test_epilogues(name, dtype, act):
    """With a bias, a residual and the gate's Y and without; the output in place of R and of Y."""
    k, dt = KERNELS[name], DT[dtype]
    M, N, K = k.M, k.N, depth(k.deep)
    g = torch.Generator(device="cuda").manual_seed(M + N)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(dt)  # noqa: E731
    x, w, bias, R = n(M, K), n(N, K, std=K ** -0.5), n(N), n(M, N)
    Y = n(M, N) if act == "glu" else None
    A, B = fl.quantize_mx4(x), fl.quantize_mx4(w)
    a, b = values_of(A), values_of(B)
    sums, size = product(a, b), product(a.abs(), b.abs())
    y64 = torch.zeros_like(sums) if Y is None else Y.double()

    def right(got, bias, R):
        s, z, terms = sums, size, K + 1
        for t in (bias, R):
            if t is not None:
                s, z, terms = s + t.double(), z + t.double().abs(), terms + 1
        return worst(got, act64(s, y64, act), act_bound(s, y64, act, terms * U32 * z), dt) <= 1.0
    for values, p, r in ((True, bias, None), (False, bias, R), (True, None, None), (False, None, R), (True, bias, R)):
        say("epilogue", name, dtype, act, values, p is not None, r is not None)
        reached(k, k.deep, values, dt)
        out, buf = guarded(M, N, dt)
        fl.fused_linear_mx4(x if values else A, B, p, Y, act=act, out=out, R=r, dtype=dt)
        assert right(out, p, r) and untouched(buf, out.numel())
    # the last, over its residual and over its gate
    want = out.clone()
    out.copy_(R)
    fl.fused_linear_mx4(x, B, bias, Y, act=act, out=out, R=out)
    assert torch.equal(out, want) and untouched(buf, out.numel())
    if Y is not None:
        out.copy_(Y)
        fl.fused_linear_mx4(x, B, bias, out, act=act, out=out, R=R)
        assert torch.equal(out, want) and untouched(buf, out.numel())


@pytest.mark.parametrize("name", KERNELS)
def test_nan_stays_in_its_row_and_column(name):
    """Scales of 255 in the first and the last block and between, in the last row and column too."""
    k = KERNELS[name]
    M, N, blocks = k.M, k.N, k.deep
    A, B = exact_operands(k, blocks, torch.Generator(device="cuda").manual_seed(1))
    want = product(values_of(A), values_of(B))
    for rows, q in (((M // 2, M - 1)[:M], A), ((0, N // 3, N - 1), B)):
        for i, row in enumerate(rows):
            q.scales[row, (0, blocks // 2, blocks - 1)[(i + 1) % 3]] = FF
            if q is A:
                want[row] = float("nan")
            else:
                want[:, row] = float("nan")
    say("NaN", name)
    for src in (A, values_of(A).float()):
        out = fl.fused_linear_mx4(src, B, act="none", dtype=torch.float32)
        assert torch.equal(torch.isnan(out), torch.isnan(want))
        if src is A:
            assert torch.equal(torch.nan_to_num(out.double()), torch.nan_to_num(want))


@pytest.mark.parametrize("name", KERNELS)
def test_again_on_another_stream_and_in_a_graph(name):
    k, dt = KERNELS[name], torch.bfloat16
    M, N, K = k.M, k.N, depth(k.deep)
    g = torch.Generator(device="cuda").manual_seed(4)
    W = operand(N, K, g, 9)
    x, R = (torch.randn(M, n, generator=g, device="cuda").bfloat16() for n in (K, N))
    bias = torch.randn(N, generator=g, device="cuda").bfloat16()
    ws = torch.empty(max(fl.mx4_workspace_bytes(M, N, K, True, dt), 1), dtype=torch.uint8, device="cuda")
    reached(k, k.deep, True, dt)
    say("again", name)

    def work(**kw):
        return fl.fused_linear_mx4(x, W, bias, act="gelu_tanh", R=R, **kw)
    first = work()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = work(stream=s)
    with torch.cuda.stream(s):
        third = work(workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(first, again) and torch.equal(first, third)
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(out=out, workspace=ws)
    for _ in range(3):
        x.normal_()
        R.normal_()
        want = work()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("one,two", [("parts_of_128x128_alone", "parts_of_256x256"), ("parts_of_128x128", "tile_128x128"),
                                     ("parts_of_128x128_alone", "stream_64x32_8"), ("tile_256x256", "stream_64x64_8")])
def test_two_streams_at_once(one, two):
    """Layers of two kernels with a workspace each, at the same time and over and over."""
    g = torch.Generator(device="cuda").manual_seed(6)
    jobs = []
    for k in (KERNELS[one], KERNELS[two]):
        x = torch.randn(k.M, depth(k.deep), generator=g, device="cuda").half()
        W = operand(k.N, depth(k.deep), g)
        jobs.append((x, W, fl.fused_linear_mx4(x, W, act="relu"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    say("two streams", one, two)
    for _ in range(5):
        outs = []
        for x, W, _, s in jobs:
            with torch.cuda.stream(s):
                outs.append([fl.fused_linear_mx4(x, W, act="relu") for _ in range(3)])
        torch.cuda.synchronize()
        for (_, _, want, _), got in zip(jobs, outs):
            assert all(torch.equal(t, want) for t in got)


def test_two_threads_two_streams():
    """Layers of two kernels, and quantising, from two host threads at the same time."""
    g = torch.Generator(device="cuda").manual_seed(6)
    jobs = []
    for name in ("parts_of_128x128_alone", "tile_128x128"):
        k = KERNELS[name]
        x = torch.randn(k.M, depth(k.deep), generator=g, device="cuda").half()
        W = operand(k.N, depth(k.deep), g)
        q = fl.quantize_mx4(x.t().contiguous(), transposed=True)
        jobs.append((x, W, (fl.fused_linear_mx4(x, W, act="relu"), q.codes, q.scales)))
    torch.cuda.synchronize()
    got, errors, start = [[], []], [], threading.Barrier(2)

    def work(i):
        try:
            x, W, _ = jobs[i]
            stream = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    q = fl.quantize_mx4(x.t().contiguous(), transposed=True)
                    got[i].append((fl.fused_linear_mx4(x, W, act="relu"), q.codes, q.scales))
                    with pytest.raises(fl.FusedLinearError, match="needs Y"):  # a message of the thread's own
                        fl.fused_linear_mx4(x, W, act="glu")
            stream.synchronize()
        except Exception as e:  # reported by the main thread
            errors.append(repr(e))
    say("two threads, two streams")
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for (_, _, want), each in zip(jobs, got):
        assert len(each) == 20 and all(torch.equal(p, q) for one in each for p, q in zip(one, want))

def test_scales_of_the_whole_range():
    """Products whose scales lie outside of fp32's range each, and inside together."""
    one = torch.tensor([[4] * 16], dtype=torch.uint8, device="cuda")  # 2, 0, 2, 0, ...: 16 twos
    at = lambda s: fl.Mx4(one, torch.tensor([[s]], dtype=torch.uint8, device="cuda"), 32)  # noqa: E731
    say("scales of the whole range")
    for s, t in ((254, 0), (0, 254), (254, 27), (200, 30), (127, 127), (254, 64), (1, 200), (0, 190)):
        got = fl.fused_linear_mx4(at(s), at(t), act="none", dtype=torch.float32)
        assert float(got) == 64.0 * 2.0 ** (s + t - 254)
