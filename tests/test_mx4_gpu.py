"""Microscaled 4-bit floating point on the GPU: codes and scales to the bit, the
linear layer against 64 bits."""
import pytest
import torch

import activation_epilogue_amd as fl
from gpu_util import say
from moe_util import DT, worst
from mx4_util import linear64, quantize64, values64

pytestmark = pytest.mark.gpu
FF = 255  # around bytes: a NaN scale, so that a read too far shows


def among(t, offset):
    """A copy of the bytes t on the device, `offset` bytes into a buffer of 255s, and the buffer."""
    buf = torch.full((t.numel() + 4096,), FF, dtype=torch.uint8, device="cuda")
    buf[offset:offset + t.numel()] = t.reshape(-1).cuda()
    return buf[offset:offset + t.numel()].view(t.shape), buf


def mx4(codes, scales, K, odd=True):
    return fl.Mx4(among(codes, 1024)[0], among(scales, 1025 if odd else 1024)[0], K)


def guarded(M, N, dtype):
    buf = torch.full((M * N + 128,), float("nan"), dtype=dtype, device="cuda")
    return buf[33:33 + M * N].view(M, N), buf


def some(rows, K, dtype, seed):
    """Values of many sizes, with blocks of zeros and of one value."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-12, 8, (rows, K), generator=g).float() / 4)
    x = x * torch.exp2(torch.randint(-9, 9, (rows, 1), generator=g).float())
    x[torch.rand(rows, K, generator=g) < 0.05] = 0.0
    if rows > 2:
        x[rows // 2] = 0.0
    if K > 64:
        x[0, 32:64] = 0.0
        x[0, 40] = -3.0
    return x.to(dtype)


def check_quantize(x, K):
    """Rows and, transposed, columns; every byte, and none around them."""
    rows = x.shape[0]
    want = quantize64(x)
    for transposed in (False, True):
        codes, cbuf = among(torch.zeros(rows, (K + 31) // 32 * 16, dtype=torch.uint8), 1024)
        scales, sbuf = among(torch.zeros(rows, (K + 31) // 32, dtype=torch.uint8), 1025)
        given = x.t().contiguous() if transposed else x
        shifted = torch.empty(given.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(given.shape)  # odd alignment
        shifted.copy_(given)
        for src in (given.cuda(), shifted):
            say("quantize", rows, K, x.dtype, transposed)
            q = fl.quantize_mx4(src, transposed=transposed, out=fl.Mx4(codes, scales, K))
            assert q.codes is codes and q.K == K
            assert torch.equal(scales.cpu(), want[1])
            assert torch.equal(codes.cpu(), want[0])
            assert (cbuf[:1024] == FF).all() and (cbuf[1024 + codes.numel():] == FF).all()
            assert (sbuf[:1025] == FF).all() and (sbuf[1025 + scales.numel():] == FF).all()
    return want


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 31), (2, 32), (3, 33), (7, 8), (64, 64), (65, 100), (33, 255), (5, 256),
                                    (257, 257), (130, 96), (1, 4096), (1000, 40), (9, 5000)])
def test_quantize(rows, K, dtype):
    x = some(rows, K, DT[dtype], rows + K)
    codes, scales = check_quantize(x, K)
    for to in ("f32", "f16", "bf16"):
        out, buf = guarded(rows, K, DT[to])
        say("dequantize", rows, K, to)
        fl.dequantize_mx4(mx4(codes, scales, K), DT[to], out=out)
        assert torch.equal(out.cpu(), values64(codes, scales, K).to(DT[to]))
        assert torch.isnan(buf[:33]).all() and torch.isnan(buf[33 + rows * K:]).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,K", [(1030, 1500), (12288, 1024), (12289, 1024), (4100, 3100), (200001, 33), (393217, 5),
                                    (1, 4200001), (3, 4194241)])
def test_columns_as_rows(rows, K, dtype):
    """Many columns, by one lane to a block and by four, to the bits of the rows they become."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, K, generator=g, device="cuda") * torch.exp2(torch.randint(-9, 9, (rows, 1), generator=g, device="cuda"))
    x = x.to(DT[dtype])
    say("columns as rows", rows, K, dtype)
    want = fl.quantize_mx4(x)
    blocks = (K + 31) // 32
    codes, cbuf = among(torch.zeros(rows, 16 * blocks, dtype=torch.uint8), 1024)
    scales, sbuf = among(torch.zeros(rows, blocks, dtype=torch.uint8), 1025)
    fl.quantize_mx4(x.t().contiguous(), transposed=True, out=fl.Mx4(codes, scales, K))
    assert torch.equal(codes, want.codes) and torch.equal(scales, want.scales)
    assert (cbuf[:1024] == FF).all() and (cbuf[1024 + codes.numel():] == FF).all()
    assert (sbuf[:1025] == FF).all() and (sbuf[1025 + scales.numel():] == FF).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_value(dtype):
    """All finite 16-bit values in blocks of their neighbours, and each below a
    largest value that puts it at another place of the grid."""
    bits = torch.arange(65536).to(torch.int32).to(torch.int16)
    x = bits.view(DT[dtype])
    x = x[torch.isfinite(x.float())]
    x = x[:x.numel() // 32 * 32].view(-1, 32)
    check_quantize(x, 32)
    for anchor in (6.0, 7.5, 0.001, 300.0):
        y = x.clone()
        y[:, 5] = torch.where(x.float().abs().amax(1) < anchor, torch.tensor(anchor).to(x.dtype), x[:, 5])
        check_quantize(y, 32)


def test_borders_in_32_bits():
    edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    edge = torch.cat([edge, torch.nextafter(edge, torch.tensor(0.0)), torch.nextafter(edge, torch.tensor(9.0)), edge[:4]])
    rows = [edge * 2.0 ** e for e in (-126, -60, -1, 0, 1, 60, 123)]
    x = torch.stack([torch.cat([r, r[:1] * 0 + r.max() * 1.0]) for r in rows])
    x = torch.cat([x, -x])
    check_quantize(x, 32)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_ends_of_the_range(dtype):
    """Denormals, the smallest and the largest values, -0, infinities and NaN:
    a block with one of the last two reads as NaN, its neighbours as they are."""
    t = torch.finfo(DT[dtype])
    x = torch.ones(12, 96, dtype=torch.float64)
    x[0, :32], x[1, :32] = t.smallest_normal, t.smallest_normal * t.eps
    x[2, :32], x[3, 3] = t.max, t.max
    x[4, :32] = -0.0
    x[5, 40], x[6, 95], x[7, 0], x[8, 64] = float("inf"), float("-inf"), float("nan"), float("nan")
    x[9] *= t.smallest_normal * 3
    x[10] = t.smallest_normal * torch.arange(96) / 8
    x = x.to(DT[dtype])
    codes, scales = check_quantize(x, 96)
    assert (scales == 255).sum() == 4
    got = fl.dequantize_mx4(mx4(codes, scales, 96), torch.float32).cpu()
    want = values64(codes, scales, 96)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got.double()), torch.nan_to_num(want.float().double()))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_every_code_at_every_scale(dtype):
    codes = torch.arange(256).to(torch.uint8).view(1, 256).expand(256, 256).contiguous()  # 512 values a row
    scales = torch.arange(256).to(torch.uint8).view(256, 1).expand(256, 16).contiguous()
    got = fl.dequantize_mx4(fl.Mx4(codes.cuda(), scales.cuda(), 512), DT[dtype]).cpu()
    want = values64(codes, scales, 512).to(DT[dtype])
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and bool(torch.isnan(got[255]).all())
    assert torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(want.float()))


# ------------------------------------------------------------ the linear layer

def bytes_of(rows, K, seed, spread=1):
    """Codes of any value and scales of 2^0 to 2^(spread-1): sums of their
    products are multiples of 1/4 below 2^22, exact in fp32 in any order."""
    g = torch.Generator().manual_seed(seed)
    blocks = (K + 31) // 32
    codes = torch.randint(0, 256, (rows, blocks * 16), generator=g).to(torch.uint8)
    if K % 32:  # what fills the last block up is zero
        live = torch.arange(blocks * 32) < K
        keep = (live.view(-1, 2).long() * torch.tensor([15, 240])).sum(1).to(torch.uint8)
        codes = codes & keep
    return codes, (127 + torch.randint(0, spread, (rows, blocks), generator=g)).to(torch.uint8)


def exact_case(M, N, K, seed=0, values=False, dtype=torch.float32):
    """Equal to the sums in 64 bits, whatever the order; nothing written around."""
    a, b = bytes_of(M, K, seed, 2), bytes_of(N, K, seed + 1, 2)
    va, vb = values64(*a, K), values64(*b, K)
    want = va @ vb.t()
    out, buf = guarded(M, N, dtype)
    A = va.to(dtype).cuda() if values else mx4(*a, K)
    say("exact", M, N, K, values, dtype)
    fl.fused_linear_mx4(A, mx4(*b, K), act="none", out=out, dtype=dtype)
    if values:  # what a block's largest value leaves of the others
        want = values64(*quantize64(va.to(dtype)), K) @ vb.t()
    assert torch.equal(out.cpu(), want.to(dtype))
    assert torch.isnan(buf[:33]).all() and torch.isnan(buf[33 + M * N:]).all()


@pytest.mark.parametrize("values", [False, True])
@pytest.mark.parametrize("K", [1, 31, 32, 33, 64, 65, 127, 128, 160, 255, 256, 257, 288, 511, 512, 513, 1000, 2049, 4096])
def test_depths(K, values):
    for M, N in ((1, 17), (16, 16), (37, 70), (300, 290)):
        exact_case(M, N, K, K, values)


@pytest.mark.parametrize("values", [False, True])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 200, 255, 256, 257, 383,
                               511, 513, 700])
def test_row_counts(M, values):
    for N, K in ((1, 64), (129, 300), (515, 1024)):
        exact_case(M, N, K, M, values)


@pytest.mark.parametrize("N", [1, 2, 3, 5, 15, 16, 17, 31, 33, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 511, 1030,
                               5000])
def test_column_counts(N):
    for M, K in ((1, 257), (20, 512), (129, 96), (260, 640)):
        exact_case(M, N, K, N)


@pytest.mark.parametrize("M,N,K", [(8, 20000, 512), (64, 9000, 1024), (128, 4096, 4096), (512, 4096, 512),
                                   (1000, 3000, 1000), (1025, 2049, 513), (2048, 2048, 256), (4097, 1030, 96),
                                   (3, 300, 8192), (70, 64, 16000), (256, 256, 8000), (33000, 40, 64)])
def test_larger(M, N, K):
    exact_case(M, N, K, 5)
    exact_case(M, N, K, 6, values=True, dtype=torch.float32)


# Sizes of several kernels (mx4_kernels.py has sizes of each, held to the choice).
@pytest.mark.parametrize("M,N,K", [(3, 1000, 2000), (9, 5001, 700), (257, 259, 100), (20, 2051, 130), (200, 1030, 65),
                                   (200, 2051, 300), (33, 4099, 8200), (300, 2051, 4100), (600, 259, 4100),
                                   (257, 4099, 8200), (3000, 5000, 65), (130, 16391, 8200), (513, 515, 16400),
                                   (4495, 11606, 65), (3331, 10282, 300)])
def test_every_kernel(M, N, K):
    exact_case(M, N, K, 7)
    exact_case(M, N, K, 8, values=True)


# A stage is 8 blocks of 32, scales come for four stages: every count of blocks in the
# last of them, with the arrays' last bytes at every place in four.
@pytest.mark.parametrize("blocks", list(range(1, 42)))
def test_tiles_at_every_depth(blocks):
    for M, N in ((1030, 514), (1025, 511), (1027, 385)):
        exact_case(M, N, 32 * blocks - blocks % 3, blocks)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 50, 45000), (2, 3000, 8200), (5, 1000, 1000), (9, 257, 4000), (11, 5000, 3000),
                                   (13, 130, 33), (16, 1000, 2800), (16, 1000, 2900), (16, 20000, 300)])
def test_few_rows_of_values(M, N, K, dtype):
    """In each block's own memory or by a launch of their own, over one run of K and over two."""
    dt = DT[dtype]
    x, b = some(M, K, dt, K), bytes_of(N, K, 2)
    va, vb = values64(*quantize64(x), K), values64(*b, K)
    out, buf = guarded(M, N, dt)
    shifted = torch.empty(M * K + 1, dtype=dt, device="cuda")[1:].view(M, K).copy_(x)
    say("few rows of values", M, N, K, dtype)
    B = mx4(*b, K)
    fl.fused_linear_mx4(shifted, B, act="none", out=out)
    want, bound = linear64(va, vb, None, None, None, "none")
    # fp16 ends at 65504: a value from half a step behind it on, 65520, rounds to an infinity, one whose
    # bound reaches there may
    far = torch.finfo(dt).max * (1 + torch.finfo(dt).eps / 4)
    must, may = want.abs() - bound > far, want.abs() + bound >= far

    def right(got):
        got = got.cpu().double()
        assert bool((got[must] == torch.copysign(torch.full_like(want, float("inf")), want)[must]).all())
        return worst(torch.where(may, torch.zeros_like(want), got), torch.where(may, torch.zeros_like(want), want),
                     bound, dt) <= 1.0
    assert right(out)
    assert torch.isnan(buf[:33]).all() and torch.isnan(buf[33 + M * N:]).all()
    # codes given instead go another way to the same products
    again = fl.fused_linear_mx4(fl.quantize_mx4(shifted), B, act="none", dtype=dt)
    assert right(again)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(700, 1, 64), (700, 7, 64), (700, 9, 64), (1030, 64, 64), (1030, 65, 64), (520, 127, 96),
                                   (520, 777, 96), (700, 1030, 96), (3001, 5001, 65), (4495, 11607, 65)])
def test_rows_of_16_bits_at_any_address(M, N, K, dtype):
    """Odd and even widths, from odd and even elements on; with a residual at another place, and over it."""
    dt = DT[dtype]
    a, b = bytes_of(M, K, 3, 1), bytes_of(N, K, 4, 1)
    sums = values64(*a, K) @ values64(*b, K).t()
    A, B = mx4(*a, K), mx4(*b, K)
    R = torch.randint(-64, 65, (M, N), generator=torch.Generator().manual_seed(1)).to(dt)
    want = sums.to(dt), (sums + R.double()).to(dt)  # exact in fp32 before they are rounded
    for first in (8, 9, 10):
        say("16-bit rows", M, N, K, dtype, first)
        for residual in (False, True):
            buf = torch.full((M * N + 64,), float("nan"), dtype=dt, device="cuda")
            out = buf[first:first + M * N].view(M, N)
            r = torch.empty(M * N + 1, dtype=dt, device="cuda")[1:].view(M, N).copy_(R) if residual else None
            fl.fused_linear_mx4(A, B, act="none", out=out, R=r, dtype=dt)
            assert torch.equal(out.cpu(), want[residual])
            assert torch.isnan(buf[:first]).all() and torch.isnan(buf[first + M * N:]).all()
        out.copy_(R)
        fl.fused_linear_mx4(A, B, act="none", out=out, R=out, dtype=dt)
        assert torch.equal(out.cpu(), want[1])


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "glu"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 100, 300), (17, 257, 1000), (64, 64, 4096), (150, 333, 257), (520, 700, 640)])
def test_against_64_bits(M, N, K, dtype, act):
    dt = DT[dtype]
    g = torch.Generator().manual_seed(M + N)
    a, w = torch.randn(M, K, generator=g).to(dt), (torch.randn(K, N, generator=g) * K ** -0.5).to(dt)
    bias, Y, R = (torch.randn(*s, generator=g).to(dt) for s in ((N,), (M, N), (M, N)))
    B = fl.quantize_mx4(w.cuda(), transposed=True)
    vb = values64(B.codes.cpu(), B.scales.cpu(), K)
    qa = quantize64(a)
    va = values64(*qa, K)
    for values, b, r in ((True, bias, None), (False, bias, R), (True, None, None), (True, bias, R)):
        y = Y if act == "glu" else None
        out, buf = guarded(M, N, dt)
        say("linear", M, N, K, dtype, act, values, r is not None)
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        fl.fused_linear_mx4(a.cuda() if values else mx4(*qa, K), B, dev(b), dev(y), act=act, out=out, R=dev(r), dtype=dt)
        want, bound = linear64(va, vb, b, y, r, act)
        assert worst(out.cpu(), want, bound, dt) <= 1.0
        assert torch.isnan(buf[:33]).all() and torch.isnan(buf[33 + M * N:]).all()


@pytest.mark.parametrize("M,N,K", [(3, 70, 100001), (130, 150, 100033), (1, 40, 600011)])
def test_long_rows(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(K)
    a, b = (torch.randn(n, K, generator=g, device="cuda") for n in (M, N))
    say("long rows", M, N, K)
    A, B = fl.quantize_mx4(a), fl.quantize_mx4(b)
    va, vb = (values64(q.codes.cpu(), q.scales.cpu(), K) for q in (A, B))
    want, bound = linear64(va, vb, None, None, None, "none")
    for src in (A, a):
        out = fl.fused_linear_mx4(src, B, act="none", dtype=torch.float32)
        assert worst(out.cpu(), want, bound, torch.float32) <= 1.0


@pytest.mark.parametrize("M,N,K", [(2, 3, 2 ** 21 + 33), (70, 40, 2 ** 21 + 33), (1, 5, 2 ** 22 - 1)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_longest_rows(M, N, K, dtype):
    """Up to the longest that are taken, whatever the type: from codes and from values of it."""
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(K)
    a, b = (torch.randn(n, K, generator=g, device="cuda").to(dt) for n in (M, N))
    say("longest rows", M, N, K, dtype)
    A, B = fl.quantize_mx4(a), fl.quantize_mx4(b)
    va, vb = (values64(q.codes.cpu(), q.scales.cpu(), K) for q in (A, B))
    want, bound = linear64(va, vb, None, None, None, "none")
    for src in (A, a):
        out = fl.fused_linear_mx4(src, B, act="none", dtype=dt)
        assert worst(out.cpu(), want, bound, dt) <= 1.0
    with pytest.raises(fl.FusedLinearError, match="2\\^22"):
        fl.mx4_workspace_bytes(M, N, 2 ** 22, True, dt)


@pytest.mark.parametrize("M,N,K", [(4, 40, 96), (64, 200, 520), (300, 280, 257), (1100, 1300, 257)])
@pytest.mark.parametrize("values", [False, True])
def test_nan_stays_in_its_row_and_column(M, N, K, values):
    a, b = bytes_of(M, K, 1), bytes_of(N, K, 2)
    clean = values64(*a, K) @ values64(*b, K).t()
    a[1][M // 2, -1] = b[1][N // 3, 0] = b[1][N - 1, 1] = FF
    A = values64(*a, K).float().cuda() if values else mx4(*a, K)
    say("NaN", M, N, K, values)
    out = fl.fused_linear_mx4(A, mx4(*b, K), act="none", dtype=torch.float32).cpu()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[M // 2], bad[:, N // 3], bad[:, N - 1] = True, True, True
    assert torch.equal(torch.isnan(out), bad)
    if not values:
        assert torch.equal(out[~bad].double(), clean[~bad])


@pytest.mark.parametrize("M,N,K", [(5, 70, 300), (100, 257, 96), (600, 513, 300)])
def test_in_place(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(3)
    a, Y, R = (torch.randn(M, n, generator=g, device="cuda").bfloat16() for n in (K, N, N))
    B = fl.quantize_mx4(torch.randn(N, K, generator=g, device="cuda").bfloat16())
    want = fl.fused_linear_mx4(a, B, None, Y, act="glu", R=R)
    for name in ("Y", "R"):
        t = {"Y": Y.clone(), "R": R.clone()}
        assert torch.equal(fl.fused_linear_mx4(a, B, None, t["Y"], act="glu", R=t["R"], out=t[name]), want)


@pytest.mark.parametrize("M,N,K", [(3, 5, 0), (0, 5, 64), (3, 0, 64), (300, 300, 0)])
def test_nothing(M, N, K):
    e = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    blocks = (K + 31) // 32
    bias = torch.arange(N, device="cuda").float() - 1
    for A in (torch.zeros(M, K, device="cuda"), fl.Mx4(e(M, 16 * blocks), e(M, blocks), K)):
        out = fl.fused_linear_mx4(A, fl.Mx4(e(N, 16 * blocks), e(N, blocks), K), bias, act="relu", dtype=torch.float32)
        assert out.shape == (M, N) and torch.equal(out, bias.clamp(min=0).expand(M, N))
    q = fl.quantize_mx4(torch.zeros(M, K, device="cuda"))
    assert q.codes.shape == (M, 16 * blocks) and fl.dequantize_mx4(q, torch.float16).shape == (M, K)
    assert fl.quantize_mx4(torch.zeros(K, M, device="cuda"), transposed=True).scales.shape == (M, blocks)


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "glu"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N", [(1, 1), (3, 5), (37, 70), (300, 515)])
def test_no_depth(M, N, dtype, act):
    """K = 0: the epilogue of nothing but zeros."""
    dt = DT[dtype]
    g = torch.Generator().manual_seed(M)
    bias, Y, R = (torch.randn(*s, generator=g).to(dt) for s in ((N,), (M, N), (M, N)))
    e = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    B = fl.Mx4(e(N, 0), e(N, 0), 0)
    y = Y if act == "glu" else None
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    say("no depth", M, N, dtype, act)
    for A in (torch.zeros(M, 0, dtype=dt, device="cuda"), fl.Mx4(e(M, 0), e(M, 0), 0)):
        for b, r in ((bias, R), (None, R), (bias, None), (None, None)):
            out, buf = guarded(M, N, dt)
            fl.fused_linear_mx4(A, B, dev(b), dev(y), act=act, out=out, R=dev(r), dtype=dt)
            want, bound = linear64(torch.zeros(M, 0).double(), torch.zeros(N, 0).double(), b, y, r, act)
            assert worst(out.cpu(), want, bound, dt) <= 1.0
            assert torch.isnan(buf[:33]).all() and torch.isnan(buf[33 + M * N:]).all()


def test_a_long_output_of_no_depth():
    """More outputs than one dimension of a launch has threads for, 16x16 of them to 512."""
    M, N = 70_001, 33_000
    e = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    bias = torch.randn(N, device="cuda").bfloat16()
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    R = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
    say("a long output of no depth")
    fl.fused_linear_mx4(fl.Mx4(e(M, 0), e(M, 0), 0), fl.Mx4(e(N, 0), e(N, 0), 0), bias, act="relu", R=R, out=out)
    want = (bias.float() + 1).clamp(min=0).bfloat16()
    assert bool((out == want).all())


def test_weights_from_a_layer_and_back():
    """The weight of a fused_linear layer, held in 4 bits: what fused_linear
    gives with the values read back, to the sums' rounding."""
    g = torch.Generator(device="cuda").manual_seed(8)
    M, N, K = 40, 300, 200
    x = torch.randn(M, K, generator=g, device="cuda").half()
    W = (torch.randn(K, N, generator=g, device="cuda") * K ** -0.5).half()
    bias = torch.randn(N, generator=g, device="cuda").half()
    B = fl.quantize_mx4(W, transposed=True)
    got = fl.fused_linear_mx4(x, B, bias, act="gelu_tanh")
    xq = fl.dequantize_mx4(fl.quantize_mx4(x), torch.float16)
    Wq = fl.dequantize_mx4(B, torch.float16).t().contiguous()
    want, bound = linear64(xq.cpu().double(), Wq.cpu().double().t(), bias.cpu(), None, None, "gelu_tanh")
    plain = fl.fused_linear(xq, Wq, bias, act="gelu_tanh")
    for out in (got, plain):
        assert worst(out.cpu(), want, bound, torch.float16) <= 1.0


@pytest.mark.parametrize("M,N,K", [(1, 3000, 2048), (48, 1000, 4096), (700, 1500, 777)])
def test_the_same_bits_again_on_another_stream_and_in_a_graph(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(4)
    W = fl.quantize_mx4(torch.randn(N, K, generator=g, device="cuda").bfloat16())
    x, R = (torch.randn(M, n, generator=g, device="cuda").bfloat16() for n in (K, N))
    bias = torch.randn(N, generator=g, device="cuda").bfloat16()
    need = fl.mx4_workspace_bytes(M, N, K, True, torch.bfloat16)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")

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


def test_two_streams_at_once():
    """Two layers with a workspace each, at the same time and over and over."""
    g = torch.Generator(device="cuda").manual_seed(6)
    jobs = []
    for M, N, K in ((64, 1030, 8000), (700, 1030, 777)):
        x = torch.randn(M, K, generator=g, device="cuda").half()
        W = fl.quantize_mx4(torch.randn(N, K, generator=g, device="cuda").half())
        jobs.append((x, W, fl.fused_linear_mx4(x, W, act="relu"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for x, W, _, s in jobs:
            with torch.cuda.stream(s):
                outs.append([fl.fused_linear_mx4(x, W, act="relu") for _ in range(3)])
        torch.cuda.synchronize()
        for (_, _, want, _), got in zip(jobs, outs):
            assert all(torch.equal(t, want) for t in got)


def test_offsets_past_32_bits():
    """A weight of more than 2^32 bytes of codes: its last rows as alone; and an
    output of more."""
    N, K = 560_007, 16384
    codes = torch.randint(0, 256, (1000, K // 2), device="cuda").to(torch.uint8)
    B = fl.Mx4(torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda"),
               torch.full((N, K // 32), 120, dtype=torch.uint8, device="cuda"), K)
    B.codes[-1000:] = codes
    last = fl.Mx4(B.codes[-1000:], B.scales[-1000:], K)
    x = torch.randn(20, K, device="cuda").bfloat16()
    for M in (1, 20):
        say("weight past 2^32 bytes", M)
        out = fl.fused_linear_mx4(x[:M], B, act="none")
        tail = fl.fused_linear_mx4(x[:M], last, act="none")
        # other columns share its launch's choices, so sums may be cut another way
        assert torch.allclose(out[:, -1000:].float(), tail.float(), rtol=2 ** -7, atol=1e-3)
        assert (out[:, :-1000] == 0).all()
    say("values past 2^32 elements of rows")
    y = fl.dequantize_mx4(B, torch.bfloat16)
    assert torch.equal(y[-1000:], fl.dequantize_mx4(last, torch.bfloat16)) and (y[:-1000] == 0).all()
    q = fl.quantize_mx4(y)
    one = fl.quantize_mx4(y[-1000:])
    assert torch.equal(q.codes[-1000:], one.codes) and torch.equal(q.scales[-1000:], one.scales)


def test_many_blocks_of_units():
    """More of them than a launch's first dimension takes: rows around its end and the last
    as they are alone."""
    rows, K = 2 ** 27 + 5003, 40
    say("units past the first dimension")
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda").normal_()
    q = fl.quantize_mx4(x)
    y = fl.dequantize_mx4(q, torch.bfloat16)
    for part in (slice(0, 1000), slice(2 ** 27 - 1000, 2 ** 27 + 1000), slice(rows - 1001, rows)):
        codes, scales = quantize64(x[part].cpu())
        assert torch.equal(q.codes[part].cpu(), codes) and torch.equal(q.scales[part].cpu(), scales)
        assert torch.equal(y[part].cpu(), values64(codes, scales, K).bfloat16())
    # every row was written: a value is off by at most half of the largest step, 1, of the scale,
    # and by 2 where it saturates: less than half of the block's largest
    assert bool(((y - x).abs().amax(1) <= x.abs().amax(1) / 2).all())


def test_a_long_output():
    M, N, K = 70_001, 33_000, 64
    a, b = bytes_of(M, K, 1), bytes_of(N, K, 2)
    say("an output past 2^32 bytes")
    out = fl.fused_linear_mx4(mx4(*a, K), mx4(*b, K), act="none", dtype=torch.bfloat16)
    va, vb = values64(*a, K), values64(*b, K)
    for rows in (slice(0, 300), slice(M - 300, M)):
        assert torch.equal(out[rows].cpu(), (va[rows] @ vb.t()).bfloat16())


def test_refusals():
    x = torch.zeros(4, 64, device="cuda")
    B = fl.quantize_mx4(torch.zeros(8, 64, device="cuda"))
    with pytest.raises(ValueError, match="rows of 32 values and B of 64"):
        fl.fused_linear_mx4(x[:, :32].contiguous(), B)
    with pytest.raises(TypeError, match="A has dtype"):
        fl.fused_linear_mx4(x, B, dtype=torch.float16)
    with pytest.raises(TypeError, match="B.codes has dtype"):
        fl.fused_linear_mx4(x, fl.Mx4(B.codes.float(), B.scales, 64))
    with pytest.raises(ValueError, match="B.scales has shape"):
        fl.fused_linear_mx4(x, fl.Mx4(B.codes, B.scales[:, :1].contiguous(), 64))
    with pytest.raises(ValueError, match="B.codes has shape"):
        fl.fused_linear_mx4(x, fl.Mx4(B.codes, B.scales, 65))
    with pytest.raises(ValueError, match="contiguous"):
        fl.quantize_mx4(x.t())
    with pytest.raises(TypeError, match="unsupported dtype"):
        fl.quantize_mx4(x.double())
    with pytest.raises(TypeError, match="unsupported dtype"):
        fl.dequantize_mx4(B, torch.int8)
    with pytest.raises(fl.FusedLinearError, match="needs Y"):
        fl.fused_linear_mx4(x, B, act="glu")
    with pytest.raises(fl.FusedLinearError, match="not aligned to 16"):
        buf = torch.zeros(8 * 32 + 1, dtype=torch.uint8, device="cuda")
        fl.fused_linear_mx4(x, fl.Mx4(buf[1:].view(8, 32), B.scales, 64))
    with pytest.raises(KeyError):
        fl.fused_linear_mx4(x, B, act="tanh")
    with pytest.raises(ValueError, match="out.K"):
        fl.quantize_mx4(x, out=fl.Mx4(B.codes, B.scales, 63))
