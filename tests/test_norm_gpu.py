"""Layer norm and its gradients on the GPU against the 64-bit plain forms."""
import threading

import pytest
import torch

import activation_epilogue_amd as fl
from activation_epilogue_amd import norm
from gpu_util import say
from norm_util import DT, U, backward64, chain, forward64, inside

pytestmark = pytest.mark.gpu


def rows(M, H, dtype, seed, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, H, generator=g) * torch.exp(0.5 * torch.randn(M, 1, generator=g)) + offset
    return (x.to(dtype), (1 + 0.3 * torch.randn(H, generator=g)).to(dtype), (0.3 * torch.randn(H, generator=g)).to(dtype),
            torch.randn(M, H, generator=g).to(dtype), torch.randn(M, H, generator=g).to(dtype))


def guarded(*shape, dtype):
    """(a tensor, the buffer around it): NaN in front and behind, odd to 16 bytes."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 128,), float("nan"), dtype=dtype, device="cuda")
    return buf[33:33 + n].view(*shape), buf


def untouched(buf, n):
    assert torch.isnan(buf[:33]).all() and torch.isnan(buf[33 + n:]).all()


def check(M, H, dtype, seed, affine=True, residual=True, offset=0.0, eps=1e-5):
    dt = DT[dtype]
    x, w, b, dy, res = rows(M, H, dt, seed, offset)
    w, b = (w, b) if affine else (None, None)
    res = res if residual else None
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    say("layer norm", M, H, dtype, affine, residual)
    out, buf = guarded(M, H, dtype=dt)
    y, mean, rstd = fl.layer_norm(dev(x), dev(w), dev(b), eps=eps, out=out, stats=True)
    assert y is out
    untouched(buf, M * H)
    y64, mean64, rstd64, (e_y, e_mean, e_rstd) = forward64(x, w, b, eps)
    inside(y, y64, e_y)
    inside(mean, mean64, e_mean)
    inside(rstd, rstd64, e_rstd)
    assert torch.equal(fl.layer_norm(dev(x), dev(w), dev(b), eps=eps), y)
    say("its gradients")
    out, buf = guarded(M, H, dtype=dt)
    dx, dw, db = fl.layer_norm_bwd(dev(dy), dev(x), mean, rstd, dev(w), R=dev(res), dX=out)
    untouched(buf, M * H)
    dx64, dw64, db64, (e_dx, e_w, e_b) = backward64(dy, x, mean.cpu(), rstd.cpu(), w, res)
    inside(dx, dx64, e_dx)
    inside(dw, dw64, e_w)
    inside(db, db64, e_b)
    only, none, _ = fl.layer_norm_bwd(dev(dy), dev(x), mean, rstd, dev(w), R=dev(res), dweight=False, dbias=None)
    assert none is None and torch.equal(only, dx)
    _, one, none = fl.layer_norm_bwd(dev(dy), dev(x), mean, rstd, dev(w), R=dev(res), dbias=False)
    assert none is None and torch.equal(one, dw)


# every team and its neighbours, whole pieces and ragged ones, one row and more than the blocks take at once
WIDTHS = (1, 2, 7, 8, 9, 31, 64, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000, 1024, 1537, 2048, 2049, 4095, 4096,
          4097, 8191, 8192, 8193, 16383, 16384, 16385, 32768, 32769, 40001)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H", WIDTHS)
def test_widths(H, dtype):
    for M in (1, 5) + ((67,) if H < 20000 else ()):
        check(M, H, dtype, seed=H + M)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,H", [(2, 512), (31, 512), (33, 64), (1025, 96), (2049, 260), (5000, 130), (300, 4096),
                                 (4097, 1537), (9001, 64), (700, 8192)])
def test_rows(M, H, dtype):
    check(M, H, dtype, seed=M)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", [100, 4096, 20000, 40001])
def test_without_weight_or_residual(H, dtype):
    check(9, H, dtype, seed=1, affine=False, residual=False)
    check(9, H, dtype, seed=2, affine=True, residual=False)
    check(9, H, dtype, seed=3, affine=False, residual=True)


@pytest.mark.parametrize("H", [64, 1000, 4096, 40001])
def test_a_mean_far_from_zero(H):
    """Squares of x would lose all of a deviation of 1 at a mean of 4000."""
    check(33, H, "f32", seed=H, offset=4000.0)


def test_one_of_weight_and_bias():
    x, w, b, _, _ = rows(12, 300, torch.float32, 5)
    for ww, bb in ((w, None), (None, b)):
        y = fl.layer_norm(x.cuda(), None if ww is None else ww.cuda(), None if bb is None else bb.cuda())
        y64, _, _, (e_y, _, _) = forward64(x, ww, bb, 1e-5)
        inside(y, y64, e_y)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H", [40, 1000, 4096, 9000, 40001])
def test_values_that_are_not_finite_stay_in_their_row(H, dtype):
    x, w, b, dy, _ = rows(8, H, DT[dtype], 11)
    y0 = fl.layer_norm(x.cuda(), w.cuda(), b.cuda())
    x[2, H // 2], x[5, 0], x[6, H - 1] = float("nan"), float("inf"), float("-inf")
    say("not finite", H, dtype)
    y, mean, rstd = fl.layer_norm(x.cuda(), w.cuda(), b.cuda(), stats=True)
    bad = [2, 5, 6]
    good = [r for r in range(8) if r not in bad]
    assert torch.isnan(y[bad]).all() and torch.equal(y[good], y0[good])
    dx, _, db = fl.layer_norm_bwd(dy.cuda(), x.cuda(), mean, rstd, w.cuda())
    assert torch.isnan(dx[bad]).all() and torch.isfinite(dx[good]).all() and torch.isfinite(db).all()


def test_rows_of_equal_values():
    """Nothing is left of them: the bias; with eps 0 it is 0 * infinity."""
    x, b = torch.full((3, 777), 2.5, device="cuda"), torch.randn(777, device="cuda")
    assert torch.equal(fl.layer_norm(x, None, b), b.expand(3, 777))
    y, mean, rstd = fl.layer_norm(x, eps=0.0, stats=True)
    assert torch.isnan(y).all() and torch.isinf(rstd).all() and (mean == 2.5).all()


@pytest.mark.parametrize("value", [0.1, 33.3, 1000.1, 12345.67, -98765.4])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H", [31, 100, 777, 2048, 4096, 4099, 8192, 16383, 16384, 16385, 32767, 40001])
def test_rows_of_any_equal_value(H, dtype, value):
    """The mean of equal values is that value, to the bit, and nothing is left of them: the bias."""
    dt = DT[dtype]
    if dtype == "f16" and abs(value) > 65504:
        value = -65504.0
    x, b = torch.full((3, H), value, device="cuda", dtype=dt), torch.randn(H, device="cuda").to(dt)
    say("equal values", H, dtype, value)
    y, mean, rstd = fl.layer_norm(x, None, b, stats=True)
    assert torch.equal(mean, x[:, 0].float()) and torch.equal(y, b.expand(3, H))
    # sqrt and the quotient: a rounding each, and one of eps
    assert bool(((rstd.double() * 1e-5 ** 0.5 - 1).abs() <= 3 * U).all())
    y, _, rstd = fl.layer_norm(x, eps=0.0, stats=True)
    assert torch.isnan(y).all() and torch.isinf(rstd).all()


@pytest.mark.parametrize("H", [64, 1000, 4096, 12000, 40001])
@pytest.mark.parametrize("offset", [300.0, -4000.0, 1e6])
def test_the_mean_is_good_to_its_last_bits(H, offset):
    """Of rows far from zero: one rounding, and what the sum of the deviations from a
    first mean (off by far less than they are) is off by: chain(H) roundings, one of each
    deviation, two of its quotient."""
    x, _, _, _, _ = rows(40, H, torch.float32, H, offset)
    say("mean", H, offset)
    _, mean, _ = fl.layer_norm(x.cuda(), stats=True)
    want = x.double().mean(1)
    spread = (x.double() - want[:, None]).abs().mean(1)
    off = (mean.cpu().double() - want).abs()
    assert bool((off <= U * want.abs() + (chain(H) + 4) * U * spread).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H", [31, 64, 100, 128, 200, 1000, 4096, 12000, 16384, 40001])
def test_rows_of_many_kinds_side_by_side(H, dtype):
    """Rows with a mean far from zero beside others, in one wave where rows are short: each as it is alone."""
    x, w, b, _, _ = rows(37, H, DT[dtype], H)
    kind = torch.arange(37) * 7 % 5
    x[kind == 1] += 4000.0
    x[kind == 2] = x[kind == 2][:, :1]
    x[3], x[11, 0] = 0.0, float("nan")
    x, w, b = x.cuda(), w.cuda(), b.cuda()
    say("kinds of rows", H, dtype)
    got = fl.layer_norm(x, w, b, stats=True)
    for r in range(37):
        alone = fl.layer_norm(x[r:r + 1], w, b, stats=True)
        assert all(torch.equal(torch.nan_to_num(p[r:r + 1]), torch.nan_to_num(q)) for p, q in zip(got, alone))
    y64, _, _, (e_y, _, _) = forward64(x.cpu(), w.cpu(), b.cpu(), 1e-5)
    keep = torch.arange(37) != 11
    inside(got[0][keep.cuda()], y64[keep], e_y[keep])
    assert torch.isnan(got[0][11]).all()

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", [64, 1024, 4096, 16384, 65536])
def test_ends_of_the_squares(H, dtype):
    """Deviations of 2^64 / sqrt(H): their squares' sum is infinite, the row its bias, its gradient the path around
    it.  Half of them, and the smallest that have squares: as any."""
    dt = DT[dtype]
    signs = torch.ones(H)
    signs[1::2] = -1.0
    most = 2.0 ** 64 / H ** 0.5
    x = torch.stack([signs * most, signs * most / 2, signs * 2.0 ** -60, signs * 2.0 ** -76, signs * 2.0 ** 127]).to(dt).cuda()
    g = torch.Generator().manual_seed(H)
    b, dy, R = (torch.randn(*s, generator=g).to(dt).cuda() for s in ((H,), x.shape, x.shape))
    say("ends of the squares", H, dtype)
    y, mean, rstd = fl.layer_norm(x, None, b, eps=0.0, stats=True)
    assert (mean == 0).all() and rstd.tolist() == [0.0, 2 / most, 2.0 ** 60, float("inf"), 0.0]
    hat = signs.cuda()
    assert torch.equal(y[0], b) and torch.equal(y[4], b)
    assert torch.equal(y[1], (hat + b.float()).to(dt)) and torch.equal(y[2], y[1])
    assert torch.isinf(y[3]).all()
    dx, _, _ = fl.layer_norm_bwd(dy, x, mean, rstd, R=R)
    assert torch.equal(dx[0], R[0]) and torch.equal(dx[4], R[4])
    only = fl.layer_norm_bwd(dy, x, mean, rstd, dweight=False, dbias=False)[0]
    assert (only[0] == 0).all() and torch.isfinite(only[1:3]).all()
    far = torch.full((2, H), torch.finfo(dt).max, dtype=dt, device="cuda")
    far[1] = 1.0
    y = fl.layer_norm(far, None, b)
    assert torch.isnan(y[0]).all() and torch.equal(y[1], b)


@pytest.mark.parametrize("M,H", [(0, 100), (3, 0), (0, 0)])
def test_nothing(M, H):
    x = torch.zeros(M, H, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(H, device="cuda", dtype=torch.bfloat16)
    y, mean, rstd = fl.layer_norm(x, w, w, stats=True)
    assert y.shape == (M, H)
    mean.zero_(), rstd.zero_()
    dw = torch.full((H,), 3.0, device="cuda")
    dx, dw, db = fl.layer_norm_bwd(x, x, mean, rstd, w, dweight=dw)
    assert dx.shape == (M, H) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("H", [65, 4096, 40001])
def test_in_place(H):
    x, w, b, dy, res = (t.cuda() for t in rows(20, H, torch.bfloat16, 3))
    y, mean, rstd = fl.layer_norm(x, w, b, stats=True)
    z = x.clone()
    assert fl.layer_norm(z, w, b, out=z) is z and torch.equal(z, y)
    want = fl.layer_norm_bwd(dy, x, mean, rstd, w, R=res)
    for name in ("dout", "X", "R"):
        args = {"dout": dy.clone(), "X": x.clone(), "R": res.clone()}
        got = fl.layer_norm_bwd(args["dout"], args["X"], mean, rstd, w, R=args["R"], dX=args[name])
        assert got[0] is args[name] and all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 5, 100, 3000])
@pytest.mark.parametrize("H", [5, 64, 216, 217, 1000, 1725, 4099, 9001, 16385, 33001])
def test_sums_where_they_belong(H, M, dtype):
    """The weight's and bias's gradients at any address of a float, nothing around them, and each alone."""
    if M * H > 2 ** 24:
        M = 300
    dt = DT[dtype]
    x, w, _, dy, _ = rows(M, H, dt, H)
    x, w, dy = x.cuda(), w.cuda(), dy.cuda()
    say("gradients' places", M, H, dtype)
    _, mean, rstd = fl.layer_norm(x, w, stats=True)
    (dw, wbuf), (db, bbuf) = guarded(H, dtype=torch.float32), guarded(H, dtype=torch.float32)
    fl.layer_norm_bwd(dy, x, mean, rstd, w, dweight=dw, dbias=db)
    untouched(wbuf, H)
    untouched(bbuf, H)
    _, dw64, db64, (_, e_w, e_b) = backward64(dy.cpu(), x.cpu(), mean.cpu(), rstd.cpu(), w.cpu(), None)
    inside(dw, dw64, e_w)
    inside(db, db64, e_b)
    _, one, none = fl.layer_norm_bwd(dy, x, mean, rstd, w, dbias=False)
    assert none is None and torch.equal(one, dw)
    _, none, one = fl.layer_norm_bwd(dy, x, mean, rstd, w, dweight=False)
    assert none is None and torch.equal(one, db)


def test_gradients_against_differences():
    """The loss sum(dy * y): its slope along each direction, by differences in
    64 bits of the formula, is what the gradients say."""
    M, H, eps = 6, 50, 1e-3
    x, w, b, dy, _ = rows(M, H, torch.float32, 17)
    y, mean, rstd = fl.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=eps, stats=True)
    dx, dw, db = (t.cpu().double() for t in fl.layer_norm_bwd(dy.cuda(), x.cuda(), mean, rstd, w.cuda()))

    def loss(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return float((dy.double() * (d * ((d * d).mean(1, keepdim=True) + eps) ** -0.5 * w + b)).sum())
    x, w, b = x.double(), w.double(), b.double()
    g = torch.Generator().manual_seed(1)
    h = 1e-4  # a central difference is off by h^2 of the third derivative, and 2^-52 of the loss over h
    for at, grad in ((0, dx), (1, dw), (2, db)):
        for _ in range(5):
            v = torch.randn(grad.shape, generator=g, dtype=torch.float64)
            up, down = [x, w, b], [x, w, b]
            up[at], down[at] = up[at] + h * v, down[at] - h * v
            slope = (loss(*up) - loss(*down)) / (2 * h)
            # fp32 gradients: 300 terms of size |grad * v|, each good to 100 roundings
            room = 100 * 2.0 ** -24 * float((grad * v).abs().sum()) + 1e-4
            assert abs(slope - float((grad * v).sum())) <= room


def test_the_same_bits_again_and_on_another_stream():
    x, w, b, dy, res = (t.cuda() for t in rows(3001, 1537, torch.bfloat16, 9))
    y, mean, rstd = fl.layer_norm(x, w, b, stats=True)
    first = fl.layer_norm_bwd(dy, x, mean, rstd, w, R=res)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = fl.layer_norm(x, w, b, stats=True, stream=s) + fl.layer_norm_bwd(dy, x, mean, rstd, w, R=res, stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((y, mean, rstd, *first), again))


def test_two_threads_two_streams():
    """Forward and backward passes of two shapes, from two host threads at the same time."""
    jobs = []
    for M, H, dt in ((3001, 1537, torch.bfloat16), (515, 12000, torch.float32)):
        x, w, b, dy, res = (t.cuda() for t in rows(M, H, dt, M))
        f = fl.layer_norm(x, w, b, stats=True)
        jobs.append(((x, w, b, dy, res), (*f, *fl.layer_norm_bwd(dy, x, f[1], f[2], w, R=res))))
    torch.cuda.synchronize()
    got, errors, start = [[], []], [], threading.Barrier(2)

    def work(i):
        try:
            x, w, b, dy, res = jobs[i][0]
            stream = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    f = fl.layer_norm(x, w, b, stats=True)
                    got[i].append((*f, *fl.layer_norm_bwd(dy, x, f[1], f[2], w, R=res)))
                    with pytest.raises(fl.FusedLinearError, match="eps"):  # a message of the thread's own
                        fl.layer_norm(x, eps=-1.0)
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
    for (_, want), each in zip(jobs, got):
        assert len(each) == 20 and all(torch.equal(p, q) for g in each for p, q in zip(g, want))

def test_workspace():
    M, H = 3001, 1537
    x, w, b, dy, _ = (t.cuda() for t in rows(M, H, torch.float16, 9))
    _, mean, rstd = fl.layer_norm(x, w, b, stats=True)
    need = fl.layer_norm_bwd_workspace_bytes(M, H, torch.float16)
    assert need > 0
    buf = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    got = fl.layer_norm_bwd(dy, x, mean, rstd, w, workspace=buf[:need])
    assert (buf[need:] == 255).all()
    assert all(torch.equal(p, q) for p, q in zip(got, fl.layer_norm_bwd(dy, x, mean, rstd, w)))
    with pytest.raises(fl.FusedLinearError, match="needed"):
        fl.layer_norm_bwd(dy, x, mean, rstd, w, workspace=buf[:need - 1])


@pytest.mark.parametrize("H", [200, 4096, 16384, 16385, 40001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_workspace_without_sums(H, dtype):
    """dX alone: what its rows need and no more, at the end of a page of the caller's."""
    M, dt = 700 if H < 20000 else 33, DT[dtype]
    x, w, _, dy, _ = (t.cuda() for t in rows(M, H, dt, 9))
    _, mean, rstd = fl.layer_norm(x, w, stats=True)
    want = fl.layer_norm_bwd(dy, x, mean, rstd, w)[0]
    need = 8 * M if H > 16384 else 0
    say("dX alone", M, H, dtype)
    buf = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(x)
    call = lambda nbytes: norm._lib().fl_layer_norm_bwd(  # noqa: E731
        dy.data_ptr(), x.data_ptr(), w.data_ptr(), mean.data_ptr(), rstd.data_ptr(), None, dx.data_ptr(), None, None, M, H,
        {"f32": 0, "bf16": 2}[dtype], buf.data_ptr() if nbytes else None, nbytes, torch.cuda.current_stream().cuda_stream)
    assert call(need) == 0
    assert torch.equal(dx, want) and (buf[need:] == 255).all()
    if need:
        assert call(need - 1) == 1
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    fl.layer_norm_bwd(dy, x, mean, rstd, w, dX=dx, dweight=False, dbias=False)
    assert torch.cuda.max_memory_allocated() - before <= need + 512  # the allocator's step


def test_captured_and_replayed():
    """A block's norm forward and backward in a graph, with new inputs and eager
    work between the replays."""
    M, H = 515, 2050
    x, w, b, dy, res = (t.cuda() for t in rows(M, H, torch.bfloat16, 21))
    ws = torch.empty(norm.layer_norm_bwd_workspace_bytes(M, H, torch.bfloat16), dtype=torch.uint8, device="cuda")
    kept = {}

    def work():
        kept["f"] = fl.layer_norm(x, w, b, stats=True)
        kept["b"] = fl.layer_norm_bwd(dy, x, kept["f"][1], kept["f"][2], w, R=res, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for seed in range(3):
        for t, new in zip((x, w, b, dy, res), rows(M, H, torch.bfloat16, 30 + seed)):
            t.copy_(new)
        f = fl.layer_norm(x, w, b, stats=True)
        want = (*f, *fl.layer_norm_bwd(dy, x, f[1], f[2], w, R=res))
        for t in (*kept["f"], *kept["b"]):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((*kept["f"], *kept["b"]), want))


def test_offsets_past_32_bits():
    """More than 2^32 bytes of rows, the last of them as the same rows alone."""
    M, H = 600_011, 4096
    x = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    x[:1000].normal_()
    x[1000:-1000] = 1.0
    x[-1000:].normal_()
    say("layer norm past 2^32 bytes")
    y, mean, rstd = fl.layer_norm(x, stats=True)
    tail = fl.layer_norm(x[-1000:], stats=True)
    assert torch.equal(y[-1000:], tail[0]) and torch.equal(mean[-1000:], tail[1])
    dy = y.clone()
    dx, _, db = fl.layer_norm_bwd(dy, x, mean, rstd)
    assert torch.equal(dx[-1000:], fl.layer_norm_bwd(dy[-1000:], x[-1000:], mean[-1000:], rstd[-1000:])[0])
    assert torch.isfinite(db).all()


@pytest.mark.parametrize("dtype,H", [("f32", 2052), ("bf16", 4104)])
def test_more_rows_than_blocks(dtype, H):
    """Blocks that go from row to row, a row to each at once: rows on both sides of the launch's 2^20 blocks."""
    M, dt = 2 ** 20 + 3001, DT[dtype]
    x = torch.empty(M, H, dtype=dt, device="cuda").normal_()
    x[::3] += 100.0
    say("more rows than blocks", M, H, dtype)
    y, mean, rstd = fl.layer_norm(x, stats=True)
    dx, _, _ = fl.layer_norm_bwd(y, x, mean, rstd, dweight=False, dbias=False)
    for part in (slice(0, 300), slice(2 ** 20 - 300, 2 ** 20 + 300), slice(M - 300, M)):
        xs, ys = x[part].cpu(), y[part].cpu()
        y64, mean64, rstd64, (e_y, e_mean, e_rstd) = forward64(xs, None, None, 1e-5)
        inside(ys, y64, e_y)
        inside(mean[part], mean64, e_mean)
        inside(rstd[part], rstd64, e_rstd)
        dx64, _, _, (e_dx, _, _) = backward64(ys, xs, mean[part].cpu(), rstd[part].cpu(), None, None)
        inside(dx[part], dx64, e_dx)

@pytest.mark.parametrize("H", [2 ** 25 + 40, 2 ** 27 + 40])
def test_sums_of_very_long_rows(H):
    """More columns than one dimension of the join's launch takes; sums of small whole numbers, exact."""
    M = 4
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dy = (torch.randint(-4, 5, (M, H), generator=g, device="cuda", dtype=torch.int8).bfloat16() for _ in range(2))
    zero, one = torch.zeros(M, device="cuda"), torch.ones(M, device="cuda")
    say("sums of rows of", H)
    (dw, wbuf), (db, bbuf) = guarded(H, dtype=torch.float32), guarded(H, dtype=torch.float32)
    fl.layer_norm_bwd(dy, x, zero, one, dweight=dw, dbias=db)
    want = torch.zeros(H, device="cuda")
    for r in range(M):
        want += dy[r].float() * x[r].float()
    assert torch.equal(dw, want) and torch.equal(db, dy.float().sum(0))
    untouched(wbuf, H)
    untouched(bbuf, H)


def test_refusals():
    x = torch.zeros(4, 8, device="cuda")
    one = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="matrix"):
        fl.layer_norm(one)
    with pytest.raises(TypeError, match="unsupported dtype"):
        fl.layer_norm(x.double())
    with pytest.raises(ValueError, match="contiguous"):
        fl.layer_norm(x.t())
    with pytest.raises(TypeError, match="weight has dtype"):
        fl.layer_norm(x, torch.zeros(8, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError, match="bias has shape"):
        fl.layer_norm(x, None, torch.zeros(9, device="cuda"))
    with pytest.raises(ValueError, match="device"):
        fl.layer_norm(torch.zeros(4, 8))
    with pytest.raises(ValueError, match="stats"):
        fl.layer_norm(x, mean=one)
    with pytest.raises(fl.FusedLinearError, match="eps"):
        fl.layer_norm(x, eps=-1.0)
    with pytest.raises(ValueError, match="mean has shape"):
        fl.layer_norm_bwd(x, x, one[:3], one)
    with pytest.raises(fl.FusedLinearError, match="mean is NULL"):
        fl.layer_norm_bwd(x, x, None, one)
