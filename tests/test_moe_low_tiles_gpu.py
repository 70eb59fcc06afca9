"""Low tiles of the experts' products where a run has one of them and where it
has several (which read the weights by different ways), forward and backward,
against 64-bit products on the GPU."""
import math

import pytest
import torch

import activation_epilogue_amd as fl
from gpu_util import say
from moe_util import DT, U32, unit

pytestmark = pytest.mark.gpu

# rows of every expert, K, N
RUNS = [
    ([500, 500], 4096, 1024), ([300], 4096, 4096), ([3] * 64, 2048, 1408), ([1, 0, 40, 31, 0, 16], 1030, 515),
    ([200, 0, 1, 7], 1029, 257), ([32] * 8, 512, 4096), ([33] * 8, 512, 4096), ([700], 2048, 64), ([150, 130], 8192, 512),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", range(len(RUNS)))
def test_low_tiles(case, dtype):
    counts, K, N = RUNS[case]
    dt, E, S = DT[dtype], len(counts), sum(counts)
    g = torch.Generator(device="cuda").manual_seed(case)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    def check(got, a, b, what):
        ref, bound = a @ b, (a.shape[1] + 20) * U32 * (a.abs() @ b.abs())
        allow = bound * (1 + unit(dt)) + unit(dt) * ref.abs() + (2.0 ** -25 if dt == torch.float16 else 2.0 ** -134)
        off = (got.double() - ref).abs()
        assert bool(torch.isfinite(got).all()) and bool((off <= allow).all()), (what, float((off / allow).max()))
    A, B, W, G = normal(S, K), normal(E, K, N, std=K ** -0.5), normal(E, N, K, std=K ** -0.5), normal(S, K)
    index = torch.randperm(S, generator=g, device="cuda").to(torch.int32)
    o = [0]
    for c in counts:
        o.append(o[-1] + c)
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    say("low tiles", counts[:6], K, N, dtype)
    out, mixed, dX = (torch.full((S, N), math.nan, dtype=dt, device="cuda") for _ in range(3))
    fl.grouped_linear(A, B, offsets, act="none", out=out)
    fl.grouped_linear(A, B, offsets, act="none", out=mixed, index=index)
    fl.grouped_linear_bwd(G, W, None, offsets, act="none", dX=dX)
    for e in range(E):
        s = slice(o[e], o[e + 1])
        b, w = B[e].double(), W[e].double().t().contiguous()
        check(out[s], A[s].double(), b, "forward")
        check(mixed[s], A[index[s].long()].double(), b, "indexed")
        check(dX[s], G[s].double(), w, "backward")
