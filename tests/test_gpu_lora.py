"""The shared projection with low-rank adapters (moe_lora_linear) against its
formula in 64 bits, from the same bf16 inputs.

Bar of y, with |.| the sums of magnitudes: one bf16 rounding of y (2^-9, taken
as 2^-8 |y|); fp32 accumulation of K terms on the tensor cores, (K + 2) 2^-22
sum |x w|, and of the adapter's, (rank + 2) 2^-22 sum |u b|; u itself is rounded
to bf16 (2^-8 |u|) after (K + 2) 2^-22 s sum |x a|, both carried through |b|."""
from __future__ import annotations

import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from gpu_common import Guarded, require_gpu

pytestmark = pytest.mark.gpu
A22 = 2.0 ** -22


def bf16(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(torch.bfloat16).cuda()


def ids_of(T, A, mix, seed=0):
    g = torch.Generator().manual_seed(seed)
    if mix == "tokens":
        i = torch.randint(-1, A, (T,), generator=g)
    elif mix == "none":
        i = torch.full((T,), -1)
    elif mix == "one":
        i = torch.full((T,), A - 1)
    else:  # runs of tokens
        i = torch.randint(-1, A, (T,), generator=g)[(torch.rand(T, generator=g) < 0.02).int().cumsum(0)]
    return i.to(torch.int32).cuda()


def reference(x, w, la, lb, sc, ids):
    """y and its bar, in 64 bits."""
    x, w = x.double(), w.double()
    K = x.shape[1]
    y, bar = x @ w.t(), (K + 2) * A22 * (x.abs() @ w.abs().t())
    for a in range(la.shape[0] if la is not None else 0):
        t = (ids == a).nonzero().view(-1)
        if not t.numel():
            continue
        s = float(sc[a]) if sc is not None else 1.0
        aa, bb = la[a].double(), lb[a].double()
        u = s * (x[t] @ aa.t())
        du = 2.0 ** -8 * u.abs() + (K + 2) * A22 * abs(s) * (x[t].abs() @ aa.abs().t())
        y[t] += u @ bb.t()
        bar[t] += du @ bb.abs().t() + (aa.shape[0] + 2) * A22 * ((u.abs() + du) @ bb.abs().t())
    return y, bar + 2.0 ** -8 * y.abs()


def run(x, w, la, lb, sc, ids, num_sms=0, stream=None):
    T, K = x.shape
    N = w.shape[0]
    A, r = (la.shape[0], la.shape[1]) if la is not None else (0, 0)
    d = B.MoeLoraDesc(T, K, N, r, A, num_sms)
    y = Guarded((T, N), torch.bfloat16, "cuda:0")
    u = Guarded((T, r), torch.bfloat16, "cuda:0") if A else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    torch.cuda.synchronize()
    B.moe_lora_linear(d, x, w, la, lb, sc, ids, u.t if A else None, y.t, err, stream=stream)
    if stream is not None:
        stream.synchronize()
    status = B.moe_get_error(err)
    assert y.guards_intact() and (u is None or u.guards_intact())
    return y.t, status


def check(T, K, N, r, A, mix, seed=0, scales=True, num_sms=0):
    require_gpu()
    x, w = bf16((T, K), seed), bf16((N, K), seed + 1, K ** -0.5)
    la, lb = bf16((A, r, K), seed + 2, K ** -0.5), bf16((A, N, r), seed + 3, r ** -0.5)
    sc = torch.rand(A, generator=torch.Generator().manual_seed(seed + 4)).add(0.25).cuda() if scales else None
    ids = ids_of(T, A, mix, seed)
    y, status = run(x, w, la, lb, sc, ids, num_sms)
    assert status == B.MOE_OK
    want, bar = reference(x, w, la, lb, sc, ids)
    assert bool(((y.double() - want).abs() <= bar).all())
    return x, w, la, lb, sc, ids, y


@pytest.mark.parametrize("mix", ["tokens", "runs"])
@pytest.mark.parametrize("T,K,N,r,A", [
    (1, 512, 512, 8, 1), (1, 4096, 4096, 16, 8), (2, 8, 8, 8, 3), (5, 72, 136, 24, 2), (31, 1000, 264, 64, 40),
    (64, 7168, 2048, 16, 32), (65, 200, 520, 40, 5), (127, 640, 384, 128, 7), (128, 512, 256, 256, 4),
    (129, 512, 256, 8, 200), (300, 328, 1032, 72, 9), (389, 2056, 4104, 24, 12), (513, 128, 4096, 16, 3),
    (200, 136, 264, 256, 5), (260, 1032, 72, 128, 30), (1000, 64, 128, 8, 1000), (16, 4096, 14336, 32, 3),
])
def test_against_the_formula(T, K, N, r, A, mix):
    check(T, K, N, r, A, mix)


@pytest.mark.parametrize("T,K,N,r,A,mix", [(2048, 512, 5128, 64, 16, "runs"), (1500, 264, 8192, 16, 128, "tokens"),
                                           (4096, 192, 2048, 136, 3, "runs"), (700, 64, 16384, 8, 2, "one")])
def test_many_tiles(T, K, N, r, A, mix):
    """Enough tiles that CTAs walk several, with both accumulators and both adapter lists in turn."""
    check(T, K, N, r, A, mix)


@pytest.mark.parametrize("T,K,N,r,A,mix", [
    (100, 16392, 264, 16, 1, "one"), (128, 8200, 72, 8, 2, "tokens"), (17, 12288, 136, 40, 3, "one"),
    (128, 4104, 520, 32, 128, "tokens"), (9, 40, 72, 24, 9, "tokens"), (33, 4096, 8, 256, 2, "one"),
    (256, 1024, 2048, 16, 8, "runs"), (1000, 4096, 1024, 24, 5, "runs"), (389, 7168, 2048, 48, 6, "tokens"),
    (700, 2056, 1032, 32, 20, "tokens"), (16, 2048, 4104, 16, 4, "tokens"), (60, 1024, 7168, 8, 60, "tokens"),
    (20, 520, 136, 16, 300, "tokens"), (20, 520, 136, 40, 21, "one"), (100, 264, 72, 8, 101, "tokens"),
    (31, 16392, 264, 16, 2, "one"), (64, 4104, 72, 40, 16, "one"), (63, 12296, 136, 8, 70, "one"), (64, 2056, 72, 256, 20, "tokens"),
])
def test_long_rows_and_every_split(T, K, N, r, A, mix):
    """Rows whose pieces take several rounds of loads and tokens that take several passes; shapes at which a tile's K
    is taken by one, two and four CTAs."""
    check(T, K, N, r, A, mix)


@pytest.mark.parametrize("mix", ["one", "none"])
@pytest.mark.parametrize("K,N,r,A", [(8, 8, 8, 1), (520, 4872, 24, 3), (2056, 8, 256, 2), (4104, 4112, 64, 5),
                                     (264, 40008, 8, 4), (16400, 72, 136, 2)])
def test_one_token(K, N, r, A, mix):
    check(1, K, N, r, A, mix)


@pytest.mark.parametrize("mix", ["none", "one"])
@pytest.mark.parametrize("T", [3, 200, 2000])
def test_no_and_one_adapter_in_use(T, mix):
    check(T, 256, 1024, 16, 6, mix)


def test_scales_are_optional():
    check(70, 256, 264, 32, 4, "tokens", scales=False)


@pytest.mark.parametrize("num_sms", [1, 7, 64])
def test_fewer_sms(num_sms):
    check(300, 264, 520, 24, 5, "tokens", num_sms=num_sms)


@pytest.mark.parametrize("T", [1, 100, 3000])
def test_projection_alone(T):
    require_gpu()
    x, w = bf16((T, 320), 1), bf16((648, 320), 2, 320 ** -0.5)
    y, status = run(x, w, None, None, None, None)
    want, bar = reference(x, w, None, None, None, None)
    assert status == B.MOE_OK and bool(((y.double() - want).abs() <= bar).all())


def test_rows_do_not_see_other_rows_or_other_adapters():
    """NaN and infinite rows, and adapters that no token uses, stay out of every other token's result."""
    require_gpu()
    T, K, N, r, A = 150, 256, 264, 16, 4
    x, w = bf16((T, K), 1), bf16((N, K), 2, K ** -0.5)
    la, lb = bf16((A, r, K), 3, K ** -0.5), bf16((A, N, r), 4, r ** -0.5)
    ids = ids_of(T, 3, "tokens", 5)  # adapter 3 is not used
    clean, _ = run(x, w, la, lb, None, ids)
    la2, lb2, x2 = la.clone(), lb.clone(), x.clone()
    la2[3], lb2[3] = float("nan"), float("inf")
    x2[7], x2[140] = float("nan"), float("inf")
    y, status = run(x2, w, la2, lb2, None, ids)
    keep = torch.ones(T, dtype=torch.bool, device="cuda:0")
    keep[7] = keep[140] = False
    assert status == B.MOE_OK and torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[7]).all()) and not bool(torch.isfinite(y[140]).any())


def test_a_token_without_an_adapter_gets_the_projection_alone():
    require_gpu()
    T, K, N, r, A = 40, 256, 264, 16, 4
    x, w = bf16((T, K), 1), bf16((N, K), 2, K ** -0.5)
    la, lb = bf16((A, r, K), 3), bf16((A, N, r), 4)
    y, _ = run(x, w, la, lb, None, torch.full((T,), -1, dtype=torch.int32, device="cuda:0"))
    alone, _ = run(x, w, None, None, None, None)
    assert torch.equal(y, alone)


def test_invalid_adapter_ids_are_reported_and_taken_as_none():
    require_gpu()
    T, K, N, r, A = 200, 128, 264, 16, 4
    x, w = bf16((T, K), 1), bf16((N, K), 2, K ** -0.5)
    la, lb = bf16((A, r, K), 3, K ** -0.5), bf16((A, N, r), 4, r ** -0.5)
    ids = ids_of(T, A, "tokens", 6)
    bad = ids.clone()
    ids[[0, 50, 199]] = -1
    bad[0], bad[50], bad[199] = 4, -2, 2 ** 31 - 1
    good, status = run(x, w, la, lb, None, ids)
    assert status == B.MOE_OK
    y, status = run(x, w, la, lb, None, bad)
    assert status == B.MOE_EINVAL and torch.equal(y, good)


def test_same_results_every_time_on_another_stream_and_in_a_graph():
    require_gpu()
    for T, N in ((33, 512), (300, 520), (2500, 2048)):
        x, w, la, lb, sc, ids, y = check(T, 520, N, 24, 6, "runs")
        assert torch.equal(run(x, w, la, lb, sc, ids)[0], y)
        assert torch.equal(run(x, w, la, lb, sc, ids, stream=torch.cuda.Stream())[0], y)
        d = B.MoeLoraDesc(T, 520, N, 24, 6, 0)
        u = torch.empty((T, 24), dtype=torch.bfloat16, device="cuda:0")
        out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda:0")
        err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
        src = torch.zeros_like(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.moe_lora_linear(d, src, w, la, lb, sc, ids, u, out, err)
            B.moe_lora_linear(d, src, w, la, lb, sc, ids, u, out, err)
        src.copy_(x)
        graph.replay()
        assert B.moe_get_error(err) == B.MOE_OK and torch.equal(out, y)


def test_input_written_by_the_kernel_before():
    """x and the ids come from kernels enqueued immediately before the call, again and again."""
    require_gpu()
    T, K, N, r, A = 96, 2048, 1024, 16, 8
    w, la, lb = bf16((N, K), 2, K ** -0.5), bf16((A, r, K), 3, K ** -0.5), bf16((A, N, r), 4, r ** -0.5)
    xs = [bf16((T, K), 20 + i) for i in range(6)]
    idl = [ids_of(T, A, "tokens", 30 + i) for i in range(6)]
    want = [run(a, w, la, lb, None, b)[0].clone() for a, b in zip(xs, idl)]
    d = B.MoeLoraDesc(T, K, N, r, A, 0)
    x, ids = torch.empty_like(xs[0]), torch.empty_like(idl[0])
    u = torch.empty((T, r), dtype=torch.bfloat16, device="cuda:0")
    ys = [torch.empty((T, N), dtype=torch.bfloat16, device="cuda:0") for _ in xs]
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    for a, b, y in zip(xs, idl, ys):
        ids.copy_(b)
        torch.mul(a, 1.0, out=x)
        B.moe_lora_linear(d, x, w, la, lb, None, ids, u, y, err)
    assert B.moe_get_error(err) == B.MOE_OK
    assert all(torch.equal(a, b) for a, b in zip(ys, want))
