"""The token sort and its way back (moe_sort, moe_sort_grad, moe_unsort,
moe_unsort_grad) against numpy.

Offsets, the forward map and the packed rows are exact. Bars of the sums, with
u = 2^-24: k terms in fp32 then one bf16 rounding (2^-9 of the result, taken as
2^-8) leave 2^-8 |sum| + (k + 1) u sum |term|; a product rounded to fp32 and
then to bf16 stays within 2^-8 of itself; a dot product over H with at most
H / 256 + 8 terms in a row per thread and 13 additions across threads is within
(H / 256 + 24) u sum |term| (H <= 8192: rows of one CTA of 256 threads, or of
fewer with at most 8 elements each; bounded here by (H / 32 + 24) u)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from combine_moe_layout_gb300 import pipeline as P
from combine_moe_layout_gb300 import workloads as wl
from gpu_common import POISON_BYTE, Guarded, require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DTYPE = {"bf16": B.MOE_BF16, "fp8": B.MOE_FP8_E4M3, "bf16q": B.MOE_BF16_TO_FP8}


def make(R, T, H, E, k, dtype="bf16"):
    return B.MoeDesc(R, T, H, E, k, max(T, 1), DTYPE[dtype], 0)


def choices(R, T, E, k, seed, masked=0.0, repeat=False):
    rng = np.random.default_rng(seed)
    n = R * T
    if repeat:
        idx = rng.integers(0, E, size=(n, k))
    else:
        idx = np.argsort(rng.random((n, E)), axis=1)[:, :k]
    idx = idx.astype(np.int32)
    if masked:
        idx[rng.random((n, k)) < masked] = -1
        idx[rng.random(n) < 0.1] = -1
    return idx


def plain_order(idx, R, E):
    """tok_packed, region offsets and (expert, token, choice) of every packed row, by counting."""
    n, k = idx.shape
    T = n // R if R else 0
    at = sorted(((int(idx[t, j]), t, j) for t in range(n) for j in range(k) if 0 <= idx[t, j] < E))
    tok = np.full((n, k), -1, dtype=np.int32)
    counts = np.zeros(E * R, dtype=np.int64)
    for p, (e, t, j) in enumerate(at):
        tok[t, j] = p
        counts[e * R + t // T] += 1
    return tok, np.concatenate([[0], np.cumsum(counts)]), at


def bf16(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def run_sort(d, idx, x, scales=None):
    R, T, H, E, k = d.num_ranks, d.tokens_per_rank, d.hidden, d.num_experts, d.topk
    n = R * T * k
    row = 2 * H if d.dtype == B.MOE_BF16 else H
    off = Guarded((E * R + 1,), torch.int32, "cuda:0")
    px = Guarded((n, row), torch.uint8, "cuda:0", POISON_BYTE)
    ps = Guarded((n, H // 128), torch.float32, "cuda:0", -7.0) if d.dtype != B.MOE_BF16 else None
    tok = Guarded((R * T, k), torch.int32, "cuda:0")
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    B.moe_sort(d, torch.from_numpy(idx).cuda(), x, scales, off.t, px.t, ps.t if ps else None, tok.t, err)
    status = B.moe_get_error(err)
    for g in (off, px, ps, tok):
        assert g is None or g.guards_intact()
    return off.t, px.t, ps.t if ps else None, tok.t, status


SHAPES = [  # R, T, H, E, k, masked
    (1, 1, 8, 1, 1, 0.0), (1, 1, 7168, 256, 8, 0.0), (2, 16, 128, 8, 2, 0.0), (1, 333, 1000, 12, 3, 0.2),
    (4, 37, 264, 60, 6, 0.5), (1, 700, 2056, 8, 8, 0.0), (3, 1, 16, 3, 3, 0.0), (1, 5000, 24, 16, 5, 0.1),
    (64, 9, 40, 64, 4, 0.3), (1, 40, 4104, 8192, 2, 0.0), (1, 3000, 64, 1000, 16, 0.05),
]


@pytest.mark.parametrize("R,T,H,E,k,masked", SHAPES)
def test_sort_bf16(R, T, H, E, k, masked):
    require_gpu()
    d = make(R, T, H, E, k)
    idx = choices(R, T, E, k, R + T, masked)
    x = bf16((R * T, H), 1)
    off, px, _, tok, status = run_sort(d, idx, x)
    assert status == B.MOE_OK
    t_ref, o_ref, at = plain_order(idx, R, E)
    assert np.array_equal(off.cpu().numpy(), o_ref)
    assert np.array_equal(tok.cpu().numpy(), t_ref)
    m = len(at)
    src = torch.tensor([t for _, t, _ in at], dtype=torch.int64, device="cuda:0")
    assert torch.equal(px[:m], x.view(torch.uint8)[src])
    assert bool((px[m:] == POISON_BYTE).all()), "a row at or above the total was written"


@pytest.mark.parametrize("dtype", ["fp8", "bf16q"])
@pytest.mark.parametrize("R,T,H,E,k,masked", [(1, 1, 128, 4, 2, 0.0), (8, 16, 7168, 256, 8, 0.0), (2, 101, 384, 24, 3, 0.3),
                                              (1, 600, 896, 8, 4, 0.1)])
def test_sort_matches_the_dispatch_path(R, T, H, E, k, masked, dtype):
    """The same packed rows, scales, offsets and map as layout, dispatch and the receive hook give."""
    require_gpu()
    w = wl.custom("sort_" + dtype, num_ranks=R, tokens_per_rank=T, hidden=H, num_experts=R * max(1, E // R), topk=k,
                  max_m=T, dtype=dtype, expert="scale", x_dist="normal")
    inp = wl.make_inputs(w)
    if masked:
        inp = wl.mask_choices(inp, masked)
    step = P.MoeStep(w, "cuda:0")
    dev = P.to_device(inp, "cuda:0")
    step.reset()
    step.layout(dev)
    step.dispatch(dev)
    packed = B.allocate_packed(step.desc, "cuda:0")
    step.recv(packed)
    assert step.error() == B.MOE_OK
    off, px, ps, tok, status = run_sort(step.desc, inp.topk_idx.reshape(R * T, k), dev.x, dev.x_scales)
    assert status == B.MOE_OK
    m = int(off[-1])
    assert torch.equal(off, packed.region_offsets)
    assert torch.equal(tok.view(-1), packed.tok_packed.view(-1))
    assert torch.equal(px[:m], packed.packed_x[:m])
    assert torch.equal(ps[:m], packed.packed_scales[:m])
    assert bool((px[m:] == POISON_BYTE).all()) and bool((ps[m:] == -7.0).all())


@pytest.mark.parametrize("R,T,E,k,masked", [(7, 1111, 301, 7, 0.1), (32, 61, 8192, 5, 0.0), (1, 40000, 2, 1, 0.3),
                                            (33, 3, 33, 4, 0.0), (3, 171, 258, 1, 0.0)])
def test_ranking_of_many_choices(R, T, E, k, masked):
    """As many CTAs as a cluster takes, source ranks that begin inside a group of 32 choices, experts of 1 to 13 bits."""
    require_gpu()
    idx = choices(R, T, E, k, E + T, masked)
    off, _, _, tok, status = run_sort(make(R, T, 8, E, k), idx, bf16((R * T, 8), 3))
    t_ref, o_ref, _ = plain_order(idx, R, E)
    assert status == B.MOE_OK
    assert np.array_equal(tok.cpu().numpy(), t_ref) and np.array_equal(off.cpu().numpy(), o_ref)


def test_sort_repeated_experts_keep_choice_order():
    require_gpu()
    d = make(2, 50, 32, 6, 6)
    idx = choices(2, 50, 6, 6, 3, 0.1, repeat=True)
    off, _, _, tok, status = run_sort(d, idx, bf16((100, 32), 2))
    t_ref, o_ref, _ = plain_order(idx, 2, 6)
    assert status == B.MOE_OK
    assert np.array_equal(tok.cpu().numpy(), t_ref) and np.array_equal(off.cpu().numpy(), o_ref)


def test_sort_reports_invalid_ids_and_masks_them():
    require_gpu()
    d = make(1, 30, 16, 5, 2)
    idx = choices(1, 30, 5, 2, 4)
    idx[3, 1], idx[7, 0], idx[9, 1] = 5, -2, 2 ** 31 - 1
    off, _, _, tok, status = run_sort(d, idx, bf16((30, 16), 2))
    t_ref, o_ref, _ = plain_order(idx, 1, 5)
    assert status == B.MOE_EINVAL
    assert np.array_equal(tok.cpu().numpy(), t_ref) and np.array_equal(off.cpu().numpy(), o_ref)


@pytest.mark.parametrize("case", ["none", "masked", "one_expert"])
def test_sort_extremes(case):
    """No tokens; every choice masked; every choice on one expert."""
    require_gpu()
    T = 0 if case == "none" else 65
    d = make(2, T, 64, 6, 2)
    idx = np.full((2 * T, 2), -1, dtype=np.int32)
    if case == "one_expert":
        idx[:, 0] = 4
    off, px, _, tok, status = run_sort(d, idx, bf16((2 * T, 64), 2))
    assert status == B.MOE_OK
    if case == "none":
        assert off.cpu().tolist() == [0] * 13
        return
    t_ref, o_ref, _ = plain_order(idx, 2, 6)
    assert np.array_equal(tok.cpu().numpy(), t_ref) and np.array_equal(off.cpu().numpy(), o_ref)


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("R,T,H,E,k,masked", SHAPES)
def test_sort_grad_and_unsort(R, T, H, E, k, masked):
    require_gpu()
    d = make(R, T, H, E, k)
    n = R * T
    idx = choices(R, T, E, k, R + T, masked)
    tok_ref, _, at = plain_order(idx, R, E)
    tok = torch.from_numpy(tok_ref).cuda()
    rows = bf16((n * k, H), 5)
    rows[len(at):] = float("nan")  # rows that no choice has are not read
    w = torch.rand((n, k), generator=torch.Generator().manual_seed(6)).cuda()
    w[tok < 0] = float("nan")  # nor the weights of masked choices
    out, gx = Guarded((n, H), torch.bfloat16, "cuda:0"), Guarded((n, H), torch.bfloat16, "cuda:0")
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    B.moe_unsort(d, rows, tok, w, out.t, err)
    B.moe_sort_grad(d, rows, tok, gx.t, err)
    assert B.moe_get_error(err) == B.MOE_OK and out.guards_intact() and gx.guards_intact()
    live = tok_ref >= 0
    v = np.where(live[:, :, None], f64(rows)[np.maximum(tok_ref, 0)], 0.0)
    wr = np.where(live, f64(w), 0.0)[:, :, None]
    for got, terms in ((out.t, v * wr), (gx.t, v)):
        want = terms.sum(1)
        assert (np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) + (k + 1) * U * np.abs(terms).sum(1)).all()


@pytest.mark.parametrize("with_gw", [True, False])
@pytest.mark.parametrize("R,T,H,E,k,masked", SHAPES)
def test_unsort_grad(R, T, H, E, k, masked, with_gw):
    require_gpu()
    d = make(R, T, H, E, k)
    n = R * T
    idx = choices(R, T, E, k, R + T, masked)
    tok_ref, _, at = plain_order(idx, R, E)
    tok = torch.from_numpy(tok_ref).cuda()
    y, go = bf16((n * k, H), 5), bf16((n, H), 7)
    y[len(at):] = float("nan")
    w = torch.rand((n, k), generator=torch.Generator().manual_seed(6)).cuda()
    w[tok < 0] = float("nan")
    gy = Guarded((n * k, H), torch.bfloat16, "cuda:0", 77.0)
    gw = Guarded((n, k), torch.float32, "cuda:0") if with_gw else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    B.moe_unsort_grad(d, y, tok, w, go, gy.t, gw.t if gw else None, err)
    assert B.moe_get_error(err) == B.MOE_OK and gy.guards_intact() and (gw is None or gw.guards_intact())
    m = len(at)
    token = np.array([t for _, t, _ in at], dtype=np.int64)
    choice = np.array([j for _, _, j in at], dtype=np.int64)
    g64, y64, w64 = f64(go), f64(y), f64(w)
    want = w64[token, choice][:, None] * g64[token]
    assert (np.abs(f64(gy.t)[:m] - want) <= 2.0 ** -8 * np.abs(want)).all()
    assert bool((gy.t[m:] == 77.0).all()), "a row at or above the total was written"
    if gw:
        terms = np.zeros((n, k, H))
        terms[token, choice] = y64[:m] * g64[token]
        bar = (H / 32 + 24) * U * np.abs(terms).sum(2)
        got = f64(gw.t)
        assert (np.abs(got - terms.sum(2)) <= bar).all() and (got[tok_ref < 0] == 0).all()


def test_gradients_against_differences():
    """The round trip sum_j w_j f(x_t) in 64 bits: central differences (h = 1e-4 of values of order 1, a bilinear
    function, so their error is rounding only) agree with the kernels' gradients to their bf16 rounding."""
    require_gpu()
    R, T, H, E, k = 1, 9, 16, 4, 2
    d = make(R, T, H, E, k)
    idx = choices(R, T, E, k, 8, 0.2)
    tok_ref, _, at = plain_order(idx, R, E)
    tok = torch.from_numpy(tok_ref).cuda()
    x, go = bf16((T, H), 9), bf16((T, H), 10)
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(11)).cuda()
    fac = np.array([1.0, -0.5, 2.0, 0.25])  # the "expert": row * fac[e], exact in bf16
    live = tok_ref >= 0
    y = torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda:0")
    for p, (e, t, _) in enumerate(at):
        y[p] = x[t] * fac[e]
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    gy, gw = torch.zeros_like(y), torch.empty_like(w)
    B.moe_unsort_grad(d, y, tok, w, go, gy, gw, err)
    gpacked = gy.clone()
    for p, (e, _, _) in enumerate(at):
        gpacked[p] = gy[p] * fac[e]  # powers of two: no rounding
    gx = torch.empty_like(x)
    B.moe_sort_grad(d, gpacked, tok, gx, err)
    assert B.moe_get_error(err) == B.MOE_OK

    def loss(xv, wv):
        f = np.where(live, fac[np.maximum(idx, 0)], 0.0) * wv
        return ((f.sum(1))[:, None] * xv * f64(go)).sum()

    x64, w64, h = f64(x), f64(w), 1e-4
    for t in range(T):
        bar = 2.0 ** -7 * np.abs(np.where(live[t], fac[np.maximum(idx[t], 0)], 0.0) * w64[t]).sum() * np.abs(f64(go)[t])
        for c in range(H):
            lo, hi = x64.copy(), x64.copy()
            lo[t, c] -= h
            hi[t, c] += h
            assert abs((loss(hi, w64) - loss(lo, w64)) / (2 * h) - float(gx[t, c])) <= bar[c] + 1e-8
        for j in range(k):
            lo, hi = w64.copy(), w64.copy()
            lo[t, j] -= h
            hi[t, j] += h
            assert abs((loss(x64, hi) - loss(x64, lo)) / (2 * h) - float(gw[t, j])) <= 1e-5


def test_unsort_calls_report_a_row_out_of_range():
    require_gpu()
    d = make(1, 4, 16, 4, 2)
    tok = torch.tensor([[0, 1], [2, 8], [3, 4], [5, -1]], dtype=torch.int32, device="cuda:0")
    rows, w = bf16((8, 16), 1), torch.ones((4, 2), device="cuda:0")
    out, gy, gw = bf16((4, 16), 2), torch.zeros((8, 16), dtype=torch.bfloat16, device="cuda:0"), torch.ones_like(w)
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    for call in (lambda: B.moe_unsort(d, rows, tok, w, out, err), lambda: B.moe_sort_grad(d, rows, tok, out, err),
                 lambda: B.moe_unsort_grad(d, rows, tok, w, out.clone(), gy, gw, err)):
        call()
        assert B.moe_get_error(err) == B.MOE_EINVAL
    assert float(gw[1, 1]) == 0.0 and torch.equal(out[1], rows[2])


def test_every_call_runs_on_its_stream_and_in_a_graph():
    """A side stream, then a captured graph replayed on new inputs in the same buffers."""
    require_gpu()
    R, T, H, E, k = 2, 150, 512, 16, 4
    d = make(R, T, H, E, k)
    idx, x = torch.from_numpy(choices(R, T, E, k, 1)).cuda(), bf16((R * T, H), 1)
    w = torch.rand((R * T, k), device="cuda:0")
    off = torch.empty(E * R + 1, dtype=torch.int32, device="cuda:0")
    px = torch.empty((R * T * k, H), dtype=torch.bfloat16, device="cuda:0")
    tok = torch.empty((R * T, k), dtype=torch.int32, device="cuda:0")
    out, gx = torch.empty_like(x), torch.empty_like(x)
    gy, gw = torch.empty_like(px), torch.empty_like(w)
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    torch.cuda.synchronize()

    def step(stream=None):
        B.moe_sort(d, idx, x, None, off, px, None, tok, err, stream=stream)
        B.moe_unsort(d, px, tok, w, out, err, stream=stream)
        B.moe_unsort_grad(d, px, tok, w, x, gy, gw, err, stream=stream)
        B.moe_sort_grad(d, gy, tok, gx, err, stream=stream)

    side = torch.cuda.Stream()
    step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    idx.copy_(torch.from_numpy(choices(R, T, E, k, 2)))
    x.copy_(bf16((R * T, H), 3))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (off, px, tok, out, gx, gy, gw)]
    step()
    assert B.moe_get_error(err) == B.MOE_OK
    for a, b in zip(got, (off, px, tok, out, gx, gy, gw)):
        assert torch.equal(a, b)
