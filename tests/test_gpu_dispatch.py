"""GPU parity of dispatch, combine and their gradients with the fp64 oracle.

Integers and copied rows must be equal.  Sums run in fp32 in slot order: with
u = 2^-24, k products and sums of magnitude <= S = sum |w y| are off by at most
(k + 1) u S, and the result is rounded once to its type (half a step, eps / 2, of
the value; below the type's normal range half its smallest step)."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from oracle import dispatch
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FLOATS = [torch.bfloat16, torch.float16, torch.float32]


def f64(t):
    return t.double().cpu().numpy()


def rounding(dtype, ref):
    """Half a step of `dtype` at ref (a hair more: the fp32 value it is rounded from may sit elsewhere)."""
    fi = torch.finfo(dtype)
    return fi.eps / 2 * (1 + 1e-3) * np.abs(ref) + fi.tiny * fi.eps / 2


def make_ids(T, k, E, gen, kind):
    if kind == "distinct":
        return torch.rand(T, E, generator=gen).topk(k, 1).indices.int()
    if kind == "repeated":                                # the same expert in several slots
        return torch.randint(0, E, (T, k), generator=gen, dtype=torch.int32)
    if kind == "one":                                     # every token to one expert
        return torch.full((T, k), E // 2, dtype=torch.int32)
    if kind == "foreign":                                 # padded slots, ids beyond the model
        ids = torch.randint(-3, E + 3, (T, k), generator=gen, dtype=torch.int32)
        ids[0] = -1
        ids[-1] = torch.iinfo(torch.int32).min if T % 2 else torch.iinfo(torch.int32).max
        return ids
    raise ValueError(kind)


def strided(rows, d, dtype, layout, fill=None):
    """A [rows, d] view on the GPU: dense, of wider rows, or of wider rows at an unaligned start."""
    if layout == "dense":
        t = torch.empty(rows, d, dtype=dtype, device="cuda")
    elif layout == "wide":
        t = torch.empty(rows, (d + 15) // 16 * 16 + 32, dtype=dtype, device="cuda")[:, 16:16 + d]
    else:
        t = torch.empty(rows, d + 5, dtype=dtype, device="cuda")[:, 3:3 + d]
    if fill is not None:
        t.fill_(fill)
    return t


def run_plan(T, k, E, offset, L, ids, d=8, dtype=torch.float32, layout="dense", seed=0):
    gen = torch.Generator().manual_seed(seed)
    p = nv.make_dispatch_problem(T, d, E, k, offset, L, dtype)
    x = strided(T, d, dtype, layout)
    x.copy_(torch.randint(0, 256, (T, d), generator=gen) if dtype == torch.uint8 else torch.randn(T, d, generator=gen))
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets = torch.full((L,), 77, **i32), torch.full((L + 1,), 77, **i32)
    perm, inv = torch.full((T * k,), -7, **i32), torch.full((T, k), -7, **i32)
    rows = strided(T * k, d, dtype, layout, fill=99)
    nv.moe_dispatch(p, ids.cuda(), x, counts, offsets, perm, inv, rows, nv.alloc_dispatch_workspace(p))
    torch.cuda.synchronize()
    return p, x, counts, offsets, perm, inv, rows


# one launch up to 16384 pairs, three above; one token a block up to 2047 tokens
SHAPES = [(1, 1, 1, 0, 1, "distinct"), (1, 8, 320, 0, 160, "distinct"), (3, 32, 1024, 100, 924, "repeated"),
          (64, 8, 320, 160, 160, "distinct"), (300, 7, 20, 5, 10, "foreign"), (2048, 8, 60, 0, 60, "distinct"),
          (2049, 8, 60, 0, 60, "repeated"), (5000, 4, 64, 60, 4, "distinct"), (4100, 32, 7, 0, 7, "foreign"),
          (20000, 1, 1024, 0, 1024, "distinct"), (700, 3, 9, 0, 9, "one"), (9000, 2, 9, 0, 9, "one"),
          (33, 5, 16, 0, 8, "one")]


@pytest.mark.parametrize("T,k,E,offset,L,kind", SHAPES)
def test_plan_and_rows_equal_the_oracle(T, k, E, offset, L, kind):
    require_gpu()
    log(f"dispatch T={T} k={k} E={E} offset={offset} L={L} {kind}")
    ids = make_ids(T, k, E, torch.Generator().manual_seed(T), kind)
    p, x, counts, offsets, perm, inv, rows = run_plan(T, k, E, offset, L, ids)
    c, o, pm, iv = dispatch.plan(ids.numpy(), offset, L)
    P = len(pm)
    assert np.array_equal(counts.cpu().numpy(), c) and np.array_equal(offsets.cpu().numpy(), o)
    assert np.array_equal(inv.cpu().numpy(), iv)
    assert np.array_equal(perm.cpu().numpy()[:P], pm) and (perm[P:] == -7).all()
    assert torch.equal(rows[:P].cpu(), x.cpu()[torch.from_numpy(pm // k)])
    assert (rows[P:] == 99).all()


@pytest.mark.parametrize("dtype", FLOATS + [torch.uint8])
@pytest.mark.parametrize("d,layout", [(1, "dense"), (7, "dense"), (64, "dense"), (1000, "dense"), (4096, "dense"),
                                      (1024, "wide"), (100, "odd"), (4096, "odd")])
def test_rows_of_every_type_width_and_stride(dtype, d, layout):
    require_gpu()
    log(f"dispatch rows {dtype} d={d} {layout}")
    for T, k, E, offset, L in ((37, 3, 12, 2, 7), (2500, 8, 40, 0, 20)):
        ids = make_ids(T, k, E, torch.Generator().manual_seed(d), "distinct")
        p, x, counts, offsets, perm, inv, rows = run_plan(T, k, E, offset, L, ids, d, dtype, layout)
        _, _, pm, _ = dispatch.plan(ids.numpy(), offset, L)
        assert torch.equal(rows[:len(pm)].cpu(), x.cpu()[torch.from_numpy(pm // k)])
        assert (rows[len(pm):] == 99).all()
        if layout != "dense":                            # nothing outside the rows is written
            whole = rows._base
            start = rows.storage_offset() % whole.shape[1]
            before = whole.clone()
            nv.moe_dispatch(p, ids.cuda(), x, None, None, None, None, rows, nv.alloc_dispatch_workspace(p))
            assert torch.equal(whole[:, :start].view(torch.uint8), before[:, :start].view(torch.uint8))
            assert torch.equal(whole[:, start + d:].view(torch.uint8), before[:, start + d:].view(torch.uint8))


def test_plan_alone_and_no_tokens():
    require_gpu()
    log("dispatch plan alone, T = 0")
    ids = make_ids(50, 4, 16, torch.Generator().manual_seed(0), "distinct")
    p = nv.make_dispatch_problem(50, 8, 16, 4, 0, 16)
    inv = torch.empty(50, 4, dtype=torch.int32, device="cuda")
    nv.moe_dispatch(p, ids.cuda(), None, None, None, None, inv, None, nv.alloc_dispatch_workspace(p))
    assert np.array_equal(inv.cpu().numpy(), dispatch.plan(ids.numpy(), 0, 16)[3])
    p = nv.make_dispatch_problem(0, 8, 16, 4, 0, 16)
    e = lambda *s, dt=torch.int32: torch.empty(*s, dtype=dt, device="cuda")          # noqa: E731
    counts, offsets, bf = e(16).fill_(5), e(17).fill_(5), torch.bfloat16
    nv.moe_dispatch(p, e(0, 4), e(0, 8, dt=bf), counts, offsets, e(0), e(0, 4), e(0, 8, dt=bf),
                    nv.alloc_dispatch_workspace(p))
    assert not counts.any() and not offsets.any()
    nv.moe_combine(p, e(0, 4), e(0, 4, dt=torch.float32), e(0, 8, dt=bf), e(0, 8, dt=bf))
    nv.moe_dispatch_backward(p, e(0, 4), e(0, 8, dt=bf), e(0, 8, dt=bf))
    nv.moe_combine_backward(p, e(0, 4), e(0, 4, dt=torch.float32), e(0, 8, dt=bf), e(0, 8, dt=bf), e(0, 8, dt=bf),
                            e(0, 4, dt=torch.float32))
    torch.cuda.synchronize()


def routed(T, k, E, offset, L, seed, kind="distinct"):
    gen = torch.Generator().manual_seed(seed)
    ids = make_ids(T, k, E, gen, kind)
    inv = dispatch.plan(ids.numpy(), offset, L)[3]
    w = torch.rand(T, k, generator=gen) - 0.25                # negative weights too
    w[torch.from_numpy(inv) < 0] = float("nan")               # a dropped slot's weight is not looked at
    return gen, inv, w


CASES = [(1, 8, 320, 0, 320, 4096, "dense"), (1, 1, 1, 0, 1, 1, "dense"), (37, 3, 12, 2, 7, 100, "odd"),
         (130, 8, 16, 0, 16, 1024, "wide"), (130, 9, 16, 3, 8, 1032, "dense"), (40, 32, 64, 0, 40, 72, "dense"),
         (515, 4, 60, 15, 30, 1000, "dense"), (66, 2, 4, 0, 1, 2056, "dense"), (9, 17, 40, 0, 40, 4097, "dense")]


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("T,k,E,offset,L,d,layout", CASES)
def test_combine_and_dispatch_backward(dtype, T, k, E, offset, L, d, layout):
    require_gpu()
    log(f"combine {dtype} T={T} k={k} L={L}/{E} d={d} {layout}")
    gen, inv, w = routed(T, k, E, offset, L, seed=d)
    p = nv.make_dispatch_problem(T, d, E, k, offset, L, dtype)
    rows = strided(T * k, d, dtype, layout, fill=float("nan"))        # rows of no pair are not looked at
    P = int((inv >= 0).sum())
    rows[:P] = torch.randn(P, d, generator=gen).to(dtype).cuda()
    inv_g, w_g = torch.from_numpy(inv).int().cuda(), w.cuda()
    for weights in (w_g, None):
        out = strided(T, d, dtype, layout, fill=float("nan"))
        if weights is None:
            nv.moe_dispatch_backward(p, inv_g, rows, out)
        else:
            nv.moe_combine(p, inv_g, weights, rows, out)
        ref, mag = dispatch.combine(inv, None if weights is None else f64(w), f64(rows))
        err = np.abs(f64(out) - ref)
        assert (err <= (k + 1) * U * mag * 1.01 + rounding(dtype, ref)).all(), float(err.max())
        empty = (inv < 0).all(axis=1)
        assert not f64(out)[empty].any()


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("T,k,E,offset,L,d,layout", CASES)
def test_combine_backward(dtype, T, k, E, offset, L, d, layout):
    require_gpu()
    log(f"combine backward {dtype} T={T} k={k} L={L}/{E} d={d} {layout}")
    gen, inv, w = routed(T, k, E, offset, L, seed=d + 1)
    p = nv.make_dispatch_problem(T, d, E, k, offset, L, dtype)
    rows = strided(T * k, d, dtype, layout, fill=float("nan"))
    P = int((inv >= 0).sum())
    rows[:P] = torch.randn(P, d, generator=gen).to(dtype).cuda()
    dout = strided(T, d, dtype, layout)
    dout.copy_(torch.randn(T, d, generator=gen))
    inv_g, w_g = torch.from_numpy(inv).int().cuda(), w.cuda()
    drows, dw = strided(T * k, d, dtype, layout, fill=3.0), torch.full((T, k), float("nan"), device="cuda")
    nv.moe_combine_backward(p, inv_g, w_g, rows, dout, drows, dw)
    ref, dref, dmag = dispatch.combine_backward(inv, f64(w), f64(rows), f64(dout))
    assert (drows[P:] == 3.0).all()
    # one fp32 product, then one rounding
    err = np.abs(f64(drows)[:P] - ref[:P])
    assert (err <= U * np.abs(ref[:P]) + rounding(dtype, ref[:P])).all()
    # d fused multiply-adds in any order, fp32
    assert (np.abs(f64(dw) - dref) <= d * U * dmag * 1.01).all()
    # each output alone gives the same bits
    drows2, dw2 = strided(T * k, d, dtype, layout, fill=3.0), torch.empty_like(dw)
    nv.moe_combine_backward(p, inv_g, w_g, None, dout, drows2, None)
    nv.moe_combine_backward(p, inv_g, w_g, rows, dout, None, dw2)
    assert torch.equal(drows, drows2) and torch.equal(dw, dw2)


def test_rows_outside_the_buffer_are_not_followed():
    """Entries of inv beyond [0, T k) count as not kept."""
    require_gpu()
    log("combine with foreign rows in inv")
    T, k, d = 5, 2, 24
    p = nv.make_dispatch_problem(T, d, 4, k, 0, 4, torch.float32)
    inv = torch.tensor([[0, 10], [-5, 3], [2 ** 31 - 1, -2 ** 31], [9, 1], [11, 12]], dtype=torch.int32)
    rows, w, dout = torch.randn(T * k, d), torch.ones(T, k), torch.randn(T, d)
    seen = np.where((inv.numpy() >= 0) & (inv.numpy() < T * k), inv.numpy(), -1)
    out, drows, dw = torch.empty(T, d, device="cuda"), torch.zeros(T * k, d, device="cuda"), torch.empty(T, k, device="cuda")
    nv.moe_combine(p, inv.cuda(), w.cuda(), rows.cuda(), out)
    nv.moe_combine_backward(p, inv.cuda(), w.cuda(), rows.cuda(), dout.cuda(), drows, dw)
    assert np.abs(f64(out) - dispatch.combine(seen, None, f64(rows))[0]).max() < 1e-6
    ref, dref, mag = dispatch.combine_backward(seen, f64(w), f64(rows), f64(dout))
    assert np.array_equal(f64(drows), np.nan_to_num(ref)) and (np.abs(f64(dw) - dref) <= d * U * mag).all()


@pytest.mark.parametrize("T", [64, 3000])
def test_another_stream_and_graph_replays(T):
    """Captured once, replayed with new ids and rows written by eager work in between."""
    require_gpu()
    log(f"dispatch/combine graph T={T}")
    k, E, d = 8, 40, 256
    p = nv.make_dispatch_problem(T, d, E, k, 10, 20)
    gen = torch.Generator().manual_seed(T)
    new = lambda: (make_ids(T, k, E, gen, "distinct").cuda(), torch.randn(T, d, generator=gen).bfloat16().cuda())  # noqa: E731
    ids, x = new()
    i32 = dict(dtype=torch.int32, device="cuda")
    bufs = dict(counts=torch.empty(20, **i32), offsets=torch.empty(21, **i32), perm=torch.zeros(T * k, **i32),
                inv=torch.empty(T, k, **i32), rows=torch.zeros(T * k, d, dtype=torch.bfloat16, device="cuda"))
    ws, w = nv.alloc_dispatch_workspace(p), torch.rand(T, k, generator=gen).cuda()
    out, drows = torch.empty_like(x), torch.zeros_like(bufs["rows"])
    dw = torch.empty(T, k, device="cuda")

    def step(b, o, dr, dwt):
        nv.moe_dispatch(p, ids, x, workspace=ws, **b)
        nv.moe_combine(p, b["inv"], w, b["rows"], o)
        nv.moe_combine_backward(p, b["inv"], w, b["rows"], x, dr, dwt)

    step(bufs, out, drows, dw)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(bufs, out, drows, dw)
    side = torch.cuda.Stream()
    for r in range(3):
        a, b = new()
        ids.copy_(a)
        x.copy_(b)
        for t in (*bufs.values(), out, drows, dw):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        e = {n: torch.zeros_like(t) for n, t in bufs.items()}
        eo, ed, ew = torch.zeros_like(out), torch.zeros_like(drows), torch.zeros_like(dw)
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            step(e, eo, ed, ew)
        side.synchronize()
        for n in e:
            assert torch.equal(e[n], bufs[n]), (r, n)
        assert torch.equal(eo, out) and torch.equal(ed, drows) and torch.equal(ew, dw), r
