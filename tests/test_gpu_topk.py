"""GPU parity of moe_route and its gradient with the fp64 oracle: ids equal, weights and
gradients within the roundings they take."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from oracle import block
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu

KIND = {"softmax": nv.ROUTE_SOFTMAX, "sigmoid": nv.ROUTE_SIGMOID}
FLOATS = [torch.bfloat16, torch.float16, torch.float32]


def draw(T, E, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * spread).to(dtype), torch.randn(E, generator=g) * 0.05


def run(logits, bias, k, kind="softmax", stride=None, **kw):
    T, E = logits.shape
    p = nv.make_route_problem(T, E, k, KIND[kind], dtype=logits.dtype, **kw)
    ids = torch.full((T, k), -77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    if stride:
        buf = torch.full((T, stride), 5.0, dtype=logits.dtype, device="cuda")
        buf[:, 1:1 + E] = logits.cuda()
        logits = buf[:, 1:1 + E]
    nv.moe_route(p, logits.cuda(), None if bias is None else bias.cuda(), ids, w)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy()


def check(logits, bias, k, kind="softmax", tokens=None, **kw):
    """Against the oracle, token by token (those of `tokens`)."""
    ids, w = run(logits, bias, k, kind, **kw)
    kw.pop("stride", None)
    l = logits.double().numpy()
    b = None if bias is None else bias.double().numpy()
    for t in range(len(l)) if tokens is None else tokens:
        want, weights, _ = block.route_token(l[t], k, kind, b, **kw)
        assert np.array_equal(ids[t], want), (t, ids[t], want)
        # fp64 throughout, one rounding to fp32
        assert (np.abs(w[t] - weights) <= 2.0 ** -24 * 1.001 * np.abs(weights) + 1e-38).all(), (t, w[t], weights)
    return ids, w


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 5), (64, 320, 8), (5, 64, 32), (7, 1024, 32), (130, 65, 3), (33, 96, 1)])
def test_choice(dtype, kind, T, E, k):
    require_gpu()
    log(f"route {dtype} {kind} T={T} E={E} k={k}")
    logits, bias = draw(T, E, dtype, T + E)
    for b in (None, bias):
        for renormalize in (True, False):
            check(logits, b, k, kind, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top_groups", [(320, 8, 8, 4), (320, 8, 8, 8), (320, 5, 5, 1), (6, 2, 3, 2),
                                                   (1024, 8, 64, 3), (1023, 16, 33, 30), (60, 7, 20, 9), (64, 3, 64, 5),
                                                   (102, 2, 17, 1), (640, 4, 2, 1), (96, 6, 3, 1)])
def test_groups(kind, E, k, groups, top_groups):
    require_gpu()
    log(f"route {kind} E={E} k={k} groups={groups}/{top_groups}")
    logits, bias = draw(40, E, torch.float32, E + groups, 1.0)
    for keys in (1, 2):
        for b in (None, bias):
            check(logits, b, k, kind, groups=groups, top_groups=top_groups, group_keys=keys)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_equal_and_nearly_equal_keys(kind):
    """Ties go to the lowest id; keys that fp32 cannot tell apart are told apart."""
    require_gpu()
    log(f"route ties {kind}")
    T, E = 64, 320
    g = torch.Generator().manual_seed(4)
    coarse = torch.randint(-2, 3, (T, E), generator=g).float()
    check(coarse, None, 8, kind)
    check(torch.zeros(T, E), None, 8, kind)
    check(coarse, torch.zeros(E), 8, kind)
    check(coarse, torch.full((E,), 0.25), 8, kind, groups=8, top_groups=3)
    check(torch.zeros(3, E), torch.zeros(E), 32, kind, groups=64, top_groups=7)
    # neighbouring fp32 logits: their scores differ by less than fp32 can hold
    base = torch.full((T, E), 3.0 if kind == "sigmoid" else 0.125)
    step = torch.randint(0, 4, (T, E), generator=g).int()
    near = (base.view(torch.int32) + step).view(torch.float32)
    check(near, None, 8, kind)
    check(near, torch.zeros(E), 8, kind)
    check(near, torch.zeros(E), 8, kind, groups=8, top_groups=2)
    # a bias that undoes most of a difference of scores
    l, _ = draw(T, E, torch.float32, 9, 1.0)
    s = np.stack([block.scores(x, kind) for x in l.double().numpy()])
    b = torch.from_numpy((s[0].max() - s[0]).astype(np.float32))
    check(l[:1].repeat(T, 1), b, 8, kind)
    check(l[:1].repeat(T, 1), b, 8, kind, groups=8, top_groups=4)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_masked_logits(kind):
    """-Inf, NaN, +Inf and the type's lowest value among the logits and the bias; rows that leave
    fewer experts than asked for, and rows that leave none."""
    require_gpu()
    log(f"route masks {kind}")
    T, E, k = 12, 40, 4
    inf = float("inf")
    l, bias = draw(T, E, torch.float32, 3)
    l[0, :] = -inf
    l[1, :] = float("nan")
    l[2, 3:] = -inf
    l[3, 1:] = float("nan")
    l[4, 5], l[4, 17] = inf, inf
    l[5, :20] = torch.finfo(torch.float32).min
    l[6, :] = torch.finfo(torch.float32).min
    l[7, 7:] = -inf
    l[8, :] = -800.0                                             # every score underflows
    l[9, ::2] = -inf
    b = bias.clone()
    b[2], b[11], b[12] = -inf, float("nan"), inf
    for m in (None, bias, b):
        for kw in (dict(), dict(renormalize=False), dict(groups=8, top_groups=2), dict(groups=8, top_groups=1, group_keys=1)):
            check(l, m, k, kind, **kw)
    ids, w = run(l, None, k, kind)
    assert (ids[:2] == -1).all() and (w[:2] == 0).all() and (ids[2, 3:] == -1).all()


def test_logits_that_are_not_aligned():
    require_gpu()
    log("route strides")
    for dtype in FLOATS:
        logits, bias = draw(30, 77, dtype, 6)
        check(logits, bias, 6, "sigmoid", stride=81)


def test_many_tokens():
    require_gpu()
    log("route many tokens")
    logits, bias = draw(9001, 320, torch.bfloat16, 8)
    check(logits, bias, 8, "sigmoid", tokens=range(0, 9001, 37), groups=8, top_groups=4, scale=2.5)
    check(logits, None, 8, "softmax", tokens=range(0, 9001, 37))
    run(torch.empty(0, 320), bias, 8)


# --------------------------------------------------------------------- gradient
def gradient(logits, ids, dw, kind, stride=None, **kw):
    T, E = logits.shape
    p = nv.make_route_problem(T, E, ids.shape[1], KIND[kind], dtype=logits.dtype, **kw)
    buf = torch.full((T, stride or E), 5.0, dtype=logits.dtype, device="cuda")
    out = buf[:, 1:1 + E] if stride else buf
    nv.moe_route_backward(p, logits.cuda(), ids.cuda(), dw.cuda(), out)
    torch.cuda.synchronize()
    if stride:
        assert (buf[:, 0] == 5).all() and (buf[:, 1 + E:] == 5).all()
    return out.double().cpu().numpy()


def check_gradient(logits, ids, dw, kind, renormalize, scale=1.0, **kw):
    got = gradient(logits, ids, dw, kind, renormalize=renormalize, scale=scale, **kw)
    l, g = logits.double().numpy(), dw.double().numpy()
    half = torch.finfo(logits.dtype).eps / 2
    T, E, k = len(l), l.shape[1], ids.shape[1]
    for t in range(T):
        i = ids[t].numpy()
        want = block.route_gradient(l[t], i, g[t], kind, renormalize, scale)
        # what is added up: share or score times (|dw| + sum |p dw|) at the chosen, score times the sum elsewhere
        sane = block._sane(l[t])
        ok = (i >= 0) & (i < E)
        s = block.scores(l[t], kind)
        share = np.zeros(E)
        if renormalize and ok.any():
            z = sane[i[ok]]
            p = np.exp(z - z.max()) if kind == "softmax" and z.max() > -np.inf else s[i[ok]]
            np.add.at(share, i[ok], p / p.sum() if p.sum() > 0 else 0)
        else:
            share = s
        hit = np.zeros(E)
        np.add.at(hit, i[ok], np.abs(g[t][ok]))
        mag = abs(scale) * share * (hit + (share[i[ok]] * np.abs(g[t][ok])).sum())
        # fp32: exponents of differences of logits round by 2^-24 of their size; sums over k and over
        # E in a tree; at most twelve more operations
        span = np.ptp(sane[np.isfinite(sane)]) if np.isfinite(sane).any() else 0.0
        terms = k + 12 + 12 + 2 * min(span, 100.0)
        lim = terms * 2.0 ** -24 * mag + half * np.abs(want) + 2e-38 + (6e-8 if logits.dtype == torch.float16 else 0)
        err = np.abs(got[t] - want)
        assert (err <= lim).all(), (t, float((err / lim).max()))
    return got


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 5), (64, 320, 8), (5, 1024, 32), (130, 65, 3), (2, 8, 2)])
def test_gradient(dtype, kind, renormalize, T, E, k):
    require_gpu()
    log(f"route gradient {dtype} {kind} renormalize={renormalize} T={T} E={E} k={k}")
    logits, bias = draw(T, E, dtype, T + E)
    ids = torch.from_numpy(run(logits, bias, k, kind)[0])
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(2))
    check_gradient(logits, ids, dw, kind, renormalize, 2.5)
    check_gradient(logits, ids, dw, kind, renormalize, stride=E + 3)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_of_masked_and_repeated_ids(kind, renormalize):
    """Ids outside the model, ids that stand twice, tokens without any; logits of +-Inf, NaN and
    far from 0; dweights of slots that are not chosen are not looked at."""
    require_gpu()
    log(f"route gradient masks {kind} {renormalize}")
    T, E, k = 8, 24, 4
    l, _ = draw(T, E, torch.float32, 5)
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(3)).int()
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(4))
    ids[0] = -1
    ids[1, 1:] = torch.tensor([E, -5, 1 << 30])
    ids[2] = 7
    ids[3, 0] = ids[3, 3]
    l[4, :] = -float("inf")
    l[5, ::2], l[5, 1] = float("nan"), -float("inf")
    l[6, :] = -300.0
    l[7, ids[7, 0].item()] = float("inf")
    clean = dw.clone()
    bad = (ids < 0) | (ids >= E)
    clean[bad] = 0.0
    dw[bad] = float("nan")
    got = gradient(l, ids, dw, kind, renormalize=renormalize)
    assert np.isfinite(got).all()
    ref = check_gradient(l, ids, clean, kind, renormalize)
    assert np.array_equal(got, ref) and (got[0] == 0).all() and (got[4] == 0).all()


def test_gradient_against_differences():
    """The library's own weights, moved by hand: sum w dw against dlogits."""
    require_gpu()
    log("route gradient differences")
    T, E, k = 6, 40, 4
    for kind in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            l, bias = draw(T, E, torch.float32, 11, 1.0)
            dw = torch.randn(T, k, generator=torch.Generator().manual_seed(6))
            kw = dict(groups=4, top_groups=4, renormalize=renormalize)
            ids, _ = run(l, bias, k, kind, **kw)
            got = gradient(l, torch.from_numpy(ids), dw, kind, **kw)
            h = 1e-2
            for t, j in ((0, 0), (1, 3), (5, 2)):
                e = ids[t, j]
                val = []
                for sign in (1, -1):
                    m = l.clone()
                    m[t, e] += sign * h
                    i2, w2 = run(m, torch.where(torch.isin(torch.arange(E), torch.from_numpy(ids[t]).long()), 10.0, -10.0),
                                 k, kind, **kw)                     # the bias holds the choice
                    order = {int(i): float(w) for i, w in zip(i2[t], w2[t])}
                    val.append(sum(order[int(i)] * float(g) for i, g in zip(ids[t], dw[t])))
                # the third derivative is at most 2 sum |dw|, a weight rounds by 2^-24
                lim = (2 * h * h / 6 + 2 ** -24 / h) * float(dw[t].abs().sum())
                assert abs((val[0] - val[1]) / (2 * h) - got[t, e]) <= lim


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_keys", [1, 2])
@pytest.mark.parametrize("groups,E,top", [(8, 320, 4), (8, 320, 1), (4, 64, 1), (2, 10, 1), (64, 128, 9), (2, 1024, 1)])
def test_biases_beyond_a_sum(kind, group_keys, groups, E, top):
    """Biases of +Inf, and of magnitudes whose sums pass fp32: a group's sum is that of the keys in fp64, equal
    sums (two of +Inf) go to the lower group."""
    require_gpu()
    log(f"route biases {kind} groups={groups} E={E} top={top} keys={group_keys}")
    n = E // groups
    for case in range(8):
        logits, bias = draw(5, E, torch.float32, 50 + case)
        if case == 0:                                            # more groups with +Inf than may serve
            bias[n - 1::n] = float("inf")
        elif case == 1:                                          # two in the last group: no more than one
            bias[0], bias[-1], bias[-2] = float("inf"), float("inf"), float("inf")
        elif case == 2:
            bias = torch.full_like(bias, 3e38)
        elif case == 3:                                          # sums of 4e38 to 6.8e38 and of the same below 0
            bias = torch.linspace(2.0e38, 3.4e38, E) * torch.where(torch.arange(E) % 3 == 0, -1.0, 1.0)
        elif case == 4:
            bias = torch.linspace(-3.4e38, -2.0e38, E)
        elif case == 5:                                          # +Inf once a group, at other places of each
            bias[torch.arange(groups) * n + torch.arange(groups - 1, -1, -1) * (n - 1) // (groups - 1)] = float("inf")
        elif case == 6:                                          # sums past fp32, equal, at other places of each
            bias[torch.arange(groups) * n + torch.arange(groups - 1, -1, -1) * (n - 1) // (groups - 1)] = 3.4e38
            bias[torch.arange(groups) * n + torch.arange(groups) * (n - 1) // (groups - 1)] = 3.4e38
        else:                                                    # the highest keys in the last groups, by little
            bias = 3.4e38 - torch.arange(E).flip(0) * 1e35
            bias[::n] = float("inf")
        check(logits, bias, min(top * n, 5), kind, groups=groups, top_groups=top, group_keys=group_keys)
        check(logits, bias, min(E, 5), kind)
