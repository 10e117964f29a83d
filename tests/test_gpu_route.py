"""GPU parity of mep_route and mep_route_grad against the 64-bit reference.

Ids are compared exactly: the kernel forms and compares the selection values
in fp64. Scores and gradients are formed in fp64 and rounded once: half a
step of the type (fp32 2^-24, bf16 2^-8, fp16 2^-11 of the value), doubled
for the fp64 arithmetic and the double rounding through fp32 of 16-bit
gradients, which together cost far less than that; plus half a step of the
type's subnormals. An unrenormalised softmax may sum its denominator in
fp32: exp to 2^-22, at most 22 roundings of the sum, under 2^-19.
"""
import numpy as np
import pytest

import expert_ref as ref
from gpu_util import note, require_gpu

pytestmark = pytest.mark.gpu

SCORE_TOL = 2.0 ** -23
SOFTMAX_TOL = 2.0 ** -19
GRAD_TOL = {"float32": 2.0 ** -23, "bfloat16": 2.0 ** -7, "float16": 2.0 ** -10}
TINY = {"float32": 2.0 ** -149, "bfloat16": 2.0 ** -133, "float16": 2.0 ** -24}


def _logits(rng, T, E, dtype, masked=0.0):
    import torch
    l = rng.standard_normal((T, E)).astype(np.float32)
    if masked:
        l[rng.random((T, E)) < masked] = -np.inf
        l[::5, 1:] = -np.inf   # one expert left
        l[::11] = -np.inf      # none left
    t = torch.from_numpy(l).to(getattr(torch, dtype))
    return t.cuda(), t.double().numpy()


def _check(l_dev, l, K, **kw):
    import torch

    import combine_balancing_amd as cba
    bias = kw.pop("bias", None)
    b = None if bias is None else torch.from_numpy(bias).cuda()
    ids, sc = cba.route(l_dev, K, bias=b, **kw)
    torch.cuda.synchronize()
    want_ids, want = ref.route(l, K, bias=bias, **kw)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = sc.cpu().numpy().astype(np.float64)
    tol = SOFTMAX_TOL if kw.get("scoring", "softmax") == "softmax" and not kw.get(
        "renormalize", True) else SCORE_TOL
    assert np.all(np.abs(got - want) <= tol * np.abs(want) + 2.0 ** -149)
    return ids, sc


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 256, 8), (3, 8, 8), (5, 7, 3), (33, 64, 64),
                                   (257, 256, 8), (64, 384, 8), (19, 1000, 16), (2, 1024, 64),
                                   (4099, 160, 6)])
def test_route_sizes(dtype, T, E, K):
    torch = require_gpu()  # noqa: F841
    note(f"route {dtype} T={T} E={E} K={K}")
    rng = np.random.default_rng(T * 7 + E)
    ld, l = _logits(rng, T, E, dtype)
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            _check(ld, l, K, scoring=scoring, renormalize=renorm, scale=2.5 if renorm else 1.0)
        _check(ld, l, K, scoring=scoring, bias=(0.2 * rng.standard_normal(E)).astype(np.float32))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("E,ng,tg,K", [(16, 1, 1, 4), (48, 1, 1, 8), (52, 1, 1, 16), (64, 4, 2, 8),
                                       (120, 1, 1, 8), (128, 8, 4, 8), (200, 1, 1, 6),
                                       (256, 8, 4, 8), (255, 1, 1, 3), (256, 2, 1, 20),
                                       (384, 1, 1, 8), (380, 1, 1, 8), (383, 1, 1, 5),
                                       (384, 8, 3, 6), (500, 1, 1, 8), (512, 16, 4, 8),
                                       (512, 1, 1, 33), (768, 1, 1, 8), (1000, 5, 2, 7),
                                       (1024, 1, 1, 8)])
def test_route_many_tokens(dtype, E, ng, tg, K):
    """Enough tokens for the variants that put several on a wave, at widths
    that fill their lanes, do not, or leave rows off the vector grid; checked
    at every 13th token and the last."""
    torch = require_gpu()
    import combine_balancing_amd as cba
    note(f"route many tokens {dtype} E={E} ng={ng} K={K}")
    T = 4099
    rng = np.random.default_rng(E + K)
    ld, l = _logits(rng, T, E, dtype, masked=0.1 if E % 3 == 0 else 0.0)
    rows = np.r_[np.arange(0, T, 13), T - 1]
    for scoring, bias in (("softmax", None), ("sigmoid", 0.2)):
        b = None if bias is None else (bias * rng.standard_normal(E)).astype(np.float32)
        ids, sc = cba.route(ld, K, bias=None if b is None else torch.from_numpy(b).cuda(),
                            scoring=scoring, n_group=ng, topk_group=tg)
        torch.cuda.synchronize()
        want_ids, want = ref.route(l[rows], K, bias=b, scoring=scoring, n_group=ng, topk_group=tg)
        assert np.array_equal(ids.cpu().numpy()[rows], want_ids)
        got = sc.cpu().numpy()[rows].astype(np.float64)
        assert np.all(np.abs(got - want) <= SCORE_TOL * np.abs(want) + 2.0 ** -149)


@pytest.mark.parametrize("T", [3, 4096])
@pytest.mark.parametrize("E,K", [(64, 4), (64, 5), (128, 9), (256, 8), (256, 9), (256, 16),
                                 (384, 8), (384, 13), (1024, 8), (1024, 17), (1024, 64)])
def test_route_chosen_side_by_side(T, E, K):
    # logits in order: one lane's experts are chosen to the last, then the next's
    torch = require_gpu()
    import combine_balancing_amd as cba
    note(f"route side by side T={T} E={E} K={K}")
    up = torch.arange(E, dtype=torch.float32) / 64 - E / 128
    l = torch.stack([up, up.flip(0), up.roll(E // 2 + 3)])
    full = l.repeat(-(-T // 3), 1)[:T].contiguous().cuda()
    ids, _ = cba.route(full, K)
    torch.cuda.synchronize()
    want = torch.argsort(l.double(), 1, descending=True)[:, :K].int()
    assert torch.equal(ids.cpu(), want.repeat(-(-T // 3), 1)[:T])


@pytest.mark.parametrize("offset", [1, 2, 4])
def test_route_off_the_vector_grid(offset):
    # logits that start inside a larger buffer, `offset` elements in
    torch = require_gpu()
    import combine_balancing_amd as cba
    note(f"route offset {offset}")
    rng = np.random.default_rng(offset)
    for dtype in (torch.float32, torch.bfloat16):
        for T, E in ((4100, 256), (7, 256), (4100, 384)):
            buf = torch.from_numpy(rng.standard_normal(T * E + 8).astype(np.float32)).to(dtype).cuda()
            l = buf[offset:offset + T * E].view(T, E)
            a = cba.route(l, 8, scoring="sigmoid")
            b = cba.route(l.clone(), 8, scoring="sigmoid")
            torch.cuda.synchronize()
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,ng,tg,K", [(256, 8, 4, 8), (256, 8, 1, 32), (64, 64, 5, 5),
                                       (160, 8, 3, 6), (48, 3, 2, 4), (1024, 16, 4, 8),
                                       (1000, 5, 2, 7), (384, 2, 1, 8), (14, 2, 2, 14)])
def test_route_groups(scoring, E, ng, tg, K):
    require_gpu()
    note(f"route groups {scoring} E={E} ng={ng} tg={tg} K={K}")
    rng = np.random.default_rng(E + ng)
    for dtype, masked in (("float32", 0.0), ("bfloat16", 0.6)):
        ld, l = _logits(rng, 67, E, dtype, masked)
        for bias in (None, (0.3 * rng.standard_normal(E)).astype(np.float32)):
            _check(ld, l, K, scoring=scoring, n_group=ng, topk_group=tg, bias=bias)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_special_values(scoring, renorm):
    torch = require_gpu()
    note(f"route special values {scoring} renorm={renorm}")
    E = 40
    rows = [np.zeros(E), np.full(E, -np.inf), np.full(E, np.nan), np.full(E, -3.0e38),
            np.where(np.arange(E) == 7, 0.0, -np.inf), np.linspace(-200, 200, E),
            np.where(np.arange(E) % 2 == 0, 1.0, np.nan), np.full(E, 1e-42),
            np.where(np.arange(E) == 3, np.inf, 1.0), np.where(np.arange(E) < 2, np.inf, -1.0),
            np.full(E, 80.0), np.full(E, -100.0)]
    l = np.array(rows, np.float32)
    ld = torch.from_numpy(l).cuda()
    for K in (1, 6):
        _check(ld, l.astype(np.float64), K, scoring=scoring, renormalize=renorm)
        bias = np.linspace(0.5, -0.5, E).astype(np.float32)
        bias[4], bias[5], bias[6] = -np.inf, np.nan, np.inf
        if scoring == "sigmoid":
            _check(ld, l.astype(np.float64), K, scoring=scoring, renormalize=renorm, bias=bias)


def test_route_near_ties_follow_64_bits():
    # sigmoid scores that agree to fp32 rounding but not in fp64, with biases
    # that make the order hang on their last bits
    torch = require_gpu()
    note("route near ties")
    rng = np.random.default_rng(3)
    T, E, K = 400, 64, 8
    base = rng.standard_normal((T, 1)).astype(np.float32)
    l = np.nextafter(base, np.float32(9)) * np.ones((1, E), np.float32)
    steps = rng.integers(-3, 4, (T, E))
    l = (l.view(np.int32) + steps).astype(np.int32).view(np.float32)
    bias = np.full(E, 0.25, np.float32)
    bias[::3] = np.nextafter(np.float32(0.25), np.float32(1))
    ld = torch.from_numpy(l).cuda()
    for b in (None, bias):
        _check(ld, l.astype(np.float64), K, scoring="sigmoid", bias=b)
    _check(ld, l.astype(np.float64), K, scoring="sigmoid", n_group=8, topk_group=4)
    # With a bias the groups are ordered by sums of two values, and sums over
    # neighbouring logits agree to second order: with u one fp32 step,
    # s(l - u) + s(l + u) - 2 s(l) is about u^2 s'' < 1e-15, which fp64 does
    # not resolve. A value s + b below 2 comes out within 4 roundings of at
    # most 2^-53 (exp, 1 + x, the quotient, the bias), a sum of two within
    # 8 * 2^-53 + 2^-53, two sums apart from each other within 2^-48.8. Rows
    # whose 4th and 5th group lie closer than 2^-48 in 80 bits are not
    # determined by fp64 and are left out.
    import combine_balancing_amd as cba
    L = np.longdouble
    c = np.sort((1 / (1 + np.exp(-l.astype(L))) + bias.astype(L)).reshape(T, 8, 8), 2)
    v = np.sort(c[:, :, -1] + c[:, :, -2], 1)
    clear = v[:, 4] - v[:, 3] > 2.0 ** -48
    assert clear.sum() > T // 4
    ids, _ = cba.route(ld, K, bias=torch.from_numpy(bias).cuda(), scoring="sigmoid", n_group=8,
                       topk_group=4)
    want, _ = ref.route(l.astype(np.float64), K, bias=bias, scoring="sigmoid", n_group=8,
                        topk_group=4)
    assert np.array_equal(ids.cpu().numpy()[clear], want[clear])


def _grad_check(ld, l, ids, d, dtype, **kw):
    import torch

    import combine_balancing_amd as cba
    got = cba.route_grad(ld, torch.from_numpy(ids).cuda(), torch.from_numpy(d).cuda(), **kw)
    torch.cuda.synchronize()
    want = ref.route_grad(l, ids, d, kw["scoring"], kw["renormalize"], kw["scale"])
    got = got.double().cpu().numpy()
    # a renormalised gradient subtracts the mean of g: fp64 rounding of it
    # against the largest g
    slack = 2.0 ** -46 * np.abs(d).max(initial=0) * kw["scale"] * ids.shape[1] * 1e3
    assert np.all(np.abs(got - want) <= GRAD_TOL[dtype] * np.abs(want) + TINY[dtype] + slack)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 256, 8), (5, 7, 3), (33, 64, 64), (257, 256, 8),
                                   (64, 384, 8), (19, 1000, 16), (1025, 160, 6)])
def test_route_grad_sizes(dtype, T, E, K):
    require_gpu()
    note(f"route_grad {dtype} T={T} E={E} K={K}")
    rng = np.random.default_rng(T + E)
    ld, l = _logits(rng, T, E, dtype)
    d = rng.standard_normal((T, K)).astype(np.float32)
    for scoring in ("softmax", "sigmoid"):
        ids = ref.route(l, K, scoring=scoring)[0]
        for renorm in (True, False):
            _grad_check(ld, l, ids, d, dtype, scoring=scoring, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("E,K", [(16, 4), (131, 8), (256, 8), (384, 16), (512, 2), (600, 8),
                                 (256, 20)])
def test_route_grad_many_tokens(dtype, E, K):
    torch = require_gpu()
    import combine_balancing_amd as cba
    note(f"route_grad many tokens {dtype} E={E} K={K}")
    T = 4099
    rng = np.random.default_rng(E * K)
    ld, l = _logits(rng, T, E, dtype, masked=0.1 if E % 2 else 0.0)
    d = rng.standard_normal((T, K)).astype(np.float32)
    rows = np.r_[np.arange(0, T, 13), T - 1]
    for scoring in ("softmax", "sigmoid"):
        ids, _ = cba.route(ld, K, scoring=scoring)
        ids[26] = ids[26, 0].item()         # one id K times
        for renorm in (True, False):
            got = cba.route_grad(ld, ids, torch.from_numpy(d).cuda(), scoring=scoring,
                                 renormalize=renorm, scale=2.5)
            torch.cuda.synchronize()
            want = ref.route_grad(l[rows], ids.cpu().numpy()[rows], d[rows], scoring, renorm, 2.5)
            got = got.double().cpu().numpy()[rows]
            slack = 2.0 ** -46 * np.abs(d).max() * 2.5 * K * 1e3
            assert np.all(np.abs(got - want) <= GRAD_TOL[dtype] * np.abs(want) + TINY[dtype] + slack)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_masked_repeated_and_bad_ids(scoring, renorm):
    require_gpu()
    note(f"route_grad masked {scoring} {renorm}")
    rng = np.random.default_rng(9)
    T, E, K = 70, 96, 6
    ld, l = _logits(rng, T, E, "float32", masked=0.4)
    ids = ref.route(l, K, scoring=scoring)[0]
    ids[3] = -1
    ids[4] = ids[4, 0]                    # one id six times
    ids[5, 2], ids[6, 1], ids[7, 0] = E, 2 ** 31 - 1, -2 ** 31
    d = rng.standard_normal((T, K)).astype(np.float32)
    _grad_check(ld, l, ids, d, "float32", scoring=scoring, renormalize=renorm, scale=1.0)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_against_differences(scoring, renorm):
    """Central differences of the scores in fp64, step 1e-5: truncation near
    1e-10, cancellation near 1e-11, against gradients of order 1; the kernel
    rounds to fp32. The bound 1e-6 covers both."""
    torch = require_gpu()
    import combine_balancing_amd as cba
    note(f"route_grad differences {scoring} {renorm}")
    rng = np.random.default_rng(4)
    T, E, K = 6, 24, 4
    l = rng.standard_normal((T, E)).astype(np.float32)
    ids = ref.route(l, K, scoring=scoring)[0]
    d = rng.standard_normal((T, K)).astype(np.float32)
    got = cba.route_grad(torch.from_numpy(l).cuda(), torch.from_numpy(ids).cuda(),
                         torch.from_numpy(d).cuda(), scoring=scoring, renormalize=renorm,
                         scale=1.5).cpu().numpy()
    h = 1e-5
    for e in range(E):
        lp, lm = l.astype(np.float64), l.astype(np.float64)
        lp[:, e] += h
        lm[:, e] -= h
        diff = (ref.route_scores(lp, ids, scoring, renorm, 1.5)
                - ref.route_scores(lm, ids, scoring, renorm, 1.5)) / (2 * h)
        assert np.all(np.abs((diff * d).sum(1) - got[:, e]) <= 1e-6)


def test_route_streams_and_graph():
    """Captured forward and gradient replay to the eager result on new
    inputs, and calls on two streams at once do not disturb each other."""
    torch = require_gpu()
    import combine_balancing_amd as cba
    note("route graph and streams")
    g = torch.Generator(device="cuda").manual_seed(1)
    l = torch.randn(300, 256, device="cuda", generator=g)
    bias = 0.1 * torch.randn(256, device="cuda", generator=g)
    ids = torch.empty(300, 8, dtype=torch.int32, device="cuda")
    sc = torch.empty(300, 8, device="cuda")
    dl = torch.empty_like(l)
    d = torch.randn(300, 8, device="cuda", generator=g)
    kw = dict(scoring="sigmoid", scale=2.5)

    def step():
        cba.route(l, 8, bias=bias, n_group=8, topk_group=4, topk_ids=ids, scores=sc, **kw)
        cba.route_grad(l, ids, d, dlogits=dl, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        l.copy_(torch.randn(300, 256, device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = ids.clone(), sc.clone(), dl.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], ids) and torch.equal(got[1], sc) and torch.equal(got[2], dl)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ls = [torch.randn(2000, 256, device="cuda", generator=g) for _ in streams]
    want = [cba.route(a, 8, **kw) for a in ls]
    torch.cuda.synchronize()
    for _ in range(4):
        outs = [cba.route(a, 8, stream=s, **kw) for a, s in zip(ls, streams)]
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_route_no_tokens():
    torch = require_gpu()
    import combine_balancing_amd as cba
    ids, sc = cba.route(torch.empty(0, 16, device="cuda"), 4)
    assert ids.shape == (0, 4) and sc.shape == (0, 4)
    assert cba.route_grad(torch.empty(0, 16, device="cuda"), ids, sc).shape == (0, 16)
