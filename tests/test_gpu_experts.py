"""GPU parity of the 4-bit packing, the experts' products and the whole
expert layer against 64-bit references (expert_ref.py, which derives the
bounds)."""
import numpy as np
import pytest

import expert_ref as ref
from gpu_util import note, require_gpu

pytestmark = pytest.mark.gpu


def _torch16(a, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(dtype)


def _q4(rng, E, N, K, kind, group, zeros, scale="bf16", exact=False):
    """(Q4Weights, float64 values, magnitudes as multiplied)."""
    import torch

    import combine_balancing_amd as cba
    G = -(-K // group)
    codes = rng.integers(0, 16, (E, N, K)).astype(np.uint8)
    s = 2.0 ** rng.integers(-3, 3, (E, N, G)) if exact else rng.random((E, N, G)) + 0.2
    dt = torch.bfloat16 if scale == "bf16" else torch.float16
    st = _torch16(s, dt)
    z = rng.integers(0, 16, (E, N, G)).astype(np.uint8) if zeros else None
    w = cba.q4_pack(torch.from_numpy(codes).cuda(), st.cuda(),
                    zeros=None if z is None else torch.from_numpy(z).cuda(), group=group,
                    kind=kind)
    sv = st.double().numpy()
    val = ref.decode(codes, sv, z, group, kind)
    # int4: |16 + q| + 24 (or 16 + z) per input
    mag = np.abs(val) if kind == "fp4" else np.repeat(sv, group, 2)[:, :, :K] * 56.0
    return w, val, mag


def _route_ids(rng, T, R, E, first, bad=0.15):
    ids = rng.integers(0, E, (T, R)).astype(np.int32) + first
    ids[rng.random((T, R)) < bad] = first - 1 - rng.integers(0, 5)
    ids[rng.random((T, R)) < bad / 2] = first + E
    return ids


KINDS = [("int4", 32, False, "bf16"), ("int4", 64, True, "fp16"), ("int4", 128, False, "fp16"),
         ("int4", 128, True, "bf16"), ("int4", 64, False, "bf16"), ("int4", 32, True, "bf16"),
         ("fp4", 32, False, "bf16"), ("fp4", 64, False, "fp16"), ("fp4", 128, False, "bf16")]


@pytest.mark.parametrize("kind,group,zeros,scale", KINDS)
@pytest.mark.parametrize("T,N,K", [(1, 1, 8), (1, 16, 128), (2, 17, 136), (16, 33, 520),
                                   (17, 100, 1000), (40, 5, 2056), (3, 1001, 264)])
def test_matvec_dense_exact(kind, group, zeros, scale, T, N, K):
    # small whole-number inputs and power-of-two scales: every partial sum is
    # a multiple of 2^-4 below 2^20, so fp32 holds all of them exactly
    torch = require_gpu()
    import combine_balancing_amd as cba
    note(f"matvec dense {kind} g={group} z={zeros} {scale} T={T} N={N} K={K}")
    rng = np.random.default_rng(T + N + K + group)
    w, val, _ = _q4(rng, 1, N, K, kind, group, zeros, scale, exact=True)
    x = rng.integers(-3, 4, (T, K)).astype(np.float32)
    got = cba.expert_matvec_q4(_torch16(x, torch.bfloat16).cuda(), w, out_dtype=torch.float32)
    torch.cuda.synchronize()
    want = x.astype(np.float64) @ val[0].T
    assert np.abs(want).max() < 2 ** 20
    assert np.array_equal(got.double().cpu().numpy(), want)


@pytest.mark.parametrize("kind,group,zeros,scale", KINDS)
@pytest.mark.parametrize("per_route", [False, True])
@pytest.mark.parametrize("T,R,E,N,K", [(1, 8, 32, 48, 256), (5, 3, 13, 50, 1024 + 88),
                                       (64, 2, 3, 20, 136), (128, 16, 40, 16, 64)])
def test_matvec_routed(kind, group, zeros, scale, per_route, T, R, E, N, K):
    torch = require_gpu()
    import combine_balancing_amd as cba
    note(f"matvec routed {kind} g={group} z={zeros} {scale} per={per_route} {(T, R, E, N, K)}")
    rng = np.random.default_rng(T + R + N + group)
    w, val, mag = _q4(rng, E, N, K, kind, group, zeros, scale)
    first = 7
    ids = _route_ids(rng, T, R, E, first)
    mask = (rng.random((T, R)) < 0.8).astype(np.uint8)
    x = ref.bf16(rng.standard_normal((T, R, K) if per_route else (T, K)))
    xd = _torch16(x, torch.bfloat16).cuda()
    for m, dt, name in ((None, torch.float32, "fp32"), (mask, torch.bfloat16, "bf16")):
        out = torch.full((T, R, N), 7.0, dtype=dt, device="cuda")
        md = None if m is None else torch.from_numpy(m).cuda()
        cba.expert_matvec_q4(xd, w, ids=torch.from_numpy(ids).cuda(), first=first, mask=md, out=out)
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        want, hit = ref.matvec(x, val, ids, first, m, np.full((T, R, N), 7.0), per_route)
        lim, _ = ref.matvec(np.abs(x), mag, ids, first, m, np.zeros((T, R, N)), per_route)
        lim = ref.product_slack(lim, K)
        assert np.array_equal(got[~hit], want[~hit])  # untouched
        assert np.all(np.abs(got - want)[hit]
                      <= (lim + ref.HALF[name] * (np.abs(want) + lim))[hit])


def test_matvec_nan_and_inf_stay_in_their_route():
    torch = require_gpu()
    import combine_balancing_amd as cba
    note("matvec nan")
    rng = np.random.default_rng(2)
    for kind in ("int4", "fp4"):
        w, val, mag = _q4(rng, 4, 40, 264, kind, 64, False)
        x = ref.bf16(rng.standard_normal((6, 264)))
        x[1, 5], x[2, 263], x[4] = np.nan, np.inf, -np.inf
        ids = np.zeros((6, 1), np.int32)
        out = cba.expert_matvec_q4(_torch16(x, torch.bfloat16).cuda(), w,
                                   ids=torch.from_numpy(ids).cuda(), out_dtype=torch.float32)
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()[:, 0]
        for t in (0, 3, 5):
            want = val[0] @ x[t].astype(np.float64)
            assert np.all(np.abs(got[t] - want)
                          <= ref.product_slack(mag[0] @ np.abs(x[t].astype(np.float64)), 264)
                          + ref.U32 * np.abs(want))
        assert not np.isfinite(got[[1, 4]]).any() and not np.isfinite(got[2]).all()


@pytest.mark.parametrize("kind", ["int4", "fp4"])
@pytest.mark.parametrize("scale", ["bfloat16", "float16"])
@pytest.mark.parametrize("E,N,K,group", [(1, 3, 8, 32), (2, 17, 136, 64), (3, 5, 1000, 128)])
def test_quantize(kind, scale, E, N, K, group):
    torch = require_gpu()
    import combine_balancing_amd as cba
    note(f"quantize {kind} {scale} {E, N, K, group}")
    rng = np.random.default_rng(K)
    w = ref.bf16(rng.standard_normal((E, N, K)) * 0.05)
    w[0, 0, :] = 0.0
    w[0, 1, :5] = [0.25, 0.5, -0.75, 1.0, 6.0]  # ties where the scale is 1
    codes, scales = cba.q4_quantize(_torch16(w, torch.bfloat16).cuda(), group=group, kind=kind,
                                    scale_dtype=getattr(torch, scale))
    torch.cuda.synchronize()
    codes, scales = codes.cpu().numpy(), scales.cpu()
    top = np.float32(6 if kind == "fp4" else 7)
    for g in range(-(-K // group)):
        b = w[:, :, g * group:(g + 1) * group]
        s = torch.from_numpy(np.abs(b).max(2) / top).to(getattr(torch, scale))
        assert torch.equal(s, scales[:, :, g])
        sf = s.float().numpy()[:, :, None]
        with np.errstate(divide="ignore", invalid="ignore"):
            v = np.where(sf > 0, b / sf, np.float32(0)).astype(np.float32)
        c = codes[:, :, g * group:(g + 1) * group]
        if kind == "int4":
            assert np.array_equal(c, np.clip(np.rint(v), -8, 7).astype(np.int32) + 8)
        else:
            # nearest value, ties to the even code: the sum of two distances
            # to the neighbours decides
            d = np.abs(np.abs(v)[..., None].astype(np.float64) - ref.FP4[:8])
            order = np.lexsort((np.broadcast_to(np.arange(8) % 2, d.shape), d), axis=-1)[..., 0]
            want = order + np.where((v < 0) & (order > 0), 8, 0)
            assert np.array_equal(c, want)


@pytest.mark.parametrize("kind", ["int4", "fp4"])
def test_quantize_past_fp16_scales(kind):
    # max |w| / 7 above fp16's range: the scale is its largest finite value
    # and the codes stop at their ends
    torch = require_gpu()
    import combine_balancing_amd as cba
    note(f"quantize past fp16 {kind}")
    w = torch.zeros(2, 64, dtype=torch.bfloat16)
    w[0, 3], w[0, 4], w[0, 40], w[1, 0] = 2.0 ** 20, -(2.0 ** 30), 65536.0, 3e38
    codes, scales = cba.q4_quantize(w.cuda(), group=32, kind=kind, scale_dtype=torch.float16)
    torch.cuda.synchronize()
    codes, scales = codes.cpu(), scales.cpu()
    low = torch.tensor(65536.0 / (6 if kind == "fp4" else 7)).half()
    assert scales[0].tolist() == [65504.0, low.item()] and scales[1].tolist() == [65504.0, 0.0]
    # 2^20 / 65504 is past either kind's largest value, as is -2^30 / 65504
    # (int4's lowest is -8)
    ends = [7, 15, 7] if kind == "fp4" else [15, 0, 15]
    assert [int(codes[0, 3]), int(codes[0, 4]), int(codes[1, 0])] == ends
    assert int(codes[0, 40]) == (7 if kind == "fp4" else 15)


def test_quantize_pack_product_chain():
    # weights through q4_quantize, q4_pack and the product: the result is the
    # product with the quantized values, and near the one with the originals
    torch = require_gpu()
    import combine_balancing_amd as cba
    note("quantize chain")
    rng = np.random.default_rng(12)
    w = ref.bf16(rng.standard_normal((70, 520)) * 0.05)
    x = ref.bf16(rng.standard_normal((9, 520)))
    for kind in ("int4", "fp4"):
        codes, scales = cba.q4_quantize(_torch16(w, torch.bfloat16).cuda(), group=32, kind=kind)
        q = cba.q4_pack(codes, scales, group=32, kind=kind)
        y = cba.expert_matvec_q4(_torch16(x, torch.bfloat16).cuda(), q, out_dtype=torch.float32)
        torch.cuda.synchronize()
        sv = scales.double().cpu().numpy()[None]
        val = ref.decode(codes.cpu().numpy()[None], sv, None, 32, kind)[0]
        mag = np.repeat(sv, 32, 2)[0, :, :520] * 56.0
        x64 = x.astype(np.float64)
        want = x64 @ val.T
        lim = ref.product_slack(np.abs(x64) @ mag.T, 520) + ref.U32 * np.abs(want)
        assert np.all(np.abs(y.double().cpu().numpy() - want) <= lim)
        # every weight is off by at most half the largest step (int4: 1, of
        # amax / 7; fp4: 2, of amax / 6) and the rounding of the scale
        amax = np.abs(w).reshape(70, -1)[:, :512].reshape(70, 16, 32).max(2)
        step = (0.5 / 7 if kind == "int4" else 1.0 / 6) + 2.0 ** -8
        err = np.abs(val[:, :512] - w[:, :512]).reshape(70, 16, 32)
        assert np.all(err <= amax[:, :, None] * step * (1 + 1e-6))


# ------------------------------------------------------------------- layer

def _layer_case(rng, T, K, E, H, I, kind, group=0, zeros=False, scale="bf16"):
    import torch
    if kind == "bf16":
        a = ref.bf16(rng.standard_normal((E, 2 * I, H)) / np.sqrt(H))
        b = ref.bf16(rng.standard_normal((E, H, I)) / np.sqrt(I))
        return (_torch16(a, torch.bfloat16).cuda(), a.astype(np.float64), None,
                _torch16(b, torch.bfloat16).cuda(), b.astype(np.float64), None)
    return (*_q4(rng, E, 2 * I, H, kind, group, zeros, scale),
            *_q4(rng, E, H, I, kind, group, zeros, scale))


def _layer_check(rng, T, K, E, H, I, kind, group=0, zeros=False, scale="bf16", ids=None,
                 first=3, mask=None, scores=None):
    import torch

    import combine_balancing_amd as cba
    w13, v13, m13, w2, v2, m2 = _layer_case(rng, T, K, E, H, I, kind, group, zeros, scale)
    if ids is None:
        ids = _route_ids(rng, T, K, E, first)
    if scores is None:
        scores = rng.standard_normal((T, K)).astype(np.float32)
    # 4-bit values are of order 4: keep h moderate
    x = ref.bf16(rng.standard_normal((T, H)) * (1.0 if kind == "bf16" else 4.0 / np.sqrt(H)))
    out_b = torch.full((T, H), 9.0, dtype=torch.bfloat16, device="cuda")
    out_f = torch.full((T, H), 9.0, device="cuda")
    ws = cba.moe_layer_workspace(T, K, I)
    ws.fill_(255)  # contents on entry do not matter
    cba.moe_layer(_torch16(x, torch.bfloat16).cuda(), torch.from_numpy(ids).cuda(),
                  torch.from_numpy(scores).cuda(), w13, w2, first=first,
                  mask=None if mask is None else torch.from_numpy(mask).cuda(), workspace=ws,
                  out_bf16=out_b, out_f32=out_f)
    torch.cuda.synchronize()
    want, lim = ref.layer(x, ids, scores, v13, v2, first, mask, m13, m2)
    for got, name in ((out_f, "fp32"), (out_b, "bf16")):
        g = got.double().cpu().numpy()
        err = np.abs(g - want)
        assert np.all(err <= lim + ref.HALF[name] * (np.abs(want) + lim)), (err - lim).max()
    return out_f, want


LAYER_KINDS = [("bf16", 0, False, "bf16")] + KINDS


@pytest.mark.parametrize("kind,group,zeros,scale", LAYER_KINDS)
@pytest.mark.parametrize("T,K,E,H,I", [(1, 1, 1, 8, 8), (1, 8, 12, 256, 136), (2, 3, 5, 136, 24),
                                       (17, 4, 3, 72, 264)])
def test_layer(kind, group, zeros, scale, T, K, E, H, I):
    require_gpu()
    note(f"layer {kind} g={group} z={zeros} {scale} {(T, K, E, H, I)}")
    _layer_check(np.random.default_rng(T + H + I + group), T, K, E, H, I, kind, group, zeros, scale)


@pytest.mark.parametrize("kind,group", [("bf16", 0), ("int4", 128), ("fp4", 32)])
@pytest.mark.parametrize("T,K,E,H,I", [(64, 8, 40, 64, 40), (128, 16, 5, 40, 16),
                                       (128, 1, 1, 1000, 344), (7, 3, 16, 1000, 344),
                                       (65, 2, 300, 24, 8), (32, 64, 64, 16, 16)])
def test_layer_sizes(kind, group, T, K, E, H, I):
    require_gpu()
    note(f"layer sizes {kind} {(T, K, E, H, I)}")
    _layer_check(np.random.default_rng(T + H), T, K, E, H, I, kind, group)


@pytest.mark.parametrize("kind,group", [("bf16", 0), ("int4", 128), ("fp4", 64)])
@pytest.mark.parametrize("T,K", [(16, 4), (13, 5), (128, 16), (1, 64), (1, 65), (32, 2)])
def test_layer_most_experts(kind, group, T, K):
    # 1024 experts, the last among them; 64 routes and one more
    require_gpu()
    note(f"layer 1024 experts {kind} {(T, K)}")
    rng = np.random.default_rng(T * K)
    ids = rng.integers(0, 1024, (T, K)).astype(np.int32)
    ids[0, 0], ids[-1, -1] = 1023, 0
    _layer_check(rng, T, K, 1024, 16, 8, kind, group, ids=ids, first=0)


def test_products_graph():
    torch = require_gpu()
    import combine_balancing_amd as cba
    note("products graph")
    rng = np.random.default_rng(77)
    w, _, _ = _q4(rng, 6, 70, 264, "int4", 64, True)
    g = torch.Generator(device="cuda").manual_seed(5)
    for T, R in ((5, 4), (40, 3)):
        x = torch.randn(T, 264, device="cuda", generator=g).bfloat16()
        ids = torch.randint(-1, 6, (T, R), device="cuda", generator=g, dtype=torch.int32)
        out = torch.zeros(T, R, 70, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            cba.expert_matvec_q4(x, w, ids=ids, out=out)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cba.expert_matvec_q4(x, w, ids=ids, out=out)
        for _ in range(3):
            x.copy_(torch.randn(T, 264, device="cuda", generator=g))
            ids.copy_(torch.randint(-1, 6, (T, R), device="cuda", generator=g, dtype=torch.int32))
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
            out.zero_()
            cba.expert_matvec_q4(x, w, ids=ids, out=out)
            torch.cuda.synchronize()
            assert torch.equal(got, out)


@pytest.mark.parametrize("kind,group", [("bf16", 0), ("int4", 64), ("fp4", 128)])
def test_layer_masks_repeats_and_empty(kind, group):
    require_gpu()
    note(f"layer masks {kind}")
    rng = np.random.default_rng(5)
    T, K, E, H, I, first = 20, 6, 9, 136, 72, 100
    ids = _route_ids(rng, T, K, E, first)
    ids[0] = first + 4                    # one expert six times
    ids[1, 0] = ids[1, 3] = ids[1, 5] = first
    ids[2] = first - 1                    # nothing held here
    ids[3] = [-2 ** 31, 2 ** 31 - 1, -1, 0, first + E, first - 1]
    mask = (rng.random((T, K)) < 0.7).astype(np.uint8)
    mask[4] = 0
    scores = rng.standard_normal((T, K)).astype(np.float32)
    scores[5] = 0.0
    scores[mask == 0] = np.nan            # a pruned route's score is not used
    out, want = _layer_check(rng, T, K, E, H, I, kind, group, ids=ids, first=first, mask=mask,
                             scores=scores)
    assert not out[2].any() and not out[3].any() and not out[4].any()
    ids[:] = -1
    out, _ = _layer_check(rng, T, K, E, H, I, kind, group, ids=ids, first=first)
    assert not out.any()


def test_layer_nan_stays_in_its_token():
    # a token with a NaN input, and an expert with NaN weights that only one
    # token takes, leave every other token's row as it was
    torch = require_gpu()
    import combine_balancing_amd as cba
    note("layer nan")
    g = torch.Generator(device="cuda").manual_seed(3)
    T, K, E, H, I = 10, 2, 6, 136, 72
    w13 = (torch.randn(E, 2 * I, H, device="cuda", generator=g) / 12).bfloat16()
    w2 = (torch.randn(E, H, I, device="cuda", generator=g) / 8).bfloat16()
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    ids = torch.randint(0, E - 1, (T, K), device="cuda", generator=g, dtype=torch.int32)
    sc = torch.rand(T, K, device="cuda", generator=g)
    clean, _ = cba.moe_layer(x, ids, sc, w13, w2)
    ids2 = ids.clone()
    ids2[7, 1] = E - 1
    w13[E - 1, 3, 5] = float("nan")
    w2[E - 1, :, 2] = float("inf")
    x2 = x.clone()
    x2[4, 9] = float("nan")
    bad, _ = cba.moe_layer(x2, ids2, sc, w13, w2)
    torch.cuda.synchronize()
    keep = [t for t in range(T) if t not in (4, 7)]
    assert torch.equal(clean[keep], bad[keep])
    assert bad[4].isnan().all() and not bad[7].isfinite().all()


def test_layer_overflow_matches_plain():
    # h beyond bf16 and fp32: infinities come out where the formula has them
    torch = require_gpu()
    import combine_balancing_amd as cba
    note("layer overflow")
    H = I = 64
    w13 = torch.zeros(1, 2 * I, H, device="cuda", dtype=torch.bfloat16)
    w13[0, :, 0] = 1.0
    w2 = torch.eye(I, device="cuda", dtype=torch.bfloat16)[None].contiguous()
    x = torch.zeros(4, H, device="cuda", dtype=torch.bfloat16)
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 1e25, -1e25, 200.0, -200.0
    ids = torch.zeros(4, 1, device="cuda", dtype=torch.int32)
    sc = torch.ones(4, 1, device="cuda")
    _, out = cba.moe_layer(x, ids, sc, w13, w2, out_bf16=False, out_f32=True)
    torch.cuda.synchronize()
    # 0 * inf of the identity's other columns is NaN, as in the formula
    assert not out[0].isfinite().any()
    xf = x[:, 0].float()
    assert torch.equal(out[1], torch.zeros_like(out[1])) or out[1].isfinite().all()
    assert torch.allclose(out[2], (xf[2] * xf[2]).expand(H), rtol=2.0 ** -15)
    assert torch.all(out[3].abs() < 1e-30)


def test_layer_is_deterministic_and_batch_graph():
    torch = require_gpu()
    import combine_balancing_amd as cba
    note("layer graph")
    g = torch.Generator(device="cuda").manual_seed(8)
    T, K, E, H, I = 24, 4, 20, 512, 200
    w13 = (torch.randn(E, 2 * I, H, device="cuda", generator=g) / 22).bfloat16()
    w2 = (torch.randn(E, H, I, device="cuda", generator=g) / 14).bfloat16()
    logits = torch.randn(T, E, device="cuda", generator=g)
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    sc = torch.empty(T, K, device="cuda")
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ws = cba.moe_layer_workspace(T, K, I)

    def step():
        cba.route(logits, K, topk_ids=ids, scores=sc)
        cba.moe_layer(x, ids, sc, w13, w2, out_bf16=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        logits.copy_(torch.randn(T, E, device="cuda", generator=g))
        x.copy_(torch.randn(T, H, device="cuda", generator=g))
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.fill_(5.0)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out)


def test_layer_two_streams():
    torch = require_gpu()
    import combine_balancing_amd as cba
    note("layer two streams")
    g = torch.Generator(device="cuda").manual_seed(9)
    E, H, I, K = 8, 256, 128, 2
    w13 = (torch.randn(E, 2 * I, H, device="cuda", generator=g) / 16).bfloat16()
    w2 = (torch.randn(E, H, I, device="cuda", generator=g) / 11).bfloat16()
    streams, args = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for T in (40, 9):
        args.append((torch.randn(T, H, device="cuda", generator=g).bfloat16(),
                     torch.randint(0, E, (T, K), device="cuda", generator=g, dtype=torch.int32),
                     torch.rand(T, K, device="cuda", generator=g)))
    want = [cba.moe_layer(*a, w13, w2)[0] for a in args]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [cba.moe_layer(*a, w13, w2, stream=s)[0] for a, s in zip(args, streams)]
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_decode_step_with_remap():
    """route -> remap_prune -> moe_layer per rank: the ranks' rows add up to
    the layer over logical experts, pruned routes left out."""
    torch = require_gpu()
    import combine_balancing_amd as cba
    note("decode step with remap")
    rng = np.random.default_rng(21)
    T, K, E, H, I, world, ppr = 12, 4, 6, 136, 72, 4, 2
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    ids, sc = cba.route(logits, K)
    # experts 0 and 1 have two instances each
    inst_of = [[0, 7], [1, 6], [2], [3], [4], [5]]
    F = 3
    table = np.zeros((E, F), np.int32)
    for e, v in enumerate(inst_of):
        table[e, 0] = len(v)
        table[e, 1:1 + len(v)] = v
    thr = torch.full((K,), 0.25, device="cuda")
    r = cba.remap_prune(ids, torch.from_numpy(table).cuda(), world, ppr, 0, 1, expert_scales=sc,
                        pruning_threshold=thr)
    w13 = ref.bf16(rng.standard_normal((E, 2 * I, H)) / 12)
    w2 = ref.bf16(rng.standard_normal((E, H, I)) / 8)
    logical = [0] * (world * ppr)
    for e, v in enumerate(inst_of):
        for i in v:
            logical[i] = e
    x = ref.bf16(rng.standard_normal((T, H)))
    total = np.zeros((T, H))
    for rank in range(world):
        mine = logical[rank * ppr:(rank + 1) * ppr]
        _, y = cba.moe_layer(_torch16(x, torch.bfloat16).cuda(), r["balanced_ids"], sc,
                             _torch16(w13[mine], torch.bfloat16).cuda(),
                             _torch16(w2[mine], torch.bfloat16).cuda(), first=rank * ppr,
                             mask=r["balanced_mask"], out_bf16=False, out_f32=True)
        total += y.double().cpu().numpy()
    torch.cuda.synchronize()
    mask = r["balanced_mask"].cpu().numpy().reshape(T, K)
    assert 0 < mask.sum() < T * K
    want, lim = ref.layer(x, ids.cpu().numpy(), sc.cpu().numpy(), w13.astype(np.float64),
                          w2.astype(np.float64), 0, mask)
    assert np.all(np.abs(total - want) <= lim + 8 * ref.U32 * (np.abs(want) + lim))


def test_products_then_combine():
    """4-bit products per route, then the library's combine over them, as an
    expert without activation would be used."""
    torch = require_gpu()
    import combine_balancing_amd as cba
    note("products then combine")
    rng = np.random.default_rng(31)
    T, K, E, N, Kin = 6, 3, 5, 64, 136
    w, val, mag = _q4(rng, E, N, Kin, "int4", 64, False)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    ids, sc = cba.route(torch.from_numpy(logits).cuda(), K, scoring="sigmoid")
    x = ref.bf16(rng.standard_normal((T, Kin)))
    y = cba.expert_matvec_q4(_torch16(x, torch.bfloat16).cuda(), w, ids=ids)
    pos = torch.arange(T * K, dtype=torch.int32, device="cuda")
    _, out = cba.combine(y.view(T * K, N), pos, sc, out_bf16=False, out_f32=True)
    torch.cuda.synchronize()
    i, s = ids.cpu().numpy(), sc.double().cpu().numpy()
    yr, _ = ref.matvec(x, val, i, 0, None, np.zeros((T, K, N)))
    lim, _ = ref.matvec(np.abs(x), mag, i, 0, None, np.zeros((T, K, N)))
    lim = ref.product_slack(lim, Kin)
    lim = lim + ref.HALF["bf16"] * (np.abs(yr) + lim)
    want = (s[:, :, None] * yr).sum(1)
    bound = (s[:, :, None] * (lim + 2 * K * ref.U32 * (np.abs(yr) + lim))).sum(1)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound)


def test_no_tokens():
    torch = require_gpu()
    import combine_balancing_amd as cba
    w13 = torch.zeros(2, 16, 8, dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros(2, 8, 8, dtype=torch.bfloat16, device="cuda")
    i32 = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    out, _ = cba.moe_layer(torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"), i32,
                           torch.empty(0, 2, device="cuda"), w13, w2)
    assert out.shape == (0, 8)


# ------------------------------------------------- sizes of the wide variants
#
# The references below run in float64 on the GPU (two-dimensional products),
# with the same bounds as expert_ref.


def _q4_gpu(g, E, N, K, kind, group, zeros, dt, exact):
    import torch

    import combine_balancing_amd as cba
    G = -(-K // group)
    codes = torch.randint(0, 16, (E, N, K), generator=g, device="cuda", dtype=torch.uint8)
    if exact:
        s = torch.exp2(torch.randint(-3, 3, (E, N, G), generator=g, device="cuda").float())
    else:
        s = (torch.rand(E, N, G, generator=g, device="cuda") + 0.2) / K ** 0.5 / 4
    s = s.to(dt)
    z = None
    if zeros:
        z = torch.randint(0, 16, (E, N, G), generator=g, device="cuda", dtype=torch.uint8)
    w = cba.q4_pack(codes, s, zeros=z, group=group, kind=kind)
    table = torch.tensor(ref.FP4, device="cuda")

    def dense(e):
        sv = s[e].double().repeat_interleave(group, 1)[:, :K]
        if kind == "fp4":
            v = table[codes[e].long()] * sv
            return v, v.abs()
        zv = 8.0 if z is None else z[e].double().repeat_interleave(group, 1)[:, :K]
        return (codes[e].double() - zv) * sv, 56.0 * sv
    return w, dense


@pytest.mark.parametrize("kind,group,zeros,scale", KINDS)
@pytest.mark.parametrize("T,R,E,N,K", [(8, 8, 32, 520, 264),      # 64 routes, one chunk a wave
                                       (20, 8, 40, 417, 264),     # more than 64 routes
                                       (40, 2, 16, 1048, 4360),   # two chunks a wave
                                       (3, 1, 3, 7000, 2056), (9, 4, 4, 600, 1000),
                                       (130, 3, 3, 90, 520), (2, 0, 1, 16500, 264)])
def test_matvec_wide_exact(kind, group, zeros, scale, T, R, E, N, K):
    # whole numbers and power-of-two scales: all partial sums are exact
    torch = require_gpu()
    import combine_balancing_amd as cba
    note(f"matvec wide {kind} g={group} z={zeros} {(T, R, E, N, K)}")
    g = torch.Generator(device="cuda").manual_seed(T + N)
    dt = torch.bfloat16 if scale == "bf16" else torch.float16
    w, dense = _q4_gpu(g, E, N, K, kind, group, zeros, dt, True)
    x = torch.randint(-3, 4, (T, K), generator=g, device="cuda").bfloat16()
    if R == 0:
        got = cba.expert_matvec_q4(x, w, out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert torch.equal(got.double(), x.double() @ dense(0)[0].t())
        return
    ids = torch.randint(-1, E, (T, R), generator=g, device="cuda", dtype=torch.int32)
    ids[::3] = ids[0, 0].clamp(0)  # one crowded expert
    got = cba.expert_matvec_q4(x, w, ids=ids, out=torch.full((T, R, N), 5.0, device="cuda"))
    torch.cuda.synchronize()
    want = torch.full((T, R, N), 5.0, device="cuda", dtype=torch.float64)
    for e in range(E):
        t, r = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            want[t, r] = x[t].double() @ dense(e)[0].t()
    assert torch.equal(got.double(), want)


@pytest.mark.parametrize("kind,group,zeros,scale", [("bf16", 0, False, "bf16"),
                                                    ("int4", 128, False, "bf16"),
                                                    ("int4", 64, True, "fp16"),
                                                    ("int4", 128, True, "bf16"),
                                                    ("fp4", 32, False, "bf16"),
                                                    ("fp4", 128, False, "fp16")])
@pytest.mark.parametrize("T,K,E,H,I", [(16, 4, 64, 1032, 264),    # held, one chunk a wave
                                       (33, 4, 64, 4104, 264),    # held, two; two tiles out
                                       (5, 3, 64, 6152, 1032),    # held, four (bf16); four tiles
                                       (40, 2, 24, 6152, 136),    # four tiles, four waves
                                       (100, 4, 6, 4104, 136),    # read in pairs of blocks
                                       (128, 8, 8, 6152, 264)])
def test_layer_wide(kind, group, zeros, scale, T, K, E, H, I):
    torch = require_gpu()
    import combine_balancing_amd as cba
    note(f"layer wide {kind} g={group} z={zeros} {(T, K, E, H, I)}")
    g = torch.Generator(device="cuda").manual_seed(T + H + I)
    dt = torch.bfloat16 if scale == "bf16" else torch.float16
    first = 11
    if kind == "bf16":
        w13 = (torch.randn(E, 2 * I, H, generator=g, device="cuda") / H ** 0.5).bfloat16()
        w2 = (torch.randn(E, H, I, generator=g, device="cuda") / I ** 0.5).bfloat16()
        d13, d2 = (lambda e: (w13[e].double(),) * 2), (lambda e: (w2[e].double(),) * 2)
    else:
        w13, d13 = _q4_gpu(g, E, 2 * I, H, kind, group, zeros, dt, False)
        w2, d2 = _q4_gpu(g, E, H, I, kind, group, zeros, dt, False)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    ids = torch.randint(-2, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    ids[::5, 0] = 3
    mask = (torch.rand(T, K, generator=g, device="cuda") < 0.9).to(torch.uint8)
    sc = torch.randn(T, K, generator=g, device="cuda")
    want = torch.zeros(T, H, device="cuda", dtype=torch.float64)
    lim = torch.zeros_like(want)
    for e in range(E):
        t, k = ((ids == e) & (mask > 0)).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        (a, am), (b, bm) = d13(e), d2(e)
        xt, s = x[t].double(), sc[t, k].double()[:, None]
        gu, d = xt @ a.t(), ref.product_slack(xt.abs() @ am.abs().t(), H)
        gate, up, dg, du = gu[:, :I], gu[:, I:], d[:, :I], d[:, I:]
        sl = gate * torch.sigmoid(gate)
        h = sl * up
        dh = (1.1 * dg + 8 * ref.U32 * sl.abs()) * (up.abs() + du) + sl.abs() * du
        dh = dh + h.abs() * 2.0 ** -16
        y = h @ b.t()
        ly = dh @ bm.abs().t() + ref.product_slack((h.abs() + dh) @ bm.abs().t(), I)
        want.index_add_(0, t, s * y)
        lim.index_add_(0, t, s.abs() * (ly + (4 + 17 * K) * ref.U32 * (y.abs() + ly)))
    for f32 in (False, True):
        ob, of = cba.moe_layer(x, ids + first, sc, w13, w2, first=first, mask=mask,
                               out_bf16=not f32, out_f32=f32)
        torch.cuda.synchronize()
        got = of if f32 else ob
        half = ref.HALF["fp32" if f32 else "bf16"]
        err = (got.double() - want).abs()
        assert bool((err <= lim + half * (want.abs() + lim)).all()), float((err - lim).max())


def test_quantize_and_pack_past_one_launch():
    # more groups than one launch has waves for: the last rows are reached too
    torch = require_gpu()
    import combine_balancing_amd as cba
    note("quantize large")
    N, K, group = 40000, 4096, 32
    g = torch.Generator(device="cuda").manual_seed(4)
    w = torch.randn(N, K, generator=g, device="cuda").bfloat16()
    codes, scales = cba.q4_quantize(w, group=group)
    tail = w[-64:].float().view(64, K // group, group)
    s = (tail.abs().amax(2) / 7).bfloat16()
    assert torch.equal(scales[-64:], s)
    want = torch.clamp(torch.round(tail / s.float()[..., None]), -8, 7) + 8
    assert torch.equal(codes[-64:].view(64, K // group, group).float(), want)
    q = cba.q4_pack(codes, scales, group=group)
    x = torch.randint(-3, 4, (2, K), generator=g, device="cuda").bfloat16()
    y = cba.expert_matvec_q4(x, q, out_dtype=torch.float32)
    torch.cuda.synchronize()
    val = (codes.double() - 8) * scales.double().repeat_interleave(group, 1)
    ref64 = x.double() @ val.t()
    lim = ref.product_slack(x.double().abs() @ (56.0 * scales.double().repeat_interleave(group, 1)).t(), K)
    assert bool(((y.double() - ref64).abs() <= lim + ref.U32 * ref64.abs()).all())
