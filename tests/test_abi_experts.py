"""Host-side refusals of the router and expert entry points (no GPU needed:
a refused call enqueues nothing)."""
import ctypes
import os

import pytest

P = 4096  # a non-null, aligned address that a refused call never reads


@pytest.fixture(scope="module")
def B():
    from combine_balancing_amd import _binding
    if not os.path.exists(_binding.LIB_PATH):
        from combine_balancing_amd import build
        build.build()
    _binding.lib()
    return _binding


def _route(B, **kw):
    a = dict(T=4, E=16, K=2, logits=P, dtype=0, bias=None, scoring=0, ng=1, tg=1, renorm=1,
             scale=1.0, ids=P, scores=P)
    a.update(kw)
    return B.mep_route(a["T"], a["E"], a["K"], a["logits"], a["dtype"], a["bias"], a["scoring"],
                       a["ng"], a["tg"], a["renorm"], a["scale"], a["ids"], a["scores"], None)


def test_route_validation(B):
    for kw in (dict(logits=None), dict(ids=None), dict(scores=None)):
        assert _route(B, **kw) == B.MEP_ERR_NULLPTR
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(K=0), dict(K=65, E=128), dict(logits=P + 2),
               dict(logits=P + 1, dtype=1), dict(T=2 ** 30, K=2)):
        assert _route(B, **kw) == B.MEP_ERR_SHAPE
    for kw in (dict(K=17), dict(dtype=3), dict(dtype=-1), dict(scoring=2), dict(ng=0), dict(ng=3),
               dict(ng=65, E=130), dict(ng=4, tg=0), dict(ng=4, tg=5), dict(ng=8, tg=1, K=3),
               dict(scale=float("inf")), dict(scale=float("nan"))):
        assert _route(B, **kw) == B.MEP_ERR_PARAM, kw
    assert _route(B, T=0, logits=None, ids=None, scores=None) == B.MEP_OK


def _grad(B, **kw):
    a = dict(T=4, E=16, K=2, logits=P, dtype=0, ids=P, d=P, scoring=0, renorm=1, scale=1.0, dl=P)
    a.update(kw)
    return B.mep_route_grad(a["T"], a["E"], a["K"], a["logits"], a["dtype"], a["ids"], a["d"],
                            a["scoring"], a["renorm"], a["scale"], a["dl"], None)


def test_route_grad_validation(B):
    for kw in (dict(logits=None), dict(ids=None), dict(d=None), dict(dl=None)):
        assert _grad(B, **kw) == B.MEP_ERR_NULLPTR
    for kw in (dict(T=-1), dict(E=0), dict(E=2000), dict(K=0), dict(K=17), dict(dl=P + 2)):
        assert _grad(B, **kw) == B.MEP_ERR_SHAPE
    for kw in (dict(dtype=7), dict(scoring=-1), dict(scale=float("-inf"))):
        assert _grad(B, **kw) == B.MEP_ERR_PARAM
    assert _grad(B, T=0, logits=None, ids=None, d=None, dl=None) == B.MEP_OK


def test_route_tokens_of_one_launch(B):
    # up to 64 threads a token, fewer than 2^32 a launch
    for T in (2 ** 26, 2 ** 31 - 1):
        assert _route(B, T=T, E=1, K=1) == B.MEP_ERR_SHAPE
        assert _grad(B, T=T, E=1, K=1) == B.MEP_ERR_SHAPE


def _w(B, kind=1, E=2, N=16, K=128, group=32, sd=1, data=P, scales=P, zeros=None):
    return B.Weights(kind, E, N, K, group, sd, data, scales, zeros)


def test_packed_sizes(B):
    # 3 tiles of 8 rows; 1 and 3 blocks of 256 inputs
    assert B.mep_packed_code_bytes(2, 17, 136) == 2 * 3 * 1 * 1024
    assert B.mep_packed_scale_count(2, 17, 520, 64) == 2 * 3 * 3 * 8 * 4
    for a in ((0, 16, 128), (1025, 16, 128), (1, 0, 128), (1, 16, 12), (1, 16, 65544),
              (1, (1 << 20) + 1, 128)):
        assert B.mep_packed_code_bytes(*a) == 0 and B.mep_packed_scale_count(*a, 32) == 0
    assert B.mep_packed_scale_count(1, 16, 128, 48) == 0


def test_pack_and_quantize_validation(B):
    ok = [1, 16, 128, 1, 32, P, P, None, P, P, None, None]

    def pack(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return B.mep_pack_weights(*a)
    for i in (5, 6, 8, 9):
        assert pack(**{f"a{i}": None}) == B.MEP_ERR_NULLPTR
    assert pack(a3=0) == pack(a3=3) == pack(a4=16) == B.MEP_ERR_PARAM
    assert pack(a7=P) == pack(a10=P) == pack(a3=2, a7=P, a10=P) == B.MEP_ERR_PARAM
    assert pack(a0=0) == pack(a2=20) == pack(a8=P + 8) == pack(a9=P + 8) == B.MEP_ERR_SHAPE
    assert pack(a5=P + 4) == B.MEP_ERR_SHAPE
    q = [1, 16, 128, 1, 32, 1, P, P, P, None]
    for i in (6, 7, 8):
        assert B.mep_quant_weights(*q[:i], None, *q[i + 1:]) == B.MEP_ERR_NULLPTR
    for i, v in ((3, 0), (4, 31), (5, 0)):
        assert B.mep_quant_weights(*q[:i], v, *q[i + 1:]) == B.MEP_ERR_PARAM
    assert B.mep_quant_weights(1, 16, 129, *q[3:]) == B.MEP_ERR_SHAPE


def _mv(B, T=4, R=2, first=0, x=P, per=0, ids=P, mask=None, w=None, ob=P, of=None):
    w = _w(B) if w is None else w
    return B.mep_expert_matvec(T, R, first, x, per, ids, mask,
                               ctypes.byref(w) if w else None, ob, of, None)


def test_expert_matvec_validation(B):
    assert _mv(B, x=None) == B.MEP_ERR_NULLPTR
    assert _mv(B, ob=None) == B.MEP_ERR_NULLPTR
    assert _mv(B, w=False) == B.MEP_ERR_NULLPTR
    assert _mv(B, w=_w(B, data=None)) == _mv(B, w=_w(B, scales=None)) == B.MEP_ERR_NULLPTR
    assert _mv(B, of=P) == B.MEP_ERR_PARAM                      # two outputs
    assert _mv(B, ids=None) == B.MEP_ERR_PARAM                  # two matrices, no ids
    one = _w(B, E=1)
    for kw in (dict(mask=P), dict(per=1), dict(first=3)):
        assert _mv(B, ids=None, w=one, **kw) == B.MEP_ERR_PARAM
    for w in (_w(B, kind=0, scales=None), _w(B, kind=3), _w(B, group=16), _w(B, sd=0),
              _w(B, kind=2, zeros=P)):
        assert _mv(B, w=w) == B.MEP_ERR_PARAM
    for kw in (dict(T=-1), dict(R=0), dict(T=1025), dict(x=P + 8), dict(ob=P + 1),
               dict(w=_w(B, K=12)), dict(w=_w(B, E=1025)), dict(w=_w(B, data=P + 8)),
               dict(w=_w(B, scales=P + 4))):
        assert _mv(B, **kw) == B.MEP_ERR_SHAPE, kw
    assert _mv(B, T=0, x=None, ob=None) == B.MEP_OK


def _layer(B, T=4, K=2, H=128, I=64, first=0, x=P, ids=P, sc=P, mask=None, w13=None, w2=None,
           ws=P, wsb=1 << 30, ob=P, of=None):
    w13 = _w(B, N=2 * 64, K=128) if w13 is None else w13
    w2 = _w(B, N=128, K=64) if w2 is None else w2
    return B.mep_moe_layer(T, K, H, I, first, x, ids, sc, mask, ctypes.byref(w13),
                           ctypes.byref(w2), ws, wsb, ob, of, None)


def test_moe_layer_validation(B):
    for kw in (dict(x=None), dict(ids=None), dict(sc=None), dict(ws=None), dict(ob=None)):
        assert _layer(B, **kw) == B.MEP_ERR_NULLPTR
    need = B.mep_moe_layer_workspace_size(4, 2, 64)
    assert need > 8 * 64 * 6
    for kw in (dict(wsb=need - 1), dict(ws=P + 16), dict(w13=_w(B, E=3, N=128, K=128)),
               dict(w13=_w(B, kind=2, N=128, K=128)), dict(w13=_w(B, group=64, N=128, K=128)),
               dict(w13=_w(B, sd=2, N=128, K=128)), dict(w2=_w(B, N=128, K=64, zeros=P))):
        assert _layer(B, **kw) == B.MEP_ERR_PARAM, kw
    for kw in (dict(T=129), dict(T=-1), dict(K=0), dict(T=128, K=17), dict(H=136), dict(I=72),
               dict(x=P + 8), dict(ob=P + 8), dict(of=P + 4), dict(H=12)):
        assert _layer(B, **kw) == B.MEP_ERR_SHAPE, kw
    assert _layer(B, T=0, x=None, ids=None, sc=None, ob=None, ws=None) == B.MEP_OK
    for a in ((129, 1, 64), (1, 0, 64), (128, 17, 64), (1, 1, 12), (1, 1, 65544), (-1, 1, 64)):
        assert B.mep_moe_layer_workspace_size(*a) == 0


def test_tensor_level_refusals():
    import torch

    import combine_balancing_amd as cba
    l = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="device tensor|GPU"):
        cba.route(l, 2)
    with pytest.raises(ValueError, match="dtype"):
        cba.route(l.double(), 2)
    with pytest.raises(ValueError, match="scoring"):
        cba.route(l, 2, scoring="relu")
    with pytest.raises(ValueError, match="different devices"):
        cba.route(l, 2, bias=torch.zeros(8, device="meta"))
    with pytest.raises(ValueError, match="required"):
        cba.route(None, 2)
    with pytest.raises(ValueError, match="kind"):
        cba.q4_pack(torch.zeros(2, 8, dtype=torch.uint8), torch.zeros(2, 1), kind="int8")
    with pytest.raises(ValueError, match="unsupported"):
        cba.q4_pack(torch.zeros(2, 12, dtype=torch.uint8), torch.zeros(2, 1))
    with pytest.raises(ValueError, match="Q4Weights"):
        cba.expert_matvec_q4(torch.zeros(2, 8), torch.zeros(2, 8))
    with pytest.raises(ValueError, match="unsupported layer"):
        cba.moe_layer_workspace(200, 8, 64)
