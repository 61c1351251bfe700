"""The operators around the expert layer on the CPU: argument checks of the C calls (nothing is
launched), checks of the binding, and the oracle's definitions against differences and
against the layer's own oracle."""

import ctypes
import itertools

import numpy as np
import pytest
import torch

import mixture_experts_ffn_02_amd as pkg
import oracle
from mixture_experts_ffn_02_amd import _lib
from mixture_experts_ffn_02_amd import moe_lora as ml
from oracle import operators_ref as ref

FAKE = 1 << 20  # 16-byte aligned, never dereferenced: validation fails first


def _scoring(**kw):
    v = dict(score=0, logits_dtype=0, renormalize=1, n_group=1, topk_group=1, group_score=1, scale=1.0, bias=None)
    v.update(kw)
    return _lib.ScoringC(*[v[f] for f, _ in _lib.ScoringC._fields_])


def _route(d, sc, logits=FAKE, ws_bytes=1 << 30, ws=FAKE):
    return pkg.load().moe_lora_route_scored(ctypes.byref(d), ctypes.byref(sc) if sc else None, logits, FAKE, FAKE, FAKE,
                                            FAKE, FAKE, ws, ws_bytes, None)


@pytest.mark.parametrize("change", [dict(score=2), dict(score=-1), dict(logits_dtype=2), dict(renormalize=2),
                                    dict(n_group=0), dict(n_group=3), dict(n_group=65), dict(n_group=4, topk_group=5),
                                    dict(n_group=4, topk_group=0), dict(group_score=0), dict(group_score=3),
                                    dict(n_group=4, topk_group=1), dict(bias=FAKE + 4)])
def test_route_scored_refusals(change):
    d = _lib.Dims(16, 8, 8, 8, 3)  # k = 3 does not fit one group of two experts
    assert _route(d, _scoring(**change)) == _lib.ERR_INVALID_ARGUMENT


def test_route_scored_refuses_bad_sizes_pointers_and_workspaces():
    lib = pkg.load()
    d = _lib.Dims(16, 8, 8, 8, 2)
    assert _route(d, None) == _lib.ERR_INVALID_ARGUMENT
    assert _route(d, _scoring(), logits=None) == _lib.ERR_INVALID_ARGUMENT
    assert _route(d, _scoring(), logits=FAKE + 8) == _lib.ERR_INVALID_ARGUMENT
    assert _route(_lib.Dims(65537, 8, 8, 8, 2), _scoring()) == _lib.ERR_UNSUPPORTED
    assert _route(_lib.Dims(16, 8, 8, 513, 2), _scoring()) == _lib.ERR_INVALID_ARGUMENT
    big = _lib.Dims(4096, 8, 8, 8, 2)
    need = lib.moe_lora_route_scored_workspace_size(ctypes.byref(big), ctypes.byref(_scoring()))
    assert need > 0
    assert _route(big, _scoring(), ws_bytes=need - 1) == _lib.ERR_WORKSPACE_TOO_SMALL
    assert _route(big, _scoring(), ws=None) == _lib.ERR_INVALID_ARGUMENT
    assert lib.moe_lora_route_scored_workspace_size(ctypes.byref(d), ctypes.byref(_scoring())) == 0
    for i in range(4):
        args = [FAKE, FAKE, FAKE, FAKE]
        args[i] = None
        assert lib.moe_lora_route_scored_backward(ctypes.byref(d), ctypes.byref(_scoring()), *args, None) == \
            _lib.ERR_INVALID_ARGUMENT
    assert lib.moe_lora_route_scored_backward(ctypes.byref(_lib.Dims(0, 8, 8, 8, 2)), ctypes.byref(_scoring()), None,
                                              None, None, None, None) == _lib.OK


def test_scoring_descriptor_refusals():
    with pytest.raises(ValueError, match="score"):
        ml.Scoring(score="tanh").to_c(torch.bfloat16, 8)
    with pytest.raises(ValueError, match="logits"):
        ml.Scoring().to_c(torch.float16, 8)
    with pytest.raises(ValueError, match="bias"):
        ml.Scoring(bias=torch.zeros(7)).to_c(torch.bfloat16, 8)


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    t = torch.zeros((4, 8))
    with pytest.raises(ValueError, match="GPU"):
        ml.moe_lora_route_scored_backward(ml.dims(4, 8, 8, 8, 2), ml.Scoring(), t, t, t, t)
    with pytest.raises(ValueError, match="elements"):
        ml._checked("x", t, torch.float32, 33)
    with pytest.raises(ValueError, match="float32"):
        ml._checked("x", t.double(), torch.float32, 32)
    with pytest.raises(ValueError, match="contiguous"):
        ml._checked("x", t.t(), torch.float32, 32)


def test_pool_descriptor_refusals():
    i32, bf16 = torch.int32, torch.bfloat16
    good = dict(token_slot=torch.zeros(5, dtype=i32), rank=torch.ones(2, dtype=i32), scaling=torch.ones(2),
                a=torch.zeros((2, 8, 16), dtype=bf16), b=torch.zeros((2, 24, 8), dtype=bf16))
    pool = ml.AdapterPool(**good)
    assert pool.to_c(5, 16, 24).max_rank == 8
    assert pool.with_slots(torch.zeros(7, dtype=i32)).to_c(7, 16, 24).num_slots == 2
    for bad in ((6, 16, 24), (5, 8, 24), (5, 16, 16)):
        with pytest.raises(ValueError, match="the pool is for"):
            pool.to_c(*bad)
    for name, t in (("token_slot", torch.zeros(5)), ("rank", torch.ones(3, dtype=i32)), ("scaling", torch.ones(2).double()),
                    ("a", torch.zeros((2, 8, 16))), ("b", torch.zeros((2, 24, 16), dtype=bf16)),
                    ("a", torch.zeros((2, 16, 8), dtype=bf16).transpose(1, 2))):
        with pytest.raises(ValueError, match=name):
            ml.AdapterPool(**{**good, name: t})
    with pytest.raises(ValueError):
        ml.AdapterPool(**{**good, "a": torch.zeros((16, 16), dtype=bf16)})
    with pytest.raises(AttributeError):
        pool.rank = torch.ones(2, dtype=i32)


def test_pool_whose_tensor_moved():
    i32, bf16 = torch.int32, torch.bfloat16
    for name in ("token_slot", "rank", "scaling", "a", "b"):
        t = dict(token_slot=torch.zeros(5, dtype=i32), rank=torch.ones(2, dtype=i32), scaling=torch.ones(2),
                 a=torch.zeros((2, 8, 16), dtype=bf16), b=torch.zeros((2, 24, 8), dtype=bf16))
        pool = ml.AdapterPool(**t)
        t[name].zero_()
        pool.to_c(5, 16, 24)  # new contents
        before = t[name].data
        t[name].data = before.clone()
        with pytest.raises(ValueError, match="moved"):
            pool.to_c(5, 16, 24)


def test_pool_with_another_order_of_ranks():
    i32, bf16 = torch.int32, torch.bfloat16
    with pytest.raises(ValueError, match="b:"):  # as many elements, other adapters
        ml.AdapterPool(torch.zeros(5, dtype=i32), torch.ones(2, dtype=i32), torch.ones(2),
                       torch.zeros((2, 8, 16), dtype=bf16), torch.zeros((4, 24, 4), dtype=bf16))



# ---- the oracle's definitions
def _logits(T, E, seed=0):
    return np.random.Generator(np.random.PCG64(seed)).standard_normal((T, E)) * 1.5


def test_scored_oracle_holds_the_named_methods():
    bits = (np.float32(_logits(9, 32)).view(np.uint32) >> 16).astype(np.uint16)
    l = oracle.bf16_bits_to_f64(bits)
    ids, w = oracle.route(bits, 4)
    got_ids, got_w = ref.route_scored(l, 4)
    assert np.array_equal(ids, got_ids)
    np.testing.assert_allclose(got_w, w, rtol=1e-12)
    bias = np.float32(_logits(1, 32, 1)[0] * 0.1)
    ids, w = oracle.route(bits, 4, "deepseek_v3", bias, 4, 2, 2.5)
    got_ids, got_w = ref.route_scored(l, 4, "sigmoid", True, 4, 2, 2, 2.5, bias)
    assert np.array_equal(ids, got_ids)
    np.testing.assert_allclose(got_w, w, rtol=1e-12)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_in_the_choice(score):
    l = np.array([[-np.inf, 0.0, 0.1, 0.2]])
    assert list(ref.route_scored(l, 3, score)[0][0]) == [3, 2, 1]
    ids, w = ref.route_scored(l, 2, score, bias=np.float32([0.3, -0.6, -0.6, 0.0]))
    assert sorted(ids[0]) == [0, 3] and (w[ids == 0] == 0).all()  # its bias alone is its key
    ids, w = ref.route_scored(l, 3, score, bias=np.float32([-np.inf, -0.6, -0.6, 0.0]))
    assert 0 not in ids[0]
    ids, w = ref.route_scored(l[:, ::-1], 2, score, n_group=2, topk_group=1)
    assert list(ids[0]) == [0, 1]                                 # groups [0.2, 0.1] and [0.0, masked]
    ids, w = ref.route_scored(np.array([[9.0, -np.inf, 1.0, 2.0]]), 2, score, n_group=2, topk_group=1)
    assert list(ids[0]) == [0, 1] and w[0, 1] == 0                # before the closed group's experts


@pytest.mark.parametrize("score,renorm", list(itertools.product(["softmax", "sigmoid"], [True, False])))
def test_scored_gradient_equals_differences(score, renorm):
    l = _logits(3, 7, 2)
    ids = np.array([[1, 4, 6], [0, 2, 3], [5, 1, 0]])
    dw = _logits(3, 3, 3)
    got = ref.route_scored_backward(l, ids, dw, score, renorm, 1.5)
    h = 1e-6
    for t, e in itertools.product(range(3), range(7)):
        up, down = l.copy(), l.copy()
        up[t, e] += h
        down[t, e] -= h
        diff = 1.5 * (dw * (ref.chosen_weights(up, ids, score, renorm) -
                            ref.chosen_weights(down, ids, score, renorm))).sum() / (2 * h)
        assert abs(diff - got[t, e]) < 1e-7


# ---- checkpoints and finalize's gradients
def test_checkpoint_refusals():
    lib = pkg.load()
    for fn in (lib.moe_lora_checkpoint_pack, lib.moe_lora_checkpoint_unpack):
        assert fn(-1, 8, FAKE, FAKE, FAKE, None) == _lib.ERR_INVALID_ARGUMENT
        assert fn(4, 0, FAKE, FAKE, FAKE, None) == _lib.ERR_INVALID_ARGUMENT
        assert fn(4, 12, FAKE, FAKE, FAKE, None) == _lib.ERR_UNSUPPORTED
        assert fn(4, 65544, FAKE, FAKE, FAKE, None) == _lib.ERR_UNSUPPORTED
        assert fn(1 << 31, 8, FAKE, FAKE, FAKE, None) == _lib.ERR_UNSUPPORTED
        assert fn(0, 8, None, None, None, None) == _lib.OK
        for i in range(3):
            args = [FAKE] * 3
            args[i] = FAKE + 8
            assert fn(4, 8, *args, None) == _lib.ERR_INVALID_ARGUMENT


def test_finalize_backward_refusals():
    lib = pkg.load()
    d = _lib.Dims(4, 64, 8, 8, 2)

    def call(dd=d, d_out=FAKE, y=FAKE, c=None, e=None, w=FAKE, e2p=FAKE, dy=FAKE, dw=FAKE):
        return lib.moe_lora_finalize_backward(ctypes.byref(dd), d_out, y, c, e, w, e2p, dy, dw, None)

    for bad in (dict(y=None), dict(c=FAKE), dict(c=FAKE, e=FAKE), dict(y=None, c=FAKE), dict(y=None, e=FAKE),
                dict(d_out=None), dict(w=None), dict(e2p=FAKE + 4), dict(dy=None), dict(dw=None)):
        assert call(**bad) == _lib.ERR_INVALID_ARGUMENT
    assert call(dd=_lib.Dims(4, 60, 8, 8, 2)) == _lib.ERR_UNSUPPORTED
    assert call(dd=_lib.Dims(0, 64, 8, 8, 2), d_out=None, y=None) == _lib.OK


def test_checkpoint_oracle_on_hand_made_blocks():
    x = np.zeros((1, 64))
    x[0, 0], x[0, 1], x[0, 2] = 448.0, 17.0, -1.0    # exponent 0: 17 is a tie of 16 and 18, taken to even
    x[0, 32], x[0, 33] = 450.0, 1.0                  # just past 448: exponent 1
    codes, exps = ref.checkpoint_pack(x)
    assert list(exps[0]) == [127, 128]
    got = ref.checkpoint_unpack(codes, exps)[0]
    assert list(got[:3]) == [448.0, 16.0, -1.0] and list(got[32:34]) == [448.0, 1.0]
    assert ref.checkpoint_exponent(0.0) == -117 and ref.checkpoint_exponent(1.75) == -8


def test_finalize_gradient_oracle_equals_differences():
    g = np.random.Generator(np.random.PCG64(0))
    T, k, H = 3, 2, 5
    y, w, d_out = g.standard_normal((T * k, H)), g.random((T, k)), g.standard_normal((T, H))
    e2p = g.permutation(T * k)

    def loss(y, w):
        return sum((w[t, j] * y[e2p[t * k + j]] * d_out[t]).sum() for t in range(T) for j in range(k))

    dy, dw = ref.finalize_backward(d_out, y, w, e2p)
    h = 1e-6
    for p, i in itertools.product(range(T * k), range(H)):
        e = np.zeros_like(y)
        e[p, i] = h
        assert abs((loss(y + e, w) - loss(y - e, w)) / (2 * h) - dy[p, i]) < 1e-8
    for t, j in itertools.product(range(T), range(k)):
        e = np.zeros_like(w)
        e[t, j] = h
        assert abs((loss(y, w + e) - loss(y, w - e)) / (2 * h) - dw[t, j]) < 1e-8


# ---- projection with pooled adapters
def _pool(**kw):
    v = dict(num_slots=2, max_rank=16, token_slot=FAKE, rank=FAKE, scaling=FAKE, a=FAKE, b=FAKE)
    v.update(kw)
    return _lib.Pool(*[v[f] for f, _ in _lib.Pool._fields_])


def _project(d, p, x=FAKE, w=FAKE, y=FAKE, v=None, ws=FAKE, ws_bytes=1 << 20):
    return pkg.load().moe_lora_project(ctypes.byref(d), x, w, ctypes.byref(p) if p else None, y, v, ws, ws_bytes, None)


@pytest.mark.parametrize("dims,status", [
    ((-1, 64, 48, 64, 48), _lib.ERR_INVALID_ARGUMENT), ((4, 0, 48, 64, 48), _lib.ERR_INVALID_ARGUMENT),
    ((4, 64, 48, 56, 48), _lib.ERR_INVALID_ARGUMENT), ((4, 64, 48, 64, 40), _lib.ERR_INVALID_ARGUMENT),
    ((4, 60, 48, 64, 48), _lib.ERR_UNSUPPORTED), ((4, 64, 44, 64, 48), _lib.ERR_UNSUPPORTED),
    ((4, 64, 48, 68, 48), _lib.ERR_UNSUPPORTED), ((4, 64, 48, 64, 1 << 23), _lib.ERR_UNSUPPORTED),
    ((4, 32768, 32768, 32768, 32768), _lib.ERR_UNSUPPORTED), (((1 << 24) + 1, 64, 48, 64, 48), _lib.ERR_UNSUPPORTED),
    ((1 << 24, 64, 1 << 19, 64, 1 << 19), _lib.ERR_UNSUPPORTED)])
def test_project_refuses_bad_sizes(dims, status):
    d = _lib.ProjDims(*dims)
    assert _project(d, _pool()) == status
    assert pkg.load().moe_lora_project_workspace_size(ctypes.byref(d), ctypes.byref(_pool())) == 0


def test_project_refuses_bad_pools_and_pointers():
    d = _lib.ProjDims(4, 64, 48, 64, 48)
    bad, no = _lib.ERR_INVALID_ARGUMENT, _lib.ERR_UNSUPPORTED
    assert _project(d, None) == bad
    assert _project(d, _pool(num_slots=-1)) == bad
    assert _project(d, _pool(num_slots=513)) == no
    assert _project(d, _pool(max_rank=0)) == bad
    assert _project(d, _pool(max_rank=12)) == no
    assert _project(d, _pool(max_rank=136)) == no
    for f in ("token_slot", "rank", "scaling", "a", "b"):
        assert _project(d, _pool(**{f: None})) == bad
        assert _project(d, _pool(**{f: FAKE + 4})) == bad
    for f in ("x", "w", "y"):
        assert _project(d, _pool(), **{f: None}) == bad
        assert _project(d, _pool(), **{f: FAKE + 8}) == bad
    assert _project(d, _pool(), v=FAKE + 4) == bad
    assert _project(d, _pool(num_slots=0), v=FAKE) == bad
    assert _project(d, _pool(), ws_bytes=8) == _lib.ERR_WORKSPACE_TOO_SMALL
    assert _project(d, _pool(), ws=None) == bad
    assert _project(_lib.ProjDims(0, 64, 48, 64, 48), _pool(), x=None, w=None, y=None, ws=None, ws_bytes=0) == _lib.OK


def test_project_oracle_is_the_merged_weight():
    g = np.random.Generator(np.random.PCG64(0))
    T, K, N, S, R = 6, 5, 4, 3, 3
    x, w, a, b = (g.standard_normal(s) for s in ((T, K), (N, K), (S, R, K), (S, N, R)))
    slot, rank, scaling = np.array([0, 1, 2, -1, 3, 0]), np.array([3, 2, 0]), np.array([0.5, 2.0, 1.0])
    y, v = ref.project(x, w, slot, rank, scaling, a, b)
    for t in range(T):
        m, s = w.copy(), slot[t]
        if 0 <= s < S:
            m += scaling[s] * b[s][:, :rank[s]] @ a[s][:rank[s]]
        np.testing.assert_allclose(y[t], m @ x[t], rtol=1e-12)
    assert (v[2:5] == 0).all() and (v[1, 2:] == 0).all()


def _back(d, p, **kw):
    v = dict(x=FAKE, c=None, e=None, w=FAKE, v=FAKE, dy=FAKE, dx=FAKE, da=FAKE, db=FAKE, ws=FAKE, ws_bytes=1 << 30)
    v.update(kw)
    return pkg.load().moe_lora_project_backward(
        ctypes.byref(d), v["x"], v["c"], v["e"], v["w"], ctypes.byref(p) if p else None, v["v"], v["dy"], v["dx"], v["da"],
        v["db"], v["ws"], v["ws_bytes"], None)


def test_project_backward_refusals():
    d = _lib.ProjDims(4, 64, 48, 64, 48)
    bad = _lib.ERR_INVALID_ARGUMENT
    for kw in (dict(dx=None, da=None, db=None), dict(x=None), dict(c=FAKE), dict(c=FAKE, e=FAKE),
               dict(x=None, c=FAKE), dict(x=None, e=FAKE), dict(w=None), dict(v=None), dict(dy=None),
               dict(ws=None), dict(dx=FAKE + 8), dict(da=FAKE + 2), dict(db=FAKE + 4), dict(x=FAKE + 8),
               dict(dy=FAKE + 8), dict(v=FAKE + 4), dict(w=FAKE + 8)):
        assert _back(d, _pool(), **kw) == bad, kw
    assert _back(d, None) == bad
    assert _back(d, _pool(), ws_bytes=64) == _lib.ERR_WORKSPACE_TOO_SMALL
    assert _back(_lib.ProjDims(4, 64, 44, 64, 48), _pool()) == _lib.ERR_UNSUPPORTED


def test_project_gradient_oracle_equals_differences():
    g = np.random.Generator(np.random.PCG64(1))
    T, K, N, S, R = 5, 4, 3, 2, 2
    x, w, a, b, dy = (g.standard_normal(s) for s in ((T, K), (N, K), (S, R, K), (S, N, R), (T, N)))
    slot, rank, scaling = np.array([0, 1, -1, 1, 0]), np.array([2, 1]), np.array([0.5, 2.0])
    _, v = ref.project(x, w, slot, rank, scaling, a, b)
    grads = ref.project_backward(dy, x, w, slot, rank, scaling, a, b, v)
    args = [x, a, b]

    def loss(x, a, b):
        return (dy * ref.project(x, w, slot, rank, scaling, a, b)[0]).sum()

    for i, got in enumerate(grads):
        for at in np.ndindex(args[i].shape):
            up, down = [m.copy() for m in args], [m.copy() for m in args]
            up[i][at] += 1e-6
            down[i][at] -= 1e-6
            assert abs((loss(*up) - loss(*down)) / 2e-6 - got[at]) < 1e-7


def test_project_backward_into_gradients_without_elements():
    none = dict(dx=None, da=None, db=None)
    assert _back(_lib.ProjDims(0, 64, 48, 64, 48), _pool(), **none) == _lib.OK
    assert _back(_lib.ProjDims(4, 64, 48, 64, 48), _pool(num_slots=0), **none) == _lib.OK
    assert _back(_lib.ProjDims(4, 64, 44, 64, 48), _pool(), **none) == _lib.ERR_UNSUPPORTED


def test_binding_refuses_what_32_bits_cut_off():
    for at in range(5):
        sizes = [8] * 5
        sizes[at] = 2 ** 32 + 8
        with pytest.raises(ValueError, match="32 bits"):
            ml._proj_dims(*sizes)
    assert ml._proj_dims(4, 8, 16, 8, 2 ** 31 - 1).ldy == 2 ** 31 - 1  # (the library's own limits come next)
    wide = torch.empty((1, 2 ** 32 + 8), dtype=torch.uint8, device="meta")
    with pytest.raises(ValueError, match="columns"):
        ml.moe_lora_checkpoint_pack(wide, wide, wide)
    with pytest.raises(ValueError, match="columns"):
        ml.moe_lora_checkpoint_unpack(wide, wide, wide)
    meta = dict(dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="pool"):
        ml.AdapterPool(torch.empty(1, dtype=torch.int32, device="meta"), torch.empty(1, dtype=torch.int32, device="meta"),
                       torch.empty(1, device="meta"), torch.empty((1, 2 ** 32 + 8, 8), **meta),
                       torch.empty((1, 8, 2 ** 32 + 8), **meta))


def test_descriptors_that_hold_tensors_compare():
    i32, bf16 = torch.int32, torch.bfloat16
    pools = [ml.AdapterPool(torch.zeros(5, dtype=i32), torch.ones(2, dtype=i32), torch.ones(2),
                            torch.zeros((2, 8, 16), dtype=bf16), torch.zeros((2, 24, 8), dtype=bf16)) for _ in range(2)]
    assert pools[0] == pools[0] and pools[0] != pools[1] and len(set(pools)) == 2
    bias = torch.zeros(8)
    assert ml.Scoring(bias=bias) == ml.Scoring(bias=bias) and ml.Scoring() == ml.Scoring()
    assert ml.Scoring(bias=bias) != ml.Scoring(bias=bias.clone()) and ml.Scoring(bias=bias) != ml.Scoring()
    assert ml.Scoring(scale=2.0) != ml.Scoring() and ml.Scoring() != ml.ROUTING_RENORMALIZE
