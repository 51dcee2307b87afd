"""The scored router and the int8 calls without a GPU: sizes, refusals (found on the
host before anything is enqueued) and the 64-bit forms against hand-made cases."""
import ctypes
import os

import numpy as np
import pytest

from oracle import int8 as o8

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_layer_02_amd",
                   "libmoe355.so")
P = 1 << 40          # a device address that nothing dereferences


@pytest.fixture(scope="module")
def abi():
    if not os.path.exists(LIB):
        pytest.fail("libmoe355.so is not built; run python -m moe_expert_layer_02_amd.build")
    from moe_expert_layer_02_amd import abi
    return abi


def i8_desc(abi, H=256, I=128, E=16, k=2, wfmt=2):
    return abi.LayerDesc(H, I, E, k, 0, 1, 1, 1.0, wfmt)


def test_sizes(abi):
    L = abi.load()
    for H, I in ((256, 128), (2048, 512), (1344, 704)):
        d = i8_desc(abi, H, I)
        assert L.moe355_expert_bytes(ctypes.byref(d)) == o8.expert_bytes(H, I)
        assert L.moe355_workspace_bytes(ctypes.byref(d), 4, abi.MODE_DECODE_I8) > 0
        assert L.moe355_workspace_bytes(ctypes.byref(d), 4, abi.MODE_PREFILL_I8) > 0
        assert L.moe355_workspace_bytes(ctypes.byref(d), 4, abi.MODE_PERMUTE) > 0
        # a mode of the other formats has no size for int8 experts, and the reverse
        for mode in (abi.MODE_DECODE, abi.MODE_PREFILL, abi.MODE_PREFILL_MX):
            assert L.moe355_workspace_bytes(ctypes.byref(d), 4, mode) == 0
        for wfmt in (0, 1):
            q = i8_desc(abi, H, I, wfmt=wfmt)
            assert L.moe355_workspace_bytes(ctypes.byref(q), 4, abi.MODE_DECODE_I8) == 0
            assert L.moe355_workspace_bytes(ctypes.byref(q), 4, abi.MODE_PREFILL_I8) == 0


@pytest.mark.parametrize("H,I,E,k", ((64, 64, 1024, 1), (64, 64, 40, 3), (256, 128, 16, 2), (1344, 704, 40, 8)))
def test_a_workspace_for_a_long_chunk_holds_a_shorter_one(abi, H, I, E, k):
    """Sizes grow with T, also where a chunk changes to another tile."""
    L, d = abi.load(), i8_desc(abi, H, I, E, k)
    for mode, last in ((abi.MODE_PREFILL_I8, 120 * E // k + 2), (abi.MODE_DECODE_I8, 256 // k), (abi.MODE_PERMUTE, 5000)):
        step = 1 if last < 20000 else 7
        sizes = [L.moe355_workspace_bytes(ctypes.byref(d), T, mode) for T in range(0, last, step)]
        assert all(x <= y for x, y in zip(sizes, sizes[1:])), mode


def test_four_bit_calls_refuse_int8_experts(abi):
    L, d = abi.load(), i8_desc(abi)
    r = ctypes.byref(d)
    assert L.moe355_pack_experts(r, P, P + (1 << 30), 1, None) == -1
    assert L.moe355_expert_ffn_prefill(r, P, 4, P, P, P, P, P, P, P, 1 << 30, None) == -1
    assert L.moe355_expert_ffn_prefill_mx(r, P, 4, P, P, P, P, P, P, P, 1 << 30, None) == -1
    out = abi.ClassifyOut()
    assert L.moe355_expert_ffn_decode(r, P, 4, P, P, None, P, 0, ctypes.byref(out), P, P, 1 << 30, None) == -1
    assert b"int8" in L.moe355_last_error()


ROUTE_BAD = {
    "no experts": (dict(n_experts=0), -1),
    "k 0": (dict(top_k=0), -1),
    "k beyond E": (dict(top_k=17), -1),
    "k beyond 32": (dict(n_experts=64, top_k=33), -3),
    "E beyond 512": (dict(n_experts=513, n_group=1, topk_group=1), -3),
    "score": (dict(score=2), -1),
    "groups do not divide": (dict(n_group=3, topk_group=1), -1),
    "no group kept": (dict(topk_group=0), -1),
    "more groups kept than there are": (dict(topk_group=5), -1),
    "groups of one": (dict(n_group=16, topk_group=8), -3),
    "k beyond the kept groups": (dict(top_k=5, topk_group=1), -1),
    "scale": (dict(scale=float("nan")), -1),
}


@pytest.mark.parametrize("case", list(ROUTE_BAD))
def test_route_scored_refusals(abi, case):
    change, want = ROUTE_BAD[case]
    f = dict(n_experts=16, top_k=2, score=1, n_group=4, topk_group=2, renorm=1, scale=1.0)
    f.update(change)
    d = abi.RouterDesc(**f)
    L = abi.load()
    assert L.moe355_route_scored(ctypes.byref(d), P, 0, 1 << 20, None, 4, P, P, None) == want, L.moe355_last_error()
    assert b"route_scored" in L.moe355_last_error()


def test_route_scored_call_refusals(abi):
    L, d = abi.load(), abi.RouterDesc(16, 2, 1, 4, 2, 1, 1.0)
    r = ctypes.byref(d)
    call = L.moe355_route_scored
    assert call(None, P, 0, 16, None, 4, P, P, None) == -1
    assert call(r, P, 2, 16, None, 4, P, P, None) == -1          # type
    assert call(r, P, 0, 15, None, 4, P, P, None) == -1          # overlapping rows
    assert call(r, P, 0, 16, None, -1, P, P, None) == -1
    for args in ((None, P, P), (P, None, P), (P, P, None)):
        assert call(r, args[0], 0, 16, None, 4, args[1], args[2], None) == -1
    assert call(r, None, 0, 16, None, 0, None, None, None) == 0   # no tokens: nothing to do


def test_quantize_and_matmul_refusals(abi):
    L = abi.load()
    q, mm = L.moe355_quantize_i8, L.moe355_matmul_i8
    assert q(P, 64, -1, 64, P, 64, P, None) == -1
    assert q(P, 64, 4, 0, P, 64, P, None) == -1
    assert q(P, 63, 4, 64, P, 64, P, None) == -1
    assert q(P, 64, 4, 64, P, 63, P, None) == -1
    assert q(None, 64, 4, 64, P, 64, P, None) == -1 and q(P, 64, 4, 64, None, 64, P, None) == -1
    assert q(P, 64, 4, 64, P, 64, None, None) == -1
    assert q(None, 64, 0, 64, None, 64, None, None) == 0
    good = dict(a=P, lda=64, sa=P, b=P, ldb=64, sb=P, M=4, N=8, K=64, out=P, t=1, ldo=8)

    def call(**c):
        v = dict(good, **c)
        return mm(v["a"], v["lda"], v["sa"], v["b"], v["ldb"], v["sb"], v["M"], v["N"], v["K"], v["out"], v["t"],
                  v["ldo"], None)

    assert call(M=-1) == -1 and call(N=0) == -1 and call(K=0) == -1 and call(t=2) == -1
    assert call(K=72, lda=80, ldb=80) == -3                       # K not a multiple of 16
    assert call(K=65552, lda=1 << 17, ldb=1 << 17) == -3          # beyond the exact sums' limit
    assert call(lda=48) == -1 and call(ldb=48) == -1 and call(ldo=7) == -1
    assert call(lda=72) == -3 and call(ldb=72) == -3              # rows not at 16 bytes
    assert call(a=P + 8) == -3 and call(b=P + 4) == -3
    assert call(lda=1 << 23) == -3 and call(ldb=1 << 23) == -3
    for name in ("a", "sa", "b", "sb", "out"):
        assert call(**{name: None}) == -1, name
    assert call(M=0, a=None, out=None) == 0


def test_expert_ffn_refusals(abi):
    L = abi.load()
    big = 1 << 34

    def pre(d, T=4, x=P, ids=P, w=P, lw=P, perm=P, off=P, out=P, ws=P, n=big):
        return L.moe355_expert_ffn_prefill_i8(ctypes.byref(d), x, T, ids, w, lw, perm, off, out, ws, n, None)

    def dec(d, T=4, x=P, ids=P, w=P, cache=None, pool=P, layer=0, exp=None, out=P, ws=P, n=big):
        return L.moe355_expert_ffn_decode_i8(ctypes.byref(d), x, T, ids, w, cache, pool, layer, exp, out, ws, n, None)

    good = i8_desc(abi)
    for call in (pre, dec):
        assert call(i8_desc(abi, wfmt=0)) == -1 and call(i8_desc(abi, wfmt=1)) == -1
        assert call(i8_desc(abi, H=96)) == -3 and call(i8_desc(abi, I=32)) == -3
        assert call(i8_desc(abi, H=16448)) == -3 and call(i8_desc(abi, E=1025)) == -3
        assert call(good, T=-1) == -1
        for name in ("x", "ids", "w", "out"):
            assert call(good, **{name: None}) == -1, name
        assert call(good, x=P + 2) == -1 and call(good, ws=P + 16) == -1
        assert call(good, n=64) == -4 and call(good, ws=None) == -4
        assert call(good, T=0, x=None, ids=None, w=None, out=None, ws=None, n=0) == 0
    assert pre(good, lw=None) == -1 and pre(good, perm=None) == -1 and pre(good, off=None) == -1
    assert pre(good, T=1 << 28) == -1
    assert pre(i8_desc(abi, H=16384, k=1), T=1 << 19) == -3       # T*H beyond 2^32
    assert dec(good, pool=None) == -1 and dec(good, layer=-1) == -1
    assert dec(good, T=129) == -3                                 # 258 pairs
    S = o8.expert_bytes(256, 128)
    lists = abi.ClassifyOut(P, P, P, P, P, P, P, P, P, 8, P, P, 64)
    cache = abi.Cache(4, 2, 16, S, P, P, P, P)
    cr, lr = ctypes.byref(cache), ctypes.byref(lists)
    assert dec(good, cache=cr) == -1                              # a cache needs the lists
    assert dec(good, cache=cr, exp=lr, layer=2) == -1
    bad = abi.Cache(4, 2, 16, S - 4, P, P, P, P)
    assert dec(good, cache=ctypes.byref(bad), exp=lr) == -1       # slots of another size
    short = abi.ClassifyOut(P, P, P, P, P, P, P, P, P, 7, P, P, 64)
    assert dec(good, exp=ctypes.byref(short)) == -4
    empty = abi.ClassifyOut(None, P, P, P, P, P, P, P, P, 8, P, P, 64)
    assert dec(good, exp=ctypes.byref(empty)) == -1


# ---- the 64-bit forms ---------------------------------------------------------

def test_oracle_quantize_by_hand():
    x = np.array([[127, -63.5, 0.5, 1.5], [0, 0, 0, 0], [1e-35, 0, 0, 0], [1, np.inf, 0, 0], [np.nan, 1, 0, 0]],
                 dtype=np.float32)
    q, s = o8.quantize(x)
    assert q[0].tolist() == [127, -64, 0, 2] and s[0] == 1.0      # ties to even
    assert not q[1:].any() and s[1] == 0 and s[2] == 0 and np.isnan(s[3:]).all()


def test_oracle_bf16_round():
    v = np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -1 - 2.0 ** -7, 0.0])
    assert o8.bf16_round(v).tolist() == [1.0, 1.0, 1 + 2.0 ** -6, -1 - 2.0 ** -7, 0.0]


def test_oracle_swiglu_against_the_float_formula():
    """The int8 layer stays within its quantisation of the unquantised formula on dequantised weights."""
    rng = np.random.default_rng(5)
    H, I = 256, 192
    blob = o8.make_expert(rng, H, I)
    x = o8.bf16_round(rng.normal(0, 1, (7, H)))
    y, b = o8.swiglu(x, blob, H, I)
    (gq, gs), (uq, us), (dq, ds) = ((q.astype(float), s.astype(float)) for q, s in o8.matrices(blob, H, I))
    g, u = x @ (gq * gs[:, None]).T, x @ (uq * us[:, None]).T
    want = (g / (1 + np.exp(-g)) * u) @ (dq * ds[:, None]).T
    assert np.linalg.norm(y - want) < 0.03 * np.linalg.norm(want)
    assert np.linalg.norm(b) < 0.01 * np.linalg.norm(want)


def test_oracle_route_scored_by_hand():
    l = np.log(np.array([[1., 2., 3., 4.]]))
    ids, w = o8.route_scored(l, None, 2, "softmax", 1, 1, False, 1.0)
    assert ids.tolist() == [[3, 2]] and np.allclose(w, [[.4, .3]])
    ids, w = o8.route_scored(l, [0, .3, 0, 0], 2, "softmax", 1, 1, True, 2.0)   # choices .1 .5 .3 .4
    assert ids.tolist() == [[1, 3]] and np.allclose(w, [[2 * .2 / .6, 2 * .4 / .6]])
    ids, _ = o8.route_scored([[0., 0., 1., -9.]], None, 2, "sigmoid", 2, 1, True, 1.0)
    assert ids.tolist() == [[0, 1]]                      # .5 + .5 beats .73 + .0001
    ids, w = o8.route_scored(np.full((1, 4), -np.inf), None, 3, "softmax", 2, 2, True, 1.0)
    assert ids.tolist() == [[0, 1, 2]] and not w.any()
