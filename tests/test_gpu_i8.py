"""The int8 operators against their 64-bit forms: codes bit for bit, products and the
expert SwiGLU within bounds derived from their roundings."""
import numpy as np
import pytest

from gpu_common import say
from oracle import int8 as o8

pytestmark = pytest.mark.gpu

# the sum is exact: int32 -> fp32 and two scalings, half a step each; bf16 once more
F32_TOL = 3 * 2.0 ** -24 * (1 + 1e-6)
BF16_TOL = F32_TOL + 2.0 ** -8 * (1 + 1e-6)


def bf16(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(torch.bfloat16)


def quantize(x, pad=0, shift=0):
    """Codes and scales of bf16 x on the device; pad: extra columns between the rows, shift: first column."""
    import torch
    import moe_expert_layer_02_amd as m
    rows, cols = x.shape
    wide = torch.full((rows, cols + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, shift:shift + cols] = x
    q = torch.full((rows, cols + pad), 77, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 1,), -7.0, dtype=torch.float32, device="cuda")
    m.quantize_i8(wide[:, shift:shift + cols], q[:, shift:shift + cols], s[:rows])
    torch.cuda.synchronize()
    assert s[rows] == -7.0
    q = q.cpu().numpy()
    assert (q[:, :shift] == 77).all() and (q[:, shift + cols:] == 77).all()
    return q[:, shift:shift + cols], s[:rows].cpu().numpy()


@pytest.mark.parametrize("rows,cols,pad,shift", [
    (1, 1, 0, 0), (3, 7, 2, 1), (5, 8, 0, 0), (2, 63, 1, 0), (300, 64, 0, 0), (9, 512, 8, 8), (4, 520, 0, 0),
    (3, 1024, 8, 0), (2, 2048, 0, 0), (1, 4096, 0, 0), (5, 4104, 0, 0), (3, 5000, 24, 16), (2, 5001, 0, 0),
    (1030, 576, 0, 0)])
def test_quantize_bit_for_bit(rows, cols, pad, shift):
    rng = np.random.default_rng(rows * 10000 + cols)
    say("quantize_i8", rows, cols, pad, shift)
    x = bf16(rng.normal(0, 1, (rows, cols)) * np.exp(rng.normal(0, 3, (rows, 1))))
    q, s = quantize(x, pad, shift)
    wq, ws = o8.quantize(x.float().cpu().numpy())
    assert np.array_equal(q, wq) and np.array_equal(s, ws)


@pytest.mark.parametrize("cols", (24, 29, 1032))
def test_quantize_special_rows(cols):
    rng = np.random.default_rng(cols)
    x = rng.normal(0, 1, (14, cols)).astype(np.float32)
    x[0] = 0
    x[1] = -0.0
    x[2, 3] = np.inf
    x[3, 4] = np.nan
    x[4, :] = -np.inf
    x[5] *= 1e-38
    x[6] *= 2.0 ** -101
    x[7] = 2.0 ** -100
    x[8] *= 1e38
    x[9] = np.arange(cols) % 9 * 0.5            # halves: ties to even
    x[9, 0] = 127
    x[10] = 3.3e38
    x[11, :] = -1
    x[12, 1:] = 0
    x[13] = -np.nan
    t = bf16(x)
    q, s = quantize(t)
    wq, ws = o8.quantize(t.float().cpu().numpy())
    assert np.array_equal(q, wq) and np.array_equal(s, ws, equal_nan=True)


def matmul(a, sa, b, sb, out_type, pads=(0, 0, 0)):
    import torch
    import moe_expert_layer_02_amd as m
    M, K = a.shape
    N = b.shape[0]

    def wide(v, pad):
        t = torch.full((v.shape[0], K + pad), 99, dtype=torch.int8, device="cuda")
        t[:, :K] = torch.from_numpy(v.astype(np.int8)).cuda()
        return t[:, :K]

    dt = torch.bfloat16 if out_type == "bf16" else torch.float32
    buf = torch.full((M + 2, N + pads[2]), -77.0, dtype=dt, device="cuda")
    m.matmul_i8(wide(a, pads[0]), torch.from_numpy(sa).cuda(), wide(b, pads[1]), torch.from_numpy(sb).cuda(),
                buf[1:M + 1, :N])
    torch.cuda.synchronize()
    assert (buf[[0, -1]] == -77).all() and (buf[:, N:] == -77).all(), "wrote outside its rows"
    return buf[1:M + 1, :N].double().cpu().numpy()


SIZES = [(1, 1, 16), (1, 16, 64), (1, 257, 80), (2, 300, 48), (7, 64, 4096), (15, 1000, 2064), (16, 33, 32),
         (17, 512, 576), (31, 255, 128), (33, 256, 112), (64, 300, 1024), (65, 129, 64), (127, 256, 96),
         (128, 257, 192), (129, 511, 256), (200, 700, 400), (257, 1025, 320), (513, 130, 2048), (1000, 96, 144)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out_type", ("f32", "bf16"))
def test_matmul_against_64_bits(M, N, K, out_type):
    rng = np.random.default_rng(M * 7919 + N * 31 + K)
    say("matmul_i8", M, N, K, out_type)
    a, b = rng.integers(-128, 128, (M, K)), rng.integers(-128, 128, (N, K))
    sa = np.exp(rng.normal(0, 1, M)).astype(np.float32)
    sb = np.exp(rng.normal(0, 1, N)).astype(np.float32)
    want = o8.product(a, sa, b, sb)
    tol = (F32_TOL if out_type == "f32" else BF16_TOL) * np.abs(want)
    for pads in ((0, 0, 0), (16, 48, 3)):
        got = matmul(a, sa, b, sb, out_type, pads)
        assert np.all(np.abs(got - want) <= tol), np.abs(got - want).max()


@pytest.mark.parametrize("M,N,K", [(520, 1025, 16), (641, 900, 48), (1024, 513, 128), (700, 1001, 400),
                                   (1025, 514, 272), (130, 9000, 1040), (2049, 4101, 16), (2300, 3500, 80),
                                   (2600, 3301, 400), (70000, 48, 144), (2700, 4097, 512)])
@pytest.mark.parametrize("out_type", ("f32", "bf16"))
def test_matmul_tiles_against_64_bits(M, N, K, out_type):
    """Sizes of the tiled forms: several tiles per block, ragged ones, K below and beside a stage."""
    test_matmul_against_64_bits(M, N, K, out_type)


def test_matmul_extremes():
    """The largest sums int32 has to hold, zero scales, and a row whose scale is NaN."""
    K = 65536
    a, b = np.full((3, K), -128), np.full((5, K), -128)
    b[1] = 127
    a[2] = 0
    sa = np.array([1.0, np.nan, 2.0], dtype=np.float32)
    sb = np.array([1.0, 0.5, 0.0, 1e-30, 1e30], dtype=np.float32)
    got, want = matmul(a, sa, b, sb, "f32"), o8.product(a, sa, b, sb)
    assert np.isnan(got[1]).all()
    # 2^14 65536 1e30 = 1.07e39 lies beyond fp32's largest value, 3.4e38: its rounding is infinity
    assert want[0, 4] > 3.5e38 and got[0, 4] == np.inf
    for r, n in ((0, 4), (2, 5)):
        assert np.all(np.abs(got[r, :n] - want[r, :n]) <= F32_TOL * np.abs(want[r, :n]))


# ---- expert SwiGLU ------------------------------------------------------------

class Layer:
    """A layer of random int8 experts on the device, with its host copies."""

    def __init__(self, H, I, E, k, seed, layers=1):
        import torch
        import moe_expert_layer_02_amd as m
        self.H, self.I, self.E, self.k = H, I, E, k
        rng = self.rng = np.random.default_rng(seed)
        self.blobs = [o8.make_expert(rng, H, I) for _ in range(layers * E)]
        self.pool = torch.from_numpy(np.concatenate(self.blobs)).cuda()
        self.desc = m.LayerDesc(H, I, E, k, m.ROUTE_SOFTMAX_TOPK, 1, 1, 1.0, m.W_INT8)

    def inputs(self, T, ids=None):
        import torch
        x = bf16(self.rng.normal(0, 1, (T, self.H)) * np.exp(self.rng.normal(0, 1, (T, 1))))
        if ids is None:
            ids = np.argsort(self.rng.random((T, self.E)), axis=1)[:, :self.k]
        ids = np.ascontiguousarray(ids, dtype=np.int32)
        w = (self.rng.random(ids.shape) + 0.05).astype(np.float32)
        return x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()

    def workspace(self, T, mode):
        import torch
        import moe_expert_layer_02_amd as m
        # no call may rely on a cleared workspace
        return torch.full((m.workspace_bytes(self.desc, T, mode),), 0xFF, dtype=torch.uint8, device="cuda")

    def prefill(self, x, ids, w, out=None, ws=None, stream=None):
        import torch
        import moe_expert_layer_02_amd as m
        T = x.shape[0]
        perm = torch.full((T * self.k,), 2 ** 30, dtype=torch.int32, device="cuda")
        offsets = torch.empty(self.E + 1, dtype=torch.int32, device="cuda")
        if out is None:
            out = torch.full((T, self.H), float("nan"), dtype=torch.bfloat16, device="cuda")
        m.permute(self.desc, ids, perm, offsets, self.workspace(T, m.MODE_PERMUTE), stream=stream)
        m.expert_ffn_prefill_i8(self.desc, x, ids, w, self.pool[:self.E * len(self.blobs[0])], perm, offsets, out,
                                self.workspace(T, m.MODE_PREFILL_I8) if ws is None else ws, stream=stream)
        return out

    def decode(self, x, ids, w, lists=None, cache=None, layer=0, out=None, ws=None, pool=None, stream=None):
        import torch
        import moe_expert_layer_02_amd as m
        if out is None:
            out = torch.full((x.shape[0], self.H), float("nan"), dtype=torch.bfloat16, device="cuda")
        m.expert_ffn_decode_i8(self.desc, x, ids, w, cache, self.pool if pool is None else pool, layer, lists, out,
                               self.workspace(x.shape[0], m.MODE_DECODE_I8) if ws is None else ws, stream=stream)
        return out

    def check(self, got, x, ids, w, y_bf16, what, layer=0):
        want, tol = o8.moe_layer(x.float().cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy(),
                                 lambda e: self.blobs[layer * self.E + e], self.H, self.I, y_bf16)
        got = got.double().cpu().numpy()
        assert np.isfinite(got).all(), what
        bad = np.abs(got - want) > tol
        rel = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-30)
        say(f"{what}: rel {rel:.2e}, largest share of its tolerance {np.max(np.abs(got - want) / np.maximum(tol, 1e-30)):.2f}")
        assert not bad.any(), (what, np.argwhere(bad)[:3], rel)


FFN = [(1, 256, 128, 16, 2), (1, 2048, 512, 8, 8), (2, 64, 64, 4, 1), (5, 320, 192, 7, 3), (16, 512, 256, 24, 6),
       (21, 1088, 448, 24, 3), (40, 192, 576, 5, 5), (64, 128, 64, 3, 2)]


@pytest.mark.parametrize("T,H,I,E,k", FFN)
def test_decode_against_64_bits(T, H, I, E, k):
    import moe_expert_layer_02_amd as m
    L = Layer(H, I, E, k, T + H)
    x, ids, w = L.inputs(T)
    out = L.decode(x, ids, w)
    L.check(out, x, ids, w, False, f"decode {T} {H} {I} {E} {k}")
    lists = m.DeviceClassifyOut(max(1, min(T * k, E)))
    m.dedup(ids, E, lists)
    assert (L.decode(x, ids, w, lists) == out).all()          # the same experts by list
    assert (L.decode(x, ids, w) == out).all()


@pytest.mark.parametrize("T,H,I,E,k", FFN + [(129, 256, 128, 4, 2), (300, 576, 320, 12, 4), (1000, 128, 192, 40, 3)])
def test_prefill_against_64_bits(T, H, I, E, k):
    L = Layer(H, I, E, k, T + I)
    x, ids, w = L.inputs(T)
    out = L.prefill(x, ids, w)
    L.check(out, x, ids, w, True, f"prefill {T} {H} {I} {E} {k}")
    assert (L.prefill(x, ids, w) == out).all()                # the same on every run


@pytest.mark.parametrize("T,H,I,E,k", [(1000, 192, 128, 6, 2), (700, 64, 64, 4, 1), (1200, 320, 448, 3, 2),
                                       (97, 128, 64, 1, 1), (2000, 128, 576, 16, 1), (513, 1024, 704, 2, 2)])
def test_prefill_long_buckets_against_64_bits(T, H, I, E, k):
    """More than 96 pairs per expert: the tall tiles, one or several a bucket."""
    test_prefill_against_64_bits(T, H, I, E, k)


@pytest.mark.parametrize("n,E", [(1, 1), (63, 7), (64, 512), (1023, 3), (4095, 512), (4096, 130), (4096, 513), (4097, 512)])
def test_permute_short(n, E):
    """The sort of few pairs in one workgroup beside the one of many; ids out of range
    stand in no bucket."""
    import torch
    import moe_expert_layer_02_amd as m
    say("permute", n, E)
    rng = np.random.default_rng(n + E)
    ids = rng.integers(0, E, n).astype(np.int32)
    d = m.LayerDesc(64, 64, E, 1, m.ROUTE_SOFTMAX_TOPK, 1, 1, 1.0, m.W_INT8)
    for bad in (False, True):
        if bad:
            ids[rng.random(n) < 0.2] = -1
            ids[n // 2] = E
        t = torch.from_numpy(ids).cuda().view(n, 1)
        perm = torch.full((n,), -5, dtype=torch.int32, device="cuda")
        off = torch.full((E + 2,), -5, dtype=torch.int32, device="cuda")
        ws = torch.empty(max(1, m.workspace_bytes(d, n, m.MODE_PERMUTE)), dtype=torch.uint8, device="cuda")
        m.permute(d, t, perm, off[:E + 1], ws)
        valid = (ids >= 0) & (ids < E)
        order = np.argsort(np.where(valid, ids, E), kind="stable")[:valid.sum()]
        starts = np.concatenate([[0], np.cumsum(np.bincount(ids[valid], minlength=E))])
        starts[E] = n
        assert (off.cpu().numpy() == np.append(starts, -5)).all()
        assert (perm.cpu().numpy() == np.append(order, np.full(n - len(order), -5))).all()


@pytest.mark.parametrize("T,k", ((300, 1), (260, 2), (900, 1), (1100, 2)))
def test_prefill_one_expert_takes_all(T, k):
    """One bucket of several tiles beside empty ones; the same expert twice in a token."""
    L = Layer(192, 128, 6, k, T)
    x, ids, w = L.inputs(T, np.full((T, k), 4))
    L.check(L.prefill(x, ids, w), x, ids, w, True, f"one expert, k={k}")


def test_decode_repeated_and_shared_experts():
    """One expert for 128 tokens, and a token that names an expert twice."""
    L = Layer(256, 128, 6, 2, 9)
    ids = np.full((128, 2), 3)
    ids[::2, 1] = 5
    x, ids, w = L.inputs(128, ids)
    L.check(L.decode(x, ids, w), x, ids, w, False, "shared experts")


@pytest.mark.parametrize("T", (1, 6, 50))
def test_padded_slots_add_nothing(T):
    L = Layer(256, 192, 8, 3, T)
    x, ids, w = L.inputs(T)
    ids[:, 2] = -1
    ids[T // 2] = -1                                           # a token with nothing left
    if T > 2:
        ids[0, 0], ids[1, 1] = 8, 2 ** 31 - 1                  # beyond the experts
    host = ids.clone()
    host[(ids < 0) | (ids >= 8)] = -1
    for name, out, y16 in (("decode", L.decode(x, ids, w), False), ("prefill", L.prefill(x, ids, w), True)):
        assert (out[T // 2] == 0).all()
        L.check(out, x, host, w, y16, f"padded {name}")


def test_rows_that_are_not_finite():
    """A token with an infinity gives a NaN row; the others are untouched by it."""
    L = Layer(256, 128, 4, 2, 3)
    x, ids, w = L.inputs(9)
    clean = {"decode": L.decode(x, ids, w), "prefill": L.prefill(x, ids, w)}
    x2 = x.clone()
    x2[4, 7] = float("inf")
    x2[6] = 0
    for name, out in (("decode", L.decode(x2, ids, w)), ("prefill", L.prefill(x2, ids, w))):
        assert out[4].isnan().all() and (out[6] == 0).all()
        rest = [i for i in range(9) if i not in (4, 6)]
        assert (out[rest] == clean[name][rest]).all()


def test_outputs_stay_inside_their_rows():
    import torch
    L = Layer(320, 128, 8, 2, 8)
    x, ids, w = L.inputs(5)
    for call in (L.decode, L.prefill):
        buf = torch.full((7, 320), -77.0, dtype=torch.bfloat16, device="cuda")
        call(x, ids, w, out=buf[1:6])
        assert (buf[[0, 6]] == -77).all()
        L.check(buf[1:6], x, ids, w, call == L.prefill, "guarded rows")


def test_empty_calls():
    import torch
    L = Layer(64, 64, 4, 2, 0)
    x, ids, w = L.inputs(0, np.zeros((0, 2)))
    assert L.decode(x, ids, w, ws=torch.empty(256, dtype=torch.uint8, device="cuda")).shape == (0, 64)
    assert L.prefill(x, ids, w, ws=torch.empty(256, dtype=torch.uint8, device="cuda")).shape == (0, 64)


def test_decode_from_the_cache():
    """Misses filled, hits from their slots, the rest in place; the pool's copies of the
    cached experts are then overwritten, so only the slots can give the result."""
    import torch
    import moe_expert_layer_02_amd as m
    H, I, E, k, T = 256, 192, 12, 3, 4
    L = Layer(H, I, E, k, 77, layers=2)
    S = len(L.blobs[0])
    cache = m.DeviceCache(5, 2, E, S)
    tick = 0
    for step in range(3):
        for layer in range(2):
            tick += 1
            x, ids, w = L.inputs(T)
            lists = m.DeviceClassifyOut(12)
            m.classify_evict(cache, layer, tick, ids, m.EvictPolicy(5, 2, 3), lists)
            m.cache_fill(cache, L.pool, layer, lists, 5)
            pool = L.pool.clone()
            table = cache.table.cpu().numpy()
            for g in np.flatnonzero(table >= 0):
                pool[g * S:(g + 1) * S] = 0
            out = L.decode(x, ids, w, lists, cache, layer, pool=pool)
            L.check(out, x, ids, w, False, f"cache step {step} layer {layer}", layer)
    # planned with the split call: hits from slots, misses from the pool
    x, ids, w = L.inputs(T)
    logits = torch.zeros((T, E), device="cuda").scatter_(1, ids.long(), 5.0 - torch.arange(k, device="cuda").float().repeat(T, 1))
    got_ids, got_w = torch.empty_like(ids), torch.empty_like(w)
    lists = m.DeviceClassifyOut(12)
    m.route_plan(L.desc, cache, 1, logits, got_ids, got_w, lists)
    assert (got_ids == ids).all()
    out = L.decode(x, ids, w, lists, cache, 1)
    L.check(out, x, ids, w, False, "planned", 1)
    m.evict_fill(L.desc, cache, L.pool, 1, None, tick + 1, ids, m.EvictPolicy(5, 1, 1), lists)
    torch.cuda.synchronize()
    table = cache.table.cpu().numpy().reshape(2, E)
    for e in np.flatnonzero(table[1] >= 0):
        s = table[1][e]
        assert (cache.data[s * S:(s + 1) * S].cpu().numpy() == L.blobs[E + e]).all()


def test_decode_from_a_pinned_host_pool():
    import torch
    L = Layer(128, 64, 6, 2, 21)
    x, ids, w = L.inputs(3)
    host = torch.empty(L.pool.numel(), dtype=torch.uint8, pin_memory=True)
    host.copy_(L.pool)
    assert (L.decode(x, ids, w, pool=host) == L.decode(x, ids, w)).all()


def test_captured_and_replayed_layer():
    """Routing, the expert SwiGLU (both forms) and a dense projection in two graphs that share
    the workspaces, replayed in turn with new inputs and other work between."""
    import torch
    import moe_expert_layer_02_amd as m
    H, I, E, k, T = 256, 128, 16, 4, 20
    L = Layer(H, I, E, k, 5)
    r = m.RouterDesc(E, k, m.SCORE_SIGMOID, 4, 2, 1, 2.5)
    dev = dict(device="cuda")
    bias = torch.zeros(E, **dev)
    ws_d, ws_p, ws_m = (L.workspace(T, mode) for mode in (m.MODE_DECODE_I8, m.MODE_PREFILL_I8, m.MODE_PERMUTE))
    wq = torch.randint(-127, 128, (96, H), dtype=torch.int8, **dev)
    sw = torch.rand(96, **dev) * 0.01
    S = o8.expert_bytes(H, I)

    def make():
        return dict(x=torch.zeros((T, H), dtype=torch.bfloat16, **dev), logits=torch.zeros((T, E), **dev),
                    ids=torch.zeros((T, k), dtype=torch.int32, **dev), w=torch.zeros((T, k), **dev),
                    perm=torch.zeros(T * k, dtype=torch.int32, **dev), off=torch.zeros(E + 1, dtype=torch.int32, **dev),
                    a=torch.zeros((T, H), dtype=torch.bfloat16, **dev), b=torch.zeros((T, H), dtype=torch.bfloat16, **dev),
                    xq=torch.zeros((T, H), dtype=torch.int8, **dev), xs=torch.zeros(T, **dev),
                    c=torch.zeros((T, 96), **dev))

    def go(s):
        m.route_scored(r, s["logits"], bias, s["ids"], s["w"])
        m.permute(L.desc, s["ids"], s["perm"], s["off"], ws_m)
        m.expert_ffn_prefill_i8(L.desc, s["x"], s["ids"], s["w"], L.pool[:E * S], s["perm"], s["off"], s["a"], ws_p)
        m.expert_ffn_decode_i8(L.desc, s["x"], s["ids"], s["w"], None, L.pool, 0, None, s["b"], ws_d)
        m.quantize_i8(s["x"], s["xq"], s["xs"])
        m.matmul_i8(s["xq"], s["xs"], wq, sw, s["c"])

    sets, graphs = [make(), make()], []
    for s in sets:
        go(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go(s)
        graphs.append(g)
    for turn in range(4):
        for s, g in zip(sets, graphs):
            gen = torch.Generator(device="cuda")
            gen.manual_seed(100 + turn)
            s["x"].copy_(torch.randn((T, H), generator=gen, **dev))
            s["logits"].copy_(torch.randn((T, E), generator=gen, **dev))
            g.replay()
            torch.cuda.synchronize()
            got = {n: s[n].clone() for n in ("ids", "w", "a", "b", "c")}
            for n in got:
                s[n].zero_()
            go(s)                                             # eager, in between
            torch.cuda.synchronize()
            for n in got:
                assert (got[n] == s[n]).all(), (turn, n)
            L.check(got["a"], s["x"], s["ids"], s["w"], True, f"replay {turn} prefill")
            L.check(got["b"], s["x"], s["ids"], s["w"], False, f"replay {turn} decode")


def test_whole_layer_with_a_shared_expert():
    """A layer as a model runs it, on a stream of its own: scored routing with a bias, the routed
    experts, and a shared expert built from the dense product, all from one quantised x."""
    import torch
    import moe_expert_layer_02_amd as m
    H, I, E, k, T = 512, 256, 32, 4, 70
    L = Layer(H, I, E, k, 31)
    shared = Layer(H, I, 1, 1, 32)
    rng = np.random.default_rng(8)
    x, _, _ = L.inputs(T)
    logits = torch.from_numpy(rng.normal(0, 1, (T, E)).astype(np.float32)).cuda()
    bias = torch.from_numpy(rng.normal(0, 0.05, E).astype(np.float32)).cuda()
    r = m.RouterDesc(E, k, m.SCORE_SIGMOID, 4, 2, 1, 2.5)
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    one = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    ones = torch.ones((T, 1), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.route_scored(r, logits, bias, ids, w, stream=side)
    routed = L.prefill(x, ids, w, stream=side)
    dense = shared.prefill(x, one, ones, stream=side)
    # the shared expert again from the dense calls
    (gq, gs), (uq, us), (dq, ds) = ((torch.from_numpy(np.array(q)).cuda(), torch.from_numpy(np.array(s)).cuda())
                                    for q, s in o8.matrices(shared.blobs[0], H, I))
    xq, xs = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    g, u = (torch.empty((T, I), device="cuda") for _ in range(2))
    hq, hs = torch.empty((T, I), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.quantize_i8(x, xq, xs)
        m.matmul_i8(xq, xs, gq, gs, g)
        m.matmul_i8(xq, xs, uq, us, u)
        h = (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)
        m.quantize_i8(h, hq, hs)
        m.matmul_i8(hq, hs, dq, ds, y)
    torch.cuda.synchronize()
    seen = logits.cpu().numpy()
    want_ids, want_w = o8.route_scored(seen, bias.cpu().numpy(), k, "sigmoid", 4, 2, True, 2.5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert np.all(np.abs(w.cpu().numpy() - want_w) <= 2.0 ** -23 * want_w)
    L.check(routed, x, ids, w, True, "routed")
    shared.check(dense, x, one, ones, True, "shared expert, grouped")
    shared.check(y, x, one, ones, True, "shared expert, dense calls")


def test_binding_refuses():
    import torch
    import moe_expert_layer_02_amd as m
    L = Layer(64, 64, 4, 2, 1)
    x, ids, w = L.inputs(3)
    with pytest.raises(TypeError):
        L.decode(x.half(), ids, w)
    with pytest.raises(ValueError):
        L.decode(x[:, :32], ids, w)
    with pytest.raises(ValueError):
        L.prefill(x, ids, w[:2])
    with pytest.raises(ValueError):
        L.decode(x, ids, w, layer=1)                           # beyond the pool
    with pytest.raises(m.Moe355Error):
        L.decode(x, ids, w, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    q, s = torch.zeros((3, 64), dtype=torch.int8, device="cuda"), torch.zeros(3, device="cuda")
    with pytest.raises(TypeError):
        m.quantize_i8(x.float(), q, s)
    with pytest.raises(ValueError):
        m.quantize_i8(x, q[:2], s)
    with pytest.raises(ValueError):
        m.matmul_i8(q, s, q[:, :32], s, torch.zeros((3, 3), device="cuda"))
    with pytest.raises(m.Moe355Error):                         # rows that do not start at 16 bytes
        m.matmul_i8(torch.zeros((3, 72), dtype=torch.int8, device="cuda")[:, :64], s, q, s,
                    torch.zeros((3, 3), device="cuda"))
