"""The operators of mixture-of-experts layers on the GPU: plan, grouped product
and combine, alone and together, against plain 64-bit implementations."""
import numpy as np
import pytest
import torch

import mx_reference as X
from gpu_helpers import dev, require_gpu
from weight_quantized_gemm_amd import qgemm as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _ids(rng, T, topk, E, skew=0.0, drop=0.0):
    """Expert ids [T][topk]: uniform, or with a few favourites; some outside [0, E)."""
    if skew:
        p = np.exp(rng.standard_normal(E) * skew)
        ids = rng.choice(E, size=(T, topk), p=p / p.sum())
    else:
        ids = rng.integers(0, E, (T, topk))
    out = rng.choice([-1, E, E + 5, -(2 ** 31), 2 ** 31 - 1], size=ids.shape)
    return np.where(rng.random(ids.shape) < drop, out, ids).astype(np.int64)


# ---------------------------------------------------------------------------
# Plan
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,topk,E", [(1, 1, 1), (1, 8, 128), (3, 2, 4), (64, 1, 64), (65, 1, 63), (16, 8, 128),
                                      (1000, 3, 7), (1024, 8, 1024), (4097, 2, 1023), (8192, 1, 5), (8193, 1, 5),
                                      (16384, 8, 128), (70001, 8, 256), (100003, 1, 1), (0, 4, 9), (5, 0, 9)])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_plan(T, topk, E, drop):
    rng = np.random.default_rng(T + topk + E)
    ids = _ids(rng, T, topk, E, skew=1.0 if E > 4 else 0.0, drop=drop)
    want = X.plan(ids, E)
    for dt in (np.int64, np.int32):
        got = Q.qgemm_group_plan(dev(ids.astype(dt)), E)
        for name, g, w in zip(("offsets", "rows", "slots"), got, want):
            assert np.array_equal(g.cpu().numpy(), w), f"{name} {dt.__name__}"


def test_plan_int64_ids_beyond_32_bits():
    """An id that only looks valid in its low word has no slot."""
    ids = np.array([[1, (1 << 32) + 1], [-(1 << 32), 0], [2, (7 << 40)]], np.int64)
    for g, w in zip(Q.qgemm_group_plan(dev(ids), 3), X.plan(ids, 3)):
        assert np.array_equal(g.cpu().numpy(), w)


def test_plan_one_expert_takes_all():
    ids = np.full((20000, 4), 17)
    for g, w in zip(Q.qgemm_group_plan(dev(ids), 64), X.plan(ids, 64)):
        assert np.array_equal(g.cpu().numpy(), w)


def test_plan_captured_with_its_workspace():
    T, topk, E = 6000, 4, 40
    rng = np.random.default_rng(1)
    ids = dev(_ids(rng, T, topk, E))
    nb = Q.qgemm_group_plan_size(T, topk, E)
    assert nb > 0
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    out = [torch.empty(s, dtype=torch.int32, device="cuda") for s in ((E + 1,), (T * topk,), (T, topk))]
    Q.qgemm_group_plan(ids, E, *out, workspace=ws, ws_bytes=nb)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Q.qgemm_group_plan(ids, E, *out, workspace=ws, ws_bytes=nb)
    for seed in range(4):
        new = _ids(np.random.default_rng(seed), T, topk, E, skew=1.0, drop=0.1)
        ids.copy_(torch.from_numpy(new))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        for o, w in zip(out, X.plan(new, E)):
            assert np.array_equal(o.cpu().numpy(), w)


# ---------------------------------------------------------------------------
# Grouped product
# ---------------------------------------------------------------------------
class Experts:
    def __init__(self, fmt, E, K, N, seed):
        rng = np.random.default_rng(seed)
        qs = [X.encode((rng.standard_normal((N, K)) * 0.02).astype(np.float32)) for _ in range(E)]
        q, s = np.stack([a for a, _ in qs]), np.stack([b for _, b in qs])
        self.fmt, self.E, self.K, self.N = fmt, E, K, N
        self.w = [X.decode(a, b) for a, b in qs]
        self.Bq, self.scales = Q.qgemm_mx_pack_device(K, N, dev(q), dev(s), E=E)

    def reference(self, A, rows, offsets):
        """float64 [S][N], NaN in rows no expert owns, and sum |a w|."""
        a = X.decode(*X.encode(A)) if self.fmt == "mxfp4a4" else A.astype(np.float64)
        C = np.full((len(rows), self.N), np.nan)
        B = np.full((len(rows), self.N), np.nan)
        for e in range(self.E):
            at = slice(offsets[e], offsets[e + 1])
            C[at] = a[rows[at]] @ self.w[e].T
            B[at] = np.abs(a[rows[at]]) @ np.abs(self.w[e]).T
        return C, B

    def run(self, A, rows, offsets, C, **kw):
        Q.qgemm_run_grouped(self.K, self.N, self.E, self.fmt, A, rows, offsets, self.Bq, self.scales, C, **kw)


def _acts(rng, T, K):
    A = rng.standard_normal((T, K)).astype(np.float16)
    A[:, rng.random(K) < 0.02] *= 20
    return A


# rows per expert: empty ones first, between and last; one, a few, a tile's edge, many
RAGGED = [[1], [0, 1, 0], [1, 1, 1, 1], [3, 0, 0, 9, 1, 8, 0], [32, 33, 31, 0, 64], [5] * 40, [0] * 70 + [2] + [0] * 60,
          [127, 128, 129, 1], [300, 0, 7, 0, 513], [0, 0, 260], [17] * 9]


@pytest.mark.parametrize("sizes", RAGGED, ids=lambda s: "-".join(map(str, s[:6])) + f"x{len(s)}")
@pytest.mark.parametrize("K,N", [(64, 33), (320, 96), (1024, 300)])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_grouped_product(fmt, K, N, sizes):
    rng = np.random.default_rng(sum(sizes) + K)
    ex = Experts(fmt, len(sizes), K, N, K + N)
    n = sum(sizes)
    T, S = max(2, n // 3), n + 5               # five slots behind the last group
    A = _acts(rng, T, K)
    rows = rng.integers(0, T, S).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    ref, sumabs = ex.reference(A, rows, offsets)
    C = torch.full((S, N), 9.0, device="cuda")
    ex.run(dev(A), dev(rows), dev(offsets), C)
    C = C.cpu().numpy()
    assert (C[n:] == 9.0).all(), "rows behind the last group were written"
    X.check_product(C[:n], ref[:n], sumabs[:n], K, what=f"{fmt} {K}x{N} {sizes[:8]}")


@pytest.mark.parametrize("kind,out", [("none", "f16"), ("silu", "f32"), ("relu", "f16")])
@pytest.mark.parametrize("K,N,sizes", [(320, 70, [3, 0, 1, 8, 5]), (640, 256, [100, 0, 200, 33]), (1024, 129, [1] * 12)])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_grouped_epilogue(fmt, K, N, sizes, kind, out):
    """Bias of each row's own expert, residual in place, activation, and the
    identity index."""
    rng = np.random.default_rng(K)
    E, S = len(sizes), sum(sizes)
    ex = Experts(fmt, E, K, N, 3)
    A = _acts(rng, S, K)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    ref, sumabs = ex.reference(A, np.arange(S), offsets)
    bias = rng.standard_normal((E, N)).astype(np.float32)
    res = rng.standard_normal((S, N)).astype(np.float16 if out == "f16" else np.float32)
    each = np.repeat(np.arange(E), sizes)
    pre = ref + bias[each] + res
    C = dev(res)
    ex.run(dev(A), None, dev(offsets), C, bias=dev(bias), residual=C, activation=kind, out_type=out)
    X.check_product(C.cpu().numpy(), X.act(pre, kind), sumabs + np.abs(bias[each]) + np.abs(res.astype(float)), K, out)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_one_group_equals_the_dense_product_closely(fmt):
    K, N, S = 512, 200, 150
    rng = np.random.default_rng(8)
    ex = Experts(fmt, 1, K, N, 5)
    A = _acts(rng, S, K)
    offsets = np.array([0, S], np.int32)
    ref, sumabs = ex.reference(A, np.arange(S), offsets)
    C, D = torch.empty((S, N), device="cuda"), torch.empty((S, N), device="cuda")
    ex.run(dev(A), None, dev(offsets), C)
    Q.qgemm_run(S, K, N, fmt, dev(A), ex.Bq, ex.scales, D)
    for c in (C, D):
        X.check_product(c.cpu().numpy(), ref, sumabs, K)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_bad_indexes_stay_inside(fmt):
    """Row indexes and offsets outside their ranges are limited to them: nothing
    outside A and C is touched, and slots with good indexes keep their values."""
    K, N, T, S = 128, 64, 6, 40
    rng = np.random.default_rng(2)
    ex = Experts(fmt, 3, K, N, 1)
    A = _acts(rng, T, K)
    rows = rng.integers(0, T, S).astype(np.int32)
    bad = rows.copy()
    bad[3], bad[20], bad[33] = -1, 2 ** 31 - 1, -(2 ** 31)
    offsets = np.array([0, 10, 30, S], np.int32)
    ref, sumabs = ex.reference(A, rows, offsets)
    buf = torch.full((S * N + 1024,), 5.0, device="cuda")
    C = buf[:S * N].view(S, N)
    ex.run(dev(A), dev(bad), dev(offsets), C)
    keep = np.setdiff1d(np.arange(S), [3, 20, 33])
    X.check_product(C.cpu().numpy()[keep], ref[keep], sumabs[keep], K)
    assert (buf[S * N:] == 5.0).all()
    wild = np.array([-7, 10, 30, 2 ** 31 - 1], np.int32)
    ex.run(dev(A), dev(rows), dev(wild), C)
    X.check_product(C.cpu().numpy(), ref, sumabs, K)
    assert (buf[S * N:] == 5.0).all()
    for wild in ([0, 30, 10, 40], [50, 60, 70, 80], [-5, -4, -3, -2]):
        ex.run(dev(A), dev(rows), dev(np.array(wild, np.int32)), C)
        torch.cuda.synchronize()
        assert (buf[S * N:] == 5.0).all()


def test_grouped_argument_checks():
    ex = Experts("mxfp4", 2, 64, 32, 1)
    A = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    C = torch.empty((4, 32), device="cuda")
    for kw in (dict(A=A.float()), dict(C=C.half()), dict(off=off[:2]), dict(rows=off), dict(A=A[:, :32]),
               dict(bias=torch.zeros(32, device="cuda")), dict(off=off.cpu()), dict(C=C.t())):
        a = dict(A=A, rows=None, off=off, C=C, bias=None)
        a.update(kw)
        with pytest.raises(ValueError):
            ex.run(a["A"], a["rows"], a["off"], a["C"], bias=a["bias"])
    with pytest.raises(Q.QGemmError):
        Q.qgemm_run_grouped(64, 32, 2, "int4b64", A, None, off, ex.Bq, ex.scales, C)


# ---------------------------------------------------------------------------
# Combine
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,topk,N", [(1, 1, 1), (1, 8, 2560), (3, 2, 33), (16, 8, 4096), (5, 4, 2056), (257, 3, 264),
                                      (9, 0, 40), (1000, 4, 1100), (2, 5, 7)])
@pytest.mark.parametrize("yt,ct", [("f32", "f32"), ("f32", "f16"), ("f16", "f32"), ("f16", "f16")])
def test_combine(T, topk, N, yt, ct):
    """fp32 sums: topk products and additions, one unit each, of sum |w y|."""
    rng = np.random.default_rng(T + topk + N)
    dt = {"f32": np.float32, "f16": np.float16}
    S = T * topk
    Y = rng.standard_normal((S, N)).astype(dt[yt])
    slots = rng.permutation(S).reshape(T, topk).astype(np.int32)
    w = rng.random((T, topk)).astype(np.float32)
    if topk > 1:
        slots[:, 0] = np.where(rng.random(T) < 0.5, -1, slots[:, 0])
        slots[T // 2] = -1                                      # a token without slots
        slots[0, 1] = S + 3                                     # outside Y
        w[slots < 0] = np.nan                                   # never used
        w[0, 1] = np.inf
    ref, mass = np.zeros((T, N)), np.zeros((T, N))
    for j in range(topk):
        on = (slots[:, j] >= 0) & (slots[:, j] < S)
        ref[on] += w[on, j, None].astype(np.float64) * Y[slots[on, j]]
        mass[on] += np.abs(w[on, j, None].astype(np.float64) * Y[slots[on, j]])
    C = torch.full((T, N), float("nan"), dtype=torch.float16 if ct == "f16" else torch.float32, device="cuda")
    Q.qgemm_group_combine(dev(Y) if S else torch.empty((0, N), dtype=getattr(torch, "float16" if yt == "f16" else
                                                                             "float32"), device="cuda"),
                          dev(slots), dev(w), C)
    bound = topk * 2.0 ** -24 * mass + 1e-40 + (2.0 ** -11 * np.abs(ref) + 2.0 ** -25 if ct == "f16" else 0.0)
    err = np.abs(C.cpu().numpy().astype(np.float64) - ref)
    assert (err <= bound * 1.001).all()


def test_combine_uses_a_slot_twice():
    Y = dev(np.arange(24, dtype=np.float32).reshape(3, 8))
    slots = dev(np.array([[2, 2], [0, 2]], np.int32))
    C = torch.empty((2, 8), device="cuda")
    Q.qgemm_group_combine(Y, slots, dev(np.array([[1, 2], [3, 4]], np.float32)), C)
    y = Y.cpu().numpy()
    assert np.array_equal(C.cpu().numpy(), np.stack([3 * y[2], 3 * y[0] + 4 * y[2]]))


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
def _layer(T, topk, E, H, I, fmt, seed, drop):
    rng = np.random.default_rng(seed)
    up, down = Experts(fmt, E, H, I, seed), Experts(fmt, E, I, H, seed + 1)
    return (up, down, _acts(rng, T, H), _ids(rng, T, topk, E, skew=1.0, drop=drop),
            rng.random((T, topk)).astype(np.float32))


def _forward(up, down, x, ids, wt, E, out):
    offsets, rows, slots = Q.qgemm_group_plan(ids, E)
    S = rows.numel()
    h = torch.zeros((S, up.N), dtype=torch.float16, device="cuda")
    y = torch.empty((S, down.N), dtype=torch.float16, device="cuda")
    up.run(x, rows, offsets, h, activation="silu", out_type="f16")
    down.run(h, None, offsets, y, out_type="f16")
    Q.qgemm_group_combine(y, slots, wt, out)


@pytest.mark.parametrize("T,topk,E,drop", [(1, 2, 8, 0.0), (5, 4, 16, 0.2), (300, 3, 6, 0.1), (1500, 4, 8, 0.0)])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_layer(fmt, T, topk, E, drop):
    """Plan, two grouped products with the activation between, combine. Each stage
    is checked from the stage before it as the GPU left it, so the bounds stay
    those of one operator."""
    H, I = 256, 320
    up, down, x, ids, wt = _layer(T, topk, E, H, I, fmt, T + E, drop)
    offsets, rows, slots = Q.qgemm_group_plan(dev(ids), E)
    off, rws, slt = X.plan(ids, E)
    assert np.array_equal(slots.cpu().numpy(), slt)
    n, S = off[-1], T * topk
    h = torch.zeros((S, I), dtype=torch.float16, device="cuda")
    up.run(dev(x), rows, offsets, h, activation="silu", out_type="f16")
    ref, mass = up.reference(x, rws, off)
    X.check_product(h.cpu().numpy()[:n], X.act(ref[:n], "silu"), mass[:n], H, "f16", "up")
    y = torch.zeros((S, H), dtype=torch.float16, device="cuda")
    down.run(h, None, offsets, y, out_type="f16")
    hn = h.cpu().numpy()
    ref, mass = down.reference(hn, np.arange(S), off)
    X.check_product(y.cpu().numpy()[:n], ref[:n], mass[:n], I, "f16", "down")
    C = torch.empty((T, H), device="cuda")
    Q.qgemm_group_combine(y, slots, dev(wt), C)
    yn = y.cpu().numpy().astype(np.float64)
    want = np.where(slt[..., None] >= 0, wt[..., None].astype(np.float64) * yn[np.maximum(slt, 0)], 0.0)
    assert (np.abs(C.cpu().numpy() - want.sum(1)) <= topk * 2.0 ** -24 * np.abs(want).sum(1) * 1.001 + 1e-40).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_layer_in_a_graph(fmt):
    """The whole layer captured once (its scratch from the caching allocator's
    graph pool or given) and replayed with other tokens and routes, with eager
    work between the replays."""
    T, topk, E, H, I = 24, 4, 10, 256, 192
    up, down, x, ids, wt = _layer(T, topk, E, H, I, fmt, 5, 0.1)
    xd, idd, wd = dev(x), dev(ids), dev(wt)
    S = T * topk
    nb = max(Q.qgemm_grouped_workspace_size(S, T, H, I, E, fmt), Q.qgemm_grouped_workspace_size(S, S, I, H, E, fmt), 16)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    rows, slots = torch.empty(S, dtype=torch.int32, device="cuda"), torch.empty((T, topk), dtype=torch.int32,
                                                                               device="cuda")
    h = torch.zeros((S, I), dtype=torch.float16, device="cuda")
    y = torch.zeros((S, H), dtype=torch.float16, device="cuda")
    out = torch.empty((T, H), device="cuda")

    def step():
        Q.qgemm_group_plan(idd, E, off, rows, slots)
        up.run(xd, rows, off, h, activation="silu", out_type="f16", workspace=ws, ws_bytes=nb)
        down.run(h, None, off, y, out_type="f16", workspace=ws, ws_bytes=nb)
        Q.qgemm_group_combine(y, slots, wd, out)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in range(4):
        rng = np.random.default_rng(seed)
        xd.copy_(torch.from_numpy(_acts(rng, T, H)))
        idd.copy_(torch.from_numpy(_ids(rng, T, topk, E, skew=1.0, drop=0.2)))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = torch.empty_like(out)
        _forward(up, down, xd, idd, wd, E, want)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_two_streams_at_once():
    """Two layers on two streams, each with its own buffers."""
    T, topk, E, H, I = 200, 4, 8, 512, 512
    sets = [_layer(T, topk, E, H, I, fmt, s, 0.0) for s, fmt in ((1, "mxfp4"), (2, "mxfp4a4"))]
    ins = [[dev(v) for v in (x, ids, wt)] for _, _, x, ids, wt in sets]
    want = []
    for (up, down, *_), (x, ids, wt) in zip(sets, ins):
        out = torch.empty((T, H), device="cuda")
        _forward(up, down, x, ids, wt, E, out)
        want.append(out)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty((T, H), device="cuda") for _ in sets]
    for _ in range(3):
        for st, (up, down, *_), (x, ids, wt), out in zip(streams, sets, ins, outs):
            with torch.cuda.stream(st):
                _forward(up, down, x, ids, wt, E, out)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_combine_more_tokens_than_one_launch_axis():
    """More workgroups than one axis of a launch may have threads for (2^32)."""
    T, S = (1 << 24) + 70001, 1000
    g = torch.Generator(device="cuda").manual_seed(5)
    Y = torch.randn((S, 1), device="cuda", generator=g)
    slots = torch.randint(0, S, (T, 1), device="cuda", generator=g, dtype=torch.int32)
    w = torch.rand((T, 1), device="cuda", generator=g)
    C = torch.full((T, 1), float("nan"), device="cuda")
    Q.qgemm_group_combine(Y, slots, w, C)
    assert torch.equal(C, w * Y[slots[:, 0].long()])     # one product, rounded once


@pytest.mark.parametrize("handle", [False, True])
def test_outputs_belong_to_the_stream_of_the_call(handle):
    """Results allocated for a call on another stream do not take memory that
    work of the current stream may still use."""
    ids = torch.randint(0, 8, (70000, 3), device="cuda", dtype=torch.int32)
    x = torch.randn((1024, 4096), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    given = side.cuda_stream if handle else side
    sizes = {"rows": 70000 * 3 * 4, "q": 1024 * 2048, "y": 1024 * 4096 * 4}
    freed = {}
    for name, n in sizes.items():
        t = torch.empty(n, dtype=torch.uint8, device="cuda")
        freed[name] = t.data_ptr()
        del t
    want = [t.clone() for t in Q.qgemm_group_plan(ids, 8)]
    torch.cuda.synchronize()
    offsets, rows, slots = Q.qgemm_group_plan(ids, 8, stream=given)
    q, s = Q.qgemm_mx_quantize_device(x, stream=given)
    y = Q.qgemm_mx_dequantize_device(q, s, stream=given)
    torch.cuda.synchronize()
    again = {n: torch.empty(b, dtype=torch.uint8, device="cuda").data_ptr() for n, b in sizes.items()}
    for t in (rows, slots, q, y):
        assert t.data_ptr() not in freed.values() and t.data_ptr() not in again.values()
    assert all(torch.equal(a, b) for a, b in zip(want, (offsets, rows, slots)))
    assert np.array_equal(y.cpu().numpy(), X.decode(*X.encode(x.cpu().numpy())).astype(np.float32))


@pytest.mark.parametrize("K", [64, 192, 448, 832, 1088, 1344])
@pytest.mark.parametrize("mean", [1, 4, 8, 40, 130, 300])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_every_tile_of_the_grouped_product(fmt, mean, K):
    """Groups of every size class (empty ones and parts of tiles among them)
    over enough columns for the large tiles, rows gathered, K of every number
    of stages left over; references on the GPU in 64 bits, bounds as in
    check_product."""
    E, N = 12, 4100
    rng = np.random.default_rng(mean + K)
    sizes = rng.integers(0, 2 * mean + 1, E)
    sizes[0], sizes[E - 1] = 2 * mean, 0
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    n = int(offsets[-1])
    T, S = max(3, n // 3), n + 7
    g = torch.Generator(device="cuda").manual_seed(mean + K)
    A = torch.randn((T, K), device="cuda", generator=g).half()
    W = torch.randn((E * N, K), device="cuda", generator=g)
    rows = torch.randint(0, T, (S,), device="cuda", generator=g, dtype=torch.int32)
    q, s = Q.qgemm_mx_quantize_device(W)
    w = Q.qgemm_mx_dequantize_device(q, s).view(E, N, K)
    Bq, Sp = Q.qgemm_mx_pack_device(K, N, q, s, E=E)
    C = torch.full((S, N), 9.0, device="cuda")
    Q.qgemm_run_grouped(K, N, E, fmt, A, rows, dev(offsets), Bq, Sp, C)
    a = Q.qgemm_mx_dequantize_device(*Q.qgemm_mx_quantize_device(A)).double() if fmt == "mxfp4a4" else A.double()
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        x, we = a[rows[lo:hi].long()], w[e].double()
        ref, mass = x @ we.t(), x.abs() @ we.abs().t()
        err = (C[lo:hi].double() - ref).abs()
        assert bool((err <= (K + 16) * 2.0 ** -23 * mass + 1e-37).all()), e
    assert bool((C[n:] == 9.0).all())


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_layer_on_a_given_stream(fmt):
    """Every call with stream= and no workspace: the library's own stream-ordered
    scratch, the same bits."""
    T, topk, E, K, N = 3000, 3, 8, 512, 384
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(0, E + 2, (T, topk), device="cuda", generator=g, dtype=torch.int32)
    wt = torch.rand((T, topk), device="cuda", generator=g)
    A = torch.randn((T, K), device="cuda", generator=g).half()
    Bq, Sp = Q.qgemm_mx_pack_device(K, N, *Q.qgemm_mx_quantize_device(
        torch.randn((E * N, K), device="cuda", generator=g)), E=E)

    def layer(stream):
        C, out = torch.zeros((T * topk, N), device="cuda"), torch.empty((T, N), device="cuda")
        torch.cuda.synchronize()
        offsets, rows, slots = Q.qgemm_group_plan(ids, E, stream=stream)
        Q.qgemm_run_grouped(K, N, E, fmt, A, rows, offsets, Bq, Sp, C, activation="relu", stream=stream)
        Q.qgemm_group_combine(C, slots, wt, out, stream=stream)
        torch.cuda.synchronize()
        return out

    want, side = layer(None), torch.cuda.Stream()
    for stream in (side, side.cuda_stream, torch.cuda.default_stream(), 0):
        assert torch.equal(layer(stream), want)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_two_threads_on_one_stream(fmt):
    """Two threads of a program on the same stream, neither giving a workspace
    nor outputs of the plan: each gets what it gets alone."""
    import threading
    T, topk, E, K, N = 3000, 2, 8, 512, 256
    sets = []
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ids = torch.randint(0, E + 1, (T, topk), device="cuda", generator=g, dtype=torch.int32)
        A = torch.randn((T, K), device="cuda", generator=g).half()
        Bq, Sp = Q.qgemm_mx_pack_device(K, N, *Q.qgemm_mx_quantize_device(
            torch.randn((E * N, K), device="cuda", generator=g)), E=E)
        sets.append((ids, A, Bq, Sp))

    def layer(ids, A, Bq, Sp):
        C = torch.zeros((T * topk, N), device="cuda")
        offsets, rows, slots = Q.qgemm_group_plan(ids, E)
        Q.qgemm_run_grouped(K, N, E, fmt, A, rows, offsets, Bq, Sp, C)
        return offsets, rows, slots, C

    want = [layer(*s) for s in sets]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        for _ in range(40):
            got[i].append(layer(*sets[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        assert len(runs) == 40
        assert all(torch.equal(a, b) for r in runs for a, b in zip(w, r))


def test_nearly_the_most_threads_of_a_launch():
    """1024 experts of one row each over 2^20 - 128 columns: 512 threads short of
    2^32 by one column of tiles, byte offsets of the weights and of C far past
    32 bits. The experts share codes and differ in scale."""
    E, K, N = 1024, 64, (1 << 20) - 128
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randint(0, 256, (N, K // 2), device="cuda", generator=g, dtype=torch.uint8)
    s = torch.full((N, K // 32), 120, device="cuda", dtype=torch.uint8)
    w = Q.qgemm_mx_dequantize_device(q, s).double()
    wp, sp = Q.qgemm_mx_pack_device(K, N, q, s)
    Bq = wp.expand(E, -1).contiguous().view(-1)
    up = (torch.arange(E, device="cuda") % 8).to(torch.uint8)
    Sp = torch.where(sp > 0, sp[None] + up[:, None], 0).to(torch.uint8).view(-1)
    A = torch.randn((E, K), device="cuda", generator=g).half()
    C = torch.full((E, N), float("nan"), dtype=torch.float16, device="cuda")
    Q.qgemm_run_grouped(K, N, E, "mxfp4", A, None, torch.arange(E + 1, device="cuda", dtype=torch.int32), Bq, Sp, C,
                        out_type="f16")
    for e in range(0, E, 64):
        a = A[e:e + 64].double() * 2.0 ** up[e:e + 64, None].double()
        ref, mass = a @ w.t(), a.abs() @ w.abs().t()
        err = (C[e:e + 64].double() - ref).abs()
        assert bool((err <= (K + 16) * 2.0 ** -23 * mass + 2.0 ** -11 * ref.abs() + 2.0 ** -25).all()), e


# average rows, experts and columns that reach the tiles between the smallest
# and the largest: 32 x 256 (four-column epilogue and an odd width), 64 x 128, 32 x
# 64, 32 x 32 and 64 x 256 (tests/test_mx_tiles.py checks what they reach)
MIDDLE = [(8, 12, 8200), (8, 12, 8203), (2, 12, 8200), (13, 13, 8200), (40, 12, 2500), (14, 12, 1300), (20, 5, 300),
          (40, 12, 8200)]
# one, two, three and no stages more than whole turns of four, of 64 elements (fp16 activations) and of 256
MIDDLE_K = [64, 128, 192, 256, 448, 640, 832, 1088, 1280]


def middle_sizes(mean, E, K):
    """Rows of each expert: none to twice the average, the last one empty."""
    sizes = np.random.default_rng(mean + K).integers(0, 2 * mean + 1, E)
    sizes[0], sizes[E - 1] = 2 * mean, 0
    return sizes


def _middle(fmt, mean, E, N, K):
    """(A, rows, offsets, Bq, scales, C, [float64 values of A's rows], [of the weights])."""
    offsets = np.concatenate([[0], np.cumsum(middle_sizes(mean, E, K))]).astype(np.int32)
    n = int(offsets[-1])
    T, S = max(3, n // 3), n + 7
    g = torch.Generator(device="cuda").manual_seed(mean + K)
    A = torch.randn((T, K), device="cuda", generator=g).half()
    rows = torch.randint(0, T, (S,), device="cuda", generator=g, dtype=torch.int32)
    q, s = Q.qgemm_mx_quantize_device(torch.randn((E * N, K), device="cuda", generator=g))
    w = Q.qgemm_mx_dequantize_device(q, s).view(E, N, K)
    a = Q.qgemm_mx_dequantize_device(*Q.qgemm_mx_quantize_device(A)).double() if fmt == "mxfp4a4" else A.double()
    return A, rows, offsets, *Q.qgemm_mx_pack_device(K, N, q, s, E=E), a, w


@pytest.mark.parametrize("K", MIDDLE_K)
@pytest.mark.parametrize("mean,E,N", MIDDLE)
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_middle_tiles_of_the_grouped_product(fmt, mean, E, N, K):
    """Ragged groups, rows gathered, K of every number of stages left over, rows
    behind the last group untouched; bounds as in check_product."""
    A, rows, offsets, Bq, Sp, a, w = _middle(fmt, mean, E, N, K)
    n, S = int(offsets[-1]), rows.numel()
    C = torch.full((S, N), 9.0, device="cuda")
    Q.qgemm_run_grouped(K, N, E, fmt, A, rows, dev(offsets), Bq, Sp, C)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        x, we = a[rows[lo:hi].long()], w[e].double()
        ref, mass = x @ we.t(), x.abs() @ we.abs().t()
        err = (C[lo:hi].double() - ref).abs()
        assert bool((err <= (K + 16) * 2.0 ** -23 * mass + 1e-37).all()), e
        assert float(err.norm()) <= 4 * (K + 16) ** 0.5 * 2.0 ** -24 * float(mass.norm()), e
    assert bool((C[n:] == 9.0).all())


@pytest.mark.parametrize("mean,E,N", MIDDLE)
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_middle_tiles_with_an_epilogue(fmt, mean, E, N):
    """Slot s reads row s, bias of the row's own expert, residual in place, ReLU
    (slope 1), fp16 result (half a step more)."""
    K = 576
    A, rows, offsets, Bq, Sp, a, w = _middle(fmt, mean, E, N, K)
    n, S = int(offsets[-1]), rows.numel()
    A, a = A[rows.long()].contiguous(), a[rows.long()]
    g = torch.Generator(device="cuda").manual_seed(N)
    bias, res = torch.randn((E, N), device="cuda", generator=g), torch.randn((S, N), device="cuda", generator=g).half()
    C = res.clone()
    Q.qgemm_run_grouped(K, N, E, fmt, A, None, dev(offsets), Bq, Sp, C, bias=bias, residual=C, activation="relu",
                        out_type="f16")
    for e in range(E):
        at = slice(int(offsets[e]), int(offsets[e + 1]))
        we, b, r = w[e].double(), bias[e].double(), res[at].double()
        ref = (a[at] @ we.t() + b + r).clamp(min=0)
        mass = a[at].abs() @ we.abs().t() + b.abs() + r.abs()
        err = (C[at].double() - ref).abs()
        assert bool((err <= (K + 16) * 2.0 ** -23 * mass + 2.0 ** -11 * ref + 2.0 ** -25).all()), e
    assert torch.equal(C[n:], res[n:])


@pytest.mark.parametrize("T,topk,E", [(150000, 8, 128), (1048577, 1, 1024), (1 << 23, 8, 7)])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_plan_of_millions_of_choices(T, topk, E, drop):
    """More than 2^20 choices, up to the most there may be (2^26)."""
    g = torch.Generator(device="cuda").manual_seed(E)
    ids = torch.randint(0, E, (T, topk), device="cuda", generator=g, dtype=torch.int32)
    ids = torch.where(torch.rand((T, topk), device="cuda", generator=g) < drop, -1 - ids, ids)
    offsets, rows, slots = Q.qgemm_group_plan(ids, E)
    key = torch.where(ids < 0, E, ids).view(-1)
    by_key, order = torch.sort(key, stable=True)
    assert torch.equal(offsets, torch.searchsorted(by_key, torch.arange(E + 1, device="cuda",
                                                                        dtype=torch.int32)).to(torch.int32))
    assert torch.equal(rows, (order // topk).to(torch.int32))
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device="cuda")
    assert torch.equal(slots.view(-1), torch.where(key < E, place, -1).to(torch.int32))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
@pytest.mark.parametrize("at", [0, 77, 127])
def test_all_rows_of_many_experts_at_one(fmt, at):
    """As many slots as a quarter of the experts, for which two-row tiles are
    planned, and every one of them the same expert's."""
    E, K, N, S = 128, 576, 100, 32
    rng = np.random.default_rng(at)
    ex = Experts(fmt, E, K, N, 7)
    A = _acts(rng, S, K)
    offsets = np.where(np.arange(E + 1) > at, S, 0).astype(np.int32)
    ref, sumabs = ex.reference(A, np.arange(S), offsets)
    C = torch.full((S, N), 9.0, device="cuda")
    ex.run(dev(A), None, dev(offsets), C)
    X.check_product(C.cpu().numpy(), ref, sumabs, K, what=f"{fmt} {at}")


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_activations_past_four_gigabytes(fmt, grouped):
    """Rows read in order: A (17 GB) and its codes (4.3 GB) far past 32-bit byte
    offsets, dense and as two groups that meet inside a tile."""
    M, K, N = (1 << 19) + 5, 16384, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    A = torch.randn((M, K), device="cuda", generator=g, dtype=torch.float16)
    q, s = Q.qgemm_mx_quantize_device(torch.randn((2 * N, K), device="cuda", generator=g))
    w = Q.qgemm_mx_dequantize_device(q, s).view(2, N, K).double()
    Bq, Sp = Q.qgemm_mx_pack_device(K, N, q, s, E=2)
    C = torch.full((M, N), float("nan"), device="cuda")
    cut = M - 41
    if grouped:
        Q.qgemm_run_grouped(K, N, 2, fmt, A, None, torch.tensor([0, cut, M], device="cuda", dtype=torch.int32), Bq, Sp, C)
    else:
        Q.qgemm_run_ex(M, K, N, fmt, A, Bq, Sp, C)
    for lo, hi in ((0, 130), (131000, 131200), (262100, 262200), (M - 200, cut), (cut, M)):
        a = Q.qgemm_mx_dequantize_device(*Q.qgemm_mx_quantize_device(A[lo:hi])) if fmt == "mxfp4a4" else A[lo:hi]
        a, we = a.double(), w[1 if grouped and lo >= cut else 0]
        err = (C[lo:hi].double() - a @ we.t()).abs()
        assert bool((err <= (K + 16) * 2.0 ** -23 * (a.abs() @ we.abs().t()) + 1e-37).all()), lo


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_two_graphs_without_a_workspace(fmt):
    """Two captured layers whose plan and products take their scratch from torch's
    allocator (each graph's own pool), replayed in turn with new inputs and
    eager calls of the same sizes between them."""
    T, topk, E, K, N = 1500, 2, 6, 320, 192
    g = torch.Generator(device="cuda").manual_seed(8)
    Bq, Sp = Q.qgemm_mx_pack_device(K, N, *Q.qgemm_mx_quantize_device(
        torch.randn((E * N, K), device="cuda", generator=g)), E=E)
    assert Q.qgemm_group_plan_size(T, topk, E) > 0

    def fresh():
        return (torch.randint(0, E + 1, (T, topk), device="cuda", generator=g, dtype=torch.int32),
                torch.randn((T, K), device="cuda", generator=g).half())

    def layer(ids, A, C):
        offsets, rows, slots = Q.qgemm_group_plan(ids, E)
        C.zero_()
        Q.qgemm_run_grouped(K, N, E, fmt, A, rows, offsets, Bq, Sp, C)
        return slots

    sets = []
    for _ in range(2):
        ids, A = fresh()
        C = torch.empty((T * topk, N), device="cuda")
        layer(ids, A, C)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            slots = layer(ids, A, C)
        sets.append((graph, ids, A, C, slots))
    for turn in range(6):
        graph, ids, A, C, slots = sets[turn % 2]
        for t, new in zip((ids, A), fresh()):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(C)
        assert torch.equal(layer(ids, A, want), slots) and torch.equal(C, want)
