"""MXFP4 on the GPU: conversions bit for bit against the 64-bit rules, and the
dense products against the 64-bit product of the same operands."""
import numpy as np
import pytest
import torch

import mx_reference as X
from gpu_helpers import dev, require_gpu
from test_mx_cpu import special_rows
from weight_quantized_gemm_amd import qgemm as Q

pytestmark = pytest.mark.gpu

NP = {"f32": np.float32, "f16": np.float16}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _rows(rng, R, K):
    x = rng.standard_normal((R, K)).astype(np.float32)
    x[:, rng.random(K) < 0.02] *= 30.0
    x[rng.random(x.shape) < 0.05] = 0.0
    return x


# ---------------------------------------------------------------------------
# Conversions
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("R,K", [(1, 32), (1, 64), (3, 96), (1, 2560), (257, 160), (33, 4096), (5000, 32),
                                 (1031, 9728)])
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_quantize_rows(R, K, t):
    x = torch.from_numpy(_rows(np.random.default_rng(R + K), R, K)).to(Q._TORCH_TYPES[Q.TYPES[t]])
    q, s = Q.qgemm_mx_quantize_device(x.cuda())
    qr, sr = X.encode(x.double().numpy())
    assert np.array_equal(s.cpu().numpy(), sr)
    assert np.array_equal(q.cpu().numpy(), qr)


def test_quantize_corners():
    """Ties, saturation, signed zeros, subnormal numbers, the ends of the exponent
    range; a NaN or an infinity takes its own block only."""
    x = special_rows()
    q, s = Q.qgemm_mx_quantize_device(dev(x))
    qr, sr = X.encode(x)
    assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(q.cpu().numpy(), qr)
    x = np.random.default_rng(3).standard_normal((6, 128)).astype(np.float32)
    x[0, 3], x[1, 40], x[2, 127], x[3, 64] = np.nan, np.inf, -np.inf, -np.nan
    for t in (torch.float32, torch.float16, torch.bfloat16):
        y = torch.from_numpy(x).to(t)
        q, s = Q.qgemm_mx_quantize_device(y.cuda())
        qr, sr = X.encode(y.double().numpy())
        assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(q.cpu().numpy(), qr)
        assert np.count_nonzero(sr == 255) == 4


def test_quantize_every_half():
    """Every finite fp16 number beside its block's largest, at several block scales."""
    h = np.arange(65536, dtype=np.uint32).astype(np.uint16).view(np.float16)
    h = h[np.isfinite(h)]
    h = h[:len(h) // 31 * 31].reshape(-1, 31)
    for top in (2.0 ** -14, 0.11, 1.0, 5.5, 300.0, 65504.0):
        x = np.concatenate([h, np.full((len(h), 1), top, np.float16)], 1)
        q, s = Q.qgemm_mx_quantize_device(dev(x))
        qr, sr = X.encode(x)
        assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(q.cpu().numpy(), qr)


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_strided_rows(t):
    """Rows inside a wider tensor, quantised and written back without touching
    what lies between them."""
    dt = Q._TORCH_TYPES[Q.TYPES[t]]
    wide = torch.randn((37, 224), dtype=torch.float32).to(dt).cuda()
    x = wide[:, 32:128]
    q, s = Q.qgemm_mx_quantize_device(x)
    qr, sr = X.encode(x.double().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(q.cpu().numpy(), qr)
    out = torch.full((37, 224), 7.0, dtype=dt, device="cuda")
    Q.qgemm_mx_dequantize_device(q, s, Y=out[:, 32:128])
    assert torch.equal(out[:, 32:128].double().cpu(), torch.from_numpy(X.decode(qr, sr)).to(dt).double())
    assert (out[:, :32] == 7).all() and (out[:, 128:] == 7).all()
    with pytest.raises(Q.QGemmError):
        Q.qgemm_mx_quantize_device(wide[:, 1:97])        # rows that do not start aligned
    with pytest.raises(ValueError):
        Q.qgemm_mx_quantize_device(wide[:, 0:192:2])
    with pytest.raises(ValueError):
        Q.qgemm_mx_quantize_device(x, q=q[:3].contiguous())


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_dequantize_every_code_and_scale(t):
    """All 16 codes at all 256 scales, each rounded once to the type."""
    q = np.tile(np.arange(256, dtype=np.uint8), (256, 1)).reshape(256, 16, 16)
    q = np.concatenate([q.reshape(256, 256)], 1)
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    y = Q.qgemm_mx_dequantize_device(dev(q), dev(s), t)
    ref = torch.from_numpy(X.decode(q, s)).to(y.dtype)
    got = y.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(torch.nan_to_num(got.double(), nan=1.0, posinf=2e308, neginf=-2e308),
                       torch.nan_to_num(ref.double(), nan=1.0, posinf=2e308, neginf=-2e308))


def test_quantize_empty():
    for shape in ((0, 64), (3, 0)):
        q, s = Q.qgemm_mx_quantize_device(torch.empty(shape, device="cuda"))
        assert q.shape == (shape[0], shape[1] // 2) and s.shape == (shape[0], shape[1] // 32)
        assert Q.qgemm_mx_dequantize_device(q, s).shape == shape


@pytest.mark.parametrize("K,N", [(64, 1), (320, 33), (576, 100), (256, 64), (4096, 96)])
def test_packed_on_the_device_equals_the_host(K, N):
    rng = np.random.default_rng(K * N)
    W = rng.standard_normal((N, K)).astype(np.float32)
    q, s = Q.qgemm_mx_quantize(W)
    wp, sp = Q.qgemm_mx_pack(K, N, q, s)
    wb, sb = Q.qgemm_packed_size(K, N, "mxfp4")
    B = torch.full((wb,), 0xA5, dtype=torch.uint8, device="cuda")
    S = torch.full((sb,), 0xA5, dtype=torch.uint8, device="cuda")
    Q.qgemm_quantize_pack_device(dev(W), "mxfp4a4", B, S)
    assert np.array_equal(B.cpu().numpy(), wp) and np.array_equal(S.cpu().numpy(), sp)
    q3 = np.stack([q, q[::-1], q ^ 0x5A])
    s3 = np.stack([s, s[::-1], s ^ 3])
    B, S = Q.qgemm_mx_pack_device(K, N, dev(q3), dev(s3), E=3)
    for e in range(3):
        wp, sp = Q.qgemm_mx_pack(K, N, q3[e], s3[e])
        assert np.array_equal(B[e * wb:(e + 1) * wb].cpu().numpy(), wp)
        assert np.array_equal(S[e * sb:(e + 1) * sb].cpu().numpy(), sp)


# ---------------------------------------------------------------------------
# Dense products
# ---------------------------------------------------------------------------
def _case(fmt, M, K, N, seed):
    rng = np.random.default_rng(seed)
    A = _rows(rng, M, K).astype(np.float16)
    W = (rng.standard_normal((N, K)) * 0.02 * np.exp2(rng.integers(-3, 4, (N, 1)))).astype(np.float32)
    q, s = X.encode(W)
    a = X.decode(*X.encode(A)) if fmt == "mxfp4a4" else A.astype(np.float64)
    w = X.decode(q, s)
    return A, Q.PackedWeight(fmt, K, N, q, s), a @ w.T, np.abs(a) @ np.abs(w).T


SHAPES = [(1, 64, 1), (1, 64, 32), (1, 4096, 300), (2, 128, 33), (3, 2560, 1024), (5, 320, 70), (8, 4096, 257),
          (9, 192, 40), (16, 1024, 129), (17, 576, 96), (31, 256, 64), (32, 2560, 256), (33, 2560, 64),
          (64, 640, 200), (65, 4096, 128), (96, 1024, 300), (128, 512, 512), (129, 832, 130), (200, 2560, 1000),
          (256, 64, 256), (300, 1088, 520), (512, 1024, 2048), (1000, 640, 2300), (1, 16384, 96), (7, 9728, 640),
          (40, 9728, 96)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_product(fmt, M, K, N):
    A, w, ref, sumabs = _case(fmt, M, K, N, M * 7 + K + N)
    C = w(dev(A))
    X.check_product(C.cpu().numpy(), ref, sumabs, K, what=f"{fmt} {M}x{K}x{N}")
    # without GEMV kernels the same shape takes the tiled ones
    if M <= 8:
        prev = Q.qgemm_set_gemv_max_m(0)
        C = w(dev(A))
        Q.qgemm_set_gemv_max_m(prev)
        X.check_product(C.cpu().numpy(), ref, sumabs, K, what=f"{fmt} {M}x{K}x{N} tiled")


@pytest.mark.parametrize("M,K,N", [(1, 4096, 300), (6, 640, 129), (33, 1024, 256), (130, 2560, 200), (700, 512, 1100)])
@pytest.mark.parametrize("parts,kind,out", [("bias", "silu", "f32"), ("residual", "gelu", "f16"),
                                            ("bias+residual", "relu", "f16"), ("inplace", "none", "f32"),
                                            ("inplace", "none", "f16"), ("", "none", "f16")])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_epilogue(fmt, M, K, N, parts, kind, out):
    A, w, ref, sumabs = _case(fmt, M, K, N, M + K + N)
    rng = np.random.default_rng(M)
    bias = rng.standard_normal(N).astype(np.float32) if "bias" in parts else None
    res = rng.standard_normal((M, N)).astype(NP[out]) if "residual" in parts or parts == "inplace" else None
    pre = ref + (0 if bias is None else bias.astype(np.float64)) + (0 if res is None else res.astype(np.float64))
    sumabs = sumabs + (0 if bias is None else np.abs(bias)) + (0 if res is None else np.abs(res.astype(np.float64)))
    C = torch.full((M, N), float("nan"), dtype=torch.float16 if out == "f16" else torch.float32, device="cuda")
    if parts == "inplace":
        C.copy_(torch.from_numpy(res))
    Q.qgemm_run_ex(M, K, N, fmt, dev(A), w.Bq, w.scales, C, bias=None if bias is None else dev(bias),
                   residual=C if parts == "inplace" else None if res is None else dev(res), activation=kind,
                   out_type=out)
    X.check_product(C.cpu().numpy(), X.act(pre, kind), sumabs, K, out, f"{fmt} {M}x{K}x{N} {parts} {kind} {out}")


@pytest.mark.parametrize("M", [1, 8, 20, 200])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_nonfinite_stays_in_its_row_and_channel(fmt, M):
    """A NaN or infinite activation reaches its own row only, a NaN scale its own
    channel only; everything else is as it would be without them."""
    K, N = 320, 72
    rng = np.random.default_rng(M)
    A = _rows(rng, M, K).astype(np.float16)
    q, s = X.encode((rng.standard_normal((N, K)) * 0.02).astype(np.float32))
    s[5, 3] = 255
    A[0, 77] = np.inf if M % 2 else np.nan
    w = Q.PackedWeight(fmt, K, N, q, s)
    C = w(dev(A)).cpu().numpy()
    assert not np.isfinite(C[0]).any() or fmt == "mxfp4"      # a zero code times infinity is NaN, else infinite
    assert not np.isfinite(C[0]).all() and np.isnan(C[:, 5]).all()
    keep = np.arange(N) != 5
    a = X.decode(*X.encode(A)) if fmt == "mxfp4a4" else A.astype(np.float64)
    wd = X.decode(q, s)[keep]
    if M > 1:
        X.check_product(C[1:, keep], a[1:] @ wd.T, np.abs(a[1:]) @ np.abs(wd).T, K, what=f"{fmt} M={M}")


def test_zero_rows_and_extreme_scales():
    """Zero activations give +-0; scales far outside fp16 work with MXFP4
    activations, whose product never forms an fp16 weight."""
    K, N, M = 256, 48, 12
    rng = np.random.default_rng(2)
    A = _rows(rng, M, K).astype(np.float16)
    A[4:9] = 0
    for scale in (2.0 ** -70, 2.0 ** 60):
        q, s = X.encode((rng.standard_normal((N, K)) * scale).astype(np.float32))
        C = Q.PackedWeight("mxfp4a4", K, N, q, s)(dev(A)).cpu().numpy()
        a, w = X.decode(*X.encode(A)), X.decode(q, s)
        X.check_product(C / np.float32(scale), a @ w.T / scale, np.abs(a) @ np.abs(w).T / scale, K)
        assert (C[4:9] == 0).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_same_result_by_every_entry_point(fmt):
    """qgemm_run, _ws, _ex with a workspace and _noalloc, on another stream, and
    twice in a row: the same bits."""
    for M, K, N in ((1, 1024, 300), (48, 2560, 320), (300, 512, 520)):
        A, w, _, _ = _case(fmt, M, K, N, 9)
        Ad = dev(A)
        C = [torch.full((M, N), float("nan"), device="cuda") for _ in range(5)]
        nb = Q.qgemm_workspace_size(M, K, N, fmt)
        ws = torch.full((max(nb, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        Q.qgemm_run(M, K, N, fmt, Ad, w.Bq, w.scales, C[0])
        Q.qgemm_run_ws(M, K, N, fmt, Ad, w.Bq, w.scales, C[1], ws, nb)
        Q.qgemm_run_ex(M, K, N, fmt, Ad, w.Bq, w.scales, C[2], workspace=ws, ws_bytes=nb)
        Q.qgemm_run_noalloc(M, K, N, fmt, Ad, w.Bq, w.scales, C[3])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            Q.qgemm_run(M, K, N, fmt, Ad, w.Bq, w.scales, C[4])
        torch.cuda.synchronize()
        assert all(torch.equal(C[0], c) for c in C[1:])


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_captured_product(fmt):
    """A captured call (no allocation) replays with new inputs, eager calls of the
    same scratch between the replays."""
    M, K, N = 40, 1024, 320
    A, w, _, _ = _case(fmt, M, K, N, 11)
    Ad, C = dev(A), torch.empty((M, N), device="cuda")
    Q.qgemm_run_noalloc(M, K, N, fmt, Ad, w.Bq, w.scales, C)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Q.qgemm_run_noalloc(M, K, N, fmt, Ad, w.Bq, w.scales, C)
    for seed in range(4):
        Ad.copy_(torch.from_numpy(_rows(np.random.default_rng(seed), M, K).astype(np.float16)))
        g.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(C)
        Q.qgemm_run_noalloc(M, K, N, fmt, Ad, w.Bq, w.scales, want)
        torch.cuda.synchronize()
        assert torch.equal(C, want)


def test_untouched_past_the_end():
    """Nothing is written behind C."""
    for fmt in ("mxfp4", "mxfp4a4"):
        for M, K, N in ((3, 128, 70), (50, 128, 33), (130, 256, 257)):
            A, w, _, _ = _case(fmt, M, K, N, 4)
            buf = torch.full((M * N + 512,), 3.0, device="cuda")
            Q.qgemm_run(M, K, N, fmt, dev(A), w.Bq, w.scales, buf[:M * N].view(M, N))
            assert (buf[M * N:] == 3.0).all()


@pytest.mark.parametrize("M", [1, 40])
def test_weights_outside_fp16(M):
    """The product with fp16 activations takes the weights in fp16: rounded
    once where they are small, infinite where they are too large."""
    K, N = 128, 64
    rng = np.random.default_rng(M)
    W = rng.standard_normal((N, K)).astype(np.float32)
    W[:32] *= (2.0 ** -rng.integers(14, 30, (32, 1))).astype(np.float32)     # down to zeros
    W[32:] *= (2.0 ** rng.integers(10, 14, (32, 1))).astype(np.float32)
    W[50] = 2.0 ** 20
    q, s = X.encode(W)
    with np.errstate(over="ignore"):
        w16 = X.decode(q, s).astype(np.float16).astype(np.float64)
    assert np.isinf(w16[50]).all() and (w16[:32] == 0).any()
    A = np.abs(rng.standard_normal((M, K))).astype(np.float16) + np.float16(0.5)
    C = Q.PackedWeight("mxfp4", K, N, q, s)(dev(A)).cpu().numpy()
    fine = np.isfinite(w16).all(1)
    assert np.isposinf(C[:, ~fine][:, :1]).all() and np.isposinf(C[:, 50]).all()
    a = A.astype(np.float64)
    X.check_product(C[:, fine], a @ w16[fine].T, np.abs(a) @ np.abs(w16[fine]).T, K)


def test_pack_refuses_strided_codes():
    q = torch.zeros((32, 64), dtype=torch.uint8, device="cuda")
    s = torch.zeros((32, 4), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        Q.qgemm_mx_pack_device(64, 32, q[:, :32], s[:, :2].contiguous())
    with pytest.raises(ValueError):
        Q.qgemm_mx_pack_device(64, 32, q[:, :32].contiguous(), s[:, :2])


# (M, N) of every tile shape the dense dispatch knows, with a ragged last tile
# of rows and of columns
TILES = [(1000, 16300), (250, 16300), (40, 18500), (30, 9300), (20, 200)]


@pytest.mark.parametrize("K", [64, 192, 320, 448, 576, 832, 1088, 1344, 2112])
@pytest.mark.parametrize("M,N", TILES)
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_every_tile_with_stages_left_over(fmt, M, N, K):
    """K of whole turns of the main loop and of every number of stages more,
    fewer stages than K groups among them; references on the GPU in 64 bits,
    bounds as in check_product."""
    g = torch.Generator(device="cuda").manual_seed(M + K)
    A = torch.randn((M, K), device="cuda", generator=g).half()
    W = torch.randn((N, K), device="cuda", generator=g)
    q, s = Q.qgemm_mx_quantize_device(W)
    w = Q.qgemm_mx_dequantize_device(q, s).double()
    Bq, Sp = Q.qgemm_mx_pack_device(K, N, q, s)
    C = torch.full((M, N), float("nan"), device="cuda")
    Q.qgemm_run_ex(M, K, N, fmt, A, Bq, Sp, C)
    a = Q.qgemm_mx_dequantize_device(*Q.qgemm_mx_quantize_device(A)).double() if fmt == "mxfp4a4" else A.double()
    ref, mass = a @ w.t(), a.abs() @ w.abs().t()
    err = (C.double() - ref).abs()
    assert bool((err <= (K + 16) * 2.0 ** -23 * mass + 1e-37).all())
    assert float(err.norm()) <= 4 * (K + 16) ** 0.5 * 2.0 ** -24 * float(mass.norm())


@pytest.mark.parametrize("M,K,N", [(1, 512, 33), (6, 576, 64), (20, 832, 130), (40, 1024, 18500), (300, 640, 257)])
@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_residual_in_place(fmt, M, K, N, out):
    """The residual may be C itself: the same bits as from a copy of it, dense
    and as one group of a grouped product."""
    g = torch.Generator(device="cuda").manual_seed(M)
    A = torch.randn((M, K), device="cuda", generator=g).half()
    Bq, Sp = Q.qgemm_mx_pack_device(K, N, *Q.qgemm_mx_quantize_device(torch.randn((N, K), device="cuda", generator=g)))
    R = torch.randn((M, N), device="cuda", generator=g).to(torch.float16 if out == "f16" else torch.float32)
    want, C = torch.empty_like(R), R.clone()
    Q.qgemm_run_ex(M, K, N, fmt, A, Bq, Sp, want, residual=R, activation="silu", out_type=out)
    Q.qgemm_run_ex(M, K, N, fmt, A, Bq, Sp, C, residual=C, activation="silu", out_type=out)
    assert torch.equal(C, want)
    offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    want, C = torch.empty_like(R), R.clone()
    Q.qgemm_run_grouped(K, N, 1, fmt, A, None, offsets, Bq, Sp, want, residual=R, activation="silu", out_type=out)
    Q.qgemm_run_grouped(K, N, 1, fmt, A, None, offsets, Bq, Sp, C, residual=C, activation="silu", out_type=out)
    assert torch.equal(C, want)


@pytest.mark.parametrize("M,K,N", [(12, 6144, 100), (33, 9728, 2560), (100, 8192, 1001), (250, 9728, 2560),
                                   (500, 9728, 2560), (17, 16384, 1024), (200, 16448, 640)])
def test_split_k(M, K, N):
    """Few tiles and a long K: K in slices, added in their order (the same bits
    every time), with every epilogue, through each entry point and its own
    scratch. (500 rows make enough tiles to stay whole: the same checks.)"""
    assert Q.qgemm_workspace_size(M, K, N, "mxfp4") >= (2 * M * N * 4 if M < 500 else 0)
    g = torch.Generator(device="cuda").manual_seed(M + N)
    A = torch.randn((M, K), device="cuda", generator=g).half()
    q, s = Q.qgemm_mx_quantize_device(torch.randn((N, K), device="cuda", generator=g))
    Bq, Sp = Q.qgemm_mx_pack_device(K, N, q, s)
    w = Q.qgemm_mx_dequantize_device(q, s).double()
    bias = torch.randn(N, device="cuda", generator=g)
    res = torch.randn((M, N), device="cuda", generator=g).half()
    ref, mass = A.double() @ w.t(), A.double().abs() @ w.abs().t()
    bound = (K + 16) * 2.0 ** -23 * mass + 1e-37
    C = torch.full((M, N), float("nan"), device="cuda")
    Q.qgemm_run(M, K, N, "mxfp4", A, Bq, Sp, C)
    assert bool(((C.double() - ref).abs() <= bound).all())
    assert float((C.double() - ref).norm()) <= 4 * (K + 16) ** 0.5 * 2.0 ** -24 * float(mass.norm())
    nb = Q.qgemm_workspace_size(M, K, N, "mxfp4")
    ws = torch.full((max(nb, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        D = torch.full((M, N), float("nan"), device="cuda")
        Q.qgemm_run_ws(M, K, N, "mxfp4", A, Bq, Sp, D, ws, nb)
        assert torch.equal(C, D)
    if nb <= Q.NOALLOC_SCRATCH_BYTES:
        D = torch.full((M, N), float("nan"), device="cuda")
        Q.qgemm_run_noalloc(M, K, N, "mxfp4", A, Bq, Sp, D)
        assert torch.equal(C, D)
    # relu has slope 1; an fp16 result rounds by half a step
    H = res.clone()
    Q.qgemm_run_ex(M, K, N, "mxfp4", A, Bq, Sp, H, bias=bias, residual=H, activation="relu", out_type="f16",
                   workspace=ws, ws_bytes=nb)
    full = (ref + bias.double() + res.double()).clamp(min=0)
    err = (H.double() - full).abs()
    assert bool((err <= bound + (K + 16) * 2.0 ** -23 * (bias.abs().double() + res.abs().double())
                 + 2.0 ** -11 * full + 2.0 ** -25).all())


# pre-activations at SiLU's corners: either side of where its exponential or
# its reciprocal leave fp32's normal numbers, far beyond, and not numbers at all
SILU_AT = np.array([-np.inf, -3.4e38, -1e30, -1e6, -300, -104, -100, -90, -88.8, -88.6, -87.5, -87.2, -80, -20, -1, -1e-3,
                    -1e-38, -0.0, 0.0, 1e-38, 1e-3, 0.5, 3, 20, 80, 88, 90, 104, 300, 1e6, 1e30, 3.4e38, np.inf, np.nan],
                   np.float32)


@pytest.mark.parametrize("M,K,N", [(1, 64, 300), (7, 512, 68), (20, 128, 257), (40, 1024, 320), (300, 512, 520),
                                   (12, 6144, 100), (200, 16448, 640)])
@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_silu_over_the_whole_range(fmt, M, K, N, out):
    """x / (1 + e^-x) for every x, by the decode, tile, split-K and grouped
    kernels (zero activations, so that the bias is x). An error of at most 4
    units: one each of the hardware's exponential and reciprocal, half each of
    three roundings, and the exponent's own; with an fp16 result |x| 2^-24 more
    (the exponent rounded once) and its own half step. Results of less than
    1.2e-36 may be zero. -infinity and NaN give NaN as the formula does."""
    x = np.resize(SILU_AT, N)
    g = torch.Generator(device="cuda").manual_seed(N)
    A = torch.zeros((M, K), dtype=torch.float16, device="cuda")
    Bq, Sp = Q.qgemm_mx_pack_device(K, N, *Q.qgemm_mx_quantize_device(
        torch.randn((N, K), device="cuda", generator=g)))
    dt = torch.float16 if out == "f16" else torch.float32
    C, D = torch.full((M, N), 7.0, dtype=dt, device="cuda"), torch.full((M, N), 7.0, dtype=dt, device="cuda")
    Q.qgemm_run_ex(M, K, N, fmt, A, Bq, Sp, C, bias=dev(x), activation="silu", out_type=out)
    Q.qgemm_run_grouped(K, N, 1, fmt, A, None, torch.tensor([0, M], dtype=torch.int32, device="cuda"), Bq, Sp, D,
                        bias=dev(x[None]), activation="silu", out_type=out)
    with np.errstate(over="ignore", invalid="ignore"):
        ref = x.astype(np.float64) / (1.0 + np.exp(-x.astype(np.float64)))
        ref = np.where(np.isneginf(x), np.nan, ref)
        want = ref.astype(np.float16 if out == "f16" else np.float32)
    num = np.isfinite(want)
    tol = 4 * 2.0 ** -23 * np.abs(ref[num]) + 1.2e-36
    if out == "f16":
        tol = tol + np.minimum(np.abs(x[num].astype(np.float64)), 128) * 2.0 ** -23 * np.abs(ref[num]) \
            + 2.0 ** -11 * np.abs(ref[num]) + 2.0 ** -25
    for got in (C.cpu().numpy(), D.cpu().numpy()):
        assert (np.isnan(got) == np.isnan(want)).all(), x[(np.isnan(got) != np.isnan(want)).any(0)]
        inf = np.isinf(want)
        assert (got[:, inf] == want[inf]).all(), x[inf]
        err = np.abs(got[:, num].astype(np.float64) - ref[num])
        assert (err <= tol).all(), (x[num][(err > tol).any(0)], got[:, num][0][(err > tol).any(0)])


# (M, N) that reach 32 x 128, 64 x 128, 64 x 256 and 128 x 256 tiles with fp16
# activations whatever K, and K of one, two, three and no stages more than whole
# turns of four, of 64 elements (fp16 activations) and of 256
# (tests/test_mx_tiles.py checks both)
MIDDLE = [(200, 4100), (500, 3620), (250, 16300), (1000, 16300)]
MIDDLE_K = [64, 128, 192, 256, 448, 640, 832, 1088, 1280]


@pytest.mark.parametrize("K", MIDDLE_K)
@pytest.mark.parametrize("M,N", MIDDLE)
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp4a4"])
def test_middle_tiles_with_stages_left_over(fmt, M, N, K):
    test_every_tile_with_stages_left_over(fmt, M, N, K)
