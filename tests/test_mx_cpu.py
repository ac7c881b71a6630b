"""MXFP4 and mixture-of-experts entry points without a GPU: the host quantiser
and packer against the 64-bit rules, sizes, and every refusal (a refused call
answers before it looks for a device)."""
import ctypes

import numpy as np
import pytest

import mx_reference as X
from weight_quantized_gemm_amd import qgemm as Q

OK, NULL, SHAPE, FMT, ALIGN, DEV, SIZE, VALUE = 0, 1, 2, 3, 4, 6, 8, 9
P = ctypes.c_void_p
A, B = P(1 << 20), P(1 << 21)          # aligned stand-ins, never followed
ODD = P((1 << 20) + 8)


def special_rows():
    """Blocks at the rule's corners: ties, saturation, signed zeros, the ends of
    the exponent range, subnormal numbers."""
    ties = np.array([0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.24999, 0.25001, 0.7499, 1.2501, 1.7499, 2.5001,
                     3.4999, 5.0001], np.float32)
    rows = []
    for e in (-126, -125, -124, -30, -3, 0, 4, 60, 120, 125):
        b = np.concatenate([ties, -ties]).astype(np.float64) * 2.0 ** e
        b[0] = 4.0 * 2.0 ** e
        rows.append(b)
        b = b.copy()
        b[0] = 7.99 * 2.0 ** e if e < 125 else 7.0 * 2.0 ** e
        rows.append(b)
    rows.append(np.zeros(32))
    rows.append(np.where(np.arange(32) % 2, -0.0, 0.0))
    rows.append(np.full(32, 2.0 ** -149))
    rows.append(np.linspace(-2.0 ** -127, 2.0 ** -127, 32))
    rows.append(np.full(32, np.float32(3.4028235e38)))
    rows.append(np.ldexp(1.0, np.arange(-16, 16)))
    return np.stack(rows).astype(np.float32)


def test_host_quantiser_follows_the_rule():
    rng = np.random.default_rng(5)
    for x in (special_rows(), rng.standard_normal((7, 320)).astype(np.float32),
              (rng.standard_normal((3, 64)) * 10.0 ** rng.uniform(-37, 37, (3, 64))).astype(np.float32)):
        q, s = Q.qgemm_mx_quantize(x)
        qr, sr = X.encode(x)
        assert np.array_equal(s, sr) and np.array_equal(q, qr)


def test_host_quantiser_error_is_within_the_format():
    """Half a step of the element's own binade, or the loss of saturation (2 x
    scale: 8 -> 6)."""
    x = np.random.default_rng(6).standard_normal((64, 256)).astype(np.float32)
    q, s = Q.qgemm_mx_quantize(x)
    scale = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)
    y = np.abs(x) / scale
    step = np.where(y < 2, 0.5, np.where(y < 4, 1.0, 2.0))
    assert (np.abs(X.decode(q, s) - x) <= np.where(y > 6, y - 6, step / 2) * scale).all()


def test_host_quantiser_refusals():
    for bad in (np.nan, np.inf, -np.inf):
        x = np.ones((2, 64), np.float32)
        x[1, 40] = bad
        with pytest.raises(Q.QGemmError) as e:
            Q.qgemm_mx_quantize(x)
        assert e.value.status == VALUE
    lib = Q.load()
    assert lib.qgemm_mx_quantize(1, 33, A, A, A) == SHAPE
    assert lib.qgemm_mx_quantize(-1, 32, A, A, A) == SHAPE
    assert lib.qgemm_mx_quantize(1, 32, None, A, A) == NULL
    assert lib.qgemm_mx_quantize(0, 32, None, None, None) == OK


@pytest.mark.parametrize("K,N", [(64, 1), (64, 33), (320, 70), (256, 32), (576, 64)])
def test_packed_layout(K, N):
    """Piece 32 h + c of record (t, b) holds the 32 codes of channel 32 t + c from
    64 b + 32 h on; the scale of that block is byte b % 4 of word 32 h + c of
    scale record (t, b / 4); everything else is zero."""
    rng = np.random.default_rng(K + N)
    q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    s = rng.integers(0, 256, (N, K // 32), dtype=np.uint8)
    wp, sp = Q.qgemm_mx_pack(K, N, q, s)
    tiles, n64, n256 = -(-N // 32), K // 64, -(-K // 256)
    assert wp.size == tiles * n64 * 1024 and sp.size == tiles * n256 * 256
    assert (wp.size, sp.size) == Q.qgemm_packed_size(K, N, "mxfp4") == Q.qgemm_packed_size(K, N, "mxfp4a4")
    qp = np.zeros((tiles * 32, K // 2), np.uint8)
    qp[:N] = q
    spd = np.zeros((tiles * 32, n256 * 8), np.uint8)
    spd[:N, :K // 32] = s
    assert np.array_equal(wp.reshape(tiles, n64, 2, 32, 16),
                          qp.reshape(tiles, 32, n64, 2, 16).transpose(0, 2, 3, 1, 4))
    assert np.array_equal(sp.reshape(tiles, n256, 2, 32, 4),
                          spd.reshape(tiles, 32, n256, 4, 2).transpose(0, 2, 4, 1, 3))


def test_pack_refusals():
    lib = Q.load()
    n = ctypes.c_size_t
    assert lib.qgemm_mx_pack(96, 8, A, A, A, n(1 << 20), A, n(1 << 20)) == SHAPE
    assert lib.qgemm_mx_pack(64, 8, A, None, A, n(1 << 20), A, n(1 << 20)) == NULL
    assert lib.qgemm_mx_pack(64, 8, A, A, A, n(1023), A, n(1 << 20)) == SIZE
    assert lib.qgemm_mx_pack(64, 0, None, None, None, n(0), None, n(0)) == OK
    with pytest.raises(ValueError):
        Q.qgemm_mx_pack(64, 8, np.zeros(10, np.uint8), np.zeros(16, np.uint8))
    f = lib.qgemm_mx_pack_device
    assert f(96, 8, 1, A, A, A, A, None) == SHAPE
    assert f(64, 8, 1025, A, A, A, A, None) == SHAPE
    assert f(64, 8, 2, A, None, A, A, None) == NULL
    assert f(64, 8, 2, A, ODD, A, A, None) == ALIGN
    assert f(64, 8, 0, None, None, None, None, None) == OK


@pytest.mark.parametrize("f", [6, 8])
def test_pair_functions_refuse_scale_byte_formats(f):
    lib = Q.load()
    n = ctypes.c_size_t
    z = ctypes.byref(ctypes.c_size_t())
    assert lib.qgemm_canonical_size(64, 8, f, z, z) == FMT
    assert lib.qgemm_quantize_weights(64, 8, f, A, A, n(1 << 20), A, n(1 << 20)) == FMT
    assert lib.qgemm_pack_weights(64, 8, f, A, A, A, n(1 << 20), A, n(1 << 20)) == FMT
    assert lib.qgemm_unpack_weights(64, 8, f, A, n(1 << 20), A, n(1 << 20), A, A) == FMT
    assert lib.qgemm_quantize_weights_device(64, 8, f, A, A, A, None) == FMT
    assert lib.qgemm_quantize_pack_device(96, 8, f, A, A, A, None) == SHAPE
    assert lib.qgemm_quantize_pack_device(64, 8, f, A, A, None, None) == NULL


@pytest.mark.parametrize("f", [6, 8])
def test_run_refusals(f):
    run = lambda M, K, N, a=A, b=A, s=A, c=A: Q.load().qgemm_run(M, K, N, f, a, b, s, c, None)
    assert run(1, 0, 8) == SHAPE
    assert run(1, 32, 8) == SHAPE and run(1, 96, 8) == SHAPE
    assert run(-1, 64, 8) == SHAPE
    assert run(1 << 24, 64, 1 << 24) == SHAPE        # more tiles than a launch can have
    assert run(0, 64, 8, None, None, None, None) == OK
    assert run(1, 64, 8, s=None) == NULL and run(1, 64, 8, a=None) == NULL
    assert run(1, 64, 8, a=ODD) == ALIGN and run(1, 64, 8, s=ODD) == ALIGN
    assert run(1, 64, 8) == DEV


def test_activation_scratch_is_reported():
    """MXFP4_A4 needs the codes (K rounded up to 256, half a byte each) and the
    scales of every row, and refuses a workspace that is too small."""
    assert Q.qgemm_workspace_size(5, 320, 64, "mxfp4a4") >= 5 * (512 // 2 + 512 // 32)
    need = Q.qgemm_workspace_size(64, 320, 64, "mxfp4a4")
    run = lambda ws, n: Q.load().qgemm_run_ws(64, 320, 64, 8, A, A, A, A, ws, ctypes.c_size_t(n), None)
    assert run(None, 0) == NULL and run(B, 15) == SIZE and run(ODD, need) == ALIGN and run(B, need) == DEV
    assert Q.qgemm_grouped_workspace_size(40, 64, 320, 64, 4, "mxfp4") == 0
    assert Q.qgemm_grouped_workspace_size(400, 64, 320, 64, 4, "mxfp4a4") >= 64 * (512 // 2 + 512 // 32)


@pytest.mark.parametrize("K", [64, 256, 320, 1024, 2560, 4096, 9728])
def test_activation_scratch_covers_the_widest_read(K):
    """The kernels fetch the scales of four 256-element groups at once, starting
    at any group of a row, so even the last row needs room for three more than
    it has (2560 elements: 13 groups of 8 bytes a row)."""
    groups = -(-K // 256)
    for M in (1, 9, 64, 200, 2048):
        codes = M * groups * 128
        assert Q.qgemm_workspace_size(M, K, 64, "mxfp4a4") >= codes + M * (groups + 3) * 8


def test_row_conversion_refusals():
    lib = Q.load()
    quant = lambda R=2, K=64, t=0, x=A, ld=64, q=A, s=A: lib.qgemm_mx_quantize_device(R, K, t, x, ld, q, s, None)
    deq = lambda R=2, K=64, t=0, x=A, ld=64, q=A, s=A: lib.qgemm_mx_dequantize_device(R, K, q, s, t, x, ld, None)
    for f in (quant, deq):
        assert f() == DEV
        assert f(t=3) == FMT and f(t=-1) == FMT
        assert f(K=48) == SHAPE and f(R=-1) == SHAPE and f(ld=32) == SHAPE and f(R=(1 << 24) + 1) == SHAPE
        assert f(x=None) == NULL and f(q=None) == NULL and f(s=None) == NULL
        assert f(x=ODD) == ALIGN and f(s=ODD) == ALIGN
        assert f(ld=66) == ALIGN and f(ld=66, R=1) == DEV       # rows must start aligned
        assert f(t=1, ld=68) == ALIGN and f(t=0, ld=68) == DEV
        assert f(R=0, x=None) == OK and f(K=0, ld=0) == OK


def test_plan_refusals():
    lib = Q.load()
    n = ctypes.c_size_t
    size = lambda T, k, E: lib.qgemm_group_plan_size(T, k, E, ctypes.byref(ctypes.c_size_t()))
    assert size(4, 2, 0) == SHAPE and size(4, 2, 1025) == SHAPE and size(-1, 2, 8) == SHAPE
    assert size(1 << 24, 8, 8) == SHAPE and size(1 << 23, 8, 8) == OK
    assert lib.qgemm_group_plan_size(4, 2, 8, None) == NULL
    f = lambda ids=A, off=A, rows=A, slots=A, ws=None, nb=0, T=4, k=2, E=8: \
        lib.qgemm_group_plan(T, k, E, ids, 1, off, rows, slots, ws, n(nb), None)
    assert f() == DEV
    assert f(E=0) == SHAPE and f(off=None) == NULL and f(ids=None) == NULL and f(slots=None) == NULL
    assert f(off=ODD) == ALIGN and f(ids=ODD) == ALIGN
    need = Q.qgemm_group_plan_size(1 << 16, 8, 8)
    assert need > 0
    assert f(T=1 << 16, k=8, ws=B, nb=need - 1) == SIZE and f(T=1 << 16, k=8, ws=ODD, nb=need) == ALIGN
    assert f(T=1 << 16, k=8, ws=None, nb=need) == NULL and f(T=1 << 16, k=8, ws=B, nb=need) == DEV
    assert f(T=0, ids=None, rows=None, slots=None) == DEV       # the offsets still have to be written


def test_grouped_refusals():
    lib = Q.load()
    n = ctypes.c_size_t
    f = lambda S=8, ar=4, K=64, N=32, E=2, fmt=6, a=A, rows=A, off=A, b=A, s=A, c=A, epi=None, ws=None, nb=0: \
        lib.qgemm_run_grouped(S, ar, K, N, E, fmt, a, rows, off, b, s, c, epi, ws, n(nb), None)
    assert f() == DEV and f(fmt=8) == DEV
    for fmt in (0, 1, 2, 3, 4, 5, 7, 9, 0x10040):
        assert f(fmt=fmt) == FMT
    assert f(K=32) == SHAPE and f(E=0) == SHAPE and f(E=1025) == SHAPE and f(S=-1) == SHAPE and f(ar=-1) == SHAPE
    assert f(S=(1 << 26) + 1) == SHAPE
    assert f(rows=None) == SHAPE and f(rows=None, ar=8) == DEV      # 8 slots cannot read 4 rows one by one
    assert f(a=None) == NULL and f(off=None) == NULL and f(b=None) == NULL and f(s=None) == NULL and f(c=None) == NULL
    assert f(a=ODD) == ALIGN and f(rows=ODD) == ALIGN and f(off=ODD) == ALIGN and f(c=ODD) == ALIGN
    assert f(S=0, a=None, c=None) == OK and f(N=0) == OK and f(ar=0, a=None) == OK
    need = Q.qgemm_grouped_workspace_size(800, 4, 64, 32, 2, "mxfp4a4")
    assert f(S=800, fmt=8, ws=B, nb=need - 1) == SIZE and f(S=800, fmt=8, ws=ODD, nb=need) == ALIGN
    bad = Q.Epilogue(None, None, 9, 0)
    assert f(epi=ctypes.byref(bad)) == FMT
    bad = Q.Epilogue((1 << 20) + 4, None, 0, 0)
    assert f(epi=ctypes.byref(bad)) == ALIGN


def test_combine_refusals():
    lib = Q.load()
    f = lambda T=4, k=2, N=32, S=8, y=A, yt=0, sl=A, w=A, c=A, ct=1: \
        lib.qgemm_group_combine(T, k, N, S, y, yt, sl, w, c, ct, None)
    assert f() == DEV and f(k=0, sl=None, w=None, y=None) == DEV and f(S=0, y=None) == DEV
    assert f(yt=2) == FMT and f(ct=2) == FMT
    assert f(T=-1) == SHAPE and f(N=-1) == SHAPE and f(S=-1) == SHAPE and f(T=1 << 26, N=1 << 20) == SHAPE
    assert f(y=None) == NULL and f(sl=None) == NULL and f(w=None) == NULL and f(c=None) == NULL
    assert f(y=ODD) == ALIGN and f(c=ODD) == ALIGN
    assert f(T=0, c=None) == OK and f(N=0, c=None) == OK


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros((2, 64))
    i = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        Q.qgemm_mx_quantize_device(x)
    with pytest.raises(ValueError):
        Q.qgemm_group_plan(i, 4)
    with pytest.raises(ValueError):
        Q.qgemm_group_combine(x, i, x[:, :2].contiguous(), x)
    with pytest.raises(ValueError):
        Q.qgemm_run_grouped(64, 32, 2, "mxfp4", x.half(), None, i, i, i, x)


def test_split_k_scratch():
    """Few tiles and a long K take partial tiles (fp32, whole slices); enough
    tiles, a short K, and MXFP4 activations do not."""
    for M, K, N in ((32, 9728, 2560), (256, 9728, 2560), (17, 16384, 1024), (12, 6144, 100)):
        need = Q.qgemm_workspace_size(M, K, N, "mxfp4")
        part = M * N * 4
        assert 2 * part <= need < 8 * part + 256
        codes = M * (-(-K // 256)) * 128
        assert codes <= Q.qgemm_workspace_size(M, K, N, "mxfp4a4") < codes + M * (K // 256 + 8) * 8 + 512
    for M, K, N in ((64, 4096, 4096), (32, 1024, 64), (2048, 9728, 2560), (512, 4096, 4096), (1, 64, 1)):
        assert Q.qgemm_workspace_size(M, K, N, "mxfp4") == 0


@pytest.mark.parametrize("call", ["plan", "grouped"])
def test_scratch_lives_until_the_call_returns(call, monkeypatch):
    """Scratch that the binding takes itself is held while the library enqueues
    its launches: freed before, another thread's call on the same stream gets
    the same memory between two of them."""
    import weakref

    import torch
    made, seen = [], []
    empty = torch.empty

    def spy(*a, **kw):
        t = empty(*a, **kw)
        made.append((weakref.ref(t), t.data_ptr(), t.numel() * t.element_size()))
        return t

    def enqueue(name, dev, stream, *args):
        ws, n = args[-2:]
        seen.append(name)
        assert any(ref() is not None and p == ws and b >= n > 0 for ref, p, b in made), "scratch was given back"

    monkeypatch.setattr(torch, "empty", spy)
    monkeypatch.setattr(Q, "_same_device", lambda **t: torch.device("cpu"))
    monkeypatch.setattr(Q, "_call", enqueue)
    if call == "plan":
        Q.qgemm_group_plan(torch.zeros((4096, 2), dtype=torch.int32), 8)
    else:
        monkeypatch.setattr(Q, "_dev_ptr", lambda t: None if t is None else t.data_ptr())
        K, N, E, S = 64, 32, 2, 800
        wb, sb = Q.qgemm_packed_size(K, N, "mxfp4a4")
        Q.qgemm_run_grouped(K, N, E, "mxfp4a4", torch.zeros((S, K), dtype=torch.float16), None,
                            torch.zeros(E + 1, dtype=torch.int32), torch.zeros(E * wb, dtype=torch.uint8),
                            torch.zeros(E * sb, dtype=torch.uint8), torch.zeros((S, N)))
    assert len(seen) == 1


def test_a_launch_that_cannot_exist_is_refused_before_anything_is_enqueued():
    """A launch has fewer than 2^32 threads along an axis. 1024 experts of one row
    each: 2^20 columns make 2^13 x 2^10 tiles of 512 threads with fp16
    activations, 2^22 columns 2^14 x 2^10 tiles of 256 with MXFP4 ones."""
    lib = Q.load()
    n = ctypes.c_size_t

    def both(S, K, N, E, fmt):
        size = lib.qgemm_grouped_workspace_size(S, S, K, N, E, fmt, ctypes.byref(ctypes.c_size_t()))
        return size, lib.qgemm_run_grouped(S, S, K, N, E, fmt, A, None, A, A, A, A, None, None, n(0), None)

    assert both(1024, 64, 1 << 20, 1024, 6) == (SHAPE, SHAPE)
    assert both(1024, 64, (1 << 20) - 128, 1024, 6) == (OK, DEV)
    assert both(1024, 64, 1 << 22, 1024, 8) == (SHAPE, SHAPE)
    assert both(1024, 64, (1 << 22) - 256, 1024, 8) == (OK, DEV)
    assert both(1 << 26, 64, 1 << 24, 1024, 8) == (SHAPE, SHAPE)
    # ordinary large calls are not
    for fmt in (6, 8):
        assert both(1 << 20, 4096, 16384, 256, fmt) == (OK, DEV)
        run = lambda M, K, N: lib.qgemm_run(M, K, N, fmt, A, A, A, A, None)
        assert run(1 << 18, 4096, 1 << 17) == DEV and run(8, 64, 1 << 24) == DEV and run(40, 64, 1 << 24) == DEV
        assert run(1 << 24, 64, 1 << 24) == SHAPE
