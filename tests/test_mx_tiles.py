"""Which tiles of the MXFP4 products the GPU tests reach (CPU): the rules of
csrc/host_pack.cpp, compiled here, answer for the tests' own shapes and for a
wide net of others. Every tile that any shape of the net takes has to be in a
test that compares it with 64 bits, so a changed rule cannot leave one out."""
import os
import shutil
import subprocess

import pytest

import test_gpu_group as G
import test_gpu_mx as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TILES = ["128x256", "64x256", "64x128", "32x256", "32x128", "32x64", "32x32"]


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("plan") / "plan")
    csrc = os.path.join(ROOT, "weight_quantized_gemm_amd", "csrc")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-D__HIP_PLATFORM_AMD__", "-I",
                        os.path.join(ROOT, "include"), "-I", csrc, "-I", "/opt/rocm/include",
                        os.path.join(ROOT, "tests", "mx_plan_driver.cpp"), os.path.join(csrc, "host_pack.cpp"),
                        "-o", exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]

    def answers(questions):
        """(tile, slices of K) of every question; tile None: the kernel for few rows."""
        text = "\n".join(" ".join(map(str, q)) for q in questions)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=300, check=True).stdout
        rows = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(rows) == len(questions)
        return [(TILES[t] if t >= 0 else None, n) for t, n in rows]

    return answers


def _values(test, names):
    """What a test is parametrised with for these names."""
    return next(m.args[1] for m in test.pytestmark if m.name == "parametrize" and m.args[0] == names)


def _kinds(ask, questions):
    return {(q[0], q[1], tile, slices > 1) for q, (tile, slices) in zip(questions, ask(questions))}


def _dense(a4, test):
    return [("d", a4, m, k, n) for m, n in _values(test, "M,N") for k in _values(test, "K")]


def test_every_tile_that_a_rule_can_choose_is_tested(ask):
    some = lambda base, top: sorted({int(base ** i) for i in range(80) if base ** i < top})
    rows, cols = some(1.35, 1 << 20), some(1.3, 1 << 20)
    net = [("d", a4, m, k, n) for a4 in (0, 1) for m in rows for k in (64, 448, 1024, 2560, 4096, 9728, 16384, 65536)
           for n in cols]
    net += [("g", a4, s, e, n) for a4 in (0, 1) for s in rows for e in (1, 2, 5, 8, 16, 32, 64, 128, 256, 1024)
            for n in cols]
    tested = []
    for a4 in (0, 1):
        tested += _dense(a4, M.test_every_tile_with_stages_left_over) + _dense(a4, M.test_middle_tiles_with_stages_left_over)
        tested += [("d", a4, m, k, n) for m, k, n in _values(M.test_split_k, "M,K,N") if not a4]
        for test, shapes in ((G.test_every_tile_of_the_grouped_product,
                              [(mean, 12, 4100) for mean in _values(G.test_every_tile_of_the_grouped_product, "mean")]),
                             (G.test_middle_tiles_of_the_grouped_product, G.MIDDLE)):
            tested += [("g", a4, int(G.middle_sizes(mean, E, K).sum()) + 7, E, N) for mean, E, N in shapes
                       for K in _values(test, "K")]
        # an expert with one or a few rows, in test_grouped_product
        tested += [("g", a4, sum(sizes) + 5, len(sizes), 300) for sizes in G.RAGGED]
    missing = _kinds(ask, net) - _kinds(ask, tested)
    assert not missing, sorted(missing, key=str)


def test_middle_shapes_reach_the_tiles_they_name(ask):
    """Each with every K, so with every number of stages left over."""
    def grouped(a4, shape):
        mean, E, N = shape
        return {t for t, _ in ask([("g", a4, int(G.middle_sizes(mean, E, K).sum()) + 7, E, N) for K in G.MIDDLE_K])}

    for a4 in (0, 1):
        for shape, tile in ((G.MIDDLE[0], "32x256"), (G.MIDDLE[1], "32x256"), (G.MIDDLE[3], "32x256"),
                            (G.MIDDLE[4], "64x128"), (G.MIDDLE[5], "32x64"), (G.MIDDLE[6], "32x32"),
                            (G.MIDDLE[7], "64x256")):
            assert grouped(a4, shape) == {tile}, (a4, shape)
    assert grouped(1, G.MIDDLE[2]) == {"32x256"}
    for (m, n), tile in zip(M.MIDDLE, ("32x128", "64x128", "64x256", "128x256")):
        assert set(ask([("d", 0, m, k, n) for k in M.MIDDLE_K])) == {(tile, 1)}
    for ks in (M.MIDDLE_K, G.MIDDLE_K):
        for step in (64, 256):
            assert {-(-k // step) % 4 for k in ks} == {0, 1, 2, 3}


def test_slices_of_the_split_shapes(ask):
    """The dense product's slices of K where C is small and K long, and two shapes
    that stay whole."""
    want = {(12, 6144, 100): ("32x32", 6), (33, 9728, 2560): ("32x64", 3), (100, 8192, 1001): ("32x64", 4),
            (250, 9728, 2560): ("64x128", 3), (500, 9728, 2560): ("64x256", 3), (17, 16384, 1024): ("32x32", 8),
            (200, 16448, 640): ("32x128", 7), (512, 4096, 4096): ("64x128", 1), (2000, 9728, 2560): ("64x256", 1)}
    assert dict(zip(want, ask([("d", 0, *s) for s in want]))) == want
