"""What the expert layer's and the norm's entry points launch, on the CPU: the host code of the kernels'
files and of the entry points, linked with a HIP runtime that only records launches (tests/host_launch/)."""
import os
import subprocess

import pytest

import tiled_dense_gemm_04_amd as tg
from tiled_dense_gemm_04_amd import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "host_launch")
CSRC = os.path.join(ROOT, "tiled_dense_gemm_04_amd", "csrc")
P = 256  # stands for an aligned device pointer; never dereferenced


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    try:
        hipcc = libbuild.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    out = str(tmp_path_factory.mktemp("host_launch"))
    include = ["-I" + os.path.join(ROOT, "include"), "-I" + CSRC]
    kernels = [os.path.join(out, name + ".o") for name in ("tgemm_expert", "tgemm_norm")]
    for cmd in (*([hipcc, "--offload-arch=" + libbuild.ARCH, "--offload-host-only", "-std=c++17", "-O1", *include, "-c",
                   os.path.join(CSRC, os.path.basename(o)[:-1] + "hip"), "-o", o] for o in kernels),
                ["/opt/rocm/llvm/bin/clang++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", *include,
                 os.path.join(CSRC, "tgemm_expert_api.cpp"), os.path.join(CSRC, "tgemm_norm_api.cpp"),
                 os.path.join(HERE, "driver.cpp"), *kernels,
                 "-Wl,--unresolved-symbols=ignore-all",  # (the device code's image, whose name is the compiler's)
                 "-o", os.path.join(out, "driver")]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-4000:]

    def call(*args):
        r = subprocess.run([os.path.join(out, "driver"), *map(str, args)], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr[-2000:]
        *launches, rc = r.stdout.split("\n")[:-1]
        return int(rc.split()[1]), [(name, int(groups), int(main)) for name, groups, main in map(str.split, launches)]

    return call


def test_gather_without_choices_reads_no_row(driver):
    """Tokens of no slots: only the workgroups that zero rows run, so x and place, which may then be null,
    are not read."""
    for tokens, H in ((5, 64), (1, 1), (4096, 4096)):
        rc, launches = driver("gather", tokens, 0, 20, H, 0, 0, P, P, 8)
        assert rc == tg.TGEMM_OK and len(launches) == 1
        name, groups, main = launches[0]
        assert "expert_gather" in name and main == 0 and groups > 0
        assert driver("gather", tokens, 0, 20, H, 0, 0, P, 0, 0) == (tg.TGEMM_OK, [])  # nothing to write
    # with slots: a workgroup for 256 chunks of eight values, and those that zero rows
    rc, launches = driver("gather", 5, 2, 10, 4096, P, P, P, P, 8)
    zeroing = groups
    assert rc == tg.TGEMM_OK and launches[0][1:] == (10 + zeroing, 10)
    rc, launches = driver("gather", 5, 2, 10, 4096, P, P, P, 0, 0)
    assert rc == tg.TGEMM_OK and launches[0][1:] == (10, 10)
    assert driver("gather", 5, 2, 10, 4096, 0, P, P, P, 8) == (tg.TGEMM_ENULL, [])


def test_combine_gradient_without_choices_reads_no_row(driver):
    rc, launches = driver("combine_grad", 5, 0, 20, 64, 0, 0, 0, P, P, 8)
    assert rc == tg.TGEMM_OK and len(launches) == 1 and launches[0][2] == 0 and launches[0][1] > 0


def test_rows_to_zero_near_the_largest_index(driver):
    """The step behind the last row may pass 2^31."""
    rows = (1 << 31) - 1
    for first, n in ((rows - 100, 64), (rows - 1, 64), (rows - 64, 64), (rows, 64), (rows - 300, 256), (5, 1 << 30)):
        rc, visited = driver("rows", first, rows, n)
        assert rc == 0 and [int(r) for _, r, _ in visited] == list(range(first, rows, n))


def test_k_tiles_of_the_longest_sums(driver):
    """An expert's rows, which the weights' form sums over, may be any number below 2^31."""
    for K in (0, 1, 31, 32, 33, 64, 65, 5000, (1 << 31) - 65, (1 << 31) - 64, (1 << 31) - 63, (1 << 31) - 31, (1 << 31) - 1):
        for BK in (32, 64):
            nk = -(-K // BK)
            assert driver("k_tiles", K, BK)[1] == [("k_tiles", nk, K - (nk - 1) * BK if nk else 0)]


def test_waves_of_the_norm(driver):
    """Six waves a row only for the widths, rows and outputs for which they measured faster."""
    def threads(rows, K, dtype, y, q):
        rc, launches = driver("norm", rows, K, dtype, y, q)
        assert rc == tg.TGEMM_OK and len(launches) == 1
        return int(launches[0][0].split("rmsnorm_rowsILi")[1].split("E")[0])

    for K in (2560, 2561, 3000, 384 * 8):
        for rows in (2048, 4095, 1 << 23):
            assert threads(rows, K, 1, P, 0) == 384 and threads(rows, K, 1, 0, P) == 384 and threads(rows, K, 0, P, 0) == 384
            assert threads(rows, K, 0, 0, P) == 256 and threads(rows, K, 0, P, P) == 256
            assert threads(rows, K, -1, P, 0) == 256 and threads(rows, K, -1, 0, P) == 256
        for rows in (1, 2047, (1 << 23) + 1):
            assert threads(rows, K, 1, P, 0) == 256 and threads(rows, K, 0, P, 0) == 256
    for K in (2559, 384 * 8 + 1, 2049, 4096):
        assert threads(4095, K, 1, P, 0) == 256
