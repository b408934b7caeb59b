"""The cross entropy's kernels and grids, on a fake runtime."""
import os
import re
import subprocess

import pytest

import sgd_gradient_all_amd as ddl
import test_gpu_cross_entropy as gpu_tests
import test_gpu_cross_entropy_edges as edge_tests

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    """launches(op, m, n, k, dtype, out, woff): [(kernel, workgroups)]"""
    tmp = tmp_path_factory.mktemp("launch_grids")
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    csrc, objects = os.path.join(ROOT, "sgd_gradient_all_amd", "csrc"), []
    for name in ("cross_entropy_loss.hip", "cross_entropy_grad.hip"):
        objects.append(str(tmp / (name + ".o")))
        subprocess.run([hipcc, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17",
                        "-fPIC", "-c", os.path.join(csrc, name), "-o", objects[-1]], check=True)
    exe = str(tmp / "launch_grids")
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    os.path.join(ROOT, "tests", "launch_grid_driver.cpp"),
                    os.path.join(csrc, "optimizer.cpp"), *objects, "-o", exe,
                    "-Wl,--unresolved-symbols=ignore-in-object-files"], check=True)

    def run(op, m, n, k, dtype, out=ddl.DDL_F32, woff=0):
        args = [exe, op, m, n, k, dtype, out, woff]
        done = subprocess.run(list(map(str, args)), capture_output=True, text=True, timeout=60)
        assert done.returncode == 0, done.stdout + done.stderr
        return [(line.split()[0], int(line.split()[1])) for line in done.stdout.splitlines()]
    return run


def tile(name):
    return tuple(map(int, re.search(r"Core.*?Li(\d+)ELi(\d+)E", name).groups()))


@pytest.mark.parametrize("dtype", [ddl.DDL_BF16, ddl.DDL_F16])
@pytest.mark.parametrize("m,n,k", [
    (1024, 1050, 2048), (1024, 1056, 1152), (512, 992, 4096), (600, 800, 4096),
    (1024, 1030, 4096), (1100, 1049, 1201), (1146, 1241, 1255), (549, 2321, 1608),
    (1024, 1024, 2048), (1, 1, 8), (3, 33, 64), (65, 97, 64), (4096, 10, 64), (300, 520, 2056)])
def test_tiles_of_dz_cover_what_the_products_read(m, n, k, dtype, launches):
    """The products' sums run over whole k tiles: 64 columns of dz at a time, those
    past the last class too, and 64 rows."""
    for out in (ddl.DDL_F32, dtype):
        got = [(tile(name), grid) for name, grid in launches(1, m, n, k, dtype, out)
               if "dz_kernel" in name]
        assert len(got) == 1
        (side_m, side_n), grid = got[0]
        across = grid // -(-m // side_m)
        assert across * side_n >= -(-n // 64) * 64
        assert -(-m // side_m) * side_m >= -(-m // 64) * 64


def test_narrow_tiles_are_among_them(launches):
    """bfloat16 operands as binary16 beside 64 x 32 tiles of dz."""
    for m, n, k in ((1024, 1050, 2048), (512, 992, 4096), (1100, 1049, 1201)):
        for out in (ddl.DDL_F32, ddl.DDL_BF16):
            names = [x for x, _ in launches(1, m, n, k, ddl.DDL_BF16, out)]
            dz = [x for x in names if "dz_kernel" in x]
            assert [tile(x) for x in dz] == [(64, 32)]


@pytest.mark.parametrize("m", [1, 3, 16, 63])
@pytest.mark.parametrize("n,k", [(1 << 22, 64), ((1 << 21) + 300, 2056), (3000000, 1001)])
def test_few_rows_need_no_more_room_than_64(m, n, k):
    """dz is held for whole k tiles of 64 rows, and a piece's size goes by those."""
    assert ddl.cross_entropy_workspace("grad", m, n, k) \
        <= ddl.cross_entropy_workspace("grad", 64, n, k)


def test_gpu_tests_take_every_tile_through_registers(launches):
    """w off 16 bytes: its rows go through registers in the loss, in dz (held in
    either type) and, unless w is converted, in dx."""
    seen = set()
    sizes = [(*s, 1) for s in gpu_tests.LARGE + gpu_tests.SIZES] + edge_tests.THROUGH_REGISTERS
    for m, n, k, first in sizes:
        for op, out in ((0, ddl.DDL_F32), (1, ddl.DDL_F32), (1, ddl.DDL_BF16)):
            for name, _ in launches(op, m, n, k, ddl.DDL_BF16, out, 2 * first):
                if "Core" not in name or "both_kernel" in name:
                    continue
                products = re.findall(r"Lb(\d)ELb(\d)EEE", name)
                what = "loss" if "loss_kernel" in name else "dz" if "dz_kernel" in name else \
                    "dx" if products[-1][0] == "1" else "dw"
                staged = re.search(r"Lb\dELb\dELb(\d)E", name).group(1) == "1"
                seen.add((what, tile(name), staged, "4Half" in name))
    for side in ((256, 256), (128, 128), (64, 64), (64, 32)):
        for held in (False, True):
            assert ("dz", side, True, held) in seen, (side, held)
        assert ("loss", side, True, False) in seen, side
    for side in ((256, 256), (128, 128), (64, 64)):
        assert ("dx", side, True, False) in seen, side
    assert ("dx", (256, 256), False, False) in seen


@pytest.mark.parametrize("m,n,k,kernel", [
    (1, 131072, 4096, "vector_kernel"), (1, 64000, 256, "vector_kernel"),
    (2, 64000, 2048, "vector_kernel"), (2, 64000, 1024, "loss_kernel"),
    (4, 64000, 256, "loss_kernel"), (4, 5000, 256, "few_kernel"),
    (1, 100, 24576, "vector_kernel"), (1, 100, 24584, "few_kernel"),
    (5, 1000, 2048, "few_kernel"), (16, 12288, 64, "few_kernel"), (16, 12289, 64, "loss_kernel"),
    (32, 8192, 64, "few_kernel"), (32, 8193, 64, "loss_kernel"), (64, 4096, 64, "few_kernel"),
    (64, 4097, 64, "loss_kernel"), (64, 131072, 4096, "loss_kernel"), (65, 16, 64, "loss_kernel")])
def test_kernels_for_few_rows(m, n, k, kernel, launches):
    for dtype in (ddl.DDL_F16, ddl.DDL_BF16):
        names = [x for x, _ in launches(0, m, n, k, dtype)]
        assert [x for x in ("vector_kernel", "few_kernel", "loss_kernel")
                if any(x in name and "pack" not in name for name in names)] == [kernel]


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 16, 17, 33, 64])
def test_room_for_the_parts_of_few_rows(m, launches):
    """A workgroup's part of each row, of every kernel that takes the call."""
    for n, k in ((1, 8), (300, 4096), (4096, 64), (12288, 64), (131072, 256), (1 << 22, 64)):
        room = ddl.cross_entropy_workspace("forward", m, n, k)
        for woff in (0, 2):
            for name, groups in launches(0, m, n, k, ddl.DDL_F16, ddl.DDL_F32, woff):
                if "vector_kernel" in name or ("few_kernel" in name and "pack" not in name):
                    parts = groups
                elif "loss_kernel" in name:
                    parts = -(-n // tile(name)[1])
                else:
                    continue
                assert 3 * 4 * parts * m <= room
