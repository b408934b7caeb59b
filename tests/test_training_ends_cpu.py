"""The cross entropy and AdamW8 without a GPU: sizes, refusals, handles, and the
kernels that sizes launch."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import sgd_gradient_all_amd as ddl
import test_gpu_cross_entropy as gpu_tests
from sgd_gradient_all_amd import _operators as ops
from test_operators_cpu import OnDevice

E_NULL, E_ARG, E_BUCKETS, E_ALIGN, E_SCRATCH = -1, -2, -3, -4, -10
# an address that is only checked, never used: every call below is refused
SOME, ROOM = 1 << 20, (1 << 21, 1 << 45)


def lib():
    return ops._lib()


def layer(**kw):
    a = ops.ddl_ce_args()
    a.m, a.n, a.k, a.dtype, a.smoothing = 4, 8, 16, ddl.DDL_F16, 0.0
    a.x, a.ldx, a.w, a.ldw = SOME, 16, SOME, 16
    a.target = a.loss = a.lse = SOME
    for k, v in kw.items():
        setattr(a, k, v)
    return a


COMMON = [
    (dict(dtype=ddl.DDL_F32), E_ARG), (dict(dtype=7), E_ARG), (dict(n=0), E_ARG),
    (dict(n=(1 << 22) + 1), E_ARG), (dict(m=(1 << 22) + 1), E_ARG),
    (dict(k=(1 << 22) + 1), E_ARG), (dict(smoothing=-0.1), E_ARG), (dict(smoothing=1.1), E_ARG),
    (dict(smoothing=float("nan")), E_ARG), (dict(ldx=15), E_ARG), (dict(ldw=15), E_ARG),
    (dict(ldw=(1 << 22) + 1), E_ARG), (dict(x=None), E_NULL), (dict(w=None), E_NULL),
    (dict(target=None), E_NULL), (dict(lse=None), E_NULL), (dict(x=SOME + 1), E_ALIGN),
    (dict(w=SOME + 1), E_ALIGN), (dict(bias=SOME + 1), E_ALIGN), (dict(target=SOME + 4), E_ALIGN),
    (dict(lse=SOME + 2), E_ALIGN),
]


@pytest.mark.parametrize("kw,code", COMMON + [(dict(loss=None), E_NULL),
                                              (dict(loss=SOME + 2), E_ALIGN)])
def test_loss_refusals(kw, code):
    assert lib().ddl_cross_entropy(ctypes.byref(layer(**kw)), *ROOM, None) == code


def grad(ws=ROOM, layer_=None, **kw):
    a = ops.ddl_ce_grad_args()
    a.layer = layer(**(layer_ or {}))
    a.scale, a.dw_dtype = 1.0, ddl.DDL_F32
    a.dx, a.lddx, a.dw, a.lddw, a.db = SOME, 16, SOME, 16, SOME
    for k, v in kw.items():
        setattr(a, k, v)
    return lib().ddl_cross_entropy_grad(ctypes.byref(a), *ws, None)


@pytest.mark.parametrize("kw,code", COMMON)
def test_gradient_refuses_the_layer(kw, code):
    assert grad(layer_=kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dw_dtype=ddl.DDL_BF16), E_ARG), (dict(accumulate=2), E_ARG),
    (dict(scale=float("inf")), E_ARG), (dict(scale=float("nan")), E_ARG), (dict(lddx=15), E_ARG),
    (dict(lddw=15), E_ARG), (dict(dx=None, dw=None, db=None), E_NULL), (dict(dx=SOME + 1), E_ALIGN),
    (dict(dw=SOME + 2), E_ALIGN), (dict(db=SOME + 2), E_ALIGN), (dict(dloss=SOME + 2), E_ALIGN),
])
def test_gradient_refusals(kw, code):
    assert grad(**kw) == code


def test_workspaces():
    a = ctypes.byref(layer())
    need = ddl.cross_entropy_workspace("forward", 4, 8, 16)
    assert need > 0 and ddl.cross_entropy_workspace("forward", 0, 8, 16) == 0
    assert lib().ddl_cross_entropy(a, None, need, None) == E_NULL
    assert lib().ddl_cross_entropy(a, SOME, need - 1, None) == E_SCRATCH
    assert lib().ddl_cross_entropy(a, SOME + 8, need, None) == E_ALIGN
    need = ddl.cross_entropy_workspace("grad", 4, 8, 16)
    assert grad(ws=(None, need)) == E_NULL
    assert grad(ws=(SOME, need - 1)) == E_SCRATCH
    assert grad(ws=(SOME + 8, need)) == E_ALIGN
    # dz of a piece in two parts, x packed, dx's sums and parts: never the logits
    big = ddl.cross_entropy_workspace("grad", 8192, 131072, 4096)
    assert big < 8192 * 131072 * 2 / 2
    with pytest.raises(ValueError):
        ddl.cross_entropy_workspace("backward", 1, 1, 1)
    with pytest.raises(ValueError):
        ddl.cross_entropy_workspace("grad", -1, 1, 1)
    with pytest.raises(ddl.DDLError) as e:
        ddl.cross_entropy_workspace("grad", 1, 0, 1)
    assert e.value.code == E_ARG
    assert lib().ddl_cross_entropy_workspace(0, 1, 1, 1, None) == E_NULL
    assert lib().ddl_cross_entropy(None, None, 0, None) == E_NULL
    assert lib().ddl_cross_entropy_grad(None, None, 0, None) == E_NULL


@pytest.mark.parametrize("op", ["forward", "grad"])
def test_a_larger_call_needs_no_less_room_than_its_rows_and_pieces(op):
    """Sizes do not wrap: the largest ones ask for more than the card has."""
    assert ddl.cross_entropy_workspace(op, 1 << 22, 1 << 22, 1 << 22) > 1 << 44
    assert ddl.cross_entropy_workspace(op, 1 << 22, 1, 0) > 1 << 24


def test_no_rows_need_nothing():
    empty = layer(m=0, x=None, target=None, loss=None, lse=None)
    assert lib().ddl_cross_entropy(ctypes.byref(empty), None, 0, None) == 0
    assert grad(ws=(None, 0), layer_=dict(m=0, x=None, target=None, lse=None), accumulate=1) == 0


def test_python_refuses(monkeypatch):
    f16, f32 = torch.float16, torch.float32
    x, w = torch.zeros(2, 3).half(), torch.zeros(4, 3).half()
    t, v = torch.zeros(2).long(), torch.zeros(2)
    with pytest.raises(ValueError, match="GPU tensor"):
        ddl.cross_entropy(x, w, t, v, v)
    with pytest.raises(ValueError, match="GPU tensor"):
        ddl.cross_entropy_grad(x, w, t, v)
    with pytest.raises(ValueError, match="two dimensions"):
        ddl.cross_entropy(x[0], w, t, v, v)
    monkeypatch.setattr(ops, "_current_device", lambda: 0)
    d = lambda *s, dtype=f16: OnDevice(0, *s, dtype=dtype)  # noqa: E731
    i64 = torch.int64
    ok = dict(x=d(2, 8), w=d(4, 8), target=d(2, dtype=i64), loss=d(2, dtype=f32),
              lse=d(2, dtype=f32))
    for kw, match in ((dict(target=d(2, dtype=torch.int32)), "int64"),
                      (dict(target=d(3, dtype=i64)), "target"), (dict(loss=d(2)), "float32"),
                      (dict(lse=d(3, dtype=f32)), "lse"), (dict(w=d(4, 9)), "w has shape"),
                      (dict(w=d(4, 8, dtype=torch.bfloat16)), "type"), (dict(bias=d(5)), "bias")):
        with pytest.raises(ValueError, match=match):
            ddl.cross_entropy(**{**ok, **kw})
    del ok["loss"]
    for kw, match in ((dict(dx=d(2, 9)), "dx"), (dict(dx=d(2, 8, dtype=f32)), "type"),
                      (dict(dw=d(4, 8, dtype=f32), db=d(4)), "db"), (dict(dloss=d(2)), "float32"),
                      (dict(dw=d(5, 8)), "dw")):
        with pytest.raises(ValueError, match=match):
            ddl.cross_entropy_grad(**{**ok, **kw})


@pytest.mark.parametrize("index,current", [(1, 0), (0, 1)])
def test_arrays_of_another_device_are_refused(index, current, monkeypatch):
    monkeypatch.setattr(ops, "_current_device", lambda: current)
    d = lambda *s, dtype=torch.float32: OnDevice(index, *s, dtype=dtype)  # noqa: E731
    h, i64 = torch.float16, torch.int64
    a = ddl.AdamW8([(0, 4)])
    m, v, s = d(4, dtype=torch.int8), d(4, dtype=torch.uint8), d(1)
    for call in (lambda: ddl.cross_entropy(d(2, 8, dtype=h), d(4, 8, dtype=h), d(2, dtype=i64),
                                           d(2), d(2)),
                 lambda: ddl.cross_entropy_grad(d(2, 8, dtype=h), d(4, 8, dtype=h),
                                                d(2, dtype=i64), d(2)),
                 lambda: a.step(d(4), m, v, s, s, [d(4)], lr=1.0),
                 lambda: a.values(m, v, s, s, d(4), d(4))):
        with pytest.raises(ValueError, match="current"):
            call()


def test_adamw8_handles():
    a = ddl.AdamW8([(5, 7), (12, 0), (20, 300), (400, 256), (700, 257)])
    assert a.need == 957 and a.blocks == 1 + 2 + 1 + 2
    h = a.handle
    n = ctypes.c_size_t()
    assert lib().ddl_adamw8_blocks(h, None) == E_NULL
    a.destroy()
    a.destroy()  # twice is once
    assert lib().ddl_adamw8_destroy(h) == E_ARG  # not a live handle
    assert lib().ddl_adamw8_blocks(h, ctypes.byref(n)) == E_ARG
    assert lib().ddl_adamw8_destroy(None) == E_NULL
    plain = ddl.AdamW([(0, 4)])
    assert lib().ddl_adamw8_values(None, *[SOME] * 6, None) == E_NULL
    plain.destroy()
    for spans in ([(0, 8), (7, 2)], [(0, 1 << 41)], [(4, 2), (4, 2)], [(0, 10), (5, 0), (6, 3)]):
        with pytest.raises(ddl.DDLError) as e:
            ddl.AdamW8(spans)
        assert e.value.code == E_BUCKETS
    with pytest.raises(ddl.DDLError) as e:
        ddl.AdamW8([(0, 1 << 39)])  # more blocks than a launch takes
    assert e.value.code == E_ARG
    with pytest.raises(ValueError):
        ddl.AdamW8([(-1, 2)])
    empty = ddl.AdamW8([])
    assert empty.blocks == 0 and step8(empty.handle, grad=None, m=None, v=None) == 0


def step8(h, **kw):
    d = dict(grad=SOME, type=0, m=SOME, v=SOME, ms=SOME, vs=SOME, w=[SOME], copy=None, copy_type=0,
             lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, step=1)
    d.update(kw)
    w = (ctypes.c_void_p * max(1, len(d["w"])))(*d["w"])
    return lib().ddl_adamw8_step(h, d["grad"], d["type"], d["m"], d["v"], d["ms"], d["vs"], w,
                                 len(d["w"]), d["copy"], d["copy_type"], d["lr"], d["b1"],
                                 d["b2"], d["eps"], d["wd"], d["step"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), E_ARG), (dict(step=0), E_ARG), (dict(b1=1.0), E_ARG), (dict(b2=-0.1), E_ARG),
    (dict(eps=-1.0), E_ARG), (dict(lr=float("nan")), E_ARG), (dict(wd=float("inf")), E_ARG),
    (dict(w=[]), E_ARG), (dict(copy=SOME, copy_type=0), E_ARG), (dict(grad=None), E_NULL),
    (dict(m=None), E_NULL), (dict(v=None), E_NULL), (dict(ms=None), E_NULL),
    (dict(vs=None), E_NULL), (dict(w=[SOME, None]), E_NULL), (dict(ms=SOME + 2), E_ALIGN),
    (dict(vs=SOME + 1), E_ALIGN), (dict(w=[SOME + 1]), E_ALIGN), (dict(grad=SOME + 2), E_ALIGN),
    (dict(copy=SOME + 1, copy_type=1), E_ALIGN),
])
def test_adamw8_refusals(kw, code):
    a = ddl.AdamW8([(0, 4)])
    assert step8(a.handle, **kw) == code


def test_adamw8_values_refusals():
    a = ddl.AdamW8([(0, 4)])
    for i in range(6):
        args = [SOME] * 6
        args[i] = None
        assert lib().ddl_adamw8_values(a.handle, *args, None) == E_NULL
        if i > 1:
            args[i] = SOME + 2
            assert lib().ddl_adamw8_values(a.handle, *args, None) == E_ALIGN


def test_adamw8_python_refuses(monkeypatch):
    monkeypatch.setattr(ops, "_current_device", lambda: 0)
    d = lambda *s, dtype=torch.float32: OnDevice(0, *s, dtype=dtype)  # noqa: E731
    a = ddl.AdamW8([(0, 300)])
    ok = dict(grad=d(300), m=d(300, dtype=torch.int8), v=d(300, dtype=torch.uint8), m_scale=d(2),
              v_scale=d(2), weights=[d(300)], lr=1.0)
    for kw, match in ((dict(m=d(300, dtype=torch.uint8)), "int8"),
                      (dict(v=d(300, dtype=torch.int8)), "uint8"), (dict(m_scale=d(1)), "m_scale"),
                      (dict(v_scale=d(2, dtype=torch.float16)), "v_scale"),
                      (dict(m=d(299, dtype=torch.int8)), "m has"), (dict(weights=[]), "replica"),
                      (dict(weights=[d(300, dtype=torch.float16)]), "weights")):
        with pytest.raises(ValueError, match=match):
            a.step(**{**ok, **kw})


@pytest.fixture(scope="module")
def host_driver(tmp_path_factory):
    """The host code on a fake runtime (training_ends_host_driver.cpp)."""
    tmp = tmp_path_factory.mktemp("training_ends_host")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    csrc, objects = os.path.join(root, "sgd_gradient_all_amd", "csrc"), []
    for name in ("adamw8_kernels.hip", "cross_entropy_loss.hip", "cross_entropy_grad.hip"):
        objects.append(str(tmp / (name + ".o")))
        subprocess.run([hipcc, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17",
                        "-fPIC", "-c", os.path.join(csrc, name), "-o", objects[-1]], check=True)
    exe = str(tmp / "training_ends_host")
    # the kernels' code and the other operators are not built here
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    os.path.join(root, "tests", "training_ends_host_driver.cpp"),
                    os.path.join(csrc, "optimizer.cpp"), *objects, "-o", exe,
                    "-Wl,--unresolved-symbols=ignore-in-object-files"], check=True)

    def run(*args):
        out = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=60)
        assert out.returncode == 0, out.stdout + out.stderr
        return out.stdout
    return run


def test_handles_where_memory_runs_out(host_driver):
    out = host_driver()
    assert re.fullmatch(r"ok \d+ refusals\n", out), out


def tile(name):
    return tuple(map(int, re.search(r"Core.*?Li(\d+)ELi(\d+)E", name).groups()))


def launched(host_driver, m, n, k):
    """{what: the kernels of the loss and of both kinds of gradient}"""
    names = []
    for op, out in ((0, ddl.DDL_F32), (1, ddl.DDL_F32), (1, ddl.DDL_F16)):
        names += host_driver("ce", op, m, n, k, ddl.DDL_F16, out).split()
    return names


def product(name):
    """(dx and not dw, dz in two parts) of a product with dz."""
    return re.findall(r"Lb(\d)ELb(\d)EEE", name)[-1]


def test_gpu_tests_reach_every_kernel(host_driver):
    """Their sizes take every tile in every product, sums whole and in parts, rows
    through registers and packed, several pieces, and the kernels for few rows."""
    sizes = gpu_tests.LARGE + gpu_tests.SIZES + [(m, 5000, 2048) for m in (1, 2, 4, 16, 33, 64)]
    names = [n for s in sizes for n in launched(host_driver, *s)]
    seen = set()
    for n in names:
        if "both_kernel" in n:  # dx by 64 x 64 beside dw
            seen.add(("both", int(re.findall(r"Li(\d+)ELi\d+ELi2ELi2E", n)[-1])))
        elif "Core" in n:
            staged = re.search(r"Lb\dELb\dELb(\d)E", n).group(1)
            what = "loss" if "loss_kernel" in n else "dz" if "dz_kernel" in n else \
                "dx" if product(n)[0] == "1" else "dw"
            seen.add((what, tile(n), staged == "1"))
    for side in ((256, 256), (128, 128), (64, 64)):
        for what in ("loss", "dz", "dx", "dw"):
            assert (what, side, False) in seen, (what, side)
    assert ("both", 64) in seen and ("both", 128) in seen
    assert ("loss", (64, 32), False) in seen and ("dz", (64, 32), False) in seen
    for part in ("rows_kernel", "11pack_kernel", "pack_few_kernel", "matrix_kernel", "grad_join",
                 "join_kernelILi1E", "join_kernelILi32E"):
        assert any(part in n for n in names), part
    for rows in (1, 2, 4):
        assert any(f"few_kernelINS_4gemm4HalfELi{rows}E" in n for n in names), rows
        assert any(f"vector_kernelINS_4gemm4HalfELi{rows}E" in n for n in names), rows
    pieces = [sum("dz_kernel" in n for n in
                  host_driver("ce", 1, *s, ddl.DDL_F16, ddl.DDL_F32).split()) for s in sizes]
    assert max(pieces) >= 2
    # bfloat16 as binary16: dx in one pass, dw in one or in two
    names = [n for s in gpu_tests.ONCE for out in (ddl.DDL_F32, ddl.DDL_BF16)
             for n in host_driver("ce", 1, *s, ddl.DDL_BF16, out).split()]
    assert any("convert_kernel" in n for n in names)
    turned = [product(n) for n in names if "grad_kernelIDF16b" in n and "4HalfE" in n]
    assert {("1", "0"), ("0", "0"), ("0", "1")} <= set(turned)
    both = [re.findall(r"Lb(\d)ELb(\d)EE", n)[-1] for n in names
            if "both_kernelIDF16b" in n and "6Bfloat" not in n]
    assert {("0", "0"), ("0", "1")} <= set(both)


@pytest.mark.parametrize("m,n,k,side", [
    (8192, 131072, 4096, (256, 256)), (512, 1000, 2048, (64, 32)), (4096, 65536, 2048, (256, 256)),
    (65, 2000, 64, (64, 32)), (100, 131072, 4096, (128, 128)),
    (40, 300, 64, (64, 32))])
def test_tiles_of_the_logits(m, n, k, side, host_driver):
    names = host_driver("ce", 1, m, n, k, ddl.DDL_BF16, ddl.DDL_F32).split()
    assert {tile(x) for x in names if "dz_kernel" in x} == {side}


def test_each_class_is_taken_once(host_driver):
    """Pieces of a gradient: one of dz and of each product for every piece."""
    for m, n, k in ((8192, 131072, 4096), (4096, 65536, 2048), (1 << 20, 1000, 8)):
        names = host_driver("ce", 1, m, n, k, ddl.DDL_BF16, ddl.DDL_F32).split()
        pieces = max(1, -(-n // max(256, (128 << 20) // m // 256 * 256)))
        assert sum("dz_kernel" in x for x in names) == pieces
        assert sum("grad_kernel" in x for x in names) + 2 * sum(
            "both_kernel" in x for x in names) == 2 * pieces
