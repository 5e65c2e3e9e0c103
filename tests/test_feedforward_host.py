"""The feed-forward entry points on the host (no GPU needed): refusals, how products are cut into units, and the package
without torch or without the compiled module of these calls."""
import ctypes
import os
import random
import shutil
import struct
import subprocess
import sys
import textwrap

import pytest

import fusion_b2b_gemm_gb300 as b2b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIGNMENT, ALIAS, NO_DEVICE = 0, 1, 2, 3, 4, (5, 6)


def gpu():
    torch = pytest.importorskip("torch")
    return torch.cuda.is_available()


@pytest.mark.parametrize("args,code", [
    ((1, 512, 1024, 512, 0), OK),     # valid: fails only on the device check below
    ((2, 8, 8, 8, 1), OK),
    ((1, 0, 1024, 512, 0), INVALID),
    ((1, 512, -8, 512, 0), INVALID),
    ((1, 512, 1024, 0, 0), INVALID),
    ((1, 512, 1024, 512, 2), INVALID),       # unknown activation
    ((9, 512, 1024, 512, 0), INVALID),       # unknown type
    ((0, 512, 1024, 512, 0), UNSUPPORTED),   # fp32 output, tf32, fp64
    ((3, 512, 1024, 512, 0), UNSUPPORTED),
    ((4, 512, 1024, 512, 0), UNSUPPORTED),
    ((1, 516, 1024, 512, 0), UNSUPPORTED),   # not multiples of 8
    ((1, 512, 1028, 512, 0), UNSUPPORTED),
    ((1, 512, 1024, 4, 0), UNSUPPORTED),
    ((1, (1 << 20) + 8, 1024, 512, 0), UNSUPPORTED),
])
def test_plan_create_validates_before_device(args, code):
    h = ctypes.c_void_p()
    got = b2b.b2b_ffn_plan_create(ctypes.byref(h), *args)
    scaled = b2b.b2b_scaled_ffn_plan_create(ctypes.byref(h), *args)
    if code == OK:
        if gpu():
            pytest.skip("a GPU is present")
        assert got in NO_DEVICE
    else:
        assert got == code and scaled == code
    assert not h.value


def test_scaled_plans_want_rows_of_16_bytes():
    h = ctypes.c_void_p()
    assert b2b.b2b_scaled_ffn_plan_create(ctypes.byref(h), 1, 520, 1024, 512, 0) == UNSUPPORTED
    assert b2b.b2b_scaled_ffn_plan_create(ctypes.byref(h), 1, 512, 1032, 512, 0) == UNSUPPORTED
    assert b2b.b2b_scaled_gemm_plan_create(ctypes.byref(h), 1, 24, 16) == UNSUPPORTED
    assert b2b.b2b_scaled_gemm_plan_create(ctypes.byref(h), 1, 32, 12) == UNSUPPORTED
    assert b2b.b2b_scaled_gemm_plan_create(ctypes.byref(h), 3, 32, 16) == UNSUPPORTED
    assert b2b.b2b_scaled_gemm_plan_create(ctypes.byref(h), 1, 0, 16) == INVALID
    if not gpu():
        assert b2b.b2b_scaled_gemm_plan_create(ctypes.byref(h), 2, 32, 8) in NO_DEVICE
    assert not h.value


def test_calls_refuse_null_plans():
    n = ctypes.c_size_t()
    assert b2b.b2b_ffn_plan_create(None, 1, 8, 8, 8, 0) == INVALID
    assert b2b.b2b_scaled_ffn_plan_create(None, 1, 16, 16, 16, 0) == INVALID
    assert b2b.b2b_scaled_gemm_plan_create(None, 1, 16, 16) == INVALID
    assert b2b.b2b_ffn_plan_destroy(None) == OK
    assert b2b.b2b_ffn_plan_device_status(None, None) == INVALID
    assert b2b.b2b_ffn_plan_set_wait_budget(None, 0) == INVALID
    assert b2b.b2b_ffn_plan_set_debug(None, 0) == INVALID
    assert b2b.b2b_ffn_workspace(None, 1, 0, ctypes.byref(n)) == INVALID
    assert b2b.b2b_ffn_kept_bytes(None, 1, ctypes.byref(n)) == INVALID
    for run in (b2b.b2b_ffn_forward, b2b.b2b_ffn_backward, b2b.b2b_scaled_ffn_run, b2b.b2b_scaled_gemm_run):
        assert run(None, None, None) == INVALID


def quantize(dtype=1, rows=10, cols=256, block_rows=1, x=(0x10000, 256), q=(0x20000, 256), scale=(0x30000, 1, 10)):
    """b2b_quantize_blocks on addresses that nothing reads: refused, or no device here."""
    return b2b.b2b_quantize_blocks(dtype, rows, cols, block_rows, struct.pack("2q", *x), struct.pack("2q", *q),
                                   struct.pack("3q", *scale), None)


def test_quantize_refusals():
    if gpu():
        pytest.skip("a GPU is present")
    assert quantize() in NO_DEVICE
    assert quantize(rows=0) == OK and quantize(cols=0) == OK
    assert quantize(block_rows=128, scale=(0x30000, 2, 1)) in NO_DEVICE
    assert quantize(dtype=9) == INVALID and quantize(rows=-1) == INVALID and quantize(cols=-8) == INVALID
    assert quantize(block_rows=64) == INVALID
    assert quantize(dtype=3) == UNSUPPORTED and quantize(cols=250) == UNSUPPORTED
    assert quantize(x=(0, 256)) == INVALID and quantize(q=(0, 256)) == INVALID and quantize(scale=(0, 1, 10)) == INVALID
    assert quantize(x=(0x10008, 256)) == ALIGNMENT and quantize(q=(0x20004, 256)) == ALIGNMENT
    assert quantize(scale=(0x30002, 1, 10)) == ALIGNMENT and quantize(x=(0x10000, 260)) == ALIGNMENT
    assert quantize(x=(0x10000, 248)) == INVALID and quantize(q=(0x20000, 0)) == INVALID  # rows that overlap
    assert quantize(scale=(0x30000, 0, 10)) == INVALID and quantize(scale=(0x30000, 1, 0)) == INVALID
    assert quantize(scale=(0x30000, -1, 10)) == INVALID
    # scales of two blocks in one place: rows 0, 1 and blocks 1, 0; every stride that keeps them apart will do
    assert quantize(scale=(0x30000, 1, 1)) == INVALID and quantize(scale=(0x30000, 1, 9)) == INVALID
    assert quantize(scale=(0x30000, 2, 1)) in NO_DEVICE and quantize(scale=(0x30000, 7, 5)) in NO_DEVICE
    assert quantize(rows=1, scale=(0x30000, 0, 1)) in NO_DEVICE and quantize(cols=128, scale=(0x30000, 1, 0)) in NO_DEVICE
    assert quantize(q=(0x10100, 512)) == ALIAS and quantize(scale=(0x10000, 1, 10)) == ALIAS
    # rows of q between those of x, in one buffer
    assert quantize(x=(0x10000, 512), q=(0x10000 + 512, 1024)) in NO_DEVICE
    assert quantize(x=(0x10000, 512), q=(0x10000 + 504, 1024)) == ALIAS
    assert b2b.b2b_quantize_blocks(1, 1, 8, 1, None, None, None, None) == INVALID


def units(sizes, gate, kpan, clusters=76):
    arr = (ctypes.c_int64 * (2 * len(sizes)))(*[v for s in sizes for v in s])
    room = 1 + 6 * 40000
    out = (ctypes.c_int64 * room)()
    assert b2b.b2b_ffn_units(len(sizes), arr, gate, kpan, clusters, out, room) == OK
    return [tuple(out[1 + 6 * i:7 + 6 * i]) for i in range(out[0])]


def check_units(sizes, gate, kpan, clusters):
    """Every panel of every tile once, parts numbered without gaps, a tile's parts in order."""
    got = units(sizes, gate, kpan, clusters)
    cover, parts = {}, []
    for prob, mt, nt, k0, k1, part in got:
        assert 0 <= k0 < k1 <= kpan
        spans = cover.setdefault((prob, mt, nt), [])
        assert k0 == (spans[-1][1] if spans else 0)
        spans.append((k0, k1))
        if part >= 0:
            parts.append(part)
        else:
            assert (k0, k1) == (0, kpan)
    assert parts == list(range(len(parts)))
    want = {(i, a, b) for i, (m, n) in enumerate(sizes) for a in range(-(-m // 256)) for b in range(-(-n // (128 if gate else 256)))}
    assert set(cover) == want and all(s[-1][1] == kpan for s in cover.values())
    return got


def test_units_cover_every_tile_once():
    rng = random.Random(1)
    for _ in range(300):
        clusters = rng.choice([76, 74, 1, 3])
        gate = rng.random() < 0.3
        sizes = [(rng.randint(1, 6000), 8 * rng.randint(1, 600)) for _ in range(1 if gate else rng.randint(1, 3))]
        check_units(sizes, gate, rng.choice([1, 2, 7, 64, 224, rng.randint(1, 500)]), clusters)


def test_few_tiles_are_cut_along_k_and_full_rounds_are_not():
    assert all(u[5] < 0 for u in check_units([(256 * 76, 256)], False, 100, 76))
    few = check_units([(256, 1024)], False, 224, 76)
    assert len(few) > 4 and all(u[5] >= 0 for u in few)
    some = check_units([(256 * 80, 256)], False, 224, 76)
    assert [u[5] for u in some[:76]] == [-1] * 76 and all(u[5] >= 0 for u in some[76:])


def test_units_refuse_bad_arguments():
    one = (ctypes.c_int64 * 2)(256, 256)
    out = (ctypes.c_int64 * 7)()
    assert b2b.b2b_ffn_units(1, one, 0, 1, 76, out, 7) == OK
    assert b2b.b2b_ffn_units(1, one, 0, 1, 76, out, 6) == INVALID
    assert b2b.b2b_ffn_units(0, one, 0, 1, 76, out, 7) == INVALID and b2b.b2b_ffn_units(4, one, 0, 1, 76, out, 7) == INVALID
    assert b2b.b2b_ffn_units(1, one, 0, 0, 76, out, 7) == INVALID and b2b.b2b_ffn_units(1, one, 0, 1, 0, out, 7) == INVALID
    assert b2b.b2b_ffn_units(1, None, 0, 1, 76, out, 7) == INVALID and b2b.b2b_ffn_units(1, one, 0, 1, 76, None, 7) == INVALID
    assert b2b.b2b_ffn_units(1, (ctypes.c_int64 * 2)(0, 256), 0, 1, 76, out, 7) == INVALID


# ----------------------------------------------------------------- the package
def python(code, root=ROOT):
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=root, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": root})
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_import_without_torch():
    out = python("""
        import sys
        sys.modules["torch"] = None
        from fusion_b2b_gemm_gb300 import *
        for make in (lambda: GatedFeedForwardPlan("f16", 8, 8), lambda: ScaledGemmPlan("f16", 16, 16), lambda: quantize_blocks(None)):
            try:
                make()
            except ImportError as e:
                print("torch" in str(e))
        """)
    assert out.split() == ["True"] * 3


@pytest.mark.parametrize("there", ["missing", "damaged"])
def test_without_the_compiled_module(tmp_path, there):
    pytest.importorskip("torch")
    copy = tmp_path / "fusion_b2b_gemm_gb300"
    package = os.path.join(ROOT, "fusion_b2b_gemm_gb300")
    shutil.copytree(package, copy, ignore=shutil.ignore_patterns("_lib", "_build", "csrc", "__pycache__"))
    (copy / "_lib").mkdir()
    os.symlink(b2b.library_path(), copy / "_lib" / "libb2b.so")
    if there == "damaged":
        (copy / "_lib" / "ffn_binding.so").write_bytes(b"not a module")
    out = python("""
        import warnings
        import fusion_b2b_gemm_gb300 as b2b
        import fusion_b2b_gemm_gb300.feedforward as f
        with warnings.catch_warnings(record=True) as seen:
            warnings.simplefilter("always")
            f._load()
        print([w.category.__name__ for w in seen if "ffn_binding.so" in str(w.message)], f._binding.__name__)
        """, str(tmp_path))
    assert "RuntimeWarning" in out and "_NoBinding" in out


def test_names_and_types_are_refused():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="unknown dtype"):
        b2b.GatedFeedForwardPlan("f64", 8, 8)
    with pytest.raises(ValueError, match="unknown dtype"):
        b2b.ScaledGemmPlan("tf32", 16, 16)
    with pytest.raises(ValueError, match="unknown activation"):
        b2b.GatedFeedForwardPlan("f16", 8, 8, activation="tanh")
    x = torch.zeros(4, 16, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU expected"):
        b2b.quantize_blocks(x)
    with pytest.raises(TypeError, match="float32"):
        b2b.quantize_blocks(x.float())
    with pytest.raises(ValueError, match="block_rows"):
        b2b.quantize_blocks(x, 2)
    with pytest.raises(ValueError, match="matrix"):
        b2b.quantize_blocks(x[0])
    with pytest.raises(RuntimeError, match="gradient"):
        b2b.quantize_blocks(x.requires_grad_())
