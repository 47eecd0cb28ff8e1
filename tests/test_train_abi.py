"""The C ABI of include/mps_train.h and its binding, without a GPU: the header
in C and C++, the exported names, every entry point's argument checks under
the host sanitizers (with stand-ins for the launchers), and the binding's own
refusals."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import mixed_precision_sharded_amd as mps
from mixed_precision_sharded_amd import binding, training

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mps_train.h")
HERE = os.path.join(ROOT, "tests", "sanitize")
CSRC = os.path.join(ROOT, "mixed_precision_sharded_amd", "csrc")


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^(?:int|size_t)\s+(\w+)\s*\(", text, flags=re.M)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from mixed_precision_sharded_amd import build
        build.build()
    return binding.lib()


def test_every_declared_function_is_exported_and_bound(lib):
    out = subprocess.run(["nm", "-D", "--defined-only", binding.LIB_PATH], check=True,
                         capture_output=True, text=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    names = declared()
    assert len(names) == 12
    assert set(names) <= exported
    assert names == sorted([*training._SIGNATURES, *training._SIZES])
    for n in names:
        assert callable(getattr(mps, n)), n


def test_signatures_have_the_header_s_argument_counts():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name, types in {**training._SIGNATURES, **training._SIZES}.items():
        args = re.search(r"\b%s\s*\(([^;]*)\)\s*;" % name, text).group(1).split(",")
        assert len(args) == len(types), name
        for a, t in zip(args, types):
            if "*" in a:
                assert t is ctypes.c_void_p, (name, a)
            else:
                want = {"int64_t": ctypes.c_int64, "double": ctypes.c_double, "size_t": ctypes.c_size_t,
                        "mps_dtype": ctypes.c_int, "int": ctypes.c_int}[a.split()[0]]
                assert t is want, (name, a)


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "mps_train.h"\n'
                   "int (*f)(const void*, mps_dtype, int64_t, int64_t, int64_t, uint8_t*, uint8_t*, void*) = act8_save;\n"
                   "typedef char row[MPS_ACT8_ROW(33) == 64 && MPS_ACT8_ROW(32) == 32 && MPS_ACT8_ROW(1) == 32 ? 1 : -1];\n"
                   "int main(void) { return (int)sizeof(row) - 1; }\n")
    inc = os.path.join(ROOT, "include")
    for cmd in (["gcc", "-std=c99"], ["g++", "-std=c++17", "-x", "c++"]):
        r = subprocess.run([*cmd, "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only", "-I", inc, str(src)],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="no g++ or ROCm headers")
def test_argument_checks_under_sanitizers(tmp_path):
    exe = str(tmp_path / "train_driver")
    subprocess.run(["g++", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-std=c++17", "-Wall",
                    "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-o", exe, os.path.join(HERE, "train_driver.cpp"),
                    os.path.join(HERE, "no_launch.cpp"), os.path.join(CSRC, "train_api.cpp"), os.path.join(CSRC, "api.cpp"),
                    "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1", UBSAN_OPTIONS="print_stacktrace=1"))
    assert r.returncode == 0 and "train driver ok" in r.stdout, r.stdout + r.stderr


def test_sizes(lib):
    assert mps.act8_row(1) == 32 and mps.act8_row(32) == 32 and mps.act8_row(33) == 64
    codes, scales = mps.act8_empty(3, 33, "cpu")
    assert codes.shape == (3, 64) and scales.shape == (3, 2) and codes.dtype == scales.dtype == torch.uint8
    assert mps.act8_rmsnorm_backward_workspace_bytes(0, 100) == 0
    assert mps.act8_rmsnorm_backward_workspace_bytes(1000, 4096) >= 4096 * 4
    assert mps.policy_loss_workspace_bytes(0, 10) == 0
    # few rows share a row's logits; the scratch stays far below one row of them
    assert 0 < mps.policy_loss_workspace_bytes(1, 128256) < 128256 * 2
    # a gradient as large as the chip's tiles is not split
    assert mps.act8_weight_grad_workspace_bytes(16384, 14336, 4096) == 0
    assert mps.act8_weight_grad_workspace_bytes(16384, 512, 512) > 0
    for bad in ((-1, 8), (1 << 31, 8), (8, 0), (8, (1 << 27) + 1)):
        with pytest.raises(mps.MpsError) as e:
            mps.policy_loss_workspace_bytes(*bad)
        assert e.value.code == -22
    with pytest.raises(ValueError):
        mps.policy_loss_workspace_bytes(1 << 70, 8)


def test_the_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 40)
    codes, scales = mps.act8_empty(4, 40, "cpu")
    with pytest.raises(ValueError, match="CUDA"):
        mps.act8_save(x, codes, scales)
    with pytest.raises(ValueError, match="dimensions"):
        mps.act8_save(x[0], codes, scales)
    with pytest.raises(ValueError, match="CUDA"):
        mps.act8_load(codes, scales, x)
    with pytest.raises(ValueError, match="CUDA"):
        mps.policy_loss(x, torch.zeros(4, dtype=torch.int64), x[:, 0], x[:, 0], x[:, 0], x[0, :1], None)


def test_matrix_checks():
    x = torch.zeros(4, 40)
    rows = lambda t, like=x, shape=None: training._rows(t, like, shape or like.shape, "t")  # noqa: E731
    assert rows(x) == 40
    wide = torch.zeros(4, 100)
    assert rows(wide[:, 3:43]) == 100
    assert rows(torch.zeros(1, 1000)[:, :40], like=torch.zeros(1, 40)) == 40  # one row: its stride says nothing
    with pytest.raises(TypeError, match="expected torch.float32"):
        rows(x.to(torch.bfloat16))
    with pytest.raises(ValueError, match=r"expected \(4, 40\)"):
        rows(torch.zeros(4, 41))
    with pytest.raises(ValueError, match="contiguous"):
        rows(torch.zeros(40, 4).t())
    with pytest.raises(ValueError, match="contiguous"):
        training._flat(torch.zeros(4, 80)[:, :40], torch.float32, (4, 40), -1, "t")
    with pytest.raises(TypeError):
        training._flat(x, torch.uint8, (4, 40), -1, "t")
    with pytest.raises(ValueError, match="must be on cuda:0"):
        training._flat(x, torch.float32, (4, 40), 0, "t")
    with pytest.raises(ValueError, match="workspace"):
        training._workspace(x, -1)
    assert training._workspace(None, -1) == (None, 0)


def test_a_missing_library_raises(monkeypatch, tmp_path):
    monkeypatch.setattr(binding, "LIB_PATH", str(tmp_path / "libmps_adamw.so"))
    monkeypatch.setattr(binding, "_lib", None)
    with pytest.raises(RuntimeError, match="missing"):
        mps.policy_loss_workspace_bytes(1, 10)
