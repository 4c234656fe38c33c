"""The host side of the feed-forward block's entry points (checks and workspace plans) under the address and
undefined-behaviour sanitizers: `tests/native/abi_validation_mlp.c` calls each with arguments it must refuse and with
the largest shapes that are accepted.  `api_mlp.hip` and the planning files are rebuilt with the sanitizers on their
host code only; nothing reaches the GPU."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "bit_quantized_finetuning_quant_amd")
SANITIZED = ["api_mlp", "norm", "gated", "gated_few"]
OBJS = ["codec", "qgemm", "lora", "gemv", "linear", "optim", "dropout", "act8", "ragged", "head", "api", "api_train"]


def test_validation_is_clean_under_host_sanitizers(tmp_path):
    from bit_quantized_finetuning_quant_amd import build

    objs = [os.path.join(PKG, "_build", f"{o}.o") for o in OBJS]
    if not all(os.path.exists(o) for o in objs):
        pytest.skip("the library objects are not built (run the build first)")
    clang = "/opt/rocm/llvm/bin/clang"
    if not os.path.exists(clang) or not shutil.which(build.hipcc()):
        pytest.skip("the ROCm compilers are not installed")
    flags = [f for f in build.HIPCC_FLAGS if f != "-O3"] + ["-O1", "-g"]
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all"]
    made = []
    for name in SANITIZED:
        made.append(str(tmp_path / f"{name}.o"))
        subprocess.run([build.hipcc(), *flags, *san, "-c", os.path.join(PKG, "csrc", f"{name}.hip"), "-o", made[-1]],
                       check=True, capture_output=True)
    drv, exe = str(tmp_path / "drv.o"), str(tmp_path / "abi_validation_mlp")
    host = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"]
    subprocess.run([clang, "-O1", "-g", *host, "-I", os.path.join(ROOT, "include"), "-c",
                    os.path.join(ROOT, "tests", "native", "abi_validation_mlp.c"), "-o", drv], check=True,
                   capture_output=True)
    subprocess.run([clang + "++", *host, drv, *made, *objs, "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib", "-o", exe], check=True, capture_output=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:protect_shadow_gap=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "all refusals as documented" in r.stdout
