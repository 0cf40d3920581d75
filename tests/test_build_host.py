"""The build and what it leaves to load (CPU)."""
import os
import subprocess
import sys

import pytest

from w4a8_quantized_gemm_token_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_the_linears_load_without_the_block_calls():
    """A _block_calls that is missing, or of another torch, takes only its own calls with it."""
    code = (
        "import sys\n"
        "sys.modules['w4a8_quantized_gemm_token_b200._block_calls'] = None\n"  # its import fails
        "from w4a8_quantized_gemm_token_b200 import binding as qk\n"
        "assert qk.qk_version() > 0 and qk.qk_w8a8_workspace_size(4, 64) > 0\n"
        "for call in (lambda: qk.qk_rmsnorm_quantize(None), lambda: qk.qk_rope(None, None, None, None)):\n"
        "    try:\n"
        "        call()\n"
        "        raise SystemExit('no error')\n"
        "    except ImportError as e:\n"
        "        assert 'w4a8_quantized_gemm_token_b200.build' in str(e), e\n"
    )
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_the_block_calls_are_built_for_this_python_and_torch(monkeypatch, tmp_path):
    """The file's name carries the ABI, and another torch or Python than it was built with builds it again."""
    import sysconfig

    assert os.path.basename(build.CALLS) == "_block_calls" + sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.exists(build.CALLS) and os.path.exists(build.CALLS_ABI)
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "CALLS", str(tmp_path / "calls.so"))
    monkeypatch.setattr(build, "CALLS_ABI", str(tmp_path / "calls.abi"))
    monkeypatch.setattr(build.subprocess, "run", run)
    build._build_calls(False)
    build._build_calls(False)
    assert len(runs) == 1 and runs[0][0] == "g++"
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "9.9.9")
    build._build_calls(False)
    build._build_calls(False)
    assert len(runs) == 2
    monkeypatch.setattr(build.sys, "version", "3.99")
    build._build_calls(False)
    assert len(runs) == 3
    (tmp_path / "calls.abi").unlink()
    build._build_calls(False)
    assert len(runs) == 4


PTXAS = """ptxas info    : 0 bytes gmem
ptxas info    : Compiling entry function '_ZN2qk63_GLOBAL__N__1_12_kv4_chunk_cu_1_221kv4_chunk_join_kernelILi64EEEvNS_7Kv4ArgsE' for 'sm_100a'
ptxas info    : Used 40 registers, used 1 barriers
ptxas info    : Compiling entry function '_ZN2qk63_GLOBAL__N__1_12_kv4_chunk_cu_1_216kv4_chunk_kernelILi64EEEvNS_7Kv4ArgsE' for 'sm_100a'
    8 bytes stack frame, 8 bytes spill stores, 8 bytes spill loads
ptxas info    : Used {} registers, used 2 barriers
ptxas info    : Compiling entry function '_ZN2qk63_GLOBAL__N__1_12_kv4_chunk_cu_1_216kv4_chunk_kernelILi128EEEvNS_7Kv4ArgsE' for 'sm_100a'
ptxas info    : Used {} registers, used 2 barriers
"""


def test_register_splits_are_checked_by_the_build(monkeypatch, tmp_path):
    """A compiler that chose another number of registers than a kernel's split is of fails the build, and not
    the first call that is large enough for that kernel."""
    assert build.launch_registers(PTXAS.format(128, 120), "kv4_chunk_kernel") == [128, 120]
    assert build.launch_registers(PTXAS.format(128, 120), "kv4_chunk_join_kernel") == [40]
    src = os.path.join(build.CSRC, "kv4_chunk.cu")
    assert build.check_split(src, PTXAS.format(128, 128)) == ""
    for bad in (PTXAS.format(128, 120), PTXAS.format(136, 128), ""):
        assert "kv4_chunk_kernel" in build.check_split(src, bad)
    # in the build: the object is not kept
    real = subprocess.run

    def run(cmd, **kw):
        if "-c" not in cmd:
            return real(["true"])
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", PTXAS.format(128, 120) if "-v" in cmd else "")

    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(RuntimeError):
        build.build()
    left = os.listdir(tmp_path)
    assert "kv4_cache.o" in left and not [s for s in build.SPLITS if s[:-3] + ".o" in left]


def test_every_split_kernel_is_in_the_list():
    for name in os.listdir(build.CSRC):
        if name.endswith(".cu"):
            with open(os.path.join(build.CSRC, name)) as f:
                text = f.read()
            assert ("regs_inc<" in text) == (name in build.SPLITS), name
