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
