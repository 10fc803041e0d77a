"""The row exchanges' entry points under AddressSanitizer + UBSan and
ThreadSanitizer, with stub kernels that check what a launch may rely on."""

import subprocess

import pytest

from test_host_sanitizers_cpu import CSRC, HOST, build


@pytest.mark.parametrize("sanitize", ["address,undefined", "thread"])
def test_rows_stress(tmp_path, sanitize):
    exe = build(tmp_path, "rows_stress", [HOST / "rows_stress.cpp"] +
                [CSRC / f for f in ("rows.cpp", "session.cpp", "validate.cpp", "plan.cpp")], sanitize)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stdout + res.stderr
    assert " 0 bad results" in res.stdout
