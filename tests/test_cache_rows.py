"""Which tokens and heads a tile of attention's rows takes where a batch's starts hold anything, on the CPU."""
import os
import shutil
import subprocess

import pytest


def test_rows_of_slots_under_address_and_undefined_behaviour_sanitizers():
    if not (os.path.exists("/opt/rocm/bin/hipcc") or shutil.which("hipcc")):
        pytest.skip("hipcc not available")
    from bit_w4a4_quantized_amd.build import BUILD_DIR, build_host_check
    exe = build_host_check(check="abi_check_rows.cpp", exe=os.path.join(BUILD_DIR, "svdq_abi_check_rows"))
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "OK: 0 failure(s)" in r.stdout, r.stdout
