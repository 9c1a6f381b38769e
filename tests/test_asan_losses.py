"""The argument checks of the adapter projection, token scoring and the losses
under AddressSanitizer: as test_asan_host.py, with every source the library is
built from and a driver for the entry points that the other one does not call
(tests/asan/losses_driver.cpp).  Host code only; no call reaches a launch."""
import concurrent.futures
import importlib.util
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "top_sampling_amd")


def _build_script():
    spec = importlib.util.spec_from_file_location("_ts_build", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


BUILD = _build_script()


def _compile(args):
    r = subprocess.run(args, capture_output=True, text=True, timeout=600)
    return r.returncode, r.stdout[-3000:] + r.stderr[-3000:]


@pytest.mark.skipif(not os.path.exists(BUILD.HIPCC), reason="hipcc not installed")
def test_losses_validation_under_asan(tmp_path):
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fno-omit-frame-pointer",
             "-Xarch_host", "-fsanitize=address", "-Wno-unused-command-line-argument",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    srcs = [os.path.join(PKG, "csrc", s) for s in BUILD.SOURCES] + [
        os.path.join(ROOT, "tests", "asan", "losses_driver.cpp")]
    objs = [str(tmp_path / (os.path.basename(s) + ".o")) for s in srcs]
    jobs = [[BUILD.HIPCC, *flags, "-x", "hip", "-c", s, "-o", o] for s, o in zip(srcs, objs)]
    with concurrent.futures.ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as ex:
        for rc, log in ex.map(_compile, jobs):
            assert rc == 0, log
    exe = tmp_path / "losses_driver"
    rc, log = _compile([BUILD.HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address",
                        *objs, "-o", str(exe)])
    assert rc == 0, log
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:exitcode=23",
               HIP_VISIBLE_DEVICES="")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "losses_driver: 0 failures" in r.stdout
    assert "AddressSanitizer" not in r.stderr
