"""What the library's host side keeps is kept per device: the table of csrc/per_device.h from a
plain C++ program, and no launch keeps an attribute or a size of one device for all."""
import glob
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_decode_attention_cache_gb300", "csrc")


def test_table_of_devices(tmp_path):
    exe = tmp_path / "per_device_example"
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-pthread", "-I", CSRC,
                        os.path.join(ROOT, "tests", "c", "per_device_example.cpp"), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "FAIL" not in r.stdout and r.stdout.count("ok ") == 7


def test_no_plain_static_holds_what_a_device_is_asked_for():
    # a plain static int or bool beside such a call would be the first device's for all of them
    for path in glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")):
        text = open(path).read()
        if re.search(r"cudaFuncSetAttribute|cudaDeviceGetAttribute", text):
            assert not re.search(r"^\s*static (int|bool) \w+ = (0|false);", text, re.M) or path.endswith("api.cu"), path
