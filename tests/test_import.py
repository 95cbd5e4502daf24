"""What building and importing need (CPU only): the C library and its ctypes calls go with any torch, or none to
build; only the 4-bit and page calls need the module built against the installed one."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    return r.stdout.strip()


def test_another_torch_leaves_the_ctypes_calls():
    out = run("""
import torch
torch.__version__ = "0.0.0+none"
import fp8_paged_kv_reshape_gb300 as kv
kv.check_scale_host(1.0)
print(kv.status_string(0), kv.paged_decode_workspace_size(4, 32, 128) > 0,
      kv.paged_attention_fp4_workspace_size(4, 32, 8, 128, 1, 256, 16) > 0)
u8, i32 = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(1, dtype=torch.int32)
for call in (lambda: kv.copy_blocks([u8], i32, i32), lambda: kv.compact_blocks([u8], i32[None], i32, 16),
             lambda: kv.dequant_fp4(u8, u8, i32.long())):
    try:
        call()
    except ImportError as e:
        assert "kvfp8_torch-0.0.0+none" in str(e) and "build()" in str(e), e
    else:
        raise AssertionError("no ImportError")
""")
    assert out == "ok True True"


def test_the_library_builds_without_torch():
    out = run("""
import importlib.util, sys
sys.modules["torch"] = None
spec = importlib.util.spec_from_file_location("b", "fp8_paged_kv_reshape_gb300/_build.py")
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
print(b.build() == b.LIB)
""")
    assert out == "True"
