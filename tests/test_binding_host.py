"""CPU checks of the binding's import and of what it asks torch for."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
import dequant_gemm_quantize_amd._lib as L

class Stream:
    cuda_stream = 4242

torch.cuda.current_stream = lambda dev: Stream if dev == 3 else None
assert L._raw_stream(3) == 4242
print("imported")
"""


def test_import_without_the_private_stream_query():
    """A torch that lacks the quick query of the stream's handle still imports the package, which then asks the public one."""
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr[-2000:]
