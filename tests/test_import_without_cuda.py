"""The wrappers on a torch that was built without CUDA: the module imports, and a
call says what it wants."""
import subprocess
import sys

from conftest import ROOT

PROGRAM = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda")]:
    delattr(torch._C, name)
from fft_long_convolution_flashconv_b200 import api
try:
    api.short_conv_fwd(torch.zeros(2, 3, 8), torch.zeros(3, 4))
except ValueError as e:
    print(e)
"""


def test_import_and_refusal():
    run = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.PIPE,
                         text=True, timeout=300)
    assert (run.returncode, run.stdout) == (0, "expected a CUDA tensor\n"), run.stderr
