"""The package imports, and its calls run, on a torch without the private symbol
that hands out a stream's handle."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WITHOUT = "import torch\ndel torch._C._cuda_getCurrentRawStream\n"


def run(code):
    r = subprocess.run([sys.executable, "-c", WITHOUT + code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split()[-1:] == ["done"], r.stdout + r.stderr


def test_import_without_the_private_symbol():
    run("import gated_delta_rule_54_amd as gdr\nassert gdr.gdr_forward and gdr.gdr_linear_forward\nprint('done')")


@pytest.mark.gpu
def test_calls_without_the_private_symbol():
    """The call's stream is the current one, the default and another."""
    run("""
import gated_delta_rule_54_amd as gdr
from gated_delta_rule_54_amd import linear as L
q = torch.randn(2, 3, 2, 64, device="cuda")
o, ht = gdr.gdr_linear_forward(q, q, q)
s = torch.cuda.Stream()
assert L._raw_stream(q.device.index) == torch.cuda.current_stream().cuda_stream
torch.cuda.synchronize()
with torch.cuda.stream(s):
    assert L._raw_stream(q.device.index) == s.cuda_stream
    o2, ht2 = gdr.gdr_linear_forward(q, q, q)
s.synchronize()
assert torch.equal(o, o2) and torch.equal(ht, ht2)
print("done")
""")
