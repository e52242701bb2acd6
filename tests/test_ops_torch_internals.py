"""The operators' binding on a torch that lacks the internal bindings it prefers:
it imports, and its calls give the same results through public ones."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WITHOUT = """
import torch
import torch._C
for at, name in ((torch._C._dynamo.guards, "_empty_strided_cuda"), (torch._C, "_cuda_getCurrentRawStream")):
    if hasattr(at, name):
        delattr(at, name)
from mixture_experts_ffn_fp32_gb300 import api as A
"""


def run(code):
    r = subprocess.run([sys.executable, "-c", WITHOUT + code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout.strip()


def test_imports():
    assert run("print(A.LayerSpec.__name__)") == "LayerSpec"


def test_public_functions_stand_in():
    from mixture_experts_ffn_fp32_gb300 import api as A
    public = object()
    assert A._internal("no_such_module.no_such_name", public) is public
    assert A._internal("_no_such_name", public) is public
    assert A._internal("_dynamo.guards", public) is torch._C._dynamo.guards


@pytest.mark.gpu
def test_same_results():
    """Every call, on the current stream and on a given one, against the preferred bindings' results."""
    code = """
import os, sys
sys.path.insert(0, os.getcwd())
g = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn(40, 64, generator=g, device="cuda")
def every(stream):
    f = A.layer_norm(x, stream=stream)
    b = A.layer_norm_backward(x, x, f["mean"], f["rstd"], stream=stream)
    r = A.group_route(x, 4, stream=stream)
    d = A.group_route_backward(r["w"], r["idx"], x, stream=stream)
    q = A.quantize_rows(x, stream=stream)
    m = A.matmul_int8(q["q"], q["scale"], q["q"][None], q["scale"][None], stream=stream)
    return [*f.values(), *b.values(), *r.values(), d, *q.values(), m]
s = torch.cuda.Stream()
s.wait_stream(torch.cuda.current_stream())
got = every(None), every(s)
torch.cuda.synchronize()
print([[float(t.double().sum()) for t in v] for v in got])
"""
    from mixture_experts_ffn_fp32_gb300 import build
    build.build()
    want = subprocess.run([sys.executable, "-c", "import torch\nfrom mixture_experts_ffn_fp32_gb300 import api as A\n" + code],
                          cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert want.returncode == 0, want.stderr[-2000:]
    got = run(code)
    assert got == want.stdout.strip() and len(eval(got)) == 2
