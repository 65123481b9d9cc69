"""A process whose first call of the library is captured into a graph: each call in a process of its own."""
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

PROGRAM = """
import sys, torch
sys.path.insert(0, sys.argv[1])
from submanifold_sparse_convolution_hash_gb300 import binding as sc
g = torch.Generator(device="cuda").manual_seed(1)
def rows(n, c):
    return torch.randn((n, c), generator=g, device="cuda").half()
x, few, W, w = rows(3000, 2056), rows(20, 2056), rows(2056, 64), torch.ones(2056, device="cuda")
gout = rows(3000, 64)
grads = [torch.randn(1000 + i, generator=g, device="cuda") for i in range(100)]
held = sc.GradList(grads, out=[torch.empty_like(t) for t in grads])
q, off = rows(200, 64).view(100, 2, 64), torch.tensor([0, 100], dtype=torch.int32, device="cuda")
call = {
    "norm": lambda: [sc.sc_add_norm_fwd(few, w)],
    "norm_grad": lambda: list(sc.sc_add_norm_bwd(x, x, w)),
    "linear_few": lambda: [sc.sc_linear_fwd(few, W)],
    "linear": lambda: [sc.sc_linear_fwd(x, W)],
    "linear_grad": lambda: list(sc.sc_linear_bwd(gout, x, W, bias=True)),
    "clip": lambda: [sc.sc_grad_clip(held, 1.0)] + held.out,
    "attention": lambda: [sc.sc_attn_fwd(q, q, q, off)],
}[sys.argv[2]]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
want = call()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
sc.sc_rows_check()
print("the same")
"""


@pytest.mark.parametrize("call", ["norm", "norm_grad", "linear_few", "linear", "linear_grad", "clip", "attention"])
def test_the_first_call_is_captured(call):
    r = subprocess.run([sys.executable, "-c", PROGRAM, ROOT, call], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "the same" in r.stdout, r.stderr[-2000:]
