"""GPU: whichever product a process calls first finds its kernels ready, and leaves
the others theirs to make: the same results in any order."""
import itertools
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALLS = ("linear", "loss", "gradient")

PROGRAM = """
import sys
import torch
import tiled_fp32_gemm_gb300 as mt

g = torch.Generator(device="cuda").manual_seed(1)
draw = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
sizes = [(3, 64, 300), (300, 64, 6000)]     # the split kernels, and pairs
ops = []
for T, K, V in sizes:
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    ops.append((draw(T, K), draw(V, K) / 8, target, torch.full((T,), 9.0, device="cuda")))
calls = {
    "linear": lambda a, b, t, f: [mt.linear(a, b, trans_b=True)],
    "loss": lambda a, b, t, f: mt.linear_cross_entropy(a, b, t, trans_b=True),
    "gradient": lambda a, b, t, f: mt.linear_cross_entropy_backward(f / 9, a, b, t, f,
                                                                    trans_b=True)}
sums = {}
for name in sys.argv[1:]:
    sums[name] = [r.double().sum().item() for o in ops for r in calls[name](*o)]
print(sorted(sums.items()))
"""


def test_any_order_of_first_calls():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    answers = set()
    for order in itertools.permutations(CALLS):
        r = subprocess.run([sys.executable, "-c", PROGRAM, *order], cwd=ROOT, text=True,
                           capture_output=True, timeout=300)
        assert r.returncode == 0, r.stderr
        answers.add(r.stdout)
    assert len(answers) == 1 and "nan" not in answers.pop()
