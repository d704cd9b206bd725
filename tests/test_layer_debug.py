"""BFP8_DEBUG: the norm and the activation with codes refuse Inf and NaN in any
input, and give the same codes of finite ones.  The variable is read once per
process, so the case runs in a child process."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import json, sys, torch
sys.path.insert(0, ROOT)
import blockwise_fp8_gemm_bfp8_amd as bfp8
gen = torch.Generator(device="cuda").manual_seed(0)
t = {n: torch.randn((128, 256), device="cuda", generator=gen).to(torch.bfloat16)
     for n in ("x", "residual", "gate", "up", "dh")}
t["w"] = torch.rand(256, device="cuda", generator=gen) + 0.5
calls = {"norm": (lambda x: bfp8.rmsnorm_quantize(x["x"], x["w"], x["residual"], transposed=True),
                  ("x", "residual", "w")),
         "norm_rows": (lambda x: bfp8.rmsnorm_quantize(x["x"][:5], x["w"]), ("w",)),
         "glu": (lambda x: bfp8.swiglu_quantize(x["gate"], x["up"]), ("gate", "up")),
         "glu_grad": (lambda x: bfp8.swiglu_backward_quantize(x["dh"], x["gate"], x["up"],
                                                              transposed=True), ("dh", "gate", "up"))}
res = {}
for name, (call, inputs) in calls.items():
    res[name] = sum(int(o.float().double().sum().item()) for o in call(t))
    for n in inputs:
        for bad in ("nan", "inf"):
            x = dict(t, **{n: t[n].clone()})
            x[n].view(-1)[200] = float(bad)
            try:
                call(x)
                torch.cuda.synchronize()
                code = 0
            except bfp8.BFP8Error as e:
                code = e.code
            res[f"{name} {n} {bad}"] = code
print("RESULT " + json.dumps(res), flush=True)
"""


def test_debug_scan():
    found = {}
    for debug in ("1", "0"):
        out = subprocess.run([sys.executable, "-c", CHILD.replace("ROOT", repr(ROOT))],
                             env=dict(os.environ, BFP8_DEBUG=debug), capture_output=True, text=True,
                             timeout=110)
        assert out.returncode == 0, out.stderr[-2000:]
        found[debug] = json.loads(out.stdout.split("RESULT ")[1])
    for name, got in found["1"].items():
        assert got == (9 if " " in name else found["0"][name]), name
        assert " " not in name or found["0"][name] == 0, name
