"""BFP8_DEBUG: attention refuses Inf and NaN in q, k, v and dout, but not in
the unused rows of a cache.  The variable is read once per process, so the
case runs in a child process."""
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
def code(fn):
    try:
        fn()
        torch.cuda.synchronize()
        return 0
    except bfp8.BFP8Error as e:
        return e.code
gen = torch.Generator(device="cuda").manual_seed(0)
new = lambda h: torch.randn((64, h, 64), device="cuda", generator=gen).to(torch.bfloat16)
t = dict(q=new(4), k=new(2).transpose(0, 1).contiguous().transpose(0, 1), v=new(2), dout=new(4))
o, lse = bfp8.attention_forward(t["q"], t["k"], t["v"])
res = {}
for name in ("none", "q", "k", "v", "dout"):
    x = {n: v.clone(memory_format=torch.preserve_format) for n, v in t.items()}
    if name != "none":
        x[name][33, 1, 5] = float("nan")
    res[name] = [code(lambda: bfp8.attention_forward(x["q"], x["k"], x["v"])),
                 code(lambda: bfp8.attention_backward(x["dout"], x["q"], x["k"], x["v"], o, lse))]
used = torch.tensor([33], dtype=torch.int32, device="cuda")
x = t["k"].clone()
x[33:] = float("nan")
res["unused"] = code(lambda: bfp8.attention_forward(t["q"][:5], x, t["v"], k_lens=used))
print("RESULT " + json.dumps(res), flush=True)
"""


def test_debug_scan():
    for debug, bad in (("1", 9), ("0", 0)):
        out = subprocess.run([sys.executable, "-c", CHILD.replace("ROOT", repr(ROOT))],
                             env=dict(os.environ, BFP8_DEBUG=debug), capture_output=True, text=True,
                             timeout=110)
        assert out.returncode == 0, out.stderr[-2000:]
        res = json.loads(out.stdout.split("RESULT ")[1])
        assert res.pop("none") == [0, 0] and res.pop("unused") == 0
        assert res.pop("dout") == [0, bad]
        assert all(v == [bad, bad] for v in res.values()), res
