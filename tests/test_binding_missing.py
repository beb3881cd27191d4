"""Without the binding of the rotary and cache operators, which is bound to one Python and one torch, the
quantizers and GEMMs work as ever; only those operators raise."""

import os
import subprocess
import sys

import pytest

pytest.importorskip("mx_block_scaled_quantize_amd", reason="libmx.so not built (run __graft_entry__.build())")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
sys.modules["mx_block_scaled_quantize_amd._bind"] = None      # importing it raises ImportError
import torch
import mx_block_scaled_quantize_amd as mxa
x, pos, t = torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int32), torch.zeros(8, 32, 2)
for f in (lambda: mxa.mx_quantize(torch.zeros(4, 64)), lambda: mxa.mm_fp8(*[torch.zeros(16, 16).to(torch.float8_e4m3fn)] * 2, t)):
    try:
        f()
    except (ValueError, RuntimeError) as e:
        assert "device" in str(e), e
    else:
        raise AssertionError("a host tensor was taken")
c = mxa.KVCache(*(torch.zeros((2, 2, 16, n), dtype=torch.uint8) for n in (64, 2, 64, 2)))
for f in (lambda: mxa.mx_rope_table(8, 64, device="cpu"), lambda: mxa.mx_rope(x, pos, t),
          lambda: mxa.mx_kv_append(x, x, c, pos.long()), lambda: mxa.mx_paged_attention(x, c, pos[None], pos, pos, max_q=1, max_kv=1)):
    try:
        f()
    except ImportError as e:
        assert "_bind" in str(e) and "build" in str(e), e
    else:
        raise AssertionError("no ImportError")
print("fine")
"""


def test_quantizers_do_not_need_the_binding():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stdout + r.stderr


def test_the_binding_is_built():
    """Its absence would otherwise show only where the operators are called."""
    import mx_block_scaled_quantize_amd as mxa
    assert os.path.exists(os.path.join(os.path.dirname(mxa.__file__), "_bind.so")), "run __graft_entry__.build()"
    assert mxa._bind.rope is not None
