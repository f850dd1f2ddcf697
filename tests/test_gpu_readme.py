"""The README's Python example, run as it is written (with a smaller slab)."""
import os
import re

import numpy as np
import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_example_runs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    text = open(os.path.join(ROOT, "README.md")).read()
    code = re.search(r"## Use from Python\n\n```python\n(.*?)```", text, re.S).group(1)
    code = code.replace("64 << 30", "1 << 30")
    assert "1 << 30" in code
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s, std=0.02: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    ins, outs = [4096] * 6 + [14336], [4096, 1024, 1024, 4096, 14336, 14336, 4096]
    T = 40
    names = dict(num_tokens=T, seg_starts=np.array([0, 25, 40], np.int32),
                 seg_adapter=np.array([7, -1], np.int32), layer=5,
                 A=[r(32, 16, i) for i in ins], B=[r(32, o, 16) for o in outs],
                 h=r(T, 4096, std=1.0), attended=r(T, 4096, std=1.0),
                 w_norm1=r(4096) + 1, w_norm2=r(4096) + 1, w_qkv=r(6144, 4096), w_o=r(4096, 4096),
                 w_gate_up=r(28672, 4096), w_down=r(4096, 14336), base_out=r(T, 6144),
                 y=torch.empty(T, 6144, dtype=torch.bfloat16, device="cuda"))
    exec(compile(code, "README.md", "exec"), names)
    torch.cuda.synchronize()
    for name, width in (("h", 4096), ("x", 4096), ("qkv", 6144), ("o", 4096), ("mid", 14336), ("y", 6144)):
        t = names[name]
        assert t.shape == (T, width) and bool(t.isfinite().all()), name
    names["pool"].close()
