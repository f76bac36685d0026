"""Wait states behind the scaled matrix instructions, on every path of every kernel in the built
library: their results are not used within 20 states, what the longest form needs (the kernels wait that
long themselves), so no count of the compiler's is relied on.  No GPU needed."""
import shutil
import subprocess

import selective_state_space_34_amd as ss
from selective_state_space_34_amd import _build
from tests import test_wait_states as waits


def test_scaled_products(tmp_path, monkeypatch):
    monkeypatch.setitem(waits.NEED, "v_mfma_scale_f32_32x32x64_f8f6f4", 20)
    if _build.stale():
        _build.build()
    shutil.copy(ss.LIB, tmp_path / "libss.so")
    subprocess.run([waits.OBJDUMP, "--offloading", "libss.so"], cwd=tmp_path, check=True, capture_output=True)
    count = 0
    for f in sorted(tmp_path.iterdir()):
        if not f.name.endswith("gfx950"):
            continue
        text = subprocess.run([waits.OBJDUMP, "-d", str(f)], check=True, capture_output=True, text=True).stdout
        for name, code in waits.functions(text).items():
            for i, (op, _, _) in enumerate(code):
                if op.startswith("v_mfma_scale"):
                    count += 1
                    assert waits.shortest(code, i) is None, (name, i, op)
    assert count >= 9
