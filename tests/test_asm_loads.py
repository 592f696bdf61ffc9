"""The compiler takes the output registers of a load in inline asm as written
at once, so it may copy them, or give them to something else, while the load is
still in flight. The weight gradients' slot ids are therefore loaded by the
compiler, which waits for what it uses: in the gfx950 assembly of every kernel
source, inline asm issues no scalar load."""

import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_grouped_moe_amd", "csrc")
HIPCC = next((c for c in ("/opt/rocm/bin/hipcc", shutil.which("hipcc")) if c and os.path.exists(c)), None)


def _asm(src, tmp):
    out = os.path.join(tmp, src + ".s")
    cmd = [HIPCC, "-O3", "-std=c++17", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", "-x", "hip",
           "--cuda-device-only", "-S", os.path.join(CSRC, src), "-o", out]
    subprocess.run(cmd, check=True, capture_output=True)
    return open(out).read().splitlines()


@pytest.mark.skipif(HIPCC is None, reason="hipcc not available")
def test_no_scalar_load_in_inline_asm(tmp_path):
    srcs = sorted(f for f in os.listdir(CSRC) if f.endswith(".hip"))
    with ThreadPoolExecutor(max_workers=4) as ex:
        listings = dict(zip(srcs, ex.map(lambda s: _asm(s, str(tmp_path)), srcs)))
    blocks = loads = 0
    for src, lines in listings.items():
        inline = False
        for l in lines:
            if "#ASMSTART" in l or "#ASMEND" in l:
                inline = "#ASMSTART" in l
                blocks += inline
            elif re.match(r"\s*s_(buffer_)?load_", l):
                assert not inline, f"{src}: {l.strip()!r} in inline asm"
                loads += 1
    assert blocks > 0 and loads > 0
