"""The kernels' assembly, built here from source: no spilled register is restored where no lane may be active.

The compiler has placed restores of spilled vector registers at the head of blocks that are entered with EXEC = 0 (the
target of s_cbranch_execz, or what follows s_cbranch_execnz), before EXEC is set again.  Such a restore does nothing for
the inactive lanes, and a value that all lanes use afterwards is stale.  Restores are vector loads from scratch and reads of
accumulation registers; scalar registers spilled into lanes of vector ones are read whatever EXEC is."""

import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from gated_deltanet_linear_verify_amd import build

RESTORE = re.compile(r"v_accvgpr_(read|mov)|scratch_load|buffer_load.*(Reload|s32)")


def restores_without_lanes(text):
    """[(kernel, label, instruction)] of the restores that a path from a block with EXEC = 0 meets before EXEC is written."""
    code, labels, kernel, owner = [], {}, None, []
    for line in text.split("\n"):
        m = re.match(r"^([.\w$]+):", line)
        if m:
            if m[1].startswith(".L"):
                labels[m[1]] = len(code)
            elif not m[1].startswith("."):
                kernel = m[1]
            continue
        c = line.split(";")[0].strip()
        if c and not c.startswith((".", "//")):
            code.append((c, line))
            owner.append(kernel)
    roots = set()
    for i, (c, _) in enumerate(code):
        if c.startswith("s_cbranch_execz"):
            roots.add(labels[c.split()[1]])
        elif c.startswith("s_cbranch_execnz"):
            roots.add(i + 1)
    found = []
    for root in sorted(roots):
        todo, seen = [root], set()
        while todo:
            i = todo.pop()
            while i < len(code) and i not in seen:
                seen.add(i)
                c, line = code[i]
                op, dest = c.split()[0], (c.split() + [""])[1]
                if "saveexec" in op or "wrexec" in op or (op.startswith("s_") and dest.rstrip(",") in ("exec", "exec_lo", "exec_hi")):
                    break
                if RESTORE.search(line):
                    found.append((owner[i], i, c))
                if op == "s_endpgm" or op == "s_setpc_b64":
                    break
                if op == "s_branch":
                    i = labels[dest]
                    continue
                if op.startswith("s_cbranch"):
                    if op != "s_cbranch_execnz":  # EXEC is 0
                        todo.append(labels[dest])
                    if op == "s_cbranch_execz":
                        break
                i += 1
    return found


HEAD = """_ZN3gdn4kernE:
\ts_and_saveexec_b64 s[0:1], vcc
\ts_cbranch_execz .LBB0_2
\tv_mov_b32 v0, 1
.LBB0_2:
"""


@pytest.mark.parametrize("tail,count", [
    ("\ts_or_b64 exec, exec, s[0:1]\n\tv_accvgpr_read_b32 v1, a0\n", 0),
    ("\tv_accvgpr_read_b32 v1, a0\n\ts_or_b64 exec, exec, s[0:1]\n", 1),
    ("\tscratch_load_dword v1, off, s32 ; 4-byte Folded Reload\n\ts_or_b64 exec, exec, s[0:1]\n", 1),
    ("\ts_cbranch_scc1 .LBB0_3\n\ts_or_b64 exec, exec, s[0:1]\n\ts_endpgm\n.LBB0_3:\n\tv_accvgpr_read_b32 v1, a0\n", 1),
    ("\tv_readlane_b32 s4, v9, 3\n\ts_or_b64 exec, exec, s[0:1]\n", 0),
    ("\ts_mov_b64 exec, -1\n.LBB0_4:\n\ts_andn2_b64 exec, exec, s[4:5]\n\ts_cbranch_execnz .LBB0_4\n\tscratch_load_dword v1, off, off\n"
     "\ts_or_b64 exec, exec, s[4:5]\n", 1),
])
def test_the_check_finds_what_it_is_for(tail, count):
    assert len(restores_without_lanes(HEAD + tail + "\ts_endpgm\n")) == count


def test_no_restore_without_lanes(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")

    def listing(src):
        out = str(tmp_path / (src + ".s"))
        cmd = [build.HIPCC] + build.COMMON + ["-x", "hip", "-S", "--cuda-device-only", os.path.join(build.CSRC, src), "-o", out]
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr
        with open(out) as f:
            return f.read()

    sources = [s for s in build.SOURCES if s.endswith(".hip")]
    with ThreadPoolExecutor(4) as pool:
        texts = list(pool.map(listing, sources))
    kernels = [text.count(".amdhsa_kernel") for text in texts]
    assert all(text.count("s_endpgm") >= n for n, text in zip(kernels, texts)) and sum(kernels) > 100
    for src, text in zip(sources, texts):
        assert restores_without_lanes(text) == [], src
