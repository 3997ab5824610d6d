"""What the compiler makes of a kernel's memory accesses and waits, for tests that hold it to the
order its source asks for.  Nothing runs: a source is compiled to gfx950 assembly."""

import functools
import os
import re
import subprocess

import pytest

from mxfp4_paged_cache_quant_amd import build


@functools.lru_cache(maxsize=None)
def kernels(source):
    """Kernel (its name and template arguments) -> its events in the order of its code, of a file of csrc/."""
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    asm = subprocess.run([build.HIPCC, *build.CFLAGS, "--cuda-device-only", "-S", "-o", "-",
                          os.path.join(build.CSRC, source)], capture_output=True, text=True, check=True).stdout
    found = dict(_functions(asm))
    names = subprocess.run(["c++filt"], input="\n".join(found), capture_output=True, text=True, check=True).stdout
    return {re.search(r"(\w+<[^()]*>)\(", n).group(1): e for n, e in zip(names.splitlines(), found.values())
            if re.search(r"\w+_kernel<[^()]*>\(", n)}


def _functions(asm):
    name, events = None, []
    for line in asm.splitlines():
        head = re.match(r"(_Z\w+):", line)
        if head:
            name, events = head.group(1), []
        elif line.startswith(".Lfunc_end"):
            yield name, events
            name = None
        elif name:
            event = _event(line.split(";")[0].strip())
            if event:
                events.append(event)


def _event(line):
    """edge: a label or branch; mfma; copy: a load to LDS; load; transpose: a transposing LDS read; wait:
    for every load, wait n: but for the youngest n; barrier; spill: a register in memory."""
    op = line.split()[0] if line else ""
    if re.match(r"\.LBB\w+:", line) or op.startswith(("s_cbranch", "s_branch")):
        return "edge"
    if op.startswith("v_mfma"):
        return "mfma"
    if op.startswith(("buffer_load", "global_load")):
        return "copy" if line.endswith(" lds") or "_lds_" in op else "load"
    if op.startswith("scratch_"):
        return "spill"
    if op.startswith("ds_read_b64_tr"):
        return "transpose"
    left = re.search(r"vmcnt\((\d+)\)", line) if op == "s_waitcnt" else None
    if left:
        return "wait" if left.group(1) == "0" else "wait " + left.group(1)
    return "barrier" if op == "s_barrier" else None
