"""Barrier ordering of the attention and 16-bit linear kernels in their generated code (CPU only:
compiles for gfx950 and reads the AMD assembly of this build).

Both keep copies into LDS in flight across a bare s_barrier, so every barrier has to be reached
with the wave's own LDS reads complete: one still in flight could be overtaken by another wave's
copy into the buffer that it reads.  These kernels leave early and loop, so the property is
followed along their branches: a read is taken to be in flight at a barrier if it is on any path
from the kernel's start to there without an lgkmcnt(0) between.
"""
import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "bit_diffusion_model_svdq_amd"))
import build  # noqa: E402  (the package's build script: flags and sources)

# the kernels of a source, and how many barriers each of their forms has at least
SOURCES = {"attention.hip": {"attention_rows": 6, "attention_keys": 2},
           "linear_bf16.hip": {"linear_tile": 2, "linear_turns": 6, "linear_rows": 1}}
assert all(src in build.HIP_SOURCES for src in SOURCES)

READ = re.compile(r"^\s+ds_(read|bpermute|swizzle|load)")
LABEL = re.compile(r"^(\.LBB\w+):")
BRANCH = re.compile(r"^\s+s_(c?)branch\w*\s+(\.LBB\w+)")


def bodies(asm):
    """(kernel, lines of its body) for every kernel of the file."""
    for name in re.findall(r"\.amdhsa_kernel (\S+)", asm):
        start = asm.index(f"\n{name}:")
        yield name, asm[start:asm.index(".Lfunc_end", start)].split("\n")[2:]


def blocks_of(lines):
    """Basic blocks in layout order: (label, instructions, labels it may go on to)."""
    out, label, code = [], "start", []
    falls = True

    def close(to, fall):
        nonlocal code
        out.append([label, code, to, fall])
        code = []

    for n, line in enumerate(lines):
        m = LABEL.match(line)
        if m:
            close([], falls)
            label, falls = m.group(1), True
            continue
        b = BRANCH.match(line)
        if b:
            close([b.group(2)], b.group(1) == "c")
            label, falls = f"after {n}", True
        elif re.match(r"^\s+s_endpgm", line):
            close([], False)
            label, falls = f"after {n}", True
        else:
            assert not re.match(r"^\s+s_(setpc|swappc|call|cbranch_\w+_fork)", line), line
            code.append(line)
    close([], False)
    return [(lb, c, to + ([out[i + 1][0]] if fall and i + 1 < len(out) else [])) for i, (lb, c, to, fall) in enumerate(out)]


def walk(code, pending):
    """(barriers, those reached with a read in flight, whether one is in flight at the end)"""
    total = bad = 0
    for line in code:
        if READ.match(line):
            pending = True
        elif "s_waitcnt" in line and "lgkmcnt(0)" in line:
            pending = False
        elif re.match(r"^\s+s_barrier\b", line):
            total += 1
            bad += pending
    return total, bad, pending


def barriers(lines):
    blocks = blocks_of(lines)
    at = {label: i for i, (label, _, _) in enumerate(blocks)}
    assert len(at) == len(blocks)
    entry = [None] * len(blocks)          # None: not reached yet
    entry[0] = False
    todo = [0]
    while todo:
        i = todo.pop()
        end = walk(blocks[i][1], entry[i])[2]
        for label in blocks[i][2]:
            j = at[label]
            if entry[j] is None or (end and not entry[j]):
                entry[j] = bool(end)
                todo.append(j)
    found = [walk(c, e)[:2] for (_, c, _), e in zip(blocks, entry) if e is not None]
    return sum(t for t, _ in found), sum(b for _, b in found)


def lines(text):
    return text.split("\n")


def test_a_read_before_the_loops_barrier_is_followed_round_the_loop():
    loop = """
	s_cbranch_scc0 .LBB0_3
.LBB0_1:
	s_barrier
	ds_read_b128 v[0:3], v4
	s_cbranch_scc1 .LBB0_1
	s_waitcnt vmcnt(4) lgkmcnt(0)
	s_barrier
	s_endpgm
.LBB0_3:
	s_endpgm
"""
    assert barriers(lines(loop)) == (2, 1)
    assert barriers(lines(loop.replace("v4\n", "v4\n\ts_waitcnt lgkmcnt(0)\n"))) == (2, 0)


def test_code_after_an_early_end_is_seen():
    early = """
	s_cbranch_execz .LBB0_2
	s_endpgm
.LBB0_2:
	ds_read_u8 v0, v1
	s_waitcnt vmcnt(0)
	s_barrier
	s_endpgm
"""
    assert barriers(lines(early)) == (1, 1)
    assert barriers(lines(early.replace("vmcnt(0)", "lgkmcnt(0)"))) == (1, 0)


@pytest.mark.parametrize("src", SOURCES)
def test_every_barrier_follows_the_waves_lds_reads(src, tmp_path):
    if not os.path.exists(build.HIPCC) and not shutil.which("hipcc"):
        pytest.skip("hipcc not available")
    out = tmp_path / (src + ".s")
    cmd = [build.HIPCC] + build.HIP_FLAGS + ["-S", "--cuda-device-only", os.path.join(build.CSRC, src), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    seen = set()
    for name, body in bodies(out.read_text()):
        total, bad = barriers(body)
        assert bad == 0, f"{name}: {bad} of {total} barriers reached with LDS reads in flight"
        for kernel, least in SOURCES[src].items():
            if kernel in name:
                seen.add(kernel)
                assert total >= least, f"{name}: only {total} barriers found"
    assert seen == set(SOURCES[src])
