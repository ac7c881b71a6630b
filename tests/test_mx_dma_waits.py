"""LDS-DMA ordering guard of the MXFP4 products (CPU only). The tiled kernel
fills an LDS ring of NS stages by DMA and waits for the next stage with an
explicit vmcnt count before the barrier that lets every wave read it; the
compiler does not order the DMA's writes against those reads. This test
compiles the kernels to assembly and replays the main loop's vector-memory
queue (loads complete in issue order; `s_waitcnt vmcnt(n)` leaves at most n
outstanding): at every barrier the DMA of at most NS - 2 stages may still be
outstanding, because the stage read next is the oldest of the NS - 1 issued
since it was itself."""
import os
import re
import shutil
import subprocess

import pytest

from weight_quantized_gemm_amd import build_lib

HIPCC = build_lib.HIPCC


def _asm(tmpdir: str, src: str) -> str:
    out = os.path.join(tmpdir, src + ".s")
    r = subprocess.run([HIPCC, *build_lib.COMMON, *build_lib.HIP_FLAGS, "-x", "hip", "-S",
                        os.path.join(build_lib.CSRC, src), "-o", out, "--offload-device-only"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return open(out).read()


def main_loops(asm: str, kernel: str):
    """(kernel name, lines from its entry to the loop, lines of the loop) of the
    loop that holds matrix instructions, for every kernel of that name."""
    lines = asm.splitlines()
    for st, ln in enumerate(lines):
        m = re.match(r"^(_Z\w*" + kernel + r"\w*):", ln)
        if not m:
            continue
        end = next(i for i in range(st, len(lines)) if ".Lfunc_end" in lines[i])
        for h in range(st, end):
            if "Loop Header" not in lines[h]:
                continue
            name = "BB" + re.match(r"^\.LBB(\w+):", lines[h]).group(1)
            member = [i for i in range(st, end) if "Header=" + name + " " in lines[i] + " "]
            last = max(member + [h])
            stop = next((i for i in range(last + 1, end) if re.match(r"^\.LBB", lines[i])), end)
            body = lines[h:stop]
            if any("v_mfma" in x for x in body):
                yield m.group(1), lines[st:h], body
                break


def replay(entry, body, most):
    """Runs the entry and the loop body twice; returns the barriers of the loop
    at which more than `most` DMA groups (the DMAs between two barriers) are
    outstanding, and the number of barriers seen in the loop."""
    queue, group, bad, barriers = [], 0, [], 0
    for k, part in enumerate((entry, body, body)):
        for ln in part:
            t = ln.strip()
            if re.match(r"(buffer|global)_load", t):
                queue.append(group if t.split(";")[0].rstrip().endswith(" lds") else None)
            elif t.startswith("s_waitcnt"):
                m = re.search(r"vmcnt\((\d+)\)", t)
                if m:
                    del queue[:max(0, len(queue) - int(m.group(1)))]
            elif t.startswith("s_barrier"):
                group += 1
                if k > 0:
                    barriers += 1
                    out = {g for g in queue if g is not None}
                    if len(out) > most:
                        bad.append(f"{len(out)} stages outstanding")
    return bad, barriers


@pytest.mark.skipif(not (shutil.which(HIPCC) or os.path.exists(HIPCC)), reason="hipcc not found")
def test_every_barrier_waits_for_the_next_stage(tmp_path):
    seen, problems = 0, []
    for name, entry, body in main_loops(_asm(str(tmp_path), "mx_gemm.hip"), "mx_tile_kernel"):
        m = re.search(r"TileILb([01])E" + r"Li(\d+)E" * 8, name)
        assert m, name
        ns = int(m.group(7))
        bad, barriers = replay(entry, body, ns - 2)
        assert barriers == 2 * ns, f"{name}: {barriers} barriers in two turns"
        problems += [f"{name[:90]}: {b}" for b in bad]
        seen += 1
    assert seen >= 10
    assert not problems, "\n".join(problems[:20])


def test_replay_catches_a_short_wait():
    dma = ["buffer_load_dwordx4 v1, s[0:3], s4 offen lds"] * 4
    load = ["buffer_load_dwordx4 v[2:5], v0, s[4:7], s8 offen"] * 2
    stage = lambda n: [f"s_waitcnt vmcnt({n}) lgkmcnt(0)", "s_barrier"] + dma + load
    entry = dma * 4 + ["s_waitcnt vmcnt(0)", "s_barrier"]
    assert replay(entry, stage(2 + 2 * 6) * 4, 2)[0] == []
    assert replay(entry, stage(2 + 3 * 6) * 4, 2)[0]


@pytest.mark.skipif(not (shutil.which(HIPCC) or os.path.exists(HIPCC)), reason="hipcc not found")
def test_the_stages_behind_the_loop_wait_as_well(tmp_path):
    """The NS - 1 stages that may follow the whole turns, with the queue that a
    turn leaves and with the one that the entry leaves (K of fewer stages)."""
    asm = _asm(str(tmp_path), "mx_gemm.hip")
    lines = asm.splitlines()
    seen, problems = 0, []
    for name, entry, body in main_loops(asm, "mx_tile_kernel"):
        ns = int(re.search(r"TileILb([01])E" + r"Li(\d+)E" * 8, name).group(7))
        start = next(i for i, ln in enumerate(lines) if ln.startswith(name + ":")) + len(entry) + len(body)
        tail, barriers = [], 0
        for ln in lines[start:]:
            tail.append(ln)
            barriers += ln.strip().startswith("s_barrier")
            if barriers == ns - 1:
                break
        assert sum("v_mfma" in ln for ln in tail) > 0 and sum(" lds" in ln for ln in tail) > 0, name
        for before in (entry, entry + body + body):
            bad, met = replay(before, tail, ns - 2)
            assert met == 2 * (ns - 1), name
            problems += [f"{name[:90]}: {b}" for b in bad]
        seen += 1
    assert seen >= 10
    assert not problems, "\n".join(problems[:20])
