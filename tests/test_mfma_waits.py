"""Matrix results are not read before they are there, in the gfx950 assembly
the compiler writes for the serving kernels.

A vector instruction that reads (or overwrites) a matrix instruction's result
too soon after it gets the old register; the hardware does not wait, the
compiler inserts the wait states.  It was seen to miss them (ROCm 7.2.0) where
the reader follows a conditional branch: a result computed before the branch
and read right behind the label it jumps to.  This test walks every path from
every matrix instruction and counts wait states (one an instruction, N + 1 for
s_nop N) up to its first reader.

The number asked for is what the compiler itself leaves on straight paths in
these kernels: 8 behind 16x16x32 (bf16, 4 passes), 10 behind 16x16x4 (float32),
12 behind 16x16x128 (8-bit, 8 passes).  A matrix instruction that takes the result as
its addend may follow at once, and one that overwrites it is ordered by the
matrix pipe.  Runs on the CPU (hipcc cross-compiles)."""
import os
import re
import shutil
import subprocess

import pytest

from token_routing_expert_amd import build as tre_build

MFMA = re.compile(r"^v_mfma_f32_(\d+x\d+x\d+)\S*\s+([av])\[(\d+):(\d+)\]")
WAIT = {"16x16x32": 8, "16x16x4": 10, "16x16x128": 12}
REG = re.compile(r"\b([av])(?:(\d+)|\[(\d+):(\d+)\])")
SOURCES = ["few.hip", "fp8_ffn.hip"]


def registers(text):
    out = set()
    for m in REG.finditer(text):
        lo, hi = (int(m[2]), int(m[2])) if m[2] else (int(m[3]), int(m[4]))
        out.update((m[1], i) for i in range(lo, hi + 1))
    return out


def early_readers(asm):
    """(matrix instructions seen, [(function, instruction, reader, wait states)])"""
    seen, bad = {}, []
    name, body, label = None, [], {}

    def check():
        for at, ins in enumerate(body):
            m = MFMA.match(ins)
            if not m:
                continue
            shape, need = m[1], WAIT[m[1]]
            seen[shape] = seen.get(shape, 0) + 1
            result = {(m[2], i) for i in range(int(m[3]), int(m[4]) + 1)}
            todo, done = [(at + 1, 0)], {}
            while todo:
                i, waited = todo.pop()
                while i < len(body) and waited < need:
                    if done.get(i, need) <= waited:
                        break
                    done[i] = waited
                    t = body[i]
                    if t.startswith("s_nop"):
                        waited += int(t.split()[1]) + 1
                        i += 1
                        continue
                    if t.startswith("v_mfma"):
                        # its addend comes through the matrix pipe; its other operands are read like a vector's
                        ops = t.split(None, 1)[1].split(",")
                        if registers(",".join(ops[1:3])) & result:
                            bad.append((name, ins, t, waited))
                        if registers(ops[0]) >= result:
                            break                     # the pipe orders it; the new result has its own walk
                    elif not t.startswith("s_") and registers(t) & result:
                        bad.append((name, ins, t, waited))
                        break
                    waited += 1
                    if t.startswith("s_cbranch") or t.startswith("s_branch"):
                        to = label.get(t.split()[1])
                        if to is not None:
                            todo.append((to, waited))
                        if t.startswith("s_branch"):
                            break
                    if t.startswith("s_endpgm"):
                        break
                    i += 1

    for line in asm.split("\n"):
        text = line.split(";")[0].strip()
        if re.match(r"^_Z\w+:$", text):
            name, body, label = text[:-1], [], {}
        elif re.match(r"^\.LBB\w+:$", text):
            label[text[:-1]] = len(body)
        elif text.startswith(".Lfunc_end") and name:
            check()
            name, body, label = None, [], {}
        elif name and text and not text.startswith("."):
            body.append(text)
    return seen, bad


def kernel(*lines):
    return "\n".join(["_Zk:"] + list(lines) + [".Lfunc_end0:"])


def test_a_read_behind_a_branch_is_seen():
    mfma = "v_mfma_f32_16x16x32_bf16 v[48:51], v[80:83], v[72:75], v[68:71]"
    seen, bad = early_readers(kernel(mfma, "s_cbranch_vccnz .LBB0_2", "s_nop 7", ".LBB0_2:", "v_fmac_f32_e32 v1, v2, v50"))
    assert seen == {"16x16x32": 1} and len(bad) == 1 and bad[0][3] == 1
    assert not early_readers(kernel(mfma, "s_cbranch_vccnz .LBB0_2", "s_nop 7", ".LBB0_2:", "s_nop 6",
                                    "v_fmac_f32_e32 v1, v2, v50"))[1]
    assert early_readers(kernel(mfma, "ds_write_b128 v9, v[48:51]"))[1]
    assert not early_readers(kernel(mfma, "v_mfma_f32_16x16x32_bf16 v[48:51], v[0:3], v[4:7], v[48:51]", "s_nop 7",
                                    "v_add_f32_e32 v1, v2, v48"))[1]
    assert early_readers(kernel(mfma, "v_mfma_f32_16x16x32_bf16 v[0:3], v[48:51], v[4:7], v[0:3]"))[1]
    # a loop's back edge
    assert early_readers(kernel(".LBB0_1:", "v_add_f32_e32 v1, v2, v49", mfma, "s_cbranch_scc1 .LBB0_1", "s_endpgm"))[1]


@pytest.mark.timeout(600)
@pytest.mark.parametrize("source", SOURCES)
def test_serving_kernels_wait(source, tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    assert os.path.exists(hipcc), "hipcc not found: the check needs the kernels' gfx950 assembly"
    out = tmp_path / "k.s"
    r = subprocess.run([hipcc, *tre_build.FLAGS, "--cuda-device-only", "-S", os.path.join(tre_build.CSRC, source), "-o",
                        str(out)], capture_output=True, text=True, timeout=540)
    assert r.returncode == 0, r.stderr[-2000:]
    asm = out.read_text()
    seen, bad = early_readers(asm)
    print(seen)
    assert seen, "no matrix instructions: the pattern changed"
    assert not bad, f"{len(bad)} matrix results read too soon, e.g. {bad[:3]}"
    for name, body in re.findall(r"\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", asm, re.S):
        scratch = int(re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", body).group(1))
        assert scratch == 0, f"{name} spills {scratch} bytes per lane"
