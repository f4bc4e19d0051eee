"""Hazards that the compiler leaves to the code, in the gfx950 assembly it
writes for the training kernels.

A 16-byte store reads its data registers some cycles after it is issued.  Behind
one without a scalar offset (buffer) or through a flat address the compiler
keeps those registers for one more instruction; behind a buffer store WITH a
scalar offset it does not, and results of the next instruction were seen in the
stored rows.  So no such store may be followed at once by an instruction that
writes its data.  Matrix results: as in the serving kernels, walked along every
path.  Runs on the CPU (hipcc cross-compiles)."""
import os
import re
import shutil
import subprocess

import pytest

import test_mfma_waits as waits
from token_routing_expert_amd import build as tre_build

STORE = re.compile(r"^(buffer|global|flat)_store_dwordx[34]\s+(.*)$")


def overwritten_stores(asm):
    """(16-byte stores seen, [(store, the next instruction)] whose data the next instruction writes)"""
    body = [t for line in asm.split("\n") if (t := line.split(";")[0].strip()) and not t.startswith(".")]
    seen, bad = 0, []
    for t, after in zip(body, body[1:]):
        m = STORE.match(t)
        if not m:
            continue
        seen += 1
        ops = m[2].split(",")
        data = waits.registers(ops[0] if m[1] == "buffer" else ops[1])
        if not after.startswith("v_"):
            continue
        args = after.split(None, 1)[1].split(",")
        written = waits.registers(",".join(args[:2]) if "swap" in after else args[0])
        if written & data:
            bad.append((t, after))
    return seen, bad


def test_an_overwritten_store_is_seen():
    store = "buffer_store_dwordx4 v[4:7], v1, s[0:3], s9 offen"
    assert overwritten_stores(store + "\n v_mov_b32_e32 v5, v9")[1]
    assert overwritten_stores(store + "\n v_permlane32_swap_b32_e32 v1, v6")[1]
    assert not overwritten_stores(store + "\n v_mov_b32_e32 v8, v5")[1]
    assert not overwritten_stores(store + "\n s_nop 0\n v_mov_b32_e32 v5, v9")[1]
    assert overwritten_stores("global_store_dwordx4 v[2:3], v[4:7], off\n v_add_f32_e32 v4, v5, v6")[1]


def assembly(source, tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    assert os.path.exists(hipcc), "hipcc not found: the check needs the kernels' gfx950 assembly"
    out = tmp_path / "k.s"
    r = subprocess.run([hipcc, *tre_build.FLAGS, "--cuda-device-only", "-S", os.path.join(tre_build.CSRC, source), "-o",
                        str(out)], capture_output=True, text=True, timeout=540)
    assert r.returncode == 0, r.stderr[-2000:]
    return out.read_text()


@pytest.mark.timeout(600)
@pytest.mark.parametrize("source", ["grouped_ffn.hip", "small_f32.hip", "train.hip", "combine.hip", "wgrad.hip"])
def test_training_kernels(source, tmp_path, monkeypatch):
    asm = assembly(source, tmp_path)
    seen, bad = overwritten_stores(asm)
    assert seen, "no 16-byte stores: the pattern changed"
    assert not bad, f"{len(bad)} stores whose data the next instruction writes, e.g. {bad[:3]}"
    for name, body in re.findall(r"\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", asm, re.S):
        scratch = int(re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", body).group(1))
        assert scratch == 0, f"{name} spills {scratch} bytes per lane"
    # what the compiler leaves on straight paths: 12 behind 32x32x16 (8 passes), 18 behind 32x32x2 (16)
    monkeypatch.setattr(waits, "WAIT", {"32x32x16": 12, "32x32x2": 18})
    mfma, early = waits.early_readers(asm)
    assert (source in ("train.hip", "combine.hip")) == (not mfma)
    assert not early, f"{len(early)} matrix results read too soon, e.g. {early[:3]}"
