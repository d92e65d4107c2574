"""What lanes hand to each other through LDS is ordered by the source itself, not by what one compiler
happens to emit. The sources are taken through the compiler's front end for gfx950 (about
2 s a file, no optimization), whose output holds the waits and fences that they ask for."""
import os
import re
import subprocess

from bit_quantized_matmul_col_amd import build

CSRC = build.CSRC


def functions(source, tmp_path):
    """{mangled name: its calls and fences in the order of the text}"""
    out = str(tmp_path / "out.ll")
    flags = [f for f in build.FLAGS if f not in ("-shared", "-fPIC") and not f.startswith("-Rpass")]
    run = subprocess.run([build.HIPCC, *flags, "-I", build.INCLUDE, "-I", CSRC,
                          "--offload-device-only", "-S", "-emit-llvm", "-Xclang",
                          "-disable-llvm-passes", os.path.join(CSRC, source), "-o", out],
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr
    found, body = {}, None
    for line in open(out):
        m = re.match(r"define .*?@([\w$.]+)\(", line)
        if m:
            body = found.setdefault(m.group(1), [])
        elif re.match(r"\s+fence ", line):
            body.append(line.strip())
        elif body is not None and " call " in line:
            body.append(line.split(" call ", 1)[1].strip())
    return found


def test_the_first_pairs_of_a_tile_have_arrived_before_other_waves_read_them(tmp_path):
    """Direct loads to LDS are in flight until the wave that issued them has waited for its vector
    memory; a barrier by itself orders LDS accesses only."""
    seen = 0
    for name, calls in functions("experts_gated.hip", tmp_path).items():
        if not name.startswith("_ZN7llmint83ffn9run_tiles"):
            continue
        barriers = [i for i, c in enumerate(calls) if "__syncthreads" in c]
        assert len(barriers) == 1, name
        assert "wait_vmILi0E" in calls[barriers[0] - 1], calls[:barriers[0] + 1]
        seen += 1
    assert seen == 4  # two types, two tiles


def test_group_values_pass_between_lanes_in_order(tmp_path):
    """A wave writes its row's values to LDS and its lanes read each other's: release before the
    meeting, acquire behind it (the meeting alone orders no memory)."""
    seen = 0
    for name, calls in functions("experts_route.hip", tmp_path).items():
        meet = [i for i, c in enumerate(calls) if "@llvm.amdgcn.wave.barrier" in c]
        for i in meet:
            assert calls[i - 1] == 'fence syncscope("wavefront") release', (name, calls[i - 1])
            assert calls[i + 1] == 'fence syncscope("wavefront") acquire', (name, calls[i + 1])
            seen += 1
    assert seen == 10  # five widths of a row, two kinds of value
