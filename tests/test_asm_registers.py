"""Assembly in the kernels says which registers it writes: the compiler keeps its own values
in what is not named."""

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mamba_selective_scan_ssm_amd", "csrc")
SPECIAL = ("m0", "vcc", "exec", "scc")


def statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        if not path.endswith((".hip", ".h")):
            continue
        text = open(path).read()
        for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\);", text, re.S):
            yield os.path.basename(path), m.group(1)


def written(body):
    """Special registers that are the first operand of an instruction of the statement."""
    code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', body.split(":")[0]))
    for line in re.split(r"\\n|;", code):
        words = line.replace("\\t", " ").replace(",", " ").split()
        for reg in SPECIAL:
            if len(words) > 1 and words[1].split("_")[0] == reg:
                yield reg


def test_written_registers_are_named():
    found = list(statements())
    assert found
    for name, body in found:
        for reg in written(body):
            assert f'"{reg}"' in body.split(":")[-1], f"{name}: {reg} is written and not named: {body}"


def test_the_reading_of_statements():
    assert list(written('"s_mov_b32 m0, %0\\n\\ts_nop 0\\n\\tv_cmp_lt_f32 vcc, %1, %2" :: "s"(a) : "memory"')) == ["m0", "vcc"]
    assert list(written('"s_waitcnt vmcnt(0)" ::: "memory"')) == []
