"""Direct global-to-LDS loads written in assembly: the load reads its LDS base from m0, and on gfx9 an instruction that
writes m0 has to lie at least one wait state before it. The compiler's hazard recognizer does not look into an asm
block, so every block must hold the state itself."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_up_projection_amd", "csrc")


def asm_lines(text):
    """Instructions of the file's string literals, in order."""
    for literal in re.findall(r'"((?:[^"\\]|\\.)*)"', text):
        for line in re.split(r"\\n\\t|\\n", literal):
            if line.strip():
                yield line.strip()


def test_a_state_between_m0_and_the_load():
    loads = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        since = None  # instructions since m0 was written
        with open(path) as f:
            text = f.read()
        for line in asm_lines(text):
            op = line.split()[0]
            if re.match(r"s_\w+ m0\b", line):
                since = 0
            elif re.match(r"(global|buffer)_load_lds|buffer_load.* lds", line):
                loads += 1
                assert since is not None and since >= 1, f"{os.path.basename(path)}: {line}"
            elif since is not None and re.match(r"[sv]_|ds_", op):
                since += 1
    assert loads >= 4
