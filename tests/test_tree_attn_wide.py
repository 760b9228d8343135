"""The written-out products of the 576/512 attention, instruction by instruction, without a GPU: that every MFMA gets the
fragment it should after the wait that brings it, that no instruction reads a result before its states are over, and
that the arithmetic between them is the softmax."""
import importlib.util
import math
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_up_projection_amd", "csrc")


def header():
    with open(os.path.join(CSRC, "tree_attn_wide.h")) as f:
        return f.read()


def block(name):
    body = re.search(r"#define %s \\\n((?:.*\\\n)*.*)" % name, header()).group(1)
    return re.findall(r'"([^"]*?)\\n\\t"', body)


def operands(line):
    op, _, rest = line.partition(" ")
    return op, [x.strip() for x in re.split(r",(?![^\[]*\])", rest)]


def registers(text):
    """v7, v[4:7] or an operand's name -> its registers."""
    m = re.fullmatch(r"v\[(\d+):(\d+)\]", text)
    if m:
        return [f"v{i}" for i in range(int(m.group(1)), int(m.group(2)) + 1)]
    return [text] if re.fullmatch(r"v\d+|%\[\w+\]", text) else []


def test_the_header_is_what_the_generator_writes():
    spec = importlib.util.spec_from_file_location("tree_attn_wide_gen", os.path.join(CSRC, "tree_attn_wide_gen.py"))
    gen = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(gen)
    assert gen.header() == header()


@pytest.mark.parametrize("name,values", [("WIDE_SCORES", False), ("WIDE_STEP", True), ("WIDE_STEP_MX", True)])
def test_every_product_gets_its_fragment(name, values):
    holds, queue, scores, sums = {}, [], [], []
    for line in block(name):
        op, args = operands(line)
        if op.startswith("ds_read"):
            addr, _, offset = args[1].partition(" offset:")
            dst = registers(args[0])
            queue.append((dst, addr, int(offset)))
            for r in dst:
                holds[r] = None  # on its way
        elif op == "s_waitcnt":
            left = int(re.fullmatch(r"lgkmcnt\((\d+)\)", args[0]).group(1))
            assert left <= 15
            while len(queue) > left:  # LDS reads return in order
                dst, addr, offset = queue.pop(0)
                for i, r in enumerate(dst):
                    holds[r] = (addr, offset, i)
        elif op.startswith("v_mfma"):
            frag = [holds[r] for r in registers(args[1])]
            assert None not in frag, line
            if args[2].startswith("%[q"):
                kk = len(scores)
                assert args[2] == f"%[q{kk}]" and args[3] == (args[0] if kk else "0")
                assert frag == [(f"%[k{kk % 4}]", kk // 4 * 4096, i) for i in range(4)], line
                scores.append(args[0])
            else:
                j = len(sums)
                n, c = j // 2, j % 2
                at = (n >> 1) * 4096 + c * 2048
                assert args[0] == args[3] == f"%[o{n}]" and registers(args[2])[0] == f"v{184 + 4 * c}"
                assert frag == [(f"%[v{e}{n & 1}]", at, i) for e in range(2) for i in range(2)], line
                sums.append(line)
    assert not queue, "reads under way at the end"
    assert len(scores) == 36 and len(set(scores)) == 1 and len(sums) == (32 if values else 0)


@pytest.mark.parametrize("name", ["WIDE_SCORES", "WIDE_STEP", "WIDE_STEP_MX"])
def test_states_between_results_and_their_use(name):
    """In instructions, of which each is a state at least and s_nop n is n + 1: two from arithmetic to an MFMA or an
    exchange of lanes, eighteen from an MFMA to anything else (an MFMA that adds to the same sum needs none), one from
    an exponential, one from vcc's compare (and one that is kept for its mask)."""
    at, written = 0, {}
    for line in block(name):
        op, args = operands(line)
        swap = op.startswith("v_permlane32_swap")
        dst = registers(args[0]) if op.startswith(("v_", "ds_read")) else []
        src = [r for a in args[0 if swap else 1:] for r in registers(a.split(" ")[0])] if op.startswith("v_") else []
        if op.startswith("v_cmp"):
            dst = ["vcc"]
        if "vcc" in args[1:]:
            src.append("vcc")
        for r in src:
            if r not in written:
                continue
            when, by = written[r]
            states = at - when - 1
            if by.startswith("v_mfma"):
                assert op.startswith("v_mfma") or states >= 18, (line, r)
            elif op.startswith("v_mfma") or swap or by.startswith(("v_permlane", "v_cmp")):
                assert states >= 2, (line, r)
            elif by.startswith("v_exp"):
                assert states >= 1 or op.startswith("v_exp"), (line, r)
        for r in dst + (registers(args[1]) if swap else []):
            if r in written and written[r][1].startswith("v_mfma") and not op.startswith("v_mfma"):
                assert at - written[r][0] - 1 >= 18, (line, r)
            written[r] = (at, op)
        at += 1 + (int(args[0]) if op == "s_nop" else 0)
    last = max(when for when, by in written.values() if by.startswith("v_mfma"))
    assert at - last - 1 >= 18


@pytest.mark.parametrize("name,loads", [("WIDE_STEP", 9), ("WIDE_STEP_MX", 5)])
def test_loads_of_a_later_tile(name, loads):
    """One for each block of a row, to its place, and every lane back at work after each."""
    seen, m0, lanes = [], None, "-1"
    for line in block(name):
        op, args = operands(line)
        if op == "s_add_u32":
            assert args[:2] == ["m0", "%[to]"]
            m0 = int(args[2])
        elif op == "s_mov_b64":
            lanes = args[1]
        elif op == "global_load_lds_dwordx4":
            offset = int(args[1].split("offset:")[1])
            seen.append((offset, m0 + offset, lanes))
        else:
            assert lanes == "-1", line
    assert lanes == "-1"
    want = [(128 * b, 4096 * b, "%[half]" if loads == 5 and b == 4 else "%[live]") for b in range(loads)]
    assert seen == want


def bf16(x):
    import numpy as np
    u = int(np.float32(x).view(np.uint32))
    return (u + 0x7FFF + ((u >> 16) & 1)) >> 16


@pytest.mark.parametrize("name", ["WIDE_STEP", "WIDE_STEP_MX"])
@pytest.mark.parametrize("m", [-math.inf, 2.0, -3.5])
def test_the_arithmetic_is_the_softmax(name, m):
    """Two lanes (the halves of one query row) through the block, all but the MFMAs carried out."""
    import random
    rng = random.Random(5)
    scores = [[rng.uniform(-6, 6) for _ in range(16)] for _ in range(2)]
    scores[0][3] = scores[1][0] = -math.inf
    nxt = [[rng.uniform(-60, 60) for _ in range(16)] for _ in range(2)]
    top, l, c = 1.25, 3.0, 0.0625
    lanes = []
    for half in range(2):
        r = {f"v{192 + i}": scores[half][i] for i in range(16)} | {f"v{208 + i}": nxt[half][i] for i in range(16)}
        lanes.append(r | {"%[m]": m, "%[top]": top, "%[l]": l, "%[c]": c, "0": 0.0, "0xff800000": -math.inf})
    for line in block(name):
        op, a = operands(line)
        if not op.startswith("v_") or op.startswith("v_mfma"):
            continue
        if op.startswith("v_permlane32_swap"):  # the upper half of the first with the lower half of the second
            lanes[1][a[0]], lanes[0][a[1]] = lanes[0][a[1]], lanes[1][a[0]]
            continue
        for r in lanes:
            if op == "v_max3_f32":
                r[a[0]] = max(r[a[1]], r[a[2]], r[a[3]])
            elif op == "v_max_f32":
                r[a[0]] = max(r[a[1]], r[a[2]])
            elif op == "v_mov_b32":
                r[a[0]] = r[a[1]]
            elif op == "v_cmp_eq_f32":
                r["vcc"] = r[a[1]] == r[a[2]]
            elif op.startswith("v_cndmask_b32"):
                r[a[0]] = r[a[2]] if r["vcc"] else r[a[1]]
            elif op == "v_sub_f32":
                r[a[0]] = r[a[1]] - r[a[2]]
            elif op == "v_add_f32":
                r[a[0]] = r[a[1]] + r[a[2]]
            elif op == "v_mul_f32":
                r[a[0]] = r[a[1]] * r[a[2]]
            elif op == "v_exp_f32":
                r[a[0]] = 2.0 ** r[a[1]]
            elif op == "v_cvt_pk_bf16_f32":
                r[a[0]] = (bf16(r[a[1]]), bf16(r[a[2]]))
            else:
                raise AssertionError(line)
    high = max(scores[0] + scores[1])
    ref = high if m == -math.inf else m
    for half, r in enumerate(lanes):
        w = [2.0 ** (s - ref) for s in scores[half]]
        assert r["%[m]"] == ref and r["%[top]"] == max(top, high)
        assert math.isclose(r["%[l]"], l + sum(w), rel_tol=1e-12)
        for i in range(8):
            got = r[f"v{184 + i}"]
            assert all(abs(g - bf16(x)) <= 1 for g, x in zip(got, w[2 * i: 2 * i + 2]))
        for i in range(16):
            assert r[f"v{192 + i}"] == nxt[half][i] * c
