"""Writes tree_attn_wide.h beside this file: python3 tree_attn_wide_gen.py.

The header's blocks are schedules: which fragment of K or V is read when and into which registers, which wait lets
which MFMA go, where the softmax's arithmetic and the loads of a later tile stand between them. All of it follows
from the few numbers and rules below, so changes are made here. A test compares the header with what this writes and
goes through its instructions one by one."""
import os

QUADS = 8             # quads that the fragments of K and V pass through
AHEAD = QUADS - 1     # fragments read ahead of their use
K_FRAGS, V_FRAGS = 36, 32
SCORES, NEXT, WEIGHTS, QUAD0 = 192, 208, 184, 224   # v192: scores of tile i, scaled; of tile i + 1; weights; quads
BLOCK, HALF = 4096, 2048                            # LDS bytes of a 64-column block and of 16 of its rows


def quad(i):
    return QUAD0 + 4 * (i % QUADS)


def regs(first, count):
    return f"v[{first}:{first + count - 1}]"


def k_read(f, at):
    """K fragment f (16 of the row's columns) to quad `at`."""
    return f"ds_read_b128 {regs(quad(at), 4)}, %[k{f % 4}] offset:{f // 4 * BLOCK}"


def v_reads(j, at):
    """V^T fragment j: value columns 32 (j // 2) .., 16 rows of half j % 2; two reads of 8 rows."""
    n, c = j // 2, j % 2
    return [f"ds_read_b64_tr_b16 {regs(quad(at) + 2 * e, 2)}, %[v{e}{n & 1}] offset:{(n >> 1) * BLOCK + c * HALF}"
            for e in range(2)]


def mfma(out, a, b, c):
    return f"v_mfma_f32_32x32x16_bf16 {out}, {a}, {b}, {c}"


def wait(issued, use):
    """Wait until the last of `issued` that is `use` has come; LDS reads return in order."""
    after = len(issued) - 1 - max(i for i, x in enumerate(issued) if x == use)
    assert after <= 15
    return f"s_waitcnt lgkmcnt({after})"


def softmax():
    """Scores of tile i to weights 2^(s - m) in bf16, with m, top and l; an exponential's result and an exchange between
    lanes take states before they are used, which other arithmetic or an s_nop fills."""
    s = [f"v{SCORES + i}" for i in range(16)]
    out = [f"v_max3_f32 %[t0], {s[0]}, {s[1]}, {s[2]}", f"v_max3_f32 %[t1], {s[3]}, {s[4]}, {s[5]}"]
    for i in (6, 10):
        out += [f"v_max3_f32 %[t0], %[t0], {s[i]}, {s[i + 1]}", f"v_max3_f32 %[t1], %[t1], {s[i + 2]}, {s[i + 3]}"]
    out += [f"v_max3_f32 %[t0], %[t0], {s[14]}, {s[15]}", "v_max_f32 %[t0], %[t0], %[t1]", "v_mov_b32 %[t1], %[t0]",
            "s_nop 1", "v_permlane32_swap_b32 %[t0], %[t1]", "s_nop 1", "v_max_f32 %[t0], %[t0], %[t1]",
            "v_max_f32 %[top], %[top], %[t0]",
            "v_cmp_eq_f32 vcc, 0xff800000, %[m]", "s_nop 1", "v_cndmask_b32 %[m], %[m], %[t0], vcc",
            "v_cmp_eq_f32 vcc, 0xff800000, %[m]", "s_nop 1", "v_cndmask_b32_e64 %[t0], %[m], 0, vcc"]
    less = [f"v_sub_f32 {x}, {x}, %[t0]" for x in s]
    out += less[:3]
    for i in range(16):
        out.append(f"v_exp_f32 {s[i]}, {s[i]}")
        if i + 3 < 16:
            out.append(less[i + 3])
        if i == 2:
            out.append(f"v_add_f32 %[t1], {s[0]}, {s[1]}")
        if i > 2:
            out.append(f"v_add_f32 %[t1], %[t1], {s[i - 1]}")
        if i >= 3 and i % 2 == 1:
            out.append(f"v_cvt_pk_bf16_f32 v{WEIGHTS + (i - 3) // 2}, {s[i - 3]}, {s[i - 2]}")
    return out + ["s_nop 1", f"v_add_f32 %[t1], %[t1], {s[15]}", f"v_cvt_pk_bf16_f32 v{WEIGHTS + 7}, {s[14]}, {s[15]}",
                  "v_add_f32 %[l], %[l], %[t1]"]


def score_products(out, loads=0, between=(), values_next=False):
    """Scores into `out`, with `between` spread evenly over the MFMAs, `loads` direct loads of a later tile (five: the
    last one half a block), and the first V fragments read at the end."""
    lines, issued, between, done = [], [], list(between), 0
    for f in range(AHEAD):
        lines.append(k_read(f, f))
        issued.append(("k", f))
    for kk in range(K_FRAGS):
        ahead = kk + AHEAD
        if ahead < K_FRAGS:
            lines.append(k_read(ahead, ahead))
            issued.append(("k", ahead))
        elif values_next:
            for r in v_reads(ahead - K_FRAGS, ahead):
                lines.append(r)
                issued.append(("v", ahead - K_FRAGS))
        if kk % 4 == 2 and kk // 4 < loads:
            b = kk // 4
            lanes = "%[half]" if loads == 5 and b == 4 else "%[live]"
            # (the instruction's offset counts for the place in LDS too)
            lines += [f"s_add_u32 m0, %[to], {b * (BLOCK - 128)}", f"s_mov_b64 exec, {lanes}",
                      f"global_load_lds_dwordx4 %[src], off offset:{b * 128}", "s_mov_b64 exec, -1"]
        due = (len(between) * (kk + 2) + K_FRAGS - 1) // K_FRAGS
        lines += between[done:due]
        done = max(done, min(due, len(between)))
        lines += [wait(issued, ("k", kk)), mfma(out, regs(quad(kk), 4), f"%[q{kk}]", out if kk else "0")]
    return lines + between[done:]


def value_products():
    """O^T += V^T P^T; the first AHEAD fragments were read by score_products. The next tile's scores are scaled between."""
    first = K_FRAGS  # V fragment j passes through quad first + j
    lines, issued = [], [("v", j) for j in range(AHEAD) for _ in range(2)]
    scale = [f"v_mul_f32 v{SCORES + i}, %[c], v{NEXT + i}" for i in range(16)]
    for j in range(V_FRAGS):
        if j + AHEAD < V_FRAGS:
            for r in v_reads(j + AHEAD, first + j + AHEAD):
                lines.append(r)
                issued.append(("v", j + AHEAD))
        if j >= 6:  # the last score product's result has come
            lines, scale = lines + scale[:2], scale[2:]
        lines.append(wait(issued, ("v", j)))
        if j == 0:
            lines.append("s_nop 1")
        o = f"%[o{j // 2}]"
        lines.append(mfma(o, regs(quad(first + j), 4), regs(WEIGHTS + 4 * (j % 2), 4), o))
    assert not scale
    return lines


END = ["s_nop 15", "s_nop 1"]  # an MFMA's result may be read


def step(loads):
    return score_products(regs(NEXT, 16), loads, softmax(), True) + value_products() + END


def macro(name, lines):
    return f"#define {name} \\\n" + " \\\n".join(f'  "{x}\\n\\t"' for x in lines)


def header():
    named = [f'"v{i}"' for i in range(NEXT, 256)]
    clobbers = " \\\n".join("  " + ", ".join(named[i:i + 12]) + ("," if i + 12 < len(named) else "")
                            for i in range(0, len(named), 12))
    return f'''// The products of a 576/512-wide tile for one wave, written out (by
// tree_attn_wide_gen.py, where changes are made).
//
// A wave that owns 32 query rows holds 144 registers of Q and 256 of O: all
// accumulation registers and more than half of the others, and the wave is alone
// on its SIMD, so nothing but its own instructions can fill the time that its
// loads and its softmax take. Left to itself the compiler moved O about (225
// moves and 77 spills a tile). Here
//  - the fragments of K and V pass through eight fixed quads, v224 to v255, each
//    read {AHEAD} fragments (about 220 cycles of MFMA) ahead of its use. LDS reads
//    return in order, so a wait names how many may still be under way;
//  - WIDE_STEP takes the softmax of tile i and the score products of tile i + 1
//    together, two or three arithmetic instructions to an MFMA, then the value
//    products of tile i;
//  - the loads of a later tile are spread over the score
//    products: 16 bytes a lane of each 64-column block. An instruction's offset
//    counts for its address and for its place in LDS.
// A block ends with all its LDS reads returned and with the states that
// arithmetic has to wait for an MFMA's result, so what the compiler puts between
// blocks cannot meet either.
//
// Operands: k0..k3 the four chunk offsets of K within a 64-column block, v00,
// v01, v10, v11 those of V ([8-row group][column half]), as LDS addresses; q0..
// q35 Q, o0..o15 O^T; c the scale; m, top, l as in tree_attn.hip; t0, t1 any.
// Scores of a tile are v192 to v207 between blocks, scaled; v208 to v223 those of
// the next; v184 to v191 the weights as bf16.
#pragma once

// The registers that the blocks use by name.
#define WIDE_CLOBBERS \\
{clobbers}

// Scores (s, not scaled) of a tile.
{macro("WIDE_SCORES", score_products("%[s]") + END)}

// Softmax and value products of tile i, scores of tile i + 1, loads of a later
// tile by the lanes in live (all or none: an instruction without lanes counts as
// one that has arrived, so waits name the same numbers to the end).
{macro("WIDE_STEP", step(9))}

// The same for a cache in 8 bits: a later tile's codes are loaded as they are,
// four blocks of 128 bytes a row and, by the lanes in half, half a block.
{macro("WIDE_STEP_MX", step(5))}
'''


if __name__ == "__main__":
    with open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "tree_attn_wide.h"), "w") as f:
        f.write(header())
