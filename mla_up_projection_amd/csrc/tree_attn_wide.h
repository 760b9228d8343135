// The products of a 576/512-wide tile for one wave, written out (by
// tree_attn_wide_gen.py, where changes are made).
//
// A wave that owns 32 query rows holds 144 registers of Q and 256 of O: all
// accumulation registers and more than half of the others, and the wave is alone
// on its SIMD, so nothing but its own instructions can fill the time that its
// loads and its softmax take. Left to itself the compiler moved O about (225
// moves and 77 spills a tile). Here
//  - the fragments of K and V pass through eight fixed quads, v224 to v255, each
//    read 7 fragments (about 220 cycles of MFMA) ahead of its use. LDS reads
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
#define WIDE_CLOBBERS \
  "v208", "v209", "v210", "v211", "v212", "v213", "v214", "v215", "v216", "v217", "v218", "v219", \
  "v220", "v221", "v222", "v223", "v224", "v225", "v226", "v227", "v228", "v229", "v230", "v231", \
  "v232", "v233", "v234", "v235", "v236", "v237", "v238", "v239", "v240", "v241", "v242", "v243", \
  "v244", "v245", "v246", "v247", "v248", "v249", "v250", "v251", "v252", "v253", "v254", "v255"

// Scores (s, not scaled) of a tile.
#define WIDE_SCORES \
  "ds_read_b128 v[224:227], %[k0] offset:0\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:0\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:0\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:0\n\t" \
  "ds_read_b128 v[240:243], %[k0] offset:4096\n\t" \
  "ds_read_b128 v[244:247], %[k1] offset:4096\n\t" \
  "ds_read_b128 v[248:251], %[k2] offset:4096\n\t" \
  "ds_read_b128 v[252:255], %[k3] offset:4096\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[224:227], %[q0], 0\n\t" \
  "ds_read_b128 v[224:227], %[k0] offset:8192\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[228:231], %[q1], %[s]\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:8192\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[232:235], %[q2], %[s]\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:8192\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[236:239], %[q3], %[s]\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:8192\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[240:243], %[q4], %[s]\n\t" \
  "ds_read_b128 v[240:243], %[k0] offset:12288\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[244:247], %[q5], %[s]\n\t" \
  "ds_read_b128 v[244:247], %[k1] offset:12288\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[248:251], %[q6], %[s]\n\t" \
  "ds_read_b128 v[248:251], %[k2] offset:12288\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[252:255], %[q7], %[s]\n\t" \
  "ds_read_b128 v[252:255], %[k3] offset:12288\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[224:227], %[q8], %[s]\n\t" \
  "ds_read_b128 v[224:227], %[k0] offset:16384\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[228:231], %[q9], %[s]\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:16384\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[232:235], %[q10], %[s]\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:16384\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[236:239], %[q11], %[s]\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:16384\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[240:243], %[q12], %[s]\n\t" \
  "ds_read_b128 v[240:243], %[k0] offset:20480\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[244:247], %[q13], %[s]\n\t" \
  "ds_read_b128 v[244:247], %[k1] offset:20480\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[248:251], %[q14], %[s]\n\t" \
  "ds_read_b128 v[248:251], %[k2] offset:20480\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[252:255], %[q15], %[s]\n\t" \
  "ds_read_b128 v[252:255], %[k3] offset:20480\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[224:227], %[q16], %[s]\n\t" \
  "ds_read_b128 v[224:227], %[k0] offset:24576\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[228:231], %[q17], %[s]\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:24576\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[232:235], %[q18], %[s]\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:24576\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[236:239], %[q19], %[s]\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:24576\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[240:243], %[q20], %[s]\n\t" \
  "ds_read_b128 v[240:243], %[k0] offset:28672\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[244:247], %[q21], %[s]\n\t" \
  "ds_read_b128 v[244:247], %[k1] offset:28672\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[248:251], %[q22], %[s]\n\t" \
  "ds_read_b128 v[248:251], %[k2] offset:28672\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[252:255], %[q23], %[s]\n\t" \
  "ds_read_b128 v[252:255], %[k3] offset:28672\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[224:227], %[q24], %[s]\n\t" \
  "ds_read_b128 v[224:227], %[k0] offset:32768\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[228:231], %[q25], %[s]\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:32768\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[232:235], %[q26], %[s]\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:32768\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[236:239], %[q27], %[s]\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:32768\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[240:243], %[q28], %[s]\n\t" \
  "s_waitcnt lgkmcnt(6)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[244:247], %[q29], %[s]\n\t" \
  "s_waitcnt lgkmcnt(5)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[248:251], %[q30], %[s]\n\t" \
  "s_waitcnt lgkmcnt(4)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[252:255], %[q31], %[s]\n\t" \
  "s_waitcnt lgkmcnt(3)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[224:227], %[q32], %[s]\n\t" \
  "s_waitcnt lgkmcnt(2)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[228:231], %[q33], %[s]\n\t" \
  "s_waitcnt lgkmcnt(1)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[232:235], %[q34], %[s]\n\t" \
  "s_waitcnt lgkmcnt(0)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[236:239], %[q35], %[s]\n\t" \
  "s_nop 15\n\t" \
  "s_nop 1\n\t"

// Softmax and value products of tile i, scores of tile i + 1, loads of a later
// tile by the lanes in live (all or none: an instruction without lanes counts as
// one that has arrived, so waits name the same numbers to the end).
#define WIDE_STEP \
  "ds_read_b128 v[224:227], %[k0] offset:0\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:0\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:0\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:0\n\t" \
  "ds_read_b128 v[240:243], %[k0] offset:4096\n\t" \
  "ds_read_b128 v[244:247], %[k1] offset:4096\n\t" \
  "ds_read_b128 v[248:251], %[k2] offset:4096\n\t" \
  "ds_read_b128 v[252:255], %[k3] offset:4096\n\t" \
  "v_max3_f32 %[t0], v192, v193, v194\n\t" \
  "v_max3_f32 %[t1], v195, v196, v197\n\t" \
  "v_max3_f32 %[t0], %[t0], v198, v199\n\t" \
  "v_max3_f32 %[t1], %[t1], v200, v201\n\t" \
  "v_max3_f32 %[t0], %[t0], v202, v203\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[224:227], %[q0], 0\n\t" \
  "ds_read_b128 v[224:227], %[k0] offset:8192\n\t" \
  "v_max3_f32 %[t1], %[t1], v204, v205\n\t" \
  "v_max3_f32 %[t0], %[t0], v206, v207\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[228:231], %[q1], v[208:223]\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:8192\n\t" \
  "s_add_u32 m0, %[to], 0\n\t" \
  "s_mov_b64 exec, %[live]\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:0\n\t" \
  "s_mov_b64 exec, -1\n\t" \
  "v_max_f32 %[t0], %[t0], %[t1]\n\t" \
  "v_mov_b32 %[t1], %[t0]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[232:235], %[q2], v[208:223]\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:8192\n\t" \
  "s_nop 1\n\t" \
  "v_permlane32_swap_b32 %[t0], %[t1]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[236:239], %[q3], v[208:223]\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:8192\n\t" \
  "s_nop 1\n\t" \
  "v_max_f32 %[t0], %[t0], %[t1]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[240:243], %[q4], v[208:223]\n\t" \
  "ds_read_b128 v[240:243], %[k0] offset:12288\n\t" \
  "v_max_f32 %[top], %[top], %[t0]\n\t" \
  "v_cmp_eq_f32 vcc, 0xff800000, %[m]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[244:247], %[q5], v[208:223]\n\t" \
  "ds_read_b128 v[244:247], %[k1] offset:12288\n\t" \
  "s_add_u32 m0, %[to], 3968\n\t" \
  "s_mov_b64 exec, %[live]\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:128\n\t" \
  "s_mov_b64 exec, -1\n\t" \
  "s_nop 1\n\t" \
  "v_cndmask_b32 %[m], %[m], %[t0], vcc\n\t" \
  "v_cmp_eq_f32 vcc, 0xff800000, %[m]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[248:251], %[q6], v[208:223]\n\t" \
  "ds_read_b128 v[248:251], %[k2] offset:12288\n\t" \
  "s_nop 1\n\t" \
  "v_cndmask_b32_e64 %[t0], %[m], 0, vcc\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[252:255], %[q7], v[208:223]\n\t" \
  "ds_read_b128 v[252:255], %[k3] offset:12288\n\t" \
  "v_sub_f32 v192, v192, %[t0]\n\t" \
  "v_sub_f32 v193, v193, %[t0]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[224:227], %[q8], v[208:223]\n\t" \
  "ds_read_b128 v[224:227], %[k0] offset:16384\n\t" \
  "v_sub_f32 v194, v194, %[t0]\n\t" \
  "v_exp_f32 v192, v192\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[228:231], %[q9], v[208:223]\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:16384\n\t" \
  "s_add_u32 m0, %[to], 7936\n\t" \
  "s_mov_b64 exec, %[live]\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:256\n\t" \
  "s_mov_b64 exec, -1\n\t" \
  "v_sub_f32 v195, v195, %[t0]\n\t" \
  "v_exp_f32 v193, v193\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[232:235], %[q10], v[208:223]\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:16384\n\t" \
  "v_sub_f32 v196, v196, %[t0]\n\t" \
  "v_exp_f32 v194, v194\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[236:239], %[q11], v[208:223]\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:16384\n\t" \
  "v_sub_f32 v197, v197, %[t0]\n\t" \
  "v_add_f32 %[t1], v192, v193\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[240:243], %[q12], v[208:223]\n\t" \
  "ds_read_b128 v[240:243], %[k0] offset:20480\n\t" \
  "v_exp_f32 v195, v195\n\t" \
  "v_sub_f32 v198, v198, %[t0]\n\t" \
  "v_add_f32 %[t1], %[t1], v194\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[244:247], %[q13], v[208:223]\n\t" \
  "ds_read_b128 v[244:247], %[k1] offset:20480\n\t" \
  "s_add_u32 m0, %[to], 11904\n\t" \
  "s_mov_b64 exec, %[live]\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:384\n\t" \
  "s_mov_b64 exec, -1\n\t" \
  "v_cvt_pk_bf16_f32 v184, v192, v193\n\t" \
  "v_exp_f32 v196, v196\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[248:251], %[q14], v[208:223]\n\t" \
  "ds_read_b128 v[248:251], %[k2] offset:20480\n\t" \
  "v_sub_f32 v199, v199, %[t0]\n\t" \
  "v_add_f32 %[t1], %[t1], v195\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[252:255], %[q15], v[208:223]\n\t" \
  "ds_read_b128 v[252:255], %[k3] offset:20480\n\t" \
  "v_exp_f32 v197, v197\n\t" \
  "v_sub_f32 v200, v200, %[t0]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[224:227], %[q16], v[208:223]\n\t" \
  "ds_read_b128 v[224:227], %[k0] offset:24576\n\t" \
  "v_add_f32 %[t1], %[t1], v196\n\t" \
  "v_cvt_pk_bf16_f32 v185, v194, v195\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[228:231], %[q17], v[208:223]\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:24576\n\t" \
  "s_add_u32 m0, %[to], 15872\n\t" \
  "s_mov_b64 exec, %[live]\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:512\n\t" \
  "s_mov_b64 exec, -1\n\t" \
  "v_exp_f32 v198, v198\n\t" \
  "v_sub_f32 v201, v201, %[t0]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[232:235], %[q18], v[208:223]\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:24576\n\t" \
  "v_add_f32 %[t1], %[t1], v197\n\t" \
  "v_exp_f32 v199, v199\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[236:239], %[q19], v[208:223]\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:24576\n\t" \
  "v_sub_f32 v202, v202, %[t0]\n\t" \
  "v_add_f32 %[t1], %[t1], v198\n\t" \
  "v_cvt_pk_bf16_f32 v186, v196, v197\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[240:243], %[q20], v[208:223]\n\t" \
  "ds_read_b128 v[240:243], %[k0] offset:28672\n\t" \
  "v_exp_f32 v200, v200\n\t" \
  "v_sub_f32 v203, v203, %[t0]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[244:247], %[q21], v[208:223]\n\t" \
  "ds_read_b128 v[244:247], %[k1] offset:28672\n\t" \
  "s_add_u32 m0, %[to], 19840\n\t" \
  "s_mov_b64 exec, %[live]\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:640\n\t" \
  "s_mov_b64 exec, -1\n\t" \
  "v_add_f32 %[t1], %[t1], v199\n\t" \
  "v_exp_f32 v201, v201\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[248:251], %[q22], v[208:223]\n\t" \
  "ds_read_b128 v[248:251], %[k2] offset:28672\n\t" \
  "v_sub_f32 v204, v204, %[t0]\n\t" \
  "v_add_f32 %[t1], %[t1], v200\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[252:255], %[q23], v[208:223]\n\t" \
  "ds_read_b128 v[252:255], %[k3] offset:28672\n\t" \
  "v_cvt_pk_bf16_f32 v187, v198, v199\n\t" \
  "v_exp_f32 v202, v202\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[224:227], %[q24], v[208:223]\n\t" \
  "ds_read_b128 v[224:227], %[k0] offset:32768\n\t" \
  "v_sub_f32 v205, v205, %[t0]\n\t" \
  "v_add_f32 %[t1], %[t1], v201\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[228:231], %[q25], v[208:223]\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:32768\n\t" \
  "s_add_u32 m0, %[to], 23808\n\t" \
  "s_mov_b64 exec, %[live]\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:768\n\t" \
  "s_mov_b64 exec, -1\n\t" \
  "v_exp_f32 v203, v203\n\t" \
  "v_sub_f32 v206, v206, %[t0]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[232:235], %[q26], v[208:223]\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:32768\n\t" \
  "v_add_f32 %[t1], %[t1], v202\n\t" \
  "v_cvt_pk_bf16_f32 v188, v200, v201\n\t" \
  "v_exp_f32 v204, v204\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[236:239], %[q27], v[208:223]\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:32768\n\t" \
  "v_sub_f32 v207, v207, %[t0]\n\t" \
  "v_add_f32 %[t1], %[t1], v203\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[240:243], %[q28], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[240:241], %[v00] offset:0\n\t" \
  "ds_read_b64_tr_b16 v[242:243], %[v10] offset:0\n\t" \
  "v_exp_f32 v205, v205\n\t" \
  "v_add_f32 %[t1], %[t1], v204\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[244:247], %[q29], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[244:245], %[v00] offset:2048\n\t" \
  "ds_read_b64_tr_b16 v[246:247], %[v10] offset:2048\n\t" \
  "s_add_u32 m0, %[to], 27776\n\t" \
  "s_mov_b64 exec, %[live]\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:896\n\t" \
  "s_mov_b64 exec, -1\n\t" \
  "v_cvt_pk_bf16_f32 v189, v202, v203\n\t" \
  "v_exp_f32 v206, v206\n\t" \
  "s_waitcnt lgkmcnt(9)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[248:251], %[q30], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[248:249], %[v01] offset:0\n\t" \
  "ds_read_b64_tr_b16 v[250:251], %[v11] offset:0\n\t" \
  "v_add_f32 %[t1], %[t1], v205\n\t" \
  "v_exp_f32 v207, v207\n\t" \
  "s_waitcnt lgkmcnt(10)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[252:255], %[q31], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[252:253], %[v01] offset:2048\n\t" \
  "ds_read_b64_tr_b16 v[254:255], %[v11] offset:2048\n\t" \
  "v_add_f32 %[t1], %[t1], v206\n\t" \
  "v_cvt_pk_bf16_f32 v190, v204, v205\n\t" \
  "s_waitcnt lgkmcnt(11)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[224:227], %[q32], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[224:225], %[v00] offset:4096\n\t" \
  "ds_read_b64_tr_b16 v[226:227], %[v10] offset:4096\n\t" \
  "s_nop 1\n\t" \
  "v_add_f32 %[t1], %[t1], v207\n\t" \
  "s_waitcnt lgkmcnt(12)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[228:231], %[q33], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[228:229], %[v00] offset:6144\n\t" \
  "ds_read_b64_tr_b16 v[230:231], %[v10] offset:6144\n\t" \
  "s_add_u32 m0, %[to], 31744\n\t" \
  "s_mov_b64 exec, %[live]\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:1024\n\t" \
  "s_mov_b64 exec, -1\n\t" \
  "v_cvt_pk_bf16_f32 v191, v206, v207\n\t" \
  "v_add_f32 %[l], %[l], %[t1]\n\t" \
  "s_waitcnt lgkmcnt(13)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[232:235], %[q34], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[232:233], %[v01] offset:4096\n\t" \
  "ds_read_b64_tr_b16 v[234:235], %[v11] offset:4096\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[236:239], %[q35], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[236:237], %[v01] offset:6144\n\t" \
  "ds_read_b64_tr_b16 v[238:239], %[v11] offset:6144\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "s_nop 1\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o0], v[240:243], v[184:187], %[o0]\n\t" \
  "ds_read_b64_tr_b16 v[240:241], %[v00] offset:8192\n\t" \
  "ds_read_b64_tr_b16 v[242:243], %[v10] offset:8192\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o0], v[244:247], v[188:191], %[o0]\n\t" \
  "ds_read_b64_tr_b16 v[244:245], %[v00] offset:10240\n\t" \
  "ds_read_b64_tr_b16 v[246:247], %[v10] offset:10240\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o1], v[248:251], v[184:187], %[o1]\n\t" \
  "ds_read_b64_tr_b16 v[248:249], %[v01] offset:8192\n\t" \
  "ds_read_b64_tr_b16 v[250:251], %[v11] offset:8192\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o1], v[252:255], v[188:191], %[o1]\n\t" \
  "ds_read_b64_tr_b16 v[252:253], %[v01] offset:10240\n\t" \
  "ds_read_b64_tr_b16 v[254:255], %[v11] offset:10240\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o2], v[224:227], v[184:187], %[o2]\n\t" \
  "ds_read_b64_tr_b16 v[224:225], %[v00] offset:12288\n\t" \
  "ds_read_b64_tr_b16 v[226:227], %[v10] offset:12288\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o2], v[228:231], v[188:191], %[o2]\n\t" \
  "ds_read_b64_tr_b16 v[228:229], %[v00] offset:14336\n\t" \
  "ds_read_b64_tr_b16 v[230:231], %[v10] offset:14336\n\t" \
  "v_mul_f32 v192, %[c], v208\n\t" \
  "v_mul_f32 v193, %[c], v209\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o3], v[232:235], v[184:187], %[o3]\n\t" \
  "ds_read_b64_tr_b16 v[232:233], %[v01] offset:12288\n\t" \
  "ds_read_b64_tr_b16 v[234:235], %[v11] offset:12288\n\t" \
  "v_mul_f32 v194, %[c], v210\n\t" \
  "v_mul_f32 v195, %[c], v211\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o3], v[236:239], v[188:191], %[o3]\n\t" \
  "ds_read_b64_tr_b16 v[236:237], %[v01] offset:14336\n\t" \
  "ds_read_b64_tr_b16 v[238:239], %[v11] offset:14336\n\t" \
  "v_mul_f32 v196, %[c], v212\n\t" \
  "v_mul_f32 v197, %[c], v213\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o4], v[240:243], v[184:187], %[o4]\n\t" \
  "ds_read_b64_tr_b16 v[240:241], %[v00] offset:16384\n\t" \
  "ds_read_b64_tr_b16 v[242:243], %[v10] offset:16384\n\t" \
  "v_mul_f32 v198, %[c], v214\n\t" \
  "v_mul_f32 v199, %[c], v215\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o4], v[244:247], v[188:191], %[o4]\n\t" \
  "ds_read_b64_tr_b16 v[244:245], %[v00] offset:18432\n\t" \
  "ds_read_b64_tr_b16 v[246:247], %[v10] offset:18432\n\t" \
  "v_mul_f32 v200, %[c], v216\n\t" \
  "v_mul_f32 v201, %[c], v217\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o5], v[248:251], v[184:187], %[o5]\n\t" \
  "ds_read_b64_tr_b16 v[248:249], %[v01] offset:16384\n\t" \
  "ds_read_b64_tr_b16 v[250:251], %[v11] offset:16384\n\t" \
  "v_mul_f32 v202, %[c], v218\n\t" \
  "v_mul_f32 v203, %[c], v219\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o5], v[252:255], v[188:191], %[o5]\n\t" \
  "ds_read_b64_tr_b16 v[252:253], %[v01] offset:18432\n\t" \
  "ds_read_b64_tr_b16 v[254:255], %[v11] offset:18432\n\t" \
  "v_mul_f32 v204, %[c], v220\n\t" \
  "v_mul_f32 v205, %[c], v221\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o6], v[224:227], v[184:187], %[o6]\n\t" \
  "ds_read_b64_tr_b16 v[224:225], %[v00] offset:20480\n\t" \
  "ds_read_b64_tr_b16 v[226:227], %[v10] offset:20480\n\t" \
  "v_mul_f32 v206, %[c], v222\n\t" \
  "v_mul_f32 v207, %[c], v223\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o6], v[228:231], v[188:191], %[o6]\n\t" \
  "ds_read_b64_tr_b16 v[228:229], %[v00] offset:22528\n\t" \
  "ds_read_b64_tr_b16 v[230:231], %[v10] offset:22528\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o7], v[232:235], v[184:187], %[o7]\n\t" \
  "ds_read_b64_tr_b16 v[232:233], %[v01] offset:20480\n\t" \
  "ds_read_b64_tr_b16 v[234:235], %[v11] offset:20480\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o7], v[236:239], v[188:191], %[o7]\n\t" \
  "ds_read_b64_tr_b16 v[236:237], %[v01] offset:22528\n\t" \
  "ds_read_b64_tr_b16 v[238:239], %[v11] offset:22528\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o8], v[240:243], v[184:187], %[o8]\n\t" \
  "ds_read_b64_tr_b16 v[240:241], %[v00] offset:24576\n\t" \
  "ds_read_b64_tr_b16 v[242:243], %[v10] offset:24576\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o8], v[244:247], v[188:191], %[o8]\n\t" \
  "ds_read_b64_tr_b16 v[244:245], %[v00] offset:26624\n\t" \
  "ds_read_b64_tr_b16 v[246:247], %[v10] offset:26624\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o9], v[248:251], v[184:187], %[o9]\n\t" \
  "ds_read_b64_tr_b16 v[248:249], %[v01] offset:24576\n\t" \
  "ds_read_b64_tr_b16 v[250:251], %[v11] offset:24576\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o9], v[252:255], v[188:191], %[o9]\n\t" \
  "ds_read_b64_tr_b16 v[252:253], %[v01] offset:26624\n\t" \
  "ds_read_b64_tr_b16 v[254:255], %[v11] offset:26624\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o10], v[224:227], v[184:187], %[o10]\n\t" \
  "ds_read_b64_tr_b16 v[224:225], %[v00] offset:28672\n\t" \
  "ds_read_b64_tr_b16 v[226:227], %[v10] offset:28672\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o10], v[228:231], v[188:191], %[o10]\n\t" \
  "ds_read_b64_tr_b16 v[228:229], %[v00] offset:30720\n\t" \
  "ds_read_b64_tr_b16 v[230:231], %[v10] offset:30720\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o11], v[232:235], v[184:187], %[o11]\n\t" \
  "ds_read_b64_tr_b16 v[232:233], %[v01] offset:28672\n\t" \
  "ds_read_b64_tr_b16 v[234:235], %[v11] offset:28672\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o11], v[236:239], v[188:191], %[o11]\n\t" \
  "ds_read_b64_tr_b16 v[236:237], %[v01] offset:30720\n\t" \
  "ds_read_b64_tr_b16 v[238:239], %[v11] offset:30720\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o12], v[240:243], v[184:187], %[o12]\n\t" \
  "s_waitcnt lgkmcnt(12)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o12], v[244:247], v[188:191], %[o12]\n\t" \
  "s_waitcnt lgkmcnt(10)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o13], v[248:251], v[184:187], %[o13]\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o13], v[252:255], v[188:191], %[o13]\n\t" \
  "s_waitcnt lgkmcnt(6)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o14], v[224:227], v[184:187], %[o14]\n\t" \
  "s_waitcnt lgkmcnt(4)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o14], v[228:231], v[188:191], %[o14]\n\t" \
  "s_waitcnt lgkmcnt(2)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o15], v[232:235], v[184:187], %[o15]\n\t" \
  "s_waitcnt lgkmcnt(0)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o15], v[236:239], v[188:191], %[o15]\n\t" \
  "s_nop 15\n\t" \
  "s_nop 1\n\t"

// The same for a cache in 8 bits: a later tile's codes are loaded as they are,
// four blocks of 128 bytes a row and, by the lanes in half, half a block.
#define WIDE_STEP_MX \
  "ds_read_b128 v[224:227], %[k0] offset:0\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:0\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:0\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:0\n\t" \
  "ds_read_b128 v[240:243], %[k0] offset:4096\n\t" \
  "ds_read_b128 v[244:247], %[k1] offset:4096\n\t" \
  "ds_read_b128 v[248:251], %[k2] offset:4096\n\t" \
  "ds_read_b128 v[252:255], %[k3] offset:4096\n\t" \
  "v_max3_f32 %[t0], v192, v193, v194\n\t" \
  "v_max3_f32 %[t1], v195, v196, v197\n\t" \
  "v_max3_f32 %[t0], %[t0], v198, v199\n\t" \
  "v_max3_f32 %[t1], %[t1], v200, v201\n\t" \
  "v_max3_f32 %[t0], %[t0], v202, v203\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[224:227], %[q0], 0\n\t" \
  "ds_read_b128 v[224:227], %[k0] offset:8192\n\t" \
  "v_max3_f32 %[t1], %[t1], v204, v205\n\t" \
  "v_max3_f32 %[t0], %[t0], v206, v207\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[228:231], %[q1], v[208:223]\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:8192\n\t" \
  "s_add_u32 m0, %[to], 0\n\t" \
  "s_mov_b64 exec, %[live]\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:0\n\t" \
  "s_mov_b64 exec, -1\n\t" \
  "v_max_f32 %[t0], %[t0], %[t1]\n\t" \
  "v_mov_b32 %[t1], %[t0]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[232:235], %[q2], v[208:223]\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:8192\n\t" \
  "s_nop 1\n\t" \
  "v_permlane32_swap_b32 %[t0], %[t1]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[236:239], %[q3], v[208:223]\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:8192\n\t" \
  "s_nop 1\n\t" \
  "v_max_f32 %[t0], %[t0], %[t1]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[240:243], %[q4], v[208:223]\n\t" \
  "ds_read_b128 v[240:243], %[k0] offset:12288\n\t" \
  "v_max_f32 %[top], %[top], %[t0]\n\t" \
  "v_cmp_eq_f32 vcc, 0xff800000, %[m]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[244:247], %[q5], v[208:223]\n\t" \
  "ds_read_b128 v[244:247], %[k1] offset:12288\n\t" \
  "s_add_u32 m0, %[to], 3968\n\t" \
  "s_mov_b64 exec, %[live]\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:128\n\t" \
  "s_mov_b64 exec, -1\n\t" \
  "s_nop 1\n\t" \
  "v_cndmask_b32 %[m], %[m], %[t0], vcc\n\t" \
  "v_cmp_eq_f32 vcc, 0xff800000, %[m]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[248:251], %[q6], v[208:223]\n\t" \
  "ds_read_b128 v[248:251], %[k2] offset:12288\n\t" \
  "s_nop 1\n\t" \
  "v_cndmask_b32_e64 %[t0], %[m], 0, vcc\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[252:255], %[q7], v[208:223]\n\t" \
  "ds_read_b128 v[252:255], %[k3] offset:12288\n\t" \
  "v_sub_f32 v192, v192, %[t0]\n\t" \
  "v_sub_f32 v193, v193, %[t0]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[224:227], %[q8], v[208:223]\n\t" \
  "ds_read_b128 v[224:227], %[k0] offset:16384\n\t" \
  "v_sub_f32 v194, v194, %[t0]\n\t" \
  "v_exp_f32 v192, v192\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[228:231], %[q9], v[208:223]\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:16384\n\t" \
  "s_add_u32 m0, %[to], 7936\n\t" \
  "s_mov_b64 exec, %[live]\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:256\n\t" \
  "s_mov_b64 exec, -1\n\t" \
  "v_sub_f32 v195, v195, %[t0]\n\t" \
  "v_exp_f32 v193, v193\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[232:235], %[q10], v[208:223]\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:16384\n\t" \
  "v_sub_f32 v196, v196, %[t0]\n\t" \
  "v_exp_f32 v194, v194\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[236:239], %[q11], v[208:223]\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:16384\n\t" \
  "v_sub_f32 v197, v197, %[t0]\n\t" \
  "v_add_f32 %[t1], v192, v193\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[240:243], %[q12], v[208:223]\n\t" \
  "ds_read_b128 v[240:243], %[k0] offset:20480\n\t" \
  "v_exp_f32 v195, v195\n\t" \
  "v_sub_f32 v198, v198, %[t0]\n\t" \
  "v_add_f32 %[t1], %[t1], v194\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[244:247], %[q13], v[208:223]\n\t" \
  "ds_read_b128 v[244:247], %[k1] offset:20480\n\t" \
  "s_add_u32 m0, %[to], 11904\n\t" \
  "s_mov_b64 exec, %[live]\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:384\n\t" \
  "s_mov_b64 exec, -1\n\t" \
  "v_cvt_pk_bf16_f32 v184, v192, v193\n\t" \
  "v_exp_f32 v196, v196\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[248:251], %[q14], v[208:223]\n\t" \
  "ds_read_b128 v[248:251], %[k2] offset:20480\n\t" \
  "v_sub_f32 v199, v199, %[t0]\n\t" \
  "v_add_f32 %[t1], %[t1], v195\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[252:255], %[q15], v[208:223]\n\t" \
  "ds_read_b128 v[252:255], %[k3] offset:20480\n\t" \
  "v_exp_f32 v197, v197\n\t" \
  "v_sub_f32 v200, v200, %[t0]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[224:227], %[q16], v[208:223]\n\t" \
  "ds_read_b128 v[224:227], %[k0] offset:24576\n\t" \
  "v_add_f32 %[t1], %[t1], v196\n\t" \
  "v_cvt_pk_bf16_f32 v185, v194, v195\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[228:231], %[q17], v[208:223]\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:24576\n\t" \
  "s_add_u32 m0, %[to], 15872\n\t" \
  "s_mov_b64 exec, %[half]\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:512\n\t" \
  "s_mov_b64 exec, -1\n\t" \
  "v_exp_f32 v198, v198\n\t" \
  "v_sub_f32 v201, v201, %[t0]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[232:235], %[q18], v[208:223]\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:24576\n\t" \
  "v_add_f32 %[t1], %[t1], v197\n\t" \
  "v_exp_f32 v199, v199\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[236:239], %[q19], v[208:223]\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:24576\n\t" \
  "v_sub_f32 v202, v202, %[t0]\n\t" \
  "v_add_f32 %[t1], %[t1], v198\n\t" \
  "v_cvt_pk_bf16_f32 v186, v196, v197\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[240:243], %[q20], v[208:223]\n\t" \
  "ds_read_b128 v[240:243], %[k0] offset:28672\n\t" \
  "v_exp_f32 v200, v200\n\t" \
  "v_sub_f32 v203, v203, %[t0]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[244:247], %[q21], v[208:223]\n\t" \
  "ds_read_b128 v[244:247], %[k1] offset:28672\n\t" \
  "v_add_f32 %[t1], %[t1], v199\n\t" \
  "v_exp_f32 v201, v201\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[248:251], %[q22], v[208:223]\n\t" \
  "ds_read_b128 v[248:251], %[k2] offset:28672\n\t" \
  "v_sub_f32 v204, v204, %[t0]\n\t" \
  "v_add_f32 %[t1], %[t1], v200\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[252:255], %[q23], v[208:223]\n\t" \
  "ds_read_b128 v[252:255], %[k3] offset:28672\n\t" \
  "v_cvt_pk_bf16_f32 v187, v198, v199\n\t" \
  "v_exp_f32 v202, v202\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[224:227], %[q24], v[208:223]\n\t" \
  "ds_read_b128 v[224:227], %[k0] offset:32768\n\t" \
  "v_sub_f32 v205, v205, %[t0]\n\t" \
  "v_add_f32 %[t1], %[t1], v201\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[228:231], %[q25], v[208:223]\n\t" \
  "ds_read_b128 v[228:231], %[k1] offset:32768\n\t" \
  "v_exp_f32 v203, v203\n\t" \
  "v_sub_f32 v206, v206, %[t0]\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[232:235], %[q26], v[208:223]\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:32768\n\t" \
  "v_add_f32 %[t1], %[t1], v202\n\t" \
  "v_cvt_pk_bf16_f32 v188, v200, v201\n\t" \
  "v_exp_f32 v204, v204\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[236:239], %[q27], v[208:223]\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:32768\n\t" \
  "v_sub_f32 v207, v207, %[t0]\n\t" \
  "v_add_f32 %[t1], %[t1], v203\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[240:243], %[q28], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[240:241], %[v00] offset:0\n\t" \
  "ds_read_b64_tr_b16 v[242:243], %[v10] offset:0\n\t" \
  "v_exp_f32 v205, v205\n\t" \
  "v_add_f32 %[t1], %[t1], v204\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[244:247], %[q29], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[244:245], %[v00] offset:2048\n\t" \
  "ds_read_b64_tr_b16 v[246:247], %[v10] offset:2048\n\t" \
  "v_cvt_pk_bf16_f32 v189, v202, v203\n\t" \
  "v_exp_f32 v206, v206\n\t" \
  "s_waitcnt lgkmcnt(9)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[248:251], %[q30], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[248:249], %[v01] offset:0\n\t" \
  "ds_read_b64_tr_b16 v[250:251], %[v11] offset:0\n\t" \
  "v_add_f32 %[t1], %[t1], v205\n\t" \
  "v_exp_f32 v207, v207\n\t" \
  "s_waitcnt lgkmcnt(10)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[252:255], %[q31], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[252:253], %[v01] offset:2048\n\t" \
  "ds_read_b64_tr_b16 v[254:255], %[v11] offset:2048\n\t" \
  "v_add_f32 %[t1], %[t1], v206\n\t" \
  "v_cvt_pk_bf16_f32 v190, v204, v205\n\t" \
  "s_waitcnt lgkmcnt(11)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[224:227], %[q32], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[224:225], %[v00] offset:4096\n\t" \
  "ds_read_b64_tr_b16 v[226:227], %[v10] offset:4096\n\t" \
  "s_nop 1\n\t" \
  "v_add_f32 %[t1], %[t1], v207\n\t" \
  "s_waitcnt lgkmcnt(12)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[228:231], %[q33], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[228:229], %[v00] offset:6144\n\t" \
  "ds_read_b64_tr_b16 v[230:231], %[v10] offset:6144\n\t" \
  "v_cvt_pk_bf16_f32 v191, v206, v207\n\t" \
  "v_add_f32 %[l], %[l], %[t1]\n\t" \
  "s_waitcnt lgkmcnt(13)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[232:235], %[q34], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[232:233], %[v01] offset:4096\n\t" \
  "ds_read_b64_tr_b16 v[234:235], %[v11] offset:4096\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 v[208:223], v[236:239], %[q35], v[208:223]\n\t" \
  "ds_read_b64_tr_b16 v[236:237], %[v01] offset:6144\n\t" \
  "ds_read_b64_tr_b16 v[238:239], %[v11] offset:6144\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "s_nop 1\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o0], v[240:243], v[184:187], %[o0]\n\t" \
  "ds_read_b64_tr_b16 v[240:241], %[v00] offset:8192\n\t" \
  "ds_read_b64_tr_b16 v[242:243], %[v10] offset:8192\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o0], v[244:247], v[188:191], %[o0]\n\t" \
  "ds_read_b64_tr_b16 v[244:245], %[v00] offset:10240\n\t" \
  "ds_read_b64_tr_b16 v[246:247], %[v10] offset:10240\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o1], v[248:251], v[184:187], %[o1]\n\t" \
  "ds_read_b64_tr_b16 v[248:249], %[v01] offset:8192\n\t" \
  "ds_read_b64_tr_b16 v[250:251], %[v11] offset:8192\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o1], v[252:255], v[188:191], %[o1]\n\t" \
  "ds_read_b64_tr_b16 v[252:253], %[v01] offset:10240\n\t" \
  "ds_read_b64_tr_b16 v[254:255], %[v11] offset:10240\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o2], v[224:227], v[184:187], %[o2]\n\t" \
  "ds_read_b64_tr_b16 v[224:225], %[v00] offset:12288\n\t" \
  "ds_read_b64_tr_b16 v[226:227], %[v10] offset:12288\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o2], v[228:231], v[188:191], %[o2]\n\t" \
  "ds_read_b64_tr_b16 v[228:229], %[v00] offset:14336\n\t" \
  "ds_read_b64_tr_b16 v[230:231], %[v10] offset:14336\n\t" \
  "v_mul_f32 v192, %[c], v208\n\t" \
  "v_mul_f32 v193, %[c], v209\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o3], v[232:235], v[184:187], %[o3]\n\t" \
  "ds_read_b64_tr_b16 v[232:233], %[v01] offset:12288\n\t" \
  "ds_read_b64_tr_b16 v[234:235], %[v11] offset:12288\n\t" \
  "v_mul_f32 v194, %[c], v210\n\t" \
  "v_mul_f32 v195, %[c], v211\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o3], v[236:239], v[188:191], %[o3]\n\t" \
  "ds_read_b64_tr_b16 v[236:237], %[v01] offset:14336\n\t" \
  "ds_read_b64_tr_b16 v[238:239], %[v11] offset:14336\n\t" \
  "v_mul_f32 v196, %[c], v212\n\t" \
  "v_mul_f32 v197, %[c], v213\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o4], v[240:243], v[184:187], %[o4]\n\t" \
  "ds_read_b64_tr_b16 v[240:241], %[v00] offset:16384\n\t" \
  "ds_read_b64_tr_b16 v[242:243], %[v10] offset:16384\n\t" \
  "v_mul_f32 v198, %[c], v214\n\t" \
  "v_mul_f32 v199, %[c], v215\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o4], v[244:247], v[188:191], %[o4]\n\t" \
  "ds_read_b64_tr_b16 v[244:245], %[v00] offset:18432\n\t" \
  "ds_read_b64_tr_b16 v[246:247], %[v10] offset:18432\n\t" \
  "v_mul_f32 v200, %[c], v216\n\t" \
  "v_mul_f32 v201, %[c], v217\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o5], v[248:251], v[184:187], %[o5]\n\t" \
  "ds_read_b64_tr_b16 v[248:249], %[v01] offset:16384\n\t" \
  "ds_read_b64_tr_b16 v[250:251], %[v11] offset:16384\n\t" \
  "v_mul_f32 v202, %[c], v218\n\t" \
  "v_mul_f32 v203, %[c], v219\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o5], v[252:255], v[188:191], %[o5]\n\t" \
  "ds_read_b64_tr_b16 v[252:253], %[v01] offset:18432\n\t" \
  "ds_read_b64_tr_b16 v[254:255], %[v11] offset:18432\n\t" \
  "v_mul_f32 v204, %[c], v220\n\t" \
  "v_mul_f32 v205, %[c], v221\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o6], v[224:227], v[184:187], %[o6]\n\t" \
  "ds_read_b64_tr_b16 v[224:225], %[v00] offset:20480\n\t" \
  "ds_read_b64_tr_b16 v[226:227], %[v10] offset:20480\n\t" \
  "v_mul_f32 v206, %[c], v222\n\t" \
  "v_mul_f32 v207, %[c], v223\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o6], v[228:231], v[188:191], %[o6]\n\t" \
  "ds_read_b64_tr_b16 v[228:229], %[v00] offset:22528\n\t" \
  "ds_read_b64_tr_b16 v[230:231], %[v10] offset:22528\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o7], v[232:235], v[184:187], %[o7]\n\t" \
  "ds_read_b64_tr_b16 v[232:233], %[v01] offset:20480\n\t" \
  "ds_read_b64_tr_b16 v[234:235], %[v11] offset:20480\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o7], v[236:239], v[188:191], %[o7]\n\t" \
  "ds_read_b64_tr_b16 v[236:237], %[v01] offset:22528\n\t" \
  "ds_read_b64_tr_b16 v[238:239], %[v11] offset:22528\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o8], v[240:243], v[184:187], %[o8]\n\t" \
  "ds_read_b64_tr_b16 v[240:241], %[v00] offset:24576\n\t" \
  "ds_read_b64_tr_b16 v[242:243], %[v10] offset:24576\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o8], v[244:247], v[188:191], %[o8]\n\t" \
  "ds_read_b64_tr_b16 v[244:245], %[v00] offset:26624\n\t" \
  "ds_read_b64_tr_b16 v[246:247], %[v10] offset:26624\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o9], v[248:251], v[184:187], %[o9]\n\t" \
  "ds_read_b64_tr_b16 v[248:249], %[v01] offset:24576\n\t" \
  "ds_read_b64_tr_b16 v[250:251], %[v11] offset:24576\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o9], v[252:255], v[188:191], %[o9]\n\t" \
  "ds_read_b64_tr_b16 v[252:253], %[v01] offset:26624\n\t" \
  "ds_read_b64_tr_b16 v[254:255], %[v11] offset:26624\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o10], v[224:227], v[184:187], %[o10]\n\t" \
  "ds_read_b64_tr_b16 v[224:225], %[v00] offset:28672\n\t" \
  "ds_read_b64_tr_b16 v[226:227], %[v10] offset:28672\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o10], v[228:231], v[188:191], %[o10]\n\t" \
  "ds_read_b64_tr_b16 v[228:229], %[v00] offset:30720\n\t" \
  "ds_read_b64_tr_b16 v[230:231], %[v10] offset:30720\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o11], v[232:235], v[184:187], %[o11]\n\t" \
  "ds_read_b64_tr_b16 v[232:233], %[v01] offset:28672\n\t" \
  "ds_read_b64_tr_b16 v[234:235], %[v11] offset:28672\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o11], v[236:239], v[188:191], %[o11]\n\t" \
  "ds_read_b64_tr_b16 v[236:237], %[v01] offset:30720\n\t" \
  "ds_read_b64_tr_b16 v[238:239], %[v11] offset:30720\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o12], v[240:243], v[184:187], %[o12]\n\t" \
  "s_waitcnt lgkmcnt(12)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o12], v[244:247], v[188:191], %[o12]\n\t" \
  "s_waitcnt lgkmcnt(10)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o13], v[248:251], v[184:187], %[o13]\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o13], v[252:255], v[188:191], %[o13]\n\t" \
  "s_waitcnt lgkmcnt(6)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o14], v[224:227], v[184:187], %[o14]\n\t" \
  "s_waitcnt lgkmcnt(4)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o14], v[228:231], v[188:191], %[o14]\n\t" \
  "s_waitcnt lgkmcnt(2)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o15], v[232:235], v[184:187], %[o15]\n\t" \
  "s_waitcnt lgkmcnt(0)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o15], v[236:239], v[188:191], %[o15]\n\t" \
  "s_nop 15\n\t" \
  "s_nop 1\n\t"
