// The two products of a 576/512-wide tile for one wave, written out.
//
// A wave that owns 32 query rows holds 144 registers of Q and 256 of O: all
// accumulation registers and more than half of the others. Left to itself the
// compiler moves O about (225 moves and 77 spills a tile). Here the fragments
// of K and V pass through eight fixed register quads, 224 to 255, each read
// 7 fragments (about 220 cycles of MFMA) ahead of its use; the last reads of
// the score block are already the first of V, so that they arrive during the
// softmax. Reads return in order, so every wait names the reads that may still
// be under way. A block ends with all its reads returned and with the states
// that arithmetic has to wait for an MFMA's result, so nothing the compiler
// puts between blocks can meet either.
//
// Operands: k0..k3 the four chunk offsets of K within a 64-column block, v00,
// v01, v10, v11 those of V ([8-row group][column half]), all as LDS addresses.
#pragma once

namespace mla {

// S^T (s) from K and Q (q0..q35); leaves V's first 7 fragments in their quads.
#define WIDE_SCORES_ASM \
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
  "ds_read_b64_tr_b16 v[240:241], %[v00] offset:0\n\t" \
  "ds_read_b64_tr_b16 v[242:243], %[v10] offset:0\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[244:247], %[q29], %[s]\n\t" \
  "ds_read_b64_tr_b16 v[244:245], %[v00] offset:2048\n\t" \
  "ds_read_b64_tr_b16 v[246:247], %[v10] offset:2048\n\t" \
  "s_waitcnt lgkmcnt(9)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[248:251], %[q30], %[s]\n\t" \
  "ds_read_b64_tr_b16 v[248:249], %[v01] offset:0\n\t" \
  "ds_read_b64_tr_b16 v[250:251], %[v11] offset:0\n\t" \
  "s_waitcnt lgkmcnt(10)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[252:255], %[q31], %[s]\n\t" \
  "ds_read_b64_tr_b16 v[252:253], %[v01] offset:2048\n\t" \
  "ds_read_b64_tr_b16 v[254:255], %[v11] offset:2048\n\t" \
  "s_waitcnt lgkmcnt(11)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[224:227], %[q32], %[s]\n\t" \
  "ds_read_b64_tr_b16 v[224:225], %[v00] offset:4096\n\t" \
  "ds_read_b64_tr_b16 v[226:227], %[v10] offset:4096\n\t" \
  "s_waitcnt lgkmcnt(12)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[228:231], %[q33], %[s]\n\t" \
  "ds_read_b64_tr_b16 v[228:229], %[v00] offset:6144\n\t" \
  "ds_read_b64_tr_b16 v[230:231], %[v10] offset:6144\n\t" \
  "s_waitcnt lgkmcnt(13)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[232:235], %[q34], %[s]\n\t" \
  "ds_read_b64_tr_b16 v[232:233], %[v01] offset:4096\n\t" \
  "ds_read_b64_tr_b16 v[234:235], %[v11] offset:4096\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[236:239], %[q35], %[s]\n\t" \
  "s_waitcnt lgkmcnt(0)\n\t" \
  "s_nop 15\n\t" \
  "s_nop 1\n\t"

// The same with the loads of a later tile's 16 bytes a lane of each 64-column
// block spread over the MFMAs (src: the lane's bytes of block 0, to: the LDS
// address of its wave's part; an instruction's offset counts for both).
#define WIDE_SCORES_LOAD_ASM \
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
  "s_add_u32 m0, %[to], 0\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:0\n\t" \
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
  "s_add_u32 m0, %[to], 3968\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:128\n\t" \
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
  "s_add_u32 m0, %[to], 7936\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:256\n\t" \
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
  "s_add_u32 m0, %[to], 11904\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:384\n\t" \
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
  "s_add_u32 m0, %[to], 15872\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:512\n\t" \
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
  "s_add_u32 m0, %[to], 19840\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:640\n\t" \
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
  "s_add_u32 m0, %[to], 23808\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:768\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[232:235], %[q26], %[s]\n\t" \
  "ds_read_b128 v[232:235], %[k2] offset:32768\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[236:239], %[q27], %[s]\n\t" \
  "ds_read_b128 v[236:239], %[k3] offset:32768\n\t" \
  "s_waitcnt lgkmcnt(7)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[240:243], %[q28], %[s]\n\t" \
  "ds_read_b64_tr_b16 v[240:241], %[v00] offset:0\n\t" \
  "ds_read_b64_tr_b16 v[242:243], %[v10] offset:0\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[244:247], %[q29], %[s]\n\t" \
  "ds_read_b64_tr_b16 v[244:245], %[v00] offset:2048\n\t" \
  "ds_read_b64_tr_b16 v[246:247], %[v10] offset:2048\n\t" \
  "s_add_u32 m0, %[to], 27776\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:896\n\t" \
  "s_waitcnt lgkmcnt(9)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[248:251], %[q30], %[s]\n\t" \
  "ds_read_b64_tr_b16 v[248:249], %[v01] offset:0\n\t" \
  "ds_read_b64_tr_b16 v[250:251], %[v11] offset:0\n\t" \
  "s_waitcnt lgkmcnt(10)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[252:255], %[q31], %[s]\n\t" \
  "ds_read_b64_tr_b16 v[252:253], %[v01] offset:2048\n\t" \
  "ds_read_b64_tr_b16 v[254:255], %[v11] offset:2048\n\t" \
  "s_waitcnt lgkmcnt(11)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[224:227], %[q32], %[s]\n\t" \
  "ds_read_b64_tr_b16 v[224:225], %[v00] offset:4096\n\t" \
  "ds_read_b64_tr_b16 v[226:227], %[v10] offset:4096\n\t" \
  "s_waitcnt lgkmcnt(12)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[228:231], %[q33], %[s]\n\t" \
  "ds_read_b64_tr_b16 v[228:229], %[v00] offset:6144\n\t" \
  "ds_read_b64_tr_b16 v[230:231], %[v10] offset:6144\n\t" \
  "s_add_u32 m0, %[to], 31744\n\t" \
  "global_load_lds_dwordx4 %[src], off offset:1024\n\t" \
  "s_waitcnt lgkmcnt(13)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[232:235], %[q34], %[s]\n\t" \
  "ds_read_b64_tr_b16 v[232:233], %[v01] offset:4096\n\t" \
  "ds_read_b64_tr_b16 v[234:235], %[v11] offset:4096\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[s], v[236:239], %[q35], %[s]\n\t" \
  "s_waitcnt lgkmcnt(0)\n\t" \
  "s_nop 15\n\t" \
  "s_nop 1\n\t"

// O^T (o0..o15) += V^T P^T (p0, p1), V's first fragments being in their quads.
#define WIDE_VALUES_ASM \
  "s_nop 1\n\t" \
  "ds_read_b64_tr_b16 v[236:237], %[v01] offset:6144\n\t" \
  "ds_read_b64_tr_b16 v[238:239], %[v11] offset:6144\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o0], v[240:243], %[p0], %[o0]\n\t" \
  "ds_read_b64_tr_b16 v[240:241], %[v00] offset:8192\n\t" \
  "ds_read_b64_tr_b16 v[242:243], %[v10] offset:8192\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o0], v[244:247], %[p1], %[o0]\n\t" \
  "ds_read_b64_tr_b16 v[244:245], %[v00] offset:10240\n\t" \
  "ds_read_b64_tr_b16 v[246:247], %[v10] offset:10240\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o1], v[248:251], %[p0], %[o1]\n\t" \
  "ds_read_b64_tr_b16 v[248:249], %[v01] offset:8192\n\t" \
  "ds_read_b64_tr_b16 v[250:251], %[v11] offset:8192\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o1], v[252:255], %[p1], %[o1]\n\t" \
  "ds_read_b64_tr_b16 v[252:253], %[v01] offset:10240\n\t" \
  "ds_read_b64_tr_b16 v[254:255], %[v11] offset:10240\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o2], v[224:227], %[p0], %[o2]\n\t" \
  "ds_read_b64_tr_b16 v[224:225], %[v00] offset:12288\n\t" \
  "ds_read_b64_tr_b16 v[226:227], %[v10] offset:12288\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o2], v[228:231], %[p1], %[o2]\n\t" \
  "ds_read_b64_tr_b16 v[228:229], %[v00] offset:14336\n\t" \
  "ds_read_b64_tr_b16 v[230:231], %[v10] offset:14336\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o3], v[232:235], %[p0], %[o3]\n\t" \
  "ds_read_b64_tr_b16 v[232:233], %[v01] offset:12288\n\t" \
  "ds_read_b64_tr_b16 v[234:235], %[v11] offset:12288\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o3], v[236:239], %[p1], %[o3]\n\t" \
  "ds_read_b64_tr_b16 v[236:237], %[v01] offset:14336\n\t" \
  "ds_read_b64_tr_b16 v[238:239], %[v11] offset:14336\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o4], v[240:243], %[p0], %[o4]\n\t" \
  "ds_read_b64_tr_b16 v[240:241], %[v00] offset:16384\n\t" \
  "ds_read_b64_tr_b16 v[242:243], %[v10] offset:16384\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o4], v[244:247], %[p1], %[o4]\n\t" \
  "ds_read_b64_tr_b16 v[244:245], %[v00] offset:18432\n\t" \
  "ds_read_b64_tr_b16 v[246:247], %[v10] offset:18432\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o5], v[248:251], %[p0], %[o5]\n\t" \
  "ds_read_b64_tr_b16 v[248:249], %[v01] offset:16384\n\t" \
  "ds_read_b64_tr_b16 v[250:251], %[v11] offset:16384\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o5], v[252:255], %[p1], %[o5]\n\t" \
  "ds_read_b64_tr_b16 v[252:253], %[v01] offset:18432\n\t" \
  "ds_read_b64_tr_b16 v[254:255], %[v11] offset:18432\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o6], v[224:227], %[p0], %[o6]\n\t" \
  "ds_read_b64_tr_b16 v[224:225], %[v00] offset:20480\n\t" \
  "ds_read_b64_tr_b16 v[226:227], %[v10] offset:20480\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o6], v[228:231], %[p1], %[o6]\n\t" \
  "ds_read_b64_tr_b16 v[228:229], %[v00] offset:22528\n\t" \
  "ds_read_b64_tr_b16 v[230:231], %[v10] offset:22528\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o7], v[232:235], %[p0], %[o7]\n\t" \
  "ds_read_b64_tr_b16 v[232:233], %[v01] offset:20480\n\t" \
  "ds_read_b64_tr_b16 v[234:235], %[v11] offset:20480\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o7], v[236:239], %[p1], %[o7]\n\t" \
  "ds_read_b64_tr_b16 v[236:237], %[v01] offset:22528\n\t" \
  "ds_read_b64_tr_b16 v[238:239], %[v11] offset:22528\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o8], v[240:243], %[p0], %[o8]\n\t" \
  "ds_read_b64_tr_b16 v[240:241], %[v00] offset:24576\n\t" \
  "ds_read_b64_tr_b16 v[242:243], %[v10] offset:24576\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o8], v[244:247], %[p1], %[o8]\n\t" \
  "ds_read_b64_tr_b16 v[244:245], %[v00] offset:26624\n\t" \
  "ds_read_b64_tr_b16 v[246:247], %[v10] offset:26624\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o9], v[248:251], %[p0], %[o9]\n\t" \
  "ds_read_b64_tr_b16 v[248:249], %[v01] offset:24576\n\t" \
  "ds_read_b64_tr_b16 v[250:251], %[v11] offset:24576\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o9], v[252:255], %[p1], %[o9]\n\t" \
  "ds_read_b64_tr_b16 v[252:253], %[v01] offset:26624\n\t" \
  "ds_read_b64_tr_b16 v[254:255], %[v11] offset:26624\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o10], v[224:227], %[p0], %[o10]\n\t" \
  "ds_read_b64_tr_b16 v[224:225], %[v00] offset:28672\n\t" \
  "ds_read_b64_tr_b16 v[226:227], %[v10] offset:28672\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o10], v[228:231], %[p1], %[o10]\n\t" \
  "ds_read_b64_tr_b16 v[228:229], %[v00] offset:30720\n\t" \
  "ds_read_b64_tr_b16 v[230:231], %[v10] offset:30720\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o11], v[232:235], %[p0], %[o11]\n\t" \
  "ds_read_b64_tr_b16 v[232:233], %[v01] offset:28672\n\t" \
  "ds_read_b64_tr_b16 v[234:235], %[v11] offset:28672\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o11], v[236:239], %[p1], %[o11]\n\t" \
  "ds_read_b64_tr_b16 v[236:237], %[v01] offset:30720\n\t" \
  "ds_read_b64_tr_b16 v[238:239], %[v11] offset:30720\n\t" \
  "s_waitcnt lgkmcnt(14)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o12], v[240:243], %[p0], %[o12]\n\t" \
  "s_waitcnt lgkmcnt(12)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o12], v[244:247], %[p1], %[o12]\n\t" \
  "s_waitcnt lgkmcnt(10)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o13], v[248:251], %[p0], %[o13]\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o13], v[252:255], %[p1], %[o13]\n\t" \
  "s_waitcnt lgkmcnt(6)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o14], v[224:227], %[p0], %[o14]\n\t" \
  "s_waitcnt lgkmcnt(4)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o14], v[228:231], %[p1], %[o14]\n\t" \
  "s_waitcnt lgkmcnt(2)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o15], v[232:235], %[p0], %[o15]\n\t" \
  "s_waitcnt lgkmcnt(0)\n\t" \
  "v_mfma_f32_32x32x16_bf16 %[o15], v[236:239], %[p1], %[o15]\n\t" \
  "s_nop 15\n\t" \
  "s_nop 1\n\t"

}  // namespace mla
