// tmaps.h - TMA tensor maps of the bf16 operands (host side).
#pragma once
#include "plan.h"

// Fill a->maps[] for every MapId; `shadow` is the bf16 parameter copy.
// Returns an mt_status.
int mt_build_tensor_maps(KArgs* a, void* shadow);

// Maps of the single-product test harness: A in MAP_R, B in MAP_WQKV and,
// when C is given, its epilogue map (MAP_E_Y for fp32 C, MAP_E_QKV for bf16).
// a_rpb / b_rpb: rows per box of the operand maps (64, or 128 / 256 for
// K-major operands loaded in taller boxes).
int mt_build_debug_maps(KArgs* a, const void* A, long long a_rows, long long a_cols, const void* B,
                        long long b_rows, long long b_cols, const void* C, long long c_rows, long long c_cols,
                        bool c_f32, int a_rpb, int b_rpb);

// One map of a row-major buffer for the stand-alone operators: `mats` matrices
// of rows x cols elements, rows `row_bytes` and matrices `mat_bytes` apart
// (mats 1: a 2-D map, mat_bytes unused; operand maps only), box of bc columns
// x br rows, 128-byte swizzle.  Output maps (F32, BF16) always have a third
// dimension.  Needs base and both strides to be multiples of 16 bytes.
enum { MT_MAP_U8 = 0, MT_MAP_BF16 = 1, MT_MAP_F32 = 2 };
int mt_encode_map(CUtensorMap* m, int type, const void* base, long long cols, long long rows, long long mats,
                  long long row_bytes, long long mat_bytes, unsigned bc, unsigned br);
