// Rules on logits before a token is chosen (logits.hip): arguments and launch.
#pragma once
#include "kv_tree.h"

namespace q4gsw {

constexpr int kLogitsHistory = 1 << 28;   // tokens of a history: their count and a path's fit 29 bits

struct LogitsArgs {
    const void* logits;
    void* out;
    int64_t rows, V, ld, out_ld;
    int batch, max_new;
    const int32_t* cu;                   // null: row r is sequence r's
    const int32_t* history;              // [batch][history_ld]; null: none
    int64_t history_ld;
    int history_cols;
    const int32_t* history_len;
    const int32_t* prompt_len;           // null: 0
    const int32_t* ids;                  // null: rows add nothing to their history
    const int32_t* parents;              // null: a row's path is the rows of its sequence up to it
    const float *repetition, *presence, *frequency;      // null: none
    const int32_t* bias_ids;             // null: none
    const float* bias;
    int64_t bias_ld;
    int bias_cols;
    const uint32_t* mask;                // null: none
    int64_t mask_ld;
    int chunks, rows_per_group;
};

hipError_t launch_logits(LogitsArgs a, int dtype, hipStream_t s);
bool logits_launch_ok(const LogitsArgs& a);

}  // namespace q4gsw
