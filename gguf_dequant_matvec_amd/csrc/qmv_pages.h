// Pages of a cache taken from and given back to a stack on the GPU.
#pragma once

#include "qmv_kv.h"

namespace qmv {

struct ReserveArgs {
    const int32_t *add;         // [n_seq] tokens wanted
    const int32_t *free_pages;  // the stack, its top at *free_count - 1
    int32_t *free_count;
    int32_t n;                  // rows there may be
    int32_t *granted;           // [n_seq]
    int32_t *start;             // [n_seq + 1]
};
hipError_t launch_kv_reserve(const KvArgs &c, int32_t *table, int32_t *seq_len, const ReserveArgs &a, int32_t *pos,
                             int64_t *slot, hipStream_t s);
hipError_t launch_kv_release(const KvArgs &c, int32_t *table, int32_t *seq_len, const int32_t *new_len,
                             int32_t *free_pages, int32_t *free_count, hipStream_t s);

}  // namespace qmv
