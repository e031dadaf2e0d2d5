// Arguments of the rotary and paged-cache launches (rotary.cu), checked by capi.cu.
// Strides are in elements.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace foak {

// Heads of T tokens on their way from one place to another.
struct HeadMove {
    const char* src;  // null: nothing to move
    char* dst;
    int64_t src_t, src_h;  // from token to token, from head to head
    int64_t dst_t, dst_h;  // dst_t of a cache: from slot to slot of a page
    int64_t dst_page;      // a cache: from page to page
    bool paged;            // the slot says where a token goes, not its index
    int H;
    int d;  // elements of a head
    int r;  // of which the first r turn (0: none)
};

struct RotaryArgs {
    HeadMove move[3];
    const int64_t* positions;  // [T]; null where nothing turns
    const uint64_t* turns;     // [r / 2] turns a position, as fractions of 2^64
    const int64_t* slots;      // [T] or null: tokens with a slot outside [0, capacity) are left out
    int32_t* err;              // null, or OR-ed with FOAK_ERRBIT_PAGE_RANGE for a slot past the capacity
    int64_t T, capacity, page_size;
    float factor, sign;
    bool interleaved;
};

// inv_freq[i] for i < r / 2 (host); scaling as FOAK_ROTARY_* of foak_ce.h.
void rotary_inv_freq(double base, int64_t r, int scaling, double factor, double low, double high, double original,
                     double* inv_freq);
// Turns a position as a fraction of 2^64 (host).
uint64_t rotary_turns(double inv_freq);

cudaError_t launch_rotary(int es, const RotaryArgs& a, cudaStream_t s);
cudaError_t launch_kv_slots(const int32_t* page_table, int64_t ld_table, int64_t max_pages, const int32_t* cache_lens,
                            const int32_t* seq_starts, int64_t B, int64_t T, int64_t page_size, int64_t num_pages,
                            int64_t* slots, int64_t* positions, int32_t* err, cudaStream_t s);

}  // namespace foak
