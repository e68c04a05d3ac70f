// The device block pool's state as its kernels see it (layout in pa.h).
#pragma once

#include <stdint.h>

#include "pa.h"

namespace pa {
namespace dpool {

// header word 5 of a state that pa_dpool_init or pa_dpool_load found sound
constexpr int32_t kMagic = 0x50414250;

// delta, last_old, writers and last_writer are scratch: 0, -1, 0 and -1 between calls.
struct Pool {
    int32_t *hdr, *ref, *ring, *delta, *last_old, *writers, *last_writer, *tail;
};

__device__ __forceinline__ Pool views(int32_t *state, int nb) {
    Pool p;
    p.hdr = state;
    p.ref = state + PA_DPOOL_HEADER_WORDS;
    p.ring = p.ref + nb;
    p.delta = p.ring + nb;
    p.last_old = p.delta + nb;
    p.writers = p.last_old + nb;
    p.last_writer = p.writers + nb;
    p.tail = p.last_writer + nb;
    return p;
}

}  // namespace dpool
}  // namespace pa
