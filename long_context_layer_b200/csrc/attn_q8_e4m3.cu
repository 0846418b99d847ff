// The 8-bit decode kernel over e4m3 payloads.
#include "q8.cuh"
#define DELTA_Q8_FMT kE4M3
#include "attn_q8_impl.cuh"
