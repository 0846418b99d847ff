// Decode attention with a sliding window and visible first tokens (sinks) over the bf16 / fp32 pools:
// o = softmax over the tokens t < sink or t >= n - window.  The decode kernels walk a computed page list
// (the sinks' pages, then the window's) and hide the tokens between the two inside a page.
//
// Bound: the bytes of the visible K and V; the pages at the window's start and the sinks' end are read
// whole, at most 30 tokens more.  The bf16 kernel carries each probability as two bf16 values (16 bits instead of
// 8), which at a few percent of the tensor pipe costs no time that shows: 16 sequences of up to 32k tokens, a
// window of 4,096 and 16 sinks, 40 query and 8 KV heads of 128 (215 MB of visible K and V) take 37 to 38 us, 5.7 TB/s;
// one sequence with a window of 1,024 takes 4.1 us in a graph of such layers, latency.

#include "host.cuh"
#include "launch_plain.cuh"

using namespace delta;

extern "C" delta_status delta_window_attn(const delta_desc* desc, const delta_page_table* pt, int32_t window_tokens,
                                          int32_t sink_tokens, const void* q, const void* k_pool, const void* v_pool,
                                          void* o, void* workspace, size_t ws_bytes, void* stream) {
    AttnCall a;
    a.mode = kModeWindow;
    a.d = desc;
    a.pt = pt;
    a.window = window_tokens;
    a.sink = sink_tokens;
    a.q = q;
    a.o = o;
    a.ws = workspace;
    a.ws_bytes = ws_bytes;
    a.stream = stream;
    return run_attention_on(PlainCache<true>{k_pool, v_pool}, a);
}
