// The kernels of attention over a paged cache in 16 or 32 bits with a window and first rows that stay visible beside it
// (kda_cache_attend_sinks). They differ from those without first rows in where a row's number says it is, and in that the
// heads of a sequence have a share together. 64 sequences of U[1,16384] rows that see the first 64 and the last 4096, 32 heads
// on 8 of 128, bf16: 136 us, 6.7 TB/s (133 at a plain copy's rate); 8 of U[1,6000] that see 5 + 777, 20 heads on 4, fp32: 11.0
// us, latency.
#include "kda_attend_kernels.cuh"

namespace kda {
namespace attend {

Kernel kernel_with_sinks(const kda_cache& c, int ht, Split split) { return kernel_of<true>(c, ht, split); }

}  // namespace attend
}  // namespace kda
