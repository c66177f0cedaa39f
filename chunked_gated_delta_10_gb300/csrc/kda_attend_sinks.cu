// The kernels of attention over a paged cache in 16 or 32 bits with a window and first rows that stay visible beside it
// (kda_cache_attend_sinks). They differ from those without first rows in where a row's number says it is.
#include "kda_attend_kernels.cuh"

namespace kda {
namespace attend {

Kernel kernel_with_sinks(const kda_cache& c, int ht, Split split) { return kernel_of<true>(c, ht, split); }

}  // namespace attend
}  // namespace kda
