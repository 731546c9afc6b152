// grouped_bf16_bf16.hip -- the grouped products of bf16 rows with bf16 outputs.
#include "grouped.hpp"

namespace ge {
namespace grouped {

hipError_t launch_bf16_bf16(const Args& a, bool gated, hipStream_t stream) { return launch<bf16, bf16>(a, gated, stream); }

}  // namespace grouped
}  // namespace ge
