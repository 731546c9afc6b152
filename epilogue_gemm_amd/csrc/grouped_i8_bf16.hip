// grouped_i8_bf16.hip -- the grouped products of i8 rows with bf16 outputs.
#include "grouped.hpp"

namespace ge {
namespace grouped {

hipError_t launch_i8_bf16(const Args& a, bool gated, hipStream_t stream) { return launch<int8_t, bf16>(a, gated, stream); }

}  // namespace grouped
}  // namespace ge
