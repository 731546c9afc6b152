// grouped_f16_f16.hip -- the grouped products of f16 rows with f16 outputs.
#include "grouped.hpp"

namespace ge {
namespace grouped {

hipError_t launch_f16_f16(const Args& a, bool gated, hipStream_t stream) { return launch<f16, f16>(a, gated, stream); }

}  // namespace grouped
}  // namespace ge
