// grouped_i8_f16.hip -- the grouped products of i8 rows with f16 outputs.
#include "grouped.hpp"

namespace ge {
namespace grouped {

hipError_t launch_i8_f16(const Args& a, bool gated, hipStream_t stream) { return launch<int8_t, f16>(a, gated, stream); }

}  // namespace grouped
}  // namespace ge
