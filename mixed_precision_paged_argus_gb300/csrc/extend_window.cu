// The kernels of extend.cuh with a sliding window and first tokens.
#include "extend.cuh"

namespace argus {
namespace extend {

ARGUS_EXTEND_FORM(kWindow)

}  // namespace extend
}  // namespace argus
