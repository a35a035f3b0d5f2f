// The kernels of extend.cuh with a tree's mask.
#include "extend.cuh"

namespace argus {
namespace extend {

ARGUS_EXTEND_FORM(kTree)

}  // namespace extend
}  // namespace argus
