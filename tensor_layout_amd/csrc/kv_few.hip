// kv_few.hip -- kv_few.hpp's kernel for sequences by themselves.
#include "kv_few.hpp"

namespace tpl {
namespace kv {

hipError_t launch_few(const AttendArgs& p, int dc, int mr, hipStream_t st) { return go_few<false>(p, dc, mr, st); }

}  // namespace kv
}  // namespace tpl
