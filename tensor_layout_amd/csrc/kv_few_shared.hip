// kv_few_shared.hip -- kv_few.hpp's kernel for sequences that share their first
// tokens: groups' rows over those, then sequences' rows over their own.
#include "kv_few.hpp"

namespace tpl {
namespace kv {

hipError_t launch_few_shared(const AttendArgs& p, int dc, int mr, hipStream_t st) { return go_few<true>(p, dc, mr, st); }

}  // namespace kv
}  // namespace tpl
