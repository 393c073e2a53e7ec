// kv_tile.hip -- kv_tile.hpp's kernels for sequences by themselves.
#include "kv_tile.hpp"

namespace tpl {
namespace kv {

hipError_t launch_tile(const AttendArgs& p, int dk, bool join, hipStream_t st) { return go_tile<false>(p, dk, join, st); }

}  // namespace kv
}  // namespace tpl
