// kv_tile_shared.hip -- kv_tile.hpp's kernels for sequences that share their
// first tokens: groups' rows over those, then sequences' rows over their own.
#include "kv_tile.hpp"

namespace tpl {
namespace kv {

hipError_t launch_tile_shared(const AttendArgs& p, int dk, bool join, hipStream_t st) { return go_tile<true>(p, dk, join, st); }

}  // namespace kv
}  // namespace tpl
