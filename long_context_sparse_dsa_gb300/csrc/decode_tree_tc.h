// decode_tree_tc.h -- host side of decode_tree_tc.cu.
#pragma once

#include "decode_tree.h"

namespace dsa {

size_t tree_tc_ws_bytes(int d);
cudaError_t launch_tree_tc(const TreeAttnArgs& a, void* ws, cudaStream_t s);

}  // namespace dsa
