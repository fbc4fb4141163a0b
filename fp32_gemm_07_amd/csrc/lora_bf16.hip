// The low-rank adapters' kernels for one element type.
#include "lora_launch_type.hpp"

const gemm::mx::LoraLaunches &gemm::mx::lora_launches_bf16() { return launches_of<kBf16>(); }
