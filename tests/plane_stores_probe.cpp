// How a tile's scales leave, compiled without HIP, as a function a test can call.
#include "plan.hpp"

extern "C" int scale_store_bytes(int64_t per, int64_t first, int codes) { return fq::scale_store_bytes(per, first, codes); }
