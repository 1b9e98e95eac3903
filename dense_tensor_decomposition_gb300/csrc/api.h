// What the files of entry points share: limits, and the calling thread's error text.
#pragma once

#include <cstdint>

namespace mk {

constexpr int64_t kMaxR = 65536;
constexpr int64_t kMaxNumel = (int64_t)1 << 40;

// Every entry point that can fail clears the text that mttkrp_last_error() returns; fail()
// writes it and returns `code`.
void clear_error();
int fail(int code, const char* fmt, ...);

}  // namespace mk
