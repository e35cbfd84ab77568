// na_machine.h -- the machine that launches are sized for.
#pragma once

namespace na {

constexpr int kSms = 152;   // multiprocessors of a GB300

}  // namespace na
