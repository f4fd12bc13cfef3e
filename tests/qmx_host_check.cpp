// Drives the argument checks of qmx_host.hpp over cases read from stdin, one
// per line ("rmsnorm ...", "router ...", "blocks ..."), for a build under
// AddressSanitizer and UndefinedBehaviorSanitizer; prints each status.
#include <cstdio>
#include <cstdlib>
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

#include "qmx_host.hpp"

int main()
{
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string what;
        in >> what;
        std::vector<double> v;
        for (double d; in >> d;) v.push_back(d);
        auto p = [&](size_t i) { return (const void *)(uintptr_t)v.at(i); };
        auto i = [&](size_t k) { return (int)v.at(k); };
        int s = -1;
        if (what == "rmsnorm")
            s = qmx_host::check_rmsnorm(i(0), p(1), i(2), p(3), p(4), i(5), p(6), (float)v.at(7), i(8), p(9), p(10),
                                        i(11), i(12));
        else if (what == "router")
            s = qmx_host::check_router(i(0), p(1), i(2), i(3), i(4), i(5), p(8), p(9));
        else if (what == "quantize")
            s = qmx_host::check_blocks(i(0), p(1), i(2), p(3), p(4), (long long)v.at(5), i(6));
        else if (what == "dequantize")
            s = qmx_host::check_blocks(i(3), p(4), i(0), p(1), p(2), (long long)v.at(5), i(6));
        else if (what == "strerror") {
            std::printf("%s\n", qmx_host::status_text(i(0)));
            continue;
        }
        std::printf("%d\n", s);
    }
    return 0;
}
