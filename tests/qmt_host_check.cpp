// Drives the argument checks and the launch plan of qmt_host.hpp over cases read
// from stdin, one per line ("weights ...", "qk ...", "logprobs ..."), for a
// build under AddressSanitizer and UndefinedBehaviorSanitizer; prints each
// status.
#include <cstdio>
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

#include "qmt_host.hpp"

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
        long long s = -1;
        if (what == "quantize")
            s = qmt_host::check_weights(i(0), p(1), p(2), p(3), i(4), i(5), i(6));
        else if (what == "dequantize")
            s = qmt_host::check_weights(i(2), p(3), p(0), p(1), i(4), i(5), i(6));
        else if (what == "qk")
            s = qmt_host::check_qk(i(0), p(1), i(2), i(3), i(4), i(5), p(6), i(7), i(8), p(9), i(10), p(11), p(12),
                                   (float)v.at(13), i(14), i(15), p(16), p(17), i(18));
        else if (what == "logprobs")
            s = qmt_host::check_logprobs(i(0), p(1), i(2), i(3), p(4), i(5), p(6), p(7), p(8), p(9));
        else if (what == "workspace")
            s = qmt_host::logprobs_workspace(i(0), i(1), i(2));
        else if (what == "covered") {
            // every group of 8 logits of a row lies in one step of one part
            const int V = i(1);
            const qmt_host::LogprobPlan l = qmt_host::plan_logprobs(i(0), V);
            const long long step = 8 * l.threads;
            s = l.parts >= 1 && l.parts <= qmt_host::kMaxParts && l.steps >= 1 && l.threads <= 1024 &&
                (l.part ? l.steps == 1 : l.threads == 512) && (l.join || l.parts == 1) &&
                l.parts * l.steps * step >= V && (l.parts - 1) * l.steps * step < V;
        }
        std::printf("%lld\n", s);
    }
    return 0;
}
