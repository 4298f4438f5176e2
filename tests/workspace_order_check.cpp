// Checks csrc/workspace_order.h on the CPU against a small model of the CUDA
// runtime (streams, events, captures), defined here in place of the library.
//
// Random programs call the workspace from several streams, capture some of the
// calls, and fork streams inside a capture.  Two calls outside any capture, or
// two of one capture, have to be ordered, the first before the second; and no
// call may wait across the border of a capture, which the runtime refuses.
#include <cstdio>
#include <cstdint>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <vector>

#include "workspace_order.h"

namespace {

struct Stream {
    std::set<int> before;  // calls that work enqueued here from now on follows
    int capture = 0;       // 0: none
};
struct Event {
    bool recorded = false;
    std::set<int> before;
    int capture = 0;
};

std::vector<Stream> streams;               // the real ones
std::map<cudaStream_t, int> by_handle;     // what a handle stands for at the moment
std::vector<Event> events;

Stream& at(cudaStream_t s) { return streams[by_handle.at(s)]; }
Event& at(cudaEvent_t e) { return events[reinterpret_cast<uintptr_t>(e) - 1]; }

}  // namespace

extern "C" {
cudaError_t CUDARTAPI cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) {
    events.emplace_back();
    *e = reinterpret_cast<cudaEvent_t>(events.size());
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t CUDARTAPI cudaEventRecord(cudaEvent_t e, cudaStream_t s) {
    at(e) = Event{true, at(s).before, at(s).capture};
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaStreamWaitEvent(cudaStream_t s, cudaEvent_t e, unsigned) {
    if (!at(e).recorded) return cudaSuccess;
    if (at(e).capture != at(s).capture)
        return at(s).capture ? cudaErrorStreamCaptureIsolation : cudaErrorCapturedEvent;
    at(s).before.insert(at(e).before.begin(), at(e).before.end());
    return cudaSuccess;
}
// ids are given once, except to the stream that each thread has of its own: what
// the model gives for that one is not to be gone by
cudaError_t CUDARTAPI cudaStreamGetId(cudaStream_t s, unsigned long long* id) {
    if (at(s).capture) return cudaErrorStreamCaptureUnsupported;
    *id = s == cudaStreamPerThread ? 1000000ull : static_cast<unsigned long long>(by_handle.at(s)) + 1;
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaStreamGetCaptureInfo(cudaStream_t s, cudaStreamCaptureStatus* status,
                                               unsigned long long* id, cudaGraph_t*, const cudaGraphNode_t**,
                                               const cudaGraphEdgeData**, size_t*) {
    *status = at(s).capture ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
    if (at(s).capture) *id = static_cast<unsigned long long>(at(s).capture);
    return cudaSuccess;
}
}

int main(int argc, char** argv) {
    // handles that stand for another stream than before; of the streams that are
    // never captured, the second has the handle of a thread's own
    const bool aliases = argc > 1;
    static_assert(sizeof(cudaStream_t) == sizeof(uintptr_t), "handles are values");
    std::mt19937 rng(7);
    const auto pick = [&](int n) { return static_cast<int>(rng() % static_cast<unsigned>(n)); };
    long calls = 0, captured_calls = 0;
    for (int program = 0; program < 20000; ++program) {
        streams.assign(5, Stream{});
        by_handle.clear();
        events.clear();
        const auto handle = [](int i) { return reinterpret_cast<cudaStream_t>(static_cast<uintptr_t>(i + 1)); };
        for (int i = 0; i < 5; ++i) by_handle[handle(i)] = i;
        hk::WorkspaceOrder order;
        order.create();
        int next_call = 0, next_capture = 0, capture = 0;
        std::vector<int> outside, inside;  // calls
        for (int step = 0; step < 24; ++step) {
            const int what = pick(10);
            const int i = pick(3);  // streams 0 to 2 are never captured, 3 and 4 may be
            if (what == 0 && !capture) {  // a capture begins; its streams have their past behind them
                capture = ++next_capture;
                streams[by_handle[handle(3)]] = Stream{{}, capture};
                inside.clear();
            } else if (what == 1 && capture) {  // and ends
                for (int k = 3; k < 5; ++k)
                    if (streams[by_handle[handle(k)]].capture) streams[by_handle[handle(k)]] = Stream{};
                capture = 0;
            } else if (what == 2 && capture) {  // stream 4 is forked from stream 3
                Stream& fork = streams[by_handle[handle(4)]];
                const Stream& from = streams[by_handle[handle(3)]];
                fork.capture = capture;
                fork.before.insert(from.before.begin(), from.before.end());
            } else if (what == 3 && aliases) {
                // the handle is destroyed and its value given to a new stream, or
                // it is a stream of each thread's own
                streams.emplace_back();
                by_handle[handle(i)] = static_cast<int>(streams.size()) - 1;
            } else {
                const bool in = capture && pick(2);
                const int which = in ? (streams[by_handle[handle(4)]].capture ? 3 + pick(2) : 3) : i;
                const cudaStream_t s = handle(which);
                cudaError_t e = order.begin(s);
                std::vector<int>& peers = in ? inside : outside;
                bool ordered = true;
                for (int c : peers) ordered = ordered && at(s).before.count(c);
                const int call = next_call++;
                at(s).before.insert(call);
                peers.push_back(call);
                if (e == cudaSuccess) e = order.end(s);
                if (e != cudaSuccess || !ordered) {
                    std::printf("program %d, step %d: %s\n", program, step,
                                ordered ? "a wait across the border of a capture" : "two calls at one time");
                    return 1;
                }
                ++calls;
                captured_calls += in;
            }
        }
    }
    std::printf("order ok: %ld calls, %ld of them captured\n", calls, captured_calls);
    return captured_calls > 10000 && calls - captured_calls > 10000 ? 0 : 1;
}
