// One user at a time for a handle's workspace: each call that uses it waits, on
// its own stream, for the call before it.  On the same stream that wait is left
// out: it would keep a call's first kernel from starting under the end of the
// kernel before it (gradients of 203 tokens at 520 x 1,400: 30.6 against 28.4 us a
// call).  Streams are told apart by their ids, which are never given twice: equal
// handle values may be different streams (each thread's own default stream, or a
// new stream that got the value of a destroyed one).
//
// Calls that are captured into a CUDA graph run when the graph is replayed, so
// they neither wait for work outside their capture (the runtime refuses that)
// nor does later work wait for them: within one capture they follow one another
// by an event of their own, and what surrounds a replay is ordered by whoever
// launches it.
#pragma once

#include <cuda_runtime_api.h>

namespace hk {

struct WorkspaceOrder {
    // The last call outside captures, and the last one of a capture.
    struct User {
        cudaEvent_t event = nullptr;
        bool some = false;
        unsigned long long stream = 0, capture = 0;
    } outside, inside;

    cudaError_t create() {
        const cudaError_t e = cudaEventCreateWithFlags(&outside.event, cudaEventDisableTiming);
        return e != cudaSuccess ? e : cudaEventCreateWithFlags(&inside.event, cudaEventDisableTiming);
    }
    void destroy() {
        if (outside.event) cudaEventDestroy(outside.event);
        if (inside.event) cudaEventDestroy(inside.event);
    }
    // Before a call's first kernel on `s`.
    cudaError_t begin(cudaStream_t s) const {
        bool in = false;
        User now;
        const cudaError_t e = describe(s, in, now);
        if (e != cudaSuccess) return e;
        const User& u = in ? inside : outside;
        if (!u.some || u.capture != now.capture) return cudaSuccess;
        if (now.stream != 0 && u.stream == now.stream) return cudaSuccess;
        return cudaStreamWaitEvent(s, u.event, 0);
    }
    // After its last.
    cudaError_t end(cudaStream_t s) {
        bool in = false;
        User now;
        cudaError_t e = describe(s, in, now);
        if (e != cudaSuccess) return e;
        User& u = in ? inside : outside;
        e = cudaEventRecord(u.event, s);
        if (e != cudaSuccess) return e;
        now.event = u.event;
        now.some = true;
        u = now;
        return cudaSuccess;
    }

private:
    // The stream's id, and the capture it takes part in.  The id is 0 for the
    // stream that is another one in every thread, and inside a capture, where it
    // may not be asked for.
    static cudaError_t describe(cudaStream_t s, bool& in, User& now) {
        cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
        const cudaError_t e = cudaStreamGetCaptureInfo(s, &status, &now.capture);
        if (e != cudaSuccess) return e;
        in = status != cudaStreamCaptureStatusNone;
        if (in || s == cudaStreamPerThread) return cudaSuccess;
        now.capture = 0;
        return cudaStreamGetId(s, &now.stream);
    }
};

}  // namespace hk
