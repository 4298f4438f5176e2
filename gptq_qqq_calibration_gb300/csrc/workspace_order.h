// One user at a time for a handle's workspace: each call that uses it waits, on
// its own stream, for the call before it.
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
    cudaEvent_t done = nullptr;      // the last call that was not captured
    cudaEvent_t captured = nullptr;  // the last call of `capture`
    cudaStream_t last = nullptr;
    bool used = false, has_capture = false;
    unsigned long long capture = 0;

    cudaError_t create() {
        const cudaError_t e = cudaEventCreateWithFlags(&done, cudaEventDisableTiming);
        return e != cudaSuccess ? e : cudaEventCreateWithFlags(&captured, cudaEventDisableTiming);
    }
    void destroy() {
        if (done) cudaEventDestroy(done);
        if (captured) cudaEventDestroy(captured);
    }
    // Before a call's first kernel on `s`.
    cudaError_t begin(cudaStream_t s) const {
        bool in = false;
        unsigned long long id = 0;
        const cudaError_t e = capturing(s, in, id);
        if (e != cudaSuccess) return e;
        if (in) return has_capture && capture == id ? cudaStreamWaitEvent(s, captured, 0) : cudaSuccess;
        return used && last != s ? cudaStreamWaitEvent(s, done, 0) : cudaSuccess;
    }
    // After its last.
    cudaError_t end(cudaStream_t s) {
        bool in = false;
        unsigned long long id = 0;
        cudaError_t e = capturing(s, in, id);
        if (e != cudaSuccess) return e;
        e = cudaEventRecord(in ? captured : done, s);
        if (e != cudaSuccess) return e;
        if (in) {
            has_capture = true;
            capture = id;
        } else {
            used = true;
            last = s;
        }
        return cudaSuccess;
    }

private:
    static cudaError_t capturing(cudaStream_t s, bool& in, unsigned long long& id) {
        cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
        const cudaError_t e = cudaStreamGetCaptureInfo(s, &status, &id);
        in = status != cudaStreamCaptureStatusNone;
        return e;
    }
};

}  // namespace hk
