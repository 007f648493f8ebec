// side_stream.h -- second streams for calls that run two of their kernels side by
// side (host code).
//
// A call forks its second stream off the caller's stream by an event and joins it
// again by another.  The second streams belong to the process: one for a caller's
// stream, so that calls on different streams are not ordered against one another
// and host threads that come and go leave nothing behind.  An entry is found by the
// stream's handle and the id of the context that it belongs to: after a device
// reset the context has another id, and the old handles are not touched again.
// The table has kSideStreams places and is never emptied; callers' streams behind
// that share the entries of their context.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

namespace m3 {

constexpr int kSideStreams = 64;

struct SideStream {
    std::mutex use;                    // held from a call's fork to its join
    unsigned long long ctx;            // 0: a free place
    cudaStream_t caller, stream;
    cudaEvent_t fork, join;
};

class SideStreams {
    std::mutex table_;
    SideStream at_[kSideStreams] = {};

    // id of the current context (0: none, or a driver without the call)
    static unsigned long long context_id() {
        using Call = CUresult (*)(CUcontext, unsigned long long*);
        static const Call call = [] {
            void* p = nullptr;
            cudaDriverEntryPointQueryResult found;
            const bool ok = cudaGetDriverEntryPoint("cuCtxGetId", &p, cudaEnableDefault, &found) == cudaSuccess &&
                            found == cudaDriverEntryPointSuccess;
            return reinterpret_cast<Call>(ok ? p : nullptr);
        }();
        unsigned long long id = 0;
        return call && call(nullptr, &id) == CUDA_SUCCESS ? id : 0;
    }
    // All of an entry's handles, or none.  Making them enqueues nothing, so that it is
    // safe while this or another thread captures, which the relaxed mode states.
    static bool make(SideStream* s) {
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return false;
        const bool ok = make_handles(s);
        cudaThreadExchangeStreamCaptureMode(&mode);
        return ok;
    }
    static bool make_handles(SideStream* s) {
        if (cudaStreamCreateWithFlags(&s->stream, cudaStreamNonBlocking) != cudaSuccess) return false;
        if (cudaEventCreateWithFlags(&s->fork, cudaEventDisableTiming) == cudaSuccess) {
            if (cudaEventCreateWithFlags(&s->join, cudaEventDisableTiming) == cudaSuccess) return true;
            cudaEventDestroy(s->fork);
        }
        cudaStreamDestroy(s->stream);
        return false;
    }
    SideStream* find(cudaStream_t st) {
        const unsigned long long ctx = context_id();
        if (!ctx) return nullptr;
        const std::lock_guard<std::mutex> hold(table_);
        int same = 0, free = -1;
        for (int i = kSideStreams - 1; i >= 0; --i) {
            if (!at_[i].ctx) free = i;
            else if (at_[i].ctx == ctx && at_[i].caller == st) return &at_[i];
            else if (at_[i].ctx == ctx) ++same;
        }
        if (free >= 0) {
            if (!make(&at_[free])) return nullptr;
            at_[free].ctx = ctx;
            at_[free].caller = st;
            return &at_[free];
        }
        if (!same) return nullptr;
        int n = (int)(((uintptr_t)st >> 4) % (unsigned)same);
        for (SideStream& s : at_)
            if (s.ctx == ctx && n-- == 0) return &s;
        return nullptr;
    }

public:
    // The second stream for a call on the current context's stream `st`, kept for the
    // caller as long as it holds `use`; null if there is none that can be used.  One
    // that an earlier call forked off the same capture stays in it until that ends,
    // and is forked off it again; one in another capture, or a broken one, is not used.
    SideStream* take(cudaStream_t st, std::unique_lock<std::mutex>* use) noexcept {
        try {
            SideStream* s = find(st);
            if (!s) return nullptr;
            *use = std::unique_lock<std::mutex>(s->use);
            cudaStreamCaptureStatus mine, its;
            unsigned long long my_id = 0, its_id = 0;
            if (cudaStreamGetCaptureInfo(s->stream, &its, &its_id) == cudaSuccess &&
                (its == cudaStreamCaptureStatusNone ||
                 (its == cudaStreamCaptureStatusActive && cudaStreamGetCaptureInfo(st, &mine, &my_id) == cudaSuccess &&
                  mine == cudaStreamCaptureStatusActive && my_id == its_id)))
                return s;
            use->unlock();
        } catch (...) {}               // (a lock that could not be had)
        return nullptr;
    }
};

}  // namespace m3
