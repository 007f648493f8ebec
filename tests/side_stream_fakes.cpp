// The second streams of side_stream.h against a fake CUDA runtime that counts what
// is made and what is given back (no GPU): fakes of the calls that it makes, and a
// main() that prints "ok" or the first check that failed.
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <utility>
#include <vector>

#include "side_stream.h"

static int streams, events, stream_frees, event_frees, fail_at = -1, made;   // fail_at: the n-th creation fails
static unsigned long long context = 7;
static cudaStreamCaptureStatus captured[4096];
static unsigned long long capture_id[4096];
static cudaStreamCaptureMode thread_mode = cudaStreamCaptureModeGlobal;
static int number(cudaStream_t s) { return (int)((uintptr_t)s >> 4); }
static bool fails() { return made++ == fail_at || thread_mode != cudaStreamCaptureModeRelaxed; }

static CUresult ctx_id(CUcontext, unsigned long long* id) {
    *id = context;
    return CUDA_SUCCESS;
}
extern "C" {
cudaError_t cudaGetDriverEntryPoint(const char*, void** p, unsigned long long, cudaDriverEntryPointQueryResult* r) {
    *p = reinterpret_cast<void*>(&ctx_id);
    *r = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t cudaStreamCreateWithFlags(cudaStream_t* s, unsigned) {
    if (fails()) return cudaErrorMemoryAllocation;
    *s = reinterpret_cast<cudaStream_t>((uintptr_t)(1000 + streams++) << 4);
    return cudaSuccess;
}
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) {
    if (fails()) return cudaErrorMemoryAllocation;
    *e = reinterpret_cast<cudaEvent_t>((uintptr_t)(1 + events++) << 4);
    return cudaSuccess;
}
cudaError_t cudaThreadExchangeStreamCaptureMode(cudaStreamCaptureMode* m) {
    std::swap(*m, thread_mode);
    return cudaSuccess;
}
cudaError_t cudaStreamDestroy(cudaStream_t) { return ++stream_frees, cudaSuccess; }
cudaError_t cudaEventDestroy(cudaEvent_t) { return ++event_frees, cudaSuccess; }
cudaError_t cudaStreamGetCaptureInfo(cudaStream_t s, cudaStreamCaptureStatus* c, unsigned long long* id, cudaGraph_t*,
                                     const cudaGraphNode_t**, size_t*) {
    *c = captured[number(s)];
    *id = capture_id[number(s)];
    return cudaSuccess;
}
}

static void check(bool ok, const char* what) {
    if (ok) return;
    std::printf("failed: %s\n", what);
    std::exit(1);
}
static cudaStream_t caller(int n) { return reinterpret_cast<cudaStream_t>((uintptr_t)n << 4); }
static m3::SideStream* take(m3::SideStreams& t, int n) {
    std::unique_lock<std::mutex> use;
    m3::SideStream* s = t.take(caller(n), &use);
    check(use.owns_lock() == (s != nullptr), "an entry comes locked, none unlocked");
    return s;
}

int main() {
    {
        static m3::SideStreams t;
        m3::SideStream* first = take(t, 1);
        check(first && streams == 1 && events == 2, "a stream and two events");
        std::vector<std::thread> threads;              // threads that come and go
        for (int i = 0; i < 40; ++i) threads.emplace_back([&] { check(take(t, 1) == first, "one entry for a caller's stream"); });
        for (std::thread& h : threads) h.join();
        check(streams == 1 && events == 2, "threads leave nothing behind");
        m3::SideStream* second = take(t, 2);
        check(second != first && second->stream != first->stream, "another caller's stream has another one");
        captured[number(first->stream)] = cudaStreamCaptureStatusInvalidated;
        check(!take(t, 1), "not one that is in a broken capture");
        captured[number(first->stream)] = cudaStreamCaptureStatusNone;
        check(take(t, 1) == first, "the same once the capture has ended");
        const int side = number(first->stream);        // forked off a capture by an earlier call
        captured[1] = captured[side] = cudaStreamCaptureStatusActive;
        capture_id[1] = capture_id[side] = 5;
        check(take(t, 1) == first && take(t, 1) == first, "again in the same capture");
        capture_id[1] = 6;
        check(!take(t, 1), "not in another one");
        captured[1] = cudaStreamCaptureStatusNone;
        check(!take(t, 1), "nor beside one");
        captured[side] = cudaStreamCaptureStatusNone;
        captured[3] = cudaStreamCaptureStatusActive;
        check(take(t, 3) && thread_mode == cudaStreamCaptureModeGlobal, "made for a caller that is captured, whose mode comes back");
        context = 8;                                   // a device reset
        m3::SideStream* after = take(t, 1);
        check(after && after->stream != first->stream, "handles of another context are not used");
        check(stream_frees == 0 && event_frees == 0, "nor touched");
        context = 0;
        check(!take(t, 1), "none without a context");
    }
    for (int n = 0; n < 3; ++n) {                      // each of the three creations fails
        static m3::SideStreams tables[3];
        m3::SideStreams& t = tables[n];
        context = 9;
        streams = events = stream_frees = event_frees = made = 0;
        fail_at = n;
        for (int again = 0; again < 5; ++again, made = 0) check(!take(t, 1), "none if one cannot be made");
        check(streams == stream_frees && events == event_frees, "what was made is given back");
        fail_at = -1;
        check(take(t, 1) && streams - stream_frees == 1 && events - event_frees == 2, "made whole later");
    }
    {
        static m3::SideStreams t;
        streams = events = stream_frees = event_frees = 0;
        for (int i = 0; i < 500; ++i) check(take(t, 1 + i), "every caller's stream has one");
        check(streams == m3::kSideStreams && stream_frees == 0, "of a bounded number");
        check(take(t, 499) == take(t, 499), "always the same");
        context = 10;
        check(!take(t, 1) && streams == m3::kSideStreams, "a full table has none for another context");
    }
    std::puts("ok");
    return 0;
}
