"""Which launches may be put in place before the one before them has ended (launch_behind in
csrc/host_common.h), against a stand-in for the CUDA runtime: only those of kernels that have run
to their end on the device, whatever threads, streams and captures the calls come from.  Nothing
runs on a GPU here."""
import ctypes
import os
import subprocess
import threading

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "softmax_topk_gb300", "csrc")

STAND_IN = r"""
#include "host_common.h"
#include <atomic>
#include <cstddef>
#include <vector>

namespace {
thread_local int device = 0;
thread_local cudaStreamCaptureMode mode = cudaStreamCaptureModeGlobal;
thread_local int attributes = -1;
std::mutex mu;
int capturing = 0, refuse_events = 0, refuse_launches = 0, live = 0, misused = 0, loads = 0;
std::vector<bool> done;  // events, by number
bool safe() { return !capturing || mode == cudaStreamCaptureModeRelaxed; }
}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes*, const void*) {
    std::lock_guard<std::mutex> lock(mu);
    ++loads;
    return cudaSuccess;
}
cudaError_t cudaThreadExchangeStreamCaptureMode(cudaStreamCaptureMode* m) {
    std::swap(*m, mode);
    return cudaSuccess;
}
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) {
    *s = capturing ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
    return cudaSuccess;
}
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) {
    std::lock_guard<std::mutex> lock(mu);
    misused += !safe();
    if (refuse_events) return cudaErrorMemoryAllocation;
    done.push_back(false);
    ++live;
    *e = reinterpret_cast<cudaEvent_t>(done.size());
    return cudaSuccess;
}
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) {
    misused += capturing != 0;
    return refuse_events ? cudaErrorUnknown : cudaSuccess;
}
cudaError_t cudaEventQuery(cudaEvent_t e) {
    std::lock_guard<std::mutex> lock(mu);
    misused += !safe();
    return done[reinterpret_cast<size_t>(e) - 1] ? cudaSuccess : cudaErrorNotReady;
}
cudaError_t cudaEventDestroy(cudaEvent_t) {
    std::lock_guard<std::mutex> lock(mu);
    --live;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void*, void**) {
    attributes = static_cast<int>(c->numAttrs);
    return refuse_launches ? cudaErrorInvalidConfiguration : cudaSuccess;
}

// 1: put in place early, 0: not, -1: the launch failed
int launch(int which, int dev) {
    static void (*const kernels[])(int) = {[](int) {}, [](int) { (void)1; }, [](int) { (void)2; },
                                           [](int) { (void)3; }};
    device = dev;
    const cudaError_t e = os::launch_behind(kernels[which], dim3(1), 32, 0, nullptr, 7);
    return e == cudaSuccess ? attributes : -1;
}
void set(int capture, int events, int launches) {
    capturing = capture, refuse_events = events, refuse_launches = launches;
}
void all_end(void) { done.assign(done.size(), true); }
int live_events(void) { return live; }
int wrong_calls(void) { return misused + (mode != cudaStreamCaptureModeGlobal); }
}
"""


@pytest.fixture
def fake(tmp_path):
    from softmax_topk_gb300 import build
    include = os.path.join(os.path.dirname(os.path.dirname(build._nvcc())), "include")
    src, lib = tmp_path / "fake.cpp", tmp_path / "fake.so"
    src.write_text(STAND_IN)
    subprocess.run(["g++", "-std=c++17", "-O0", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", CSRC,
                    "-I", include, str(src), "-o", str(lib), "-lpthread"], check=True)
    f = ctypes.CDLL(str(lib))
    yield f
    assert f.wrong_calls() == 0


def test_not_before_the_first_launch_has_ended(fake):
    assert fake.launch(0, 0) == 0
    assert [fake.launch(0, 0) for _ in range(3)] == [0, 0, 0]  # asked for, not ended
    fake.all_end()
    assert [fake.launch(0, 0) for _ in range(3)] == [1, 1, 1]
    assert fake.live_events() == 0


def test_kernels_and_devices_are_their_own(fake):
    fake.launch(0, 0)
    fake.all_end()
    assert fake.launch(0, 0) == 1 and fake.launch(1, 0) == 0 and fake.launch(0, 1) == 0
    assert fake.launch(0, 0) == 1 and fake.launch(0, 1) == 0
    fake.all_end()
    assert fake.launch(1, 0) == 1 and fake.launch(0, 1) == 1 and fake.live_events() == 0


def test_a_captured_launch_has_not_run(fake):
    fake.set(1, 0, 0)
    assert [fake.launch(0, 0) for _ in range(3)] == [0, 0, 0] and fake.live_events() == 0
    fake.set(0, 0, 0)
    fake.all_end()
    assert fake.launch(0, 0) == 0
    # its end is found inside a capture too
    fake.set(1, 0, 0)
    assert fake.launch(0, 0) == 0
    fake.all_end()
    assert fake.launch(0, 0) == 1 and fake.live_events() == 0
    fake.set(0, 0, 0)


def test_errors_leave_it_unknown(fake):
    fake.set(0, 0, 1)
    assert fake.launch(0, 0) == -1 and fake.live_events() == 0
    fake.set(0, 1, 0)
    assert fake.launch(0, 0) == 0
    fake.all_end()
    assert fake.launch(0, 0) == 0 and fake.live_events() == 0
    fake.set(0, 0, 0)
    assert fake.launch(0, 0) == 0
    fake.all_end()
    assert fake.launch(0, 0) == 1


def test_threads(fake):
    """A second thread's launch does not count on the first one's, which may come later on the GPU."""
    got, start = [], threading.Barrier(8)

    def calls():
        start.wait()
        got.extend(fake.launch(i % 4, 0) for i in range(200))

    for early in (0, 1):
        threads = [threading.Thread(target=calls) for _ in range(8)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert got == [early] * 1600
        got.clear()
        fake.all_end()
    assert fake.live_events() == 0
