"""The per-device tables that calls on several threads share (csrc/device_once.h): a host program
with a fake of the CUDA runtime, built with the thread sanitizer, which reports a data race by its
exit code.  Callers hold no lock (the entry points run without the GIL)."""
import os
import shutil
import subprocess

import pytest

from gated_softmax_attention_gqa_gb300 import build

PROGRAM = r"""
#include <atomic>
#include <thread>
#include <vector>

#include "device_once.h"

static std::atomic<int> sets[100];
static thread_local int current = 0;

extern "C" cudaError_t cudaGetDevice(int* dev) { *dev = current; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int bytes) {
    if (bytes < 0) return cudaErrorInvalidValue;
    sets[(const char*)f - (const char*)0x1000]++;
    return cudaSuccess;
}
extern "C" cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int dev) { *v = 100 + dev; return cudaSuccess; }

static const void* kernel(int i) { return (const char*)0x1000 + i; }

int main() {
    std::atomic<int> ready{0}, wrong{0};
    std::vector<std::thread> threads;
    for (int t = 0; t < 8; ++t)
        threads.emplace_back([&, t] {
            current = t % 3;
            for (ready++; ready < 8;) {}
            for (int n = 0; n < 200; ++n)
                for (int i = 0; i < 12; ++i) {
                    if (gattn::set_smem_once(kernel((i + t) % 12), 1) != cudaSuccess) wrong++;
                    if (gattn::sm_count() != 100 + current) wrong++;
                }
        });
    for (auto& t : threads) t.join();
    if (wrong) return 3;
    // every kernel on every device at least once, at most once a thread, and never again
    int before[12];
    for (int i = 0; i < 12; ++i) {
        before[i] = sets[i];
        if (before[i] < 3 || before[i] > 8) return 4;
    }
    for (current = 0; current < 3; ++current)
        for (int i = 0; i < 12; ++i) gattn::set_smem_once(kernel(i), 1);
    for (int i = 0; i < 12; ++i)
        if (sets[i] != before[i]) return 5;
    // an error is passed on and not remembered; a kernel past the table is set on every call
    current = 0;
    if (gattn::set_smem_once(kernel(50), -1) != cudaErrorInvalidValue) return 6;
    if (gattn::set_smem_once(kernel(50), 1) != cudaSuccess || sets[50] != 1) return 7;
    for (int n = 0; n < 2; ++n)
        for (int i = 0; i < 100; ++i)
            if (gattn::set_smem_once(kernel(i), 1) != cudaSuccess) return 8;
    for (int i = 0; i < 100; ++i)
        if (sets[i] == 0) return 9;
    return 0;
}
"""


def test_tables_shared_by_threads(tmp_path):
    gxx = shutil.which("g++")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    empty = tmp_path / "empty.cpp"
    empty.write_text("int main() {}\n")
    if not gxx or subprocess.run([gxx, "-fsanitize=thread", "-o", str(tmp_path / "empty"), str(empty)]).returncode:
        pytest.skip("no thread sanitizer")
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fsanitize=thread", f"-I{build.CSRC}", f"-I{cuda}", str(src), "-o", str(exe),
                    "-pthread"], check=True)
    r = subprocess.run([str(exe)], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[-4000:]
