"""Answers that are kept by device (CPU only: a fake of the runtime's question for the current device)."""
import os
import shutil
import subprocess

from linear_recurrence_ssm_gb300 import _build

PROGRAM = r"""
#include "kept_by_device.cuh"

#include <initializer_list>

static int current = 0, asked = 0;
extern "C" cudaError_t CUDARTAPI cudaGetDevice(int *device) {
    *device = current;
    return cudaSuccess;
}
static ssm::KeptByDevice<3> kept;
static int get(int device, int place, cudaError_t status = cudaSuccess) {
    current = device;
    int answer = -1;
    const cudaError_t e = kept.get(place, &answer, [&](int d, int *a) {
        ++asked;
        *a = 100 * d + place + 1;
        return status;
    });
    return e == status || e == cudaSuccess ? (e ? -int(e) : answer) : -1000;
}
int main() {
    if (get(0, 2, cudaErrorNotReady) != -int(cudaErrorNotReady) || asked != 1) return 1;    // not kept
    for (int turn = 0; turn < 3; ++turn)
        for (int d : {0, 1, 63})
            for (int place = 0; place < 3; ++place)
                if (get(d, place) != 100 * d + place + 1) return 2;     // each device its own answer
    if (asked != 1 + 9) return 3;                                       // and asked once
    if (get(64, 1) != 6402 || get(64, 1) != 6402 || get(700, 2) != 70003) return 4;
    return asked == 1 + 9 + 3 ? 0 : 5;
}
"""


def test_each_device_keeps_its_own_answer(tmp_path):
    source, program = tmp_path / "kept.cpp", tmp_path / "kept"
    source.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build._nvcc()))), "include")
    subprocess.run([shutil.which("g++"), "-std=c++17", "-I" + _build.CSRC, "-I" + cuda, str(source), "-o", str(program)],
                   check=True)
    assert subprocess.run([str(program)]).returncode == 0
