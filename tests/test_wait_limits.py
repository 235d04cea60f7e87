"""How long the prompt and tree kernels' waits last: kf_wait.cuh run on the host, and the
kernels' sources."""
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_kf_gb300", "csrc")
POLL = 3.75e-6          # a failed try_wait (kf_check_bounded_wait: 2^16 of them in 246 ms)
KEY = 40e-9             # of a unit: a 128-key tile in 5 us, with three value products

MODEL = r"""
#include <stdio.h>
#include <stdlib.h>
#include "kf_wait.cuh"
// argv: polls after which the barrier completes, polls after which another role gives up (-1: never)
int main(int, char **v) {
    const long long comes = atoll(v[1]), stops = atoll(v[2]);
    long long polls = 0;
    auto slice = [&] {
        for (unsigned i = 0; i < kf::kPollsASlice; ++i) {
            ++polls;
            if (comes >= 0 && polls > comes) return true;
        }
        return false;
    };
    auto wait = [&] { KF_WAIT_IN_SLICES(slice(), stops >= 0 && polls >= stops); };
    const bool ok = wait();
    printf("%d %lld\n", ok, polls);
}
"""


@pytest.fixture(scope="module")
def wait(tmp_path_factory):
    d = tmp_path_factory.mktemp("wait")
    (d / "wait.cpp").write_text(MODEL)
    exe = str(d / "wait")
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, str(d / "wait.cpp"), "-o", exe], check=True)

    def run(comes=-1, stops=-1):
        ok, polls = subprocess.run([exe, str(comes), str(stops)], check=True, capture_output=True,
                                   text=True).stdout.split()
        return bool(int(ok)), int(polls)
    return run


def test_a_lost_hand_off_is_given_up(wait):
    """Within some half a minute, and not before a unit of 2^29 keys has had its time."""
    ok, polls = wait()
    assert not ok
    assert (1 << 29) * KEY <= polls * POLL <= 32


def test_a_wait_ends_when_it_can(wait):
    assert wait(comes=0) == (True, 1)
    assert wait(comes=5000) == (True, 5001)
    # another role's giving up is seen within 5 ms
    ok, polls = wait(stops=100000)
    assert not ok and (polls - 100000) * POLL <= 5e-3


@pytest.mark.parametrize("name", ["kf_prompt.cu", "kf_tree.cu"])
def test_the_kernels_wait_no_longer(name):
    """The two kernels' long waits are kf_wait.cuh's; the others give up after 2^22 polls; no loop goes
    round a bounded wait a fixed number of times."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    body = re.search(r"auto long_wait = \[&\]\(uint32_t bar, uint32_t parity\) \{(.*?)\n    \};", src, re.S).group(1)
    assert re.search(r"KF_WAIT_IN_SLICES\(.*mbar_wait\(bar, parity, kPollsASlice\).*abort_flag != 0", body, re.S)
    for m in re.finditer(r"for \(int i = 0; i < (\d+); \+\+i\) \{([^}]*)\}", src):
        assert "_wait(" not in m.group(2), m.group(0)
