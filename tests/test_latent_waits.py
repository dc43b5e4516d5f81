"""The clock arithmetic of the latent-cache attention's waits, on the CPU."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_07_b200", "csrc")

# A wait that nothing ends, against a clock of which it sees 32 bits: it gives up
# no earlier than asked (or than the largest limit) and at most one look later.
PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "sa_wait.h"
int main() {
    const uint64_t step = 250'000'000;  // a quarter of a second between looks at the clock
    for (uint64_t start : {0ull, 4'000'000'000ull, 0xFFFFFFFFull, 123'456'789'012ull})
        for (uint32_t asked : {1u, 200u, 1'000'000'000u, 2'147'483'647u, 2'147'483'648u, 4'294'000'000u, 0xFFFFFFFEu, 0xFFFFFFFFu}) {
            const uint32_t limit = sa::wait32_limit(asked);
            uint64_t t = start;
            while (!sa::wait32_over(uint32_t(start), uint32_t(t), limit)) {
                t += step;
                if (t - start > 60'000'000'000ull) {
                    std::printf("a limit of %u ns never runs out\n", asked);
                    return 1;
                }
            }
            const uint64_t want = asked < sa::kMaxWait32Ns ? asked : sa::kMaxWait32Ns;
            if (t - start <= want || t - start > want + step) {
                std::printf("a limit of %u ns ran out after %llu\n", asked, static_cast<unsigned long long>(t - start));
                return 1;
            }
        }
    return 0;
}
"""


def test_every_limit_runs_out(tmp_path):
    compiler = shutil.which("g++") or shutil.which("c++")
    if compiler is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "waits.cpp", tmp_path / "waits"
    src.write_text(PROGRAM)
    subprocess.run([compiler, "-std=c++17", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True)
    assert got.returncode == 0, got.stdout


def test_the_kernel_uses_the_checked_limit():
    with open(os.path.join(CSRC, "mla_latent.cu")) as f:
        source = f.read()
    assert "wait32_limit(wait_limit_of(" in source
    assert "wait_limit_of(" not in source.replace("wait32_limit(wait_limit_of(", "")


def test_reports_between_the_ctas_of_a_pair_order_their_operands():
    """The thread that issues a pair's products reads operands of both CTAs: reports release, and its waits
    acquire, at cluster scope (a release at CTA scope would order them for the writing CTA's threads only)."""
    with open(os.path.join(CSRC, "sa_device.cuh")) as f:
        device = f.read()

    def body(name):
        start = device.index(f" {name}(")
        return device[start:device.index("\n}", start)]

    arrive = body("mbar_arrive_remote")
    assert "fence.release.sync_restrict::shared::cta.cluster" in arrive or "arrive.release.cluster" in arrive
    assert ".cta;" not in arrive.replace("shared::cta.cluster;", "")
    assert "try_wait.parity.acquire.cluster" in body("mbar_try_wait_acq_cluster")
    with open(os.path.join(CSRC, "mla_latent.cu")) as f:
        source = f.read()
    for bar in ("bar_kfull", "bar_vfull", "bar_pfull", "bar_query"):
        assert f"wait.pair(&{bar}" in source and f"wait(&{bar}" not in source, bar
