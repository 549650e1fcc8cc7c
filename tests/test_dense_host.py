"""Host side of the dense path, and the parts of its kernels that also run on the host (CPU)."""
import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from binary_rank_linear_lb_b200 import build
from oracle import dense

# ------------------------------------------------------------ waits that give up
# The tile loop of the 8-bit linear's draining warps against barriers with phases, the
# issuing warp and the draining warps as threads.  The issuer stops before tile `stop`, or
# warp 0 gives up at tile `quit` by itself: then every wait that is not over gives up.  No
# tile may be stored as summed whose sums are not in its accumulator while it is read.
DRAIN_PROGRAM = r"""
#include <condition_variable>
#include <cstdio>
#include <mutex>
#include <thread>
#include <vector>
#include "lb_drain.h"

struct Barrier {                                   // an mbarrier: phases of `need` arrivals
    int need, left, phase = 0;
    explicit Barrier(int n) : need(n), left(n) {}
    void arrive() { if (--left == 0) { left = need; ++phase; } }
    bool done(uint32_t parity) const { return (uint32_t)(phase & 1) != parity; }
};

// 0 when all went as it should
int run(int tiles, int warps, int stop, int quit) {
    std::mutex mu;
    std::condition_variable cv;
    Barrier full[2] = {Barrier(1), Barrier(1)}, empty[2] = {Barrier(warps), Barrier(warps)};
    int held[2] = {-1, -1}, bad = 0;
    bool abort = false;
    auto wait = [&](Barrier& b, uint32_t parity) { // the barrier first, then the abort flag
        std::unique_lock<std::mutex> l(mu);
        cv.wait(l, [&] { return b.done(parity) || abort; });
        return b.done(parity);
    };
    std::vector<std::vector<int>> summed(warps, std::vector<int>(tiles, -1));
    std::thread issuer([&] {
        for (int i = 0; i < tiles; ++i) {
            const uint32_t buf = i & 1;
            if (!wait(empty[buf], ((uint32_t)(i >> 1) & 1u) ^ 1u)) return;
            std::lock_guard<std::mutex> l(mu);
            if (i == stop) {
                held[buf] = -1;                    // (partial sums)
                abort = true;
                cv.notify_all();
                return;
            }
            held[buf] = i;
            full[buf].arrive();
            cv.notify_all();
        }
    });
    std::vector<std::thread> drains;
    for (int w = 0; w < warps; ++w)
        drains.emplace_back([&, w] {
            lb::DrainTurn turn;
            for (int t = 0; t < tiles; ++t, turn.next()) {
                const uint32_t buf = turn.buf();
                if (w == 0 && t == quit) {         // gives up by itself: the others find out later
                    std::lock_guard<std::mutex> l(mu);
                    abort = true;
                    cv.notify_all();
                }
                const bool ok = turn.full([&](uint32_t parity) { return wait(full[buf], parity); });
                for (int look = 0; look < 3; ++look) {
                    std::this_thread::yield();
                    std::lock_guard<std::mutex> l(mu);
                    if (ok && held[buf] != t) ++bad;
                }
                summed[w][t] = ok;
                if (!turn.alive) continue;
                std::lock_guard<std::mutex> l(mu);
                empty[buf].arrive();
                cv.notify_all();
            }
        });
    issuer.join();
    for (auto& d : drains) d.join();
    for (int w = 0; w < warps; ++w)
        for (int t = 0; t < tiles; ++t) {
            if (summed[w][t] < 0) ++bad;           // every tile is stored, as sums or as NaN
            if (stop < 0 && quit < 0 && !summed[w][t]) ++bad;
            if (stop >= 0 && quit < 0 && summed[w][t] && t >= stop) ++bad;
            if (t > 0 && summed[w][t] && !summed[w][t - 1]) ++bad;
        }
    return bad;
}

int main() {
    int bad = 0;
    for (int rep = 0; rep < 20; ++rep)
        for (int tiles : {1, 2, 3, 7, 12}) {
            bad += run(tiles, 8, -1, -1);
            for (int at = 0; at < tiles; ++at) {
                bad += run(tiles, 8, at, -1);
                bad += run(tiles, 8, -1, at);
                bad += run(tiles, 1, at, -1);
            }
        }
    std::printf("%d\n", bad);
    return bad != 0;
}
"""


def compile_and_run(tmp_path, program, name):
    src, exe = tmp_path / (name + ".cpp"), tmp_path / name
    src.write_text(program)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-pthread", "-I" + build.CSRC, str(src), "-o", str(exe)])
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)


def test_a_wait_that_gave_up_leaves_every_later_tile_unsummed(tmp_path):
    r = compile_and_run(tmp_path, DRAIN_PROGRAM, "drain")
    assert r.returncode == 0, r.stdout + r.stderr


# ------------------------------------------------------------ the oracle's codes at a tie
def test_oracle_codes_of_ties_with_48_bit_products():
    """v = (2 k + 1) peak / 254 exactly: code k or k + 1, whichever is even."""
    rng = np.random.default_rng(3)
    for m in range(1, 254, 2):
        u, w0 = int(rng.integers(1 << 15, 66000)) | 1, int(rng.integers(1 << 23, 1 << 24)) | 1
        s = np.array([[254 * u, m * u, -m * u, m * u + 1, m * u - 1]], dtype=np.float64) * 2.0 ** -20
        w = np.full(5, w0 * 2.0 ** -30)
        even = m // 2 + (m // 2) % 2
        assert Fraction(s[0, 1] * w[1]) * 127 / Fraction(s[0, 0] * w[0]) == Fraction(m, 2)
        q, _ = dense.rmsnorm_quantize(s, w)
        assert q.tolist() == [[127, even, -even, m // 2 + 1, m // 2]], m


# ------------------------------------------------------------ building
def test_the_c_library_is_built_where_the_torch_binding_cannot_be(tmp_path, monkeypatch):
    """No g++: liblb.so stands, a binding of other sources goes, and the caller is told."""
    build.build()
    stale = tmp_path / "lb_torch.so"
    stale.write_bytes(b"")
    os.utime(stale, (1, 1))
    monkeypatch.setattr(build, "EXT", str(stale))
    monkeypatch.setenv("PATH", str(tmp_path))
    with pytest.warns(UserWarning, match="lb_torch.so.*g\\+\\+"):
        assert build.build() == build.LIB
    assert not stale.exists()


def test_the_binding_is_built_again_for_another_torch_or_python(tmp_path, monkeypatch):
    build.build()
    assert build.up_to_date()
    built = []
    monkeypatch.setattr(build, "STAMP", str(tmp_path / "stamp"))
    monkeypatch.setattr(build, "compile_ext", lambda: built.append(1))
    for made_for in (None, "torch 0.1 cpython-27\n"):      # an older tree's build, another torch's
        if made_for is not None:
            (tmp_path / "stamp").write_text(made_for)
        assert not build.up_to_date()
        build.build()
        assert built.pop() and build.up_to_date()
        build.build()
        assert not built
