"""What the windowed kernels do once a wait has run out, as far as integer
arithmetic decides it (compiled from csrc/mla_window.cuh for the host).  The
failure itself is not made on a GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mla_decode_attention_gb300", "csrc")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("aborts")
    (d / "a.cpp").write_text('#include "mla_window.cuh"\nextern "C" unsigned loads(unsigned n, int i) { return mla::q_box_loads(n, i); }\n')
    out = str(d / "a.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "a.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


def test_query_boxes_in_flight_when_a_wait_fails(lib):
    """The key producer requests four query boxes a piece through three ring
    slots and may stop before any slot: each box is then waited for in the phase
    of its own last request, and one never requested is not waited for."""
    for pieces in range(6):
        for slots in range(3):                     # slots passed in the last piece, that failed
            requests = [[], [], [], []]            # phases requested of each box
            total = 0
            for piece in range(pieces + 1):
                for g in range(3 if piece < pieces else slots):
                    for box in ([0], [2, 1], [3])[g]:
                        requests[box].append(piece & 1)
                        total += 1
            for box in range(4):
                n = lib.loads(total, box)
                assert n == len(requests[box])
                if n:
                    assert (n - 1) & 1 == requests[box][-1]


def test_the_producer_counts_boxes_in_that_order():
    """The request loop of the kernel, read from its source: slot 0 asks for box
    0, slot 1 for 2 and 1, slot 2 for 3, and each is counted as it is asked for."""
    text = " ".join(open(os.path.join(CSRC, "mla_pair.cuh")).read().split())
    assert ("load_q_box(g == 0 ? 0 : g + 1, q); if (g == 1) load_q_box(1, q); q_boxes += g == 1 ? 2 : 1;") in text
    assert "const uint32_t loads = q_box_loads(q_boxes, i);" in text


def one_sm_kernel():
    text = open(os.path.join(CSRC, "mla_splitkv.cuh")).read()
    return " ".join(text[text.index("mla_splitkv_kernel("):].split())


def test_every_role_of_the_one_sm_kernel_comes_for_every_batch():
    """A role that leaves its loop over the pieces after a failed wait would not
    arrive at the work list, and the others would wait there for as long as that
    wait may take.  So it goes through the rest of the list before the teardown."""
    text = one_sm_kernel()
    teardown = text[text.index("// ---- teardown"):]
    walk = teardown.index("walk_list_out(p);")
    assert "__any_sync(0xffffffffu, *abort_flag != 0u) && (warp < kProducerWarp || lane == 0)" in teardown[:walk]
    assert walk < teardown.index("__syncthreads();")


def test_softmax_warps_leave_together_or_not_at_all():
    """Without the FP8 caches' barriers of all softmax warps, a warp whose wait
    failed must reach every barrier of its warpgroup, since a wait may fail for
    one warp and not for another: the loops have no way out that is not the FP8
    caches' own, behind a vote of all sixteen."""
    text = one_sm_kernel()
    softmax = text[text.index("// Thread = one token row r of the tile"):text.index("// ---- teardown")]
    assert "while ((!is_fp8(kMode) || ok) && pc.next()) {" in softmax
    waits = softmax.split("if (is_fp8(kMode) || ok) ok = mbar_wait(")[1:]   # for the scores, for the output
    assert len(waits) == 2
    for after in waits:
        fp8, rest = after.split("} else {", 1)
        assert "if constexpr (is_fp8(kMode)) {" in fp8 and "named_barrier_or(kDequantBarrier" in fp8 and "if (!ok) break;" in fp8
        other = rest.split("}", 1)[0]
        assert "ok = __all_sync(0xffffffffu, ok);" in other and "break" not in other
    # besides those two: the FP8 conversion's vote, its tile loop, its pieces
    assert softmax.count("break;") == 5
    assert "ok = !named_barrier_or(kDequantBarrier, 128 * kSoftmaxGroups, !ok); if (!ok) break; convert_unit" in softmax
    assert "if (!ok) break; } // windowed" in softmax and "if (is_fp8(kMode) && !ok) break; // ---- epilogue" in softmax


@pytest.mark.parametrize("source", ["mla_splitkv.cuh", "mla_pair.cuh"])
def test_copies_in_flight_land_before_the_block_ends(source):
    """Not every role counts what it has left in flight (the FP8 producer's codes,
    query rows, copies into the peer, products on TMEM), so after an abort every
    block pauses once its own roles have ended, before it lets the peer go, and
    once more after the peer's have, before it gives up TMEM and ends."""
    text = " ".join(open(os.path.join(CSRC, source)).read().split())
    teardown = text[text.index("// ---- teardown"):]
    order = ["__syncthreads();", "if (*abort_flag) settle_after_abort();", "cluster_sync();", "if (*abort_flag) settle_after_abort();", "tmem_dealloc("]
    at = 0
    for step in order:
        at = teardown.index(step, at) + len(step)
