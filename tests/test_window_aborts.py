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
