"""The arithmetic of the decode by independent warps that compiles for the host as well
(csrc/cut_entries.h): which entries its merge follows, and the length of a range."""
import ctypes
import itertools
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_cache_86_gb300", "csrc")
SHIM = """
#include "cut_entries.h"
extern "C" int merges_entry(int seq, int first, int last, int at, int by_seq, int num_seqs, int ranges) {
  return pkv::merges_entry(seq, first, last, at, by_seq != 0, num_seqs, ranges);
}
extern "C" int range_length(int total, int ranges, int least) { return pkv::range_length(total, ranges, least); }
"""
LARGE = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    where = tmp_path_factory.mktemp("cut_entries")
    src, so = where / "shim.cpp", where / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + CSRC, str(src), "-o", str(so)],
                   check=True)
    return ctypes.CDLL(str(so))


def test_what_the_kernels_write_is_followed(lib):
    """(sequence, first, last): cut ones merge, whole ones and (-1, 0, 0) do not."""
    for by_seq in (0, 1):
        for seq, ranges in itertools.product((0, 1, 6), (2, 5, 304)):
            for first in range(min(ranges, 6)):
                for last in range(first, min(ranges, 8)):
                    assert lib.merges_entry(seq, first, last, seq, by_seq, 7, ranges) == (last > first)
        assert not lib.merges_entry(-1, 0, 0, 3, by_seq, 7, 5)
    assert lib.merges_entry(6, 1, 2, 2, 0, 7, 5)             # an entry of range 2 has any sequence
    assert lib.merges_entry(0, 0, 303, 0, 1, 1, 304)


def test_what_was_never_written_is_not(lib):
    """Whatever bytes an entry holds, what is followed lies in the records, the output and the line."""
    words = [-LARGE - 1, -5, -1, 0, 1, 2, 3, 4, 5, 6, 7, 303, 304, 0x3F800000, 0x7FC00000, LARGE]
    for seq, first, last in itertools.product(words, repeat=3):
        for by_seq, at in itertools.product((0, 1), (0, 3)):
            if lib.merges_entry(seq, first, last, at, by_seq, 7, 5):
                assert 0 <= seq < 7 and 0 <= first < last < 5
                assert not by_seq or seq == at
    for byte in range(256):                                  # a workspace filled with one byte
        word = int.from_bytes(bytes([byte]) * 4, "little", signed=True)
        assert not lib.merges_entry(word, word, word, 0, 1, 7, 5)


def test_the_merge_asks(lib):
    """The kernel follows an entry behind the condition alone."""
    text = open(os.path.join(CSRC, "decode_warp.cu")).read()
    body = text[text.index("decode_warp_combine_kernel"):]
    assert "if (!merges_entry(seq, r0, r1, " in body[:body.index("p.ml[")]


@pytest.mark.parametrize("ranges", [1, 2, 7, 152, 304, 1216, 65535])
def test_ranges_hold_the_whole_line(lib, ranges):
    """Up to the longest line that a call may have (16 sequences of 2^31 - 512 tokens are 2^31 - 480 tiles)."""
    for total in [0, 1, 3, 4, 5, 100, ranges, 4 * ranges, 4 * ranges + 1, 10**6, LARGE - ranges, LARGE - ranges + 1,
                  LARGE - 479, LARGE]:
        n = lib.range_length(total, ranges, 4)
        assert n * ranges >= total and n >= 4
        assert n == 4 or (n - 1) * ranges < total
