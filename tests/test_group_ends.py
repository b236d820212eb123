"""The two ends of a group of fa_prefix_decode_paged may be any 32-bit numbers: csrc/groups.h says which of them lengths are
read by, compiled here by itself (no GPU needed), and the call reports the others."""

import ctypes
import itertools
import os
import random
import shutil
import subprocess

import pytest
import torch

import attention_fa2_attn_gb300 as fa
from attention_fa2_attn_gb300 import _lib

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_fa2_attn_gb300", "csrc")
LOW, HIGH = -2**31, 2**31 - 1
# pairs whose difference is not a 32-bit number among them
ENDS = [LOW, LOW + 1, -1_500_000_000, -2, -1, 0, 1, 2, 7, 8, 9, 1_500_000_000, HIGH - 1, HIGH]


@pytest.fixture(scope="module")
def several(tmp_path_factory):
    cxx = os.environ.get("CXX", "g++")
    if not shutil.which(cxx):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("groups")
    (d / "t.cpp").write_text('#include "groups.h"\nextern "C" int several(int s0, int s1, int B) { return fa::group_of_several(s0, s1, B); }\n')
    # a sum or difference that leaves 32 bits ends the process
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-ftrapv", "-shared", "-fPIC", f"-I{CSRC}", "-o", str(d / "t.so"),
                    str(d / "t.cpp")], check=True)
    return ctypes.CDLL(str(d / "t.so")).several


def test_lengths_are_read_by_ends_inside_the_batch_only(several):
    rng = random.Random(1)
    pairs = list(itertools.product(ENDS, ENDS)) + [(rng.randint(LOW, HIGH), rng.randint(LOW, HIGH)) for _ in range(20000)]
    seen = [0, 0]
    for B in (1, 2, 8, 45_000, 2**30, HIGH):
        for s0, s1 in pairs:
            want = 0 <= s0 and s1 <= B and s1 - s0 >= 2
            assert bool(several(s0, s1, B)) == want, (s0, s1, B)
            seen[want] += 1
    assert min(seen) > 1000


def test_the_kernel_asks_nothing_else():
    # every length that is read by a group's first sequence stands behind this question
    code = open(os.path.join(CSRC, "prefix.cu")).read()
    assert code.count("group_of_several(s0, s1, p.B) ? max(0, min(") == 2 and "s1 - s0 < 2" not in code


@pytest.mark.gpu
def test_ends_that_are_no_sequences_are_reported_and_the_result_is_the_same():
    from parity import compare
    from test_gpu_prefix import _call, _case, _i32, _ref

    c = _case(8, 2, 1, 64, [(320, [10, 30, 2, 400])], 6)
    want = _ref(c)
    for s0, s1 in itertools.product(ENDS, ENDS):
        for starts in ([s0, s1], [0, s0, s1], [s0, s1, 4]):
            o, lse = _call(dict(c, starts=_i32(starts), lens=_i32([320] * (len(starts) - 1))))
            fine = starts == sorted(starts) and 0 <= starts[0] and starts[-1] <= 4
            assert fa.fa_get_last_device_error()[0] == (_lib.FA_OK if fine else _lib.FA_ERR_BOUNDS), starts
            compare(o, lse, *want, what=str(starts))
    # more sequences than a block has room for the lengths of: they come from memory then
    n = 45_000
    table = torch.zeros(n, 1, dtype=torch.int32, device="cuda:0")
    q = torch.randn(n, 1, 1, 64, device="cuda:0").bfloat16()
    pool = torch.randn(2, 16, 1, 64, device="cuda:0").bfloat16()
    one = torch.ones(n, dtype=torch.int32, device="cuda:0")
    for s0, s1 in itertools.product(ENDS, ENDS):
        o, _ = fa.fa_prefix_decode_paged(q, pool, pool, table, one, _i32([s0, s1]), _i32([16]))
        assert fa.fa_get_last_device_error()[0] == (_lib.FA_OK if 0 <= s0 <= s1 <= n else _lib.FA_ERR_BOUNDS), (s0, s1)
        assert torch.equal(o, pool[0, 0].expand(n, 1, 1, 64))  # one key: its value
