"""Workspace sizes of attention's backward pass, as include/eqattn.h states them.
No call here reaches the GPU."""
import ctypes
import os

import pytest

import group_dft_structured_amd as eq
from group_dft_structured_amd import attention
from group_dft_structured_amd.attention import PackingStruct

A = 1 << 20  # an aligned address, never read


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(eq.LIB_PATH):
        pytest.skip("libeqlinear.so not built (run __graft_entry__.build())")
    return attention._lib()


@pytest.mark.parametrize("seqs,tokens,heads,dim,span", [(256, 262144, 16, 64, 1023), (1024, 524288, 32, 64, 128),
                                                         (512, 65536, 16, 128, 128)])
def test_sums_over_offsets_follow_the_tokens(lib, seqs, tokens, heads, dim, span):
    # not the longest sequence: a part for each tile of 64 queries or more, and one a sequence
    plan = eq.eqattn_plan_create(heads, heads, dim, 0.125, True, 32, span, eq.EQL_F16)
    most = heads * tokens * 4 + (tokens // 64 + seqs) * heads * (2 * span + 1) * 4 \
        + 16 * heads * (2 * span + 1) * 8 + 1024
    sizes = []
    for longest in (256, 2048, 8192, 65536):
        packing = PackingStruct(seqs, tokens, tokens, longest, longest, A, A, None, None)
        sizes.append(lib.eqattn_backward_workspace(plan, ctypes.addressof(packing)))
    eq.eqattn_plan_destroy(plan)
    assert all(0 < s <= most for s in sizes), (sizes, most)
