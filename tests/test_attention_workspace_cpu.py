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


@pytest.mark.parametrize("buckets,span", [(0, 0), (8, 1000)])
def test_a_call_without_dtable_needs_no_place_for_its_sums(lib, buckets, span):
    # no sequence: arguments are checked, nothing is launched
    heads, tokens = 6, 100
    plan = eq.eqattn_plan_create(heads, heads, 64, 0.125, False, buckets, span, eq.EQL_F16)
    packing = PackingStruct(0, tokens, tokens, 90, 90, None, None, None, None)
    view = attention.View(A, 64 * heads, 64)
    p, v, bias = ctypes.addressof(packing), ctypes.addressof(view), A if buckets else None
    need = heads * tokens * 4  # delta

    def call(nbytes, dtable=None):
        return lib.eqattn_backward(plan, p, v, v, v, v, v, A, bias, bias, v, v, v, dtable, A, nbytes, None)

    got = lib.eqattn_backward_workspace_no_dtable(plan, p)
    assert need <= got < need + 256 and lib.eqattn_backward_workspace_no_dtable(plan, None) == 0
    assert call(got) == 0 and call(got - 1) == 5
    full = lib.eqattn_backward_workspace(plan, p)
    assert full == got if buckets == 0 else full > got
    if buckets:
        assert call(full - 1, A) == 5
    eq.eqattn_plan_destroy(plan)
