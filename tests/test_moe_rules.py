"""Which form of quest_moe_fwd a call takes: the library's own rule against its definition (no GPU)."""
from __future__ import annotations

import ctypes

import pytest

import quantization_aware_amd as qa


@pytest.fixture(scope="module")
def is_few():
    """quest::moe_is_few(int n, int experts, int top, int k, int m, bool packed)."""
    f = qa.load_library()._ZN5quest10moe_is_fewEiiiiib
    f.argtypes, f.restype = [ctypes.c_int] * 5 + [ctypes.c_bool], ctypes.c_bool
    return f


@pytest.mark.parametrize("experts,top,k,m,packed", [(4, 4, 4096, 7168, False), (8, 8, 4096, 4096, False),
                                                    (1, 1, 32768, 8192, False), (64, 8, 2048, 1024, True),
                                                    (256, 8, 2048, 5632, True), (2, 1, 64, 64, False)])
def test_one_token_reads_no_expert_twice(is_few, experts, top, k, m, packed):
    assert is_few(1, experts, top, k, m, packed)


@pytest.mark.parametrize("n,experts,top,k,m,packed,few", [
    # as measured: the faster form
    (6, 64, 8, 2048, 1024, True, True), (8, 64, 8, 2048, 1024, True, False), (16, 13, 3, 704, 448, False, True),
    (24, 13, 3, 704, 448, False, False), (12, 32, 4, 1024, 512, True, True), (16, 32, 4, 1024, 512, True, False),
    (4, 8, 2, 2048, 5632, False, True), (5, 8, 2, 2048, 5632, False, False), (2, 4, 4, 4096, 7168, False, False),
    # what the form cannot hold
    (33, 256, 1, 64, 64, False, False), (1, 32, 32, 2048, 2304, True, False)])
def test_the_form_of_a_call(is_few, n, experts, top, k, m, packed, few):
    assert is_few(n, experts, top, k, m, packed) == few


@pytest.mark.parametrize("n", [2, 3, 7, 16, 30])
@pytest.mark.parametrize("experts,top", [(8, 2), (64, 8), (128, 8), (5, 5), (13, 3)])
def test_the_estimate(is_few, n, experts, top):
    """Bytes read again: those of n top expert reads less those of the experts that some token takes, a token's being
    distinct; a workgroup of 16 columns counts as 32 KB at least."""
    k, few = 1024, []
    for m in range(64, 8192 // top * 8, 64):
        if top * m > 65536 or m > 8192:
            break
        each = max(3 * m * k, 32000 * m // 16)
        again = n * top * each - experts * (1 - (1 - top / experts) ** n) * 3 * m * k
        most = 100e6 if n <= 4 else 42e6
        if abs(again - most) > 1:
            few.append(is_few(n, experts, top, k, m, False) == (again <= most))
    assert few and all(few)
