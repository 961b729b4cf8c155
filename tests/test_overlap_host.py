"""Outputs that may lie on an input and outputs that may not, as the library's
entry points answer without a GPU: a refused overlap is AG_ERR_INVALID_ARG, an
allowed one goes on to the check of the device (any other error here)."""
import ctypes

import pytest

INVALID = 1
A, B, C, D, E = (i << 24 for i in range(1, 6))   # addresses far apart; nothing is read


@pytest.fixture(scope="module")
def agb():
    from __graft_entry__ import build_library
    build_library()
    import gnn_sparse_aggregation_b200 as m
    return m


def test_resnorm_outputs_on_matrices_and_vectors(agb):
    def fwd(X, Z, N, H, dtype, **vectors):
        op = agb.ResNorm(eps=1e-5, **vectors)
        return agb.lib.ag_resnorm_fwd(ctypes.byref(op), A, B, C, X, Z, N, H, dtype, None)
    for X, Z in ((D, E), (A, B), (C, D), (D, A)):
        assert fwd(X, Z, 4, 8, 0) != INVALID
    assert fwd(A, A, 4, 8, 0) == INVALID and fwd(A + 32, D, 4, 8, 0) == INVALID
    # one row of fp32 or two of bf16 are as long as a vector, which every row reads
    for N, dtype in ((1, 0), (2, 1)):
        for v in ("gamma1", "beta1", "scale", "gamma2", "beta2"):
            assert fwd(D, E, N, 2048, dtype, **{v: E}) == INVALID
            assert fwd(E, D, N, 2048, dtype, **{v: E}) == INVALID


def test_resnorm_gradients_on_matrices_vectors_and_scratch(agb):
    need = agb.lib.ag_resnorm_scratch_bytes(1, 64)

    def bwd(dR, dB, sums=(None,) * 5, scratch=None, N=1, H=64, **vectors):
        op = agb.ResNorm(eps=1e-5, **vectors)
        return agb.lib.ag_resnorm_backward(ctypes.byref(op), A, B, None, C, C, dR, dB, None, *sums, N, H, 0, scratch,
                                           need, None)
    assert bwd(D, E) != INVALID and bwd(A, B) != INVALID and bwd(C, D) != INVALID
    assert bwd(D, E, gamma1=D) == INVALID and bwd(D, E, gamma2=E) == INVALID
    # a vector's gradient is written when every row has been read: it may lie on the vector
    far = 9 << 24
    assert bwd(D, E, (far + 4096, None, None, None, None), far, gamma1=far + 4096) != INVALID
    assert bwd(D, E, (far + 4096, far + 4096, None, None, None), far) == INVALID
    # scratch lies on no matrix, of its own length neither
    N = 5 * 8 * 148
    need = agb.lib.ag_resnorm_scratch_bytes(N, 64)
    assert need == N * 64 * 4
    assert bwd(D, E, (far + (8 << 20), None, None, None, None), far, N=N) != INVALID
    for matrix in (A, B, C, D):
        assert bwd(D, E, (far + (8 << 20), None, None, None, None), matrix, N=N) == INVALID


def test_rotary_outputs_on_either_matrix_but_not_on_its_table(agb):
    def call(q, k, qo, ko, N=4, H=16, pos=E, freq=E + 4096, dtype=0):
        return agb.lib.ag_rotary(q, k, pos, freq, qo, ko, N, H, 2, 8, 0, 1.0, 0, dtype, None)
    for qo, ko in ((C, D), (A, B), (B, A), (B, C)):
        assert call(A, B, qo, ko) != INVALID
    assert call(A, B, C, C) == INVALID and call(A, B, A + 64, C) == INVALID
    # two bf16 rows of 64 are as long as the table of 32 frequencies, and four of 4 as their positions
    assert agb.lib.ag_rotary(A, None, C, D, D, None, 2, 64, 1, 64, 0, 1.0, 0, 1, None) == INVALID
    assert agb.lib.ag_rotary(A, None, C, D, C, None, 4, 4, 1, 4, 0, 1.0, 0, 1, None) == INVALID
