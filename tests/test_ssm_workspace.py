"""The workspace that the selective scan's backward asks for, without a GPU."""
import ctypes

import pytest

import recurrent_state_memory_amd as gdr


def _need(B, T, C, N, G):
    def P(i):
        return (i + 1) << 44     # far apart, never dereferenced
    a = gdr.SsmBwdArgs(B=B, T=T, C=C, N=N, G=G, io_dtype=gdr.GDR_F32, softplus=1, x=P(0), dt=P(1), A=P(2), Bv=P(3), Cv=P(4),
                       ckpt=P(5), grad_y=P(6), grad_x=P(7), grad_dt=P(8), grad_A=P(9), grad_Bv=P(10), grad_Cv=P(11))
    need = gdr.load_library().gdr_ssm_bwd_workspace(ctypes.byref(a))
    assert need > 0
    return need


@pytest.mark.parametrize("N", [1, 3, 8, 16, 17, 33, 50, 64])
def test_as_many_planes_as_states(N):
    """Partial sums of the vectors' gradients: two fp32 numbers for every state (those of a wave
    that holds two of them count as pairs, the waves of 9 to 16 states all), token and
    workgroup; on top a row [N + 2][C] and rounding."""
    B, T, C = 4, 4096, 8192
    G = C if N <= 8 else 1024                        # groups of one channel or eight: a workgroup each
    states = N if N <= 8 else 16 if N <= 16 else N + N % 2
    assert _need(B, T, C, N, G) <= 2 * 4 * B * T * G * states + B * (N + 2) * C * 4 + 1024
