"""The library's choice of a kernel for MXFP4 products, on the host: the sizes
that stand for each kernel in the GPU tests take it."""
import pytest

import _ffn_mx_choice as mx


@pytest.mark.parametrize("kernel,M,N,K,act,bias,residual,preact", mx.DENSE)
@pytest.mark.parametrize("f16", [False, True])
def test_dense(kernel, M, N, K, act, bias, residual, preact, f16):
    assert mx.choice(M, N, K, 0, act, bias, residual, preact, f16) == kernel


@pytest.mark.parametrize("kernel,R,E,N,K,act,bias,preact", mx.GROUPED)
@pytest.mark.parametrize("f16", [False, True])
def test_grouped(kernel, R, E, N, K, act, bias, preact, f16):
    assert mx.choice(R, N, K, E, act, bias, False, preact, f16) == kernel


def test_every_kernel_is_taken():
    assert {c[0] for c in mx.DENSE} == {1, 16, 64, 65, 128, 256} and {c[0] for c in mx.GROUPED} == {16, 64, 65, 128, 256}


@pytest.mark.parametrize("M", [1, 16, 17, 100, 4096])
@pytest.mark.parametrize("N", [8, 4096, 65536])
@pytest.mark.parametrize("K", [0, 32, 160, 256, 4096])
def test_tiles_of_256_rows_take_whole_slices(M, N, K):
    for groups in (0, 1, 100):
        kernel = mx.choice(M, N, K, groups)
        assert kernel in (1, 16, 64, 65, 128, 256) and (kernel != 256 or K in (256, 4096))
