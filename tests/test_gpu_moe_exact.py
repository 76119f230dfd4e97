"""awq_w4a16_moe against bounds that a lost part of a sum cannot pass: layers whose
every value is exact, bit for bit, and the rows' distance from the fp64 form."""

import numpy as np
import pytest

from gpu_helpers import need_cuda
from serving_exact import ROW_BOUND, layer, row_distance
from serving_oracle import moe
from test_gpu_moe import _case, _Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    need_cuda()


@pytest.mark.parametrize("T,hidden,inter,E,k,group", [
    (1, 512, 256, 8, 1, 128), (2, 64, 1024, 4, 2, 64), (3, 576, 192, 4, 4, 32), (5, 1024, 2816, 6, 2, 64),
    (8, 512, 8192, 4, 1, 128), (8, 1088, 64, 64, 4, 32), (9, 512, 512, 6, 1, 64), (16, 128, 4160, 8, 2, 64),
    (24, 512, 704, 1, 1, 64), (33, 1024, 1408, 2, 1, 128), (37, 640, 320, 16, 4, 32), (64, 512, 1088, 20, 2, 64),
    (64, 192, 64, 256, 4, 64), (64, 256, 8192, 2, 2, 128)])
def test_moe_exact_layers(T, hidden, inter, E, k, group):
    X, router, gu, dn, Y, ids = layer(T, hidden, inter, E, k, group, T + hidden + inter)
    got = _Layer(X, router, gu, dn, group, k, True).run()
    assert np.array_equal(got[1], ids) and np.all(got[2] == 1 / k)
    assert np.array_equal(got[0].view(np.uint16), Y.view(np.uint16))


@pytest.mark.parametrize("T,hidden,inter,E,k,group", [
    (1, 512, 256, 8, 1, 128), (2, 576, 1024, 4, 2, 64), (3, 128, 2816, 4, 4, 32), (4, 1024, 640, 2, 1, 64),
    (4, 64, 8192, 4, 2, 64)])
def test_moe_few_tokens_keep_what_h_loses(T, hidden, inter, E, k, group):
    """Up to four tokens of an expert: H of 15 bits stays exact."""
    X, router, gu, dn, Y, ids = layer(T, hidden, inter, E, k, group, T + hidden + inter, free=True)
    got = _Layer(X, router, gu, dn, group, k, True).run()
    assert np.array_equal(got[1], ids)
    assert np.array_equal(got[0].view(np.uint16), Y.view(np.uint16))


@pytest.mark.parametrize("T,hidden,inter,E,k,group,ren", [
    (1, 512, 256, 8, 2, 128, True), (5, 2048, 384, 64, 8, 128, False), (7, 8192, 64, 4, 2, 64, True),
    (4, 64, 8192, 4, 2, 64, True), (8, 1024, 640, 4, 1, 128, True), (16, 576, 320, 3, 2, 32, False),
    (37, 1024, 256, 40, 4, 128, False), (64, 512, 384, 8, 2, 128, True), (64, 1088, 704, 18, 16, 32, True)])
def test_moe_rows_are_near(T, hidden, inter, E, k, group, ren):
    X, router, gu, dn = _case(T, hidden, inter, E, group, T + hidden + E)
    Y, ids, _, _ = moe(X, router, gu, dn, group, k, ren)
    got = _Layer(X, router, gu, dn, group, k, ren).run()
    assert np.array_equal(got[1], ids)
    d = row_distance(got[0], Y)
    assert d.max() < ROW_BOUND, d
