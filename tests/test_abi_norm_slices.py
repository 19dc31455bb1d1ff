"""gdn_add_rmsnorm on column slices of one wider buffer: not an overlap unless
the columns do, on the host with addresses that are never used (without a GPU)
and with real ones."""

import ctypes

import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from gated_delta_net_causal_gb300 import _build

ALIAS = 4


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer validation runs only without a GPU")
def test_only_columns_that_meet_are_refused():
    _build.build()
    lib = gdn.library()
    base, W = 0x100000, 256  # rows of 256 bf16: slices of 64

    def call(x, out, residual=None, sum_out=None, xs=W, os=W, q=None, qs=0):
        p = lambda col: None if col is None else ctypes.c_void_p(base + 2 * col)
        return lib.gdn_add_rmsnorm(5, 64, 1, p(x), xs, p(residual), W, p(sum_out), W, None, 1e-6, p(out), os, p(q), qs,
                                   None if q is None else ctypes.c_void_p(0x900000), None)

    for x, out in ((0, 64), (64, 0), (128, 64), (0, 192), (192, 128)):
        assert call(x, out) not in (0, ALIAS)  # nothing to launch on here: the checks are passed
    assert call(0, 64, residual=128, sum_out=192) != ALIAS
    assert call(0, 64, residual=128, sum_out=128) != ALIAS  # in place
    assert call(0, 128, q=64, qs=2 * W) != ALIAS  # codes in rows of as many bytes
    for x, out in ((0, 0), (0, 56), (64, 8), (0, 200), (200, 0), (0, W)):  # 200 + 64 runs into the next row
        assert call(x, out) == ALIAS, (x, out)
    assert call(0, 64, residual=128, sum_out=72) == ALIAS and call(0, 64, residual=120) == ALIAS
    assert call(0, 64, os=W + 8) == ALIAS and call(0, 64, xs=W + 8) == ALIAS  # other strides: somewhere they meet
    assert call(0, 128, q=64, qs=W) == ALIAS


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(3, 64), (2000, 1024), (7, 51), (2, 20000)])
def test_slices_of_one_buffer(rows, cols):
    gen = torch.Generator().manual_seed(cols)
    pitch = (cols + 7) // 8 * 8
    wide = torch.randn((rows, 4 * pitch), generator=gen).to(torch.bfloat16).cuda()
    part = lambda t, i: t[:, i * pitch:i * pitch + cols]
    before = wide.clone()
    w = (1 + 0.2 * torch.randn(cols, generator=gen)).cuda()
    want, want_sum = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda"), torch.empty_like(part(wide, 0))
    x, r = part(before, 0).contiguous(), part(before, 1).contiguous()
    gdn.gdn_add_rmsnorm(x, w, residual=r, sum_out=want_sum, out=want)
    gdn.gdn_add_rmsnorm(part(wide, 0), w, residual=part(wide, 1), sum_out=part(wide, 2), out=part(wide, 3))
    close = lambda a, b: ((a.float() - b.float()).abs() <= 2.02 * 2.0 ** -8 * b.float().abs() + 2.0 ** -133).all()
    assert torch.equal(part(wide, 2), want_sum) and close(part(wide, 3), want)
    for i in range(4):
        part(wide, i)[:] = part(before, i)
    assert torch.equal(wide, before)  # nothing between the slices was touched
