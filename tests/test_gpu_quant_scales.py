"""pd_attn_chunk_quant where the scales of V are as small or as large as they can be: the softmax's sum is then
near the ends of what fp32 holds."""
import math

import pytest
import torch

import step_ref as ref
from test_gpu_chunk_quant import BF16, E4M3, F32, Batch, i32

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import decode_ragged_paged_gb300 as pd


@pytest.mark.parametrize("hq,new,B,d", [(4, 1, 912, 64), (4, 1, 608, 128), (16, 16, 304, 64), (16, 16, 304, 128),
                                        (16, 2, 304, 128)])
def test_many_keys_of_the_smallest_scale(hq, new, B, d):
    # Every block of V has the smallest scale, 2^-100, and all keys but the first 128 a score of 5.1875 where those
    # have 0: 2^7.48, just less than raises the maximum of the first. So the weights over their scales come to more than
    # 2^128. All requests have the same pages, so that a CTA has a request's keys.
    page, kv = 64, 300_000
    pages = kv // page + 1
    k = torch.zeros(pages, 1, page, d, device="cuda")
    k[..., 0] = 1.0
    k[:2] = 0.0
    v = (torch.arange(d, device="cuda") % 16 - 8.0).expand(pages, 1, page, d)
    k, v = k.to(E4M3), v.to(E4M3).contiguous()
    ks, vs = torch.ones(pages, 1, 1, device="cuda"), torch.full((pages, 1, 1), 2.0 ** -100, device="cuda")
    q = torch.zeros(B * new, hq, d, device="cuda", dtype=BF16)
    q[..., 0] = 5.1875
    px = torch.arange(pages, device="cuda", dtype=torch.int32).repeat(B)
    for o_dtype in (F32, BF16):
        o, lse = pd.pd_attn_chunk_quant(q, k, v, ks, vs, i32([kv] * B), i32([i * pages for i in range(B + 1)]), px,
                                        i32([i * new for i in range(B + 1)]), max_qo_len=new, max_kv_len=kv, sm_scale=1.0,
                                        o_dtype=o_dtype)
        seen = torch.arange(kv - new + 1, kv + 1, device="cuda", dtype=torch.float64)
        want = torch.log(128 + (seen - 128) * math.exp(5.1875)).repeat(B)[:, None].expand(-1, hq)
        # the sum over n keys is off by n 2^-23 of itself at most
        assert bool(((lse.double() - want).abs() <= kv * 2.0 ** -23).all())
        exact = v[0, 0, 0].double() * 2.0 ** -100
        bound = (2 * kv * 2.0 ** -23 + 2.0 ** -11 + ref.U[o_dtype]) * exact.abs()
        assert bool(((o.double() - exact).abs() <= bound).all())


@pytest.mark.parametrize("dt,d,page,block", [(BF16, 128, 16, 16), (BF16, 64, 32, 8), (BF16, 128, 6, 3), (F32, 64, 16, 16)])
@pytest.mark.parametrize("new,kv", [([40, 3], [300, 128]), ([1, 2], [300, 128]), ([2], [9000]), ([9], [9000])])
@pytest.mark.parametrize("e", [110, 116, 120, 126])
def test_scales_up_to_the_largest(dt, d, page, block, new, kv, e):
    # values of 2^-9 to 2^-4 times scales of up to 1.9 2^126
    if e > 116 and (dt == F32 or page % 8):
        pytest.skip("on the CUDA cores the sum of 9000 such values leaves fp32")
    b = Batch(51, new, kv, 4, 2, d, page, block, dt)
    codes = b.v.view(torch.uint8)
    codes[:] = torch.where((codes & 0x7f) == 0x7f, codes, (codes & 0x80) | (codes & 0x7f) % 24)
    g = torch.Generator(device="cuda").manual_seed(e)
    top = 1.0 + 0.9 * torch.rand(b.vs.shape, device="cuda", generator=g)
    b.vs = torch.where(torch.isnan(b.vs), b.vs, top * 2.0 ** e)
    b.check()
    b.check(o_dtype=F32)
    b.vs = torch.where(torch.isnan(b.vs), b.vs, torch.full_like(b.vs, 2.0 ** e))
    b.check(o_dtype=F32)
