"""pd_attn_chunk_quant held to what include/pd.h says of it: weights off by 2^-11 of themselves (quant_ref.attention
allows the 2^-8 of bf16 weights), and pools whose offsets pass 32 bits in each of its kernels and in the append; the
append's one rounding where scales are a caller's own."""
import pytest
import torch

import quant_ref as qref
import step_ref as ref
from test_gpu_chunk_quant import BF16, E4M3, F32, Batch, i32
from test_gpu_kvquant import Cache

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import decode_ragged_paged_gb300 as pd


def check_weights(b, causal=True, window=-1):
    """b's outputs in fp32, within quant_ref.attention's bound with 2^-11 a weight in place of 2^-8: of the weights'
    sum of the values' sizes."""
    o, lse = b.run(causal=causal, window_left=window, o_dtype=F32)
    ro, rl, ob, lb = b.ref(causal, window)
    k, v = (qref.dequant(x, s, b.layout) for x, s in ((b.k, b.ks), (b.v, b.vs)))
    sizes = ref.attention(b.q, k, torch.nan_to_num(v).abs(), b.qo, b.kv, b.pp, b.px, causal=causal, window=window,
                          layout=b.layout)[0]
    ref.check_attention(o, lse, (ro, rl, ob - (2.0 ** -8 - 2.0 ** -11) * sizes, lb))


@pytest.mark.parametrize("d,page,block", [(128, 16, 16), (64, 32, 8), (128, 64, 32), (64, 24, 24)])
@pytest.mark.parametrize("hq,hkv,new,kv", [
    (8, 2, [1, 1, 2, 2, 1], [1, 17, 64, 700, 2000]),
    (28, 4, [1] * 6, [1, 2, 64, 127, 300, 3000]),
    (8, 2, [5, 33, 12, 1], [5, 40, 1000, 2]),
    (16, 1, [1] * 5, [3, 17, 200, 5, 900]),
    (8, 2, [130, 64, 300], [130, 500, 2000]),
])
def test_weights_of_fp16(d, page, block, hq, hkv, new, kv):
    b = Batch(61, new, kv, hq, hkv, d, page, block, BF16)
    check_weights(b)
    check_weights(b, causal=False)
    check_weights(b, window=30)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("new", [1, 2, 9, 200])
def test_attention_past_32_bit_offsets(dt, new):
    # 1 and 2 tokens: the kernel for few rows; 9 and 200: the tensor cores; fp32: the CUDA cores
    d, hkv, page = 128, 8, 64
    pages = (1 << 32) // (hkv * page * d) + 40
    k, v = (torch.zeros(pages, hkv, page, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, hkv, 2), 2.0 ** -7, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(62)
    px = torch.tensor([pages - 1, 0, pages - 2, 1, pages - 30], device="cuda", dtype=torch.int32)
    for pool in (k, v):
        pool[px.long()] = (100 * torch.randn(5, hkv, page, d, device="cuda", generator=g)).clamp(-448, 448).to(E4M3).view(
            torch.uint8)
    q = torch.randn(new, 32, d, device="cuda", generator=g).to(dt)
    at = torch.arange(5, device="cuda", dtype=torch.int32)
    for layout in ("HND", "NHD"):
        kk, vv = (x if layout == "HND" else x.view(pages, page, hkv, d) for x in (k, v))
        o, lse = pd.pd_attn_chunk_quant(q, kk, vv, ks, vs, i32([300]), i32([0, 5]), px, i32([0, new]), max_qo_len=new,
                                        max_kv_len=300, layout=layout)
        few = [x[px.long()] for x in (kk, vv, ks, vs)]
        ref.check_attention(o, lse, qref.attention(q, *few, [0, new], [300], [0, 5], at, layout=layout))


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_append_past_32_bit_offsets(dt, layout):
    heads, d, page, block = 8, 128, 64, 16
    pages = (1 << 32) // (heads * page * d) + 40
    shape = (pages, heads, page, d) if layout == "HND" else (pages, page, heads, d)
    k, v = (torch.zeros(*shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, heads, page // block), 2.0 ** -9, device="cuda") for _ in range(2))
    px = i32([pages - 1, 0, pages - 2])
    g = torch.Generator(device="cuda").manual_seed(63)
    kn, vn = (torch.randn(150, heads, d, device="cuda", generator=g).to(dt) for _ in range(2))
    at = [0, 1, 2]
    want = []
    for x, pool, scale in ((kn, k, ks), (vn, v, vs)):
        few = pool[px.long()].view(E4M3), scale[px.long()]
        want.append(qref.append(x, *few, [0, 150], [170], [0, 3], at, page, block, layout))
    pd.pd_kv_append_quant(kn, vn, k, v, ks, vs, i32([0, 150]), i32([170]), i32([0, 3]), px, max_kv_len=170, layout=layout)
    torch.cuda.synchronize()
    for pool, scale, (codes, scales) in ((k, ks, want[0]), (v, vs, want[1])):
        assert torch.equal(pool[px.long()].view(E4M3).double(), codes)
        assert torch.equal(scale[px.long()].double(), scales)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("factor", [1.3, 1.7, 300.0, 0.01])
def test_append_to_callers_scales_rounds_once(dt, factor):
    # scales that are no powers of two: values are those of the exact quotients, to the nearest e4m3
    for seed in range(3):
        c = Cache(64 + seed, [3, 5, 40, 7], [20, 30, 47, 8], 4, 128, 16, 16, dt)
        c.ks *= factor
        c.vs *= factor
        want = c.want()
        c.run()
        c.check(want)
