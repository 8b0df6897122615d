"""A cache held in 4 bits in pages of very many rows, one for each request: rows
past 2^32 bytes of codes of a head (GPU)."""
import pytest
import torch

import kva_int4_reference as Q
import kva_reference as R
from test_gpu_kva_int4 import Call, kva, lengths  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("head", [64, 96, 128, 256])
@pytest.mark.parametrize("extra,small", [(256, 256), (16 * 9, 16 * 17)])  # copies of 64, 16 rows
def test_rows_past_32_bit_offsets(kva, head, extra, small):
    """The same rows around row 2^32 / (head / 2) of a page give the same bits as
    in a small page, written, read back and attended to."""
    edge = -(-(1 << 32) // (head // 2) // 64) * 64  # whole tiles
    page, shift = edge + extra, edge - 128
    c = Q.Int4(210, *lengths(169), kv_heads=1, head=head, page=small, layers=1, layer=0,
               spare_pages=0).fill()
    x = Call(kva, c, 6, window=100)
    codes = torch.zeros((1, 2, 1, 1, page, head // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((1, 2, 1, 1, c.groups, page), dtype=torch.bfloat16, device="cuda")
    codes[..., shift:shift + 200, :] = c.codes[0, :, 0, :, :200].cuda()[None, :, None]
    scales[..., shift:shift + 200] = c.scales[0, :, 0, :, :, :200].cuda()[None, :, None]
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    lens = torch.tensor([168 + shift], dtype=torch.int32, device="cuda")
    far = kva.int4_cache(codes, scales, table, lens)
    near = x.cache, x.scales

    qkv = c.normal(1, 8 * head).cuda()
    q = [torch.empty(1, 6, head, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rows = [torch.empty(40, 1, head, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    off = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    for i, (d, first) in enumerate(((near, 129), (far, 129 + shift))):
        kva.kva_append_qkv_int4(q[i], qkv, x.keep[4], *d, None, 0, err_flags=x.flags)
        kva.kva_gather_kv_int4(rows[2 * i], rows[2 * i + 1], off, *d, 0, first_positions=torch.tensor(
            [first], dtype=torch.int32, device="cuda"), err_flags=x.flags)
    assert torch.equal(*q)
    assert torch.equal(rows[0], rows[2]) and torch.equal(rows[1], rows[3])
    x.call()
    want = x.out.clone()
    x.out.fill_(7.0)
    x.cache, x.scales = far
    x.call()
    torch.cuda.synchronize()
    assert int(x.flags) == 0 and torch.equal(x.out, want)
