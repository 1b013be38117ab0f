"""The 4-bit insert on one buffer that holds queries, keys and k_out side by side: the same bits as on buffers of their own."""
import pytest
import torch

import sparse_mla_decode_combine_gb300 as pkg
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [1, 5, 16])
@pytest.mark.parametrize("T", [1, 2, 77])
def test_queries_in_place_beside_keys(T, H):
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(T + H)
    row = torch.randn((T, (H + 2) * 576), generator=g, device="cuda").bfloat16()
    q, kv, ko = row[:, :H * 576].view(T, H, 576), row[:, H * 576:(H + 1) * 576], row[:, (H + 1) * 576:]
    cs = torch.randn((16, 64), generator=g, device="cuda")
    pos, slots = torch.arange(T, device="cuda") % 16, torch.randperm(T, generator=g, device="cuda")
    caches = [torch.zeros((T, 400), dtype=torch.uint8, device="cuda") for _ in range(2)]
    kept = kv.clone()
    q2 = torch.empty((T, H, 576), dtype=torch.bfloat16, device="cuda")
    k2 = torch.empty((T, 576), dtype=torch.bfloat16, device="cuda")
    pkg.check(pkg.dsv4_qk_norm_rope_kv_insert_fp4(q.clone(), q2, kept, pos, slots, cs, caches[0], k2))
    pkg.check(pkg.dsv4_qk_norm_rope_kv_insert_fp4(q, q, kv, pos, slots, cs, caches[1], ko))
    assert torch.equal(q, q2) and torch.equal(ko, k2) and torch.equal(kv, kept) and torch.equal(*caches)
    across = row[:, H * 576 + 2:(H + 1) * 576 + 2]
    assert pkg.dsv4_qk_norm_rope_kv_insert_fp4(q, q, kv, pos, slots, cs, caches[1], across) == pkg.DSV4_ERR_INVALID_ARG
    assert pkg.dsv4_get_device_status() == pkg.DSV4_OK
