"""kvx.store_kv and kvx.load_kv: an axis of one element has no stride that counts, so K and V that differ there alone are
taken (no GPU is needed: the calls end at their missing workspace)."""
import pytest
import torch

from disaggregated_paged_kv_gb300 import kvx
from tests.test_quant_abi import A, lib  # noqa: F401


def reaches_the_library(pool, k, v, n):
    for f in (kvx.store_kv, kvx.load_kv):
        with pytest.raises(kvx.KvxError) as e:
            f(pool, 0, k, v, torch.zeros(n, dtype=torch.int32), None, torch.zeros(1, dtype=torch.int32), ws_bytes=0, stream=0)
        assert e.value.code == kvx.ERR_NO_WORKSPACE


def refused(pool, k, v, n):
    for f in (kvx.store_kv, kvx.load_kv):
        with pytest.raises(ValueError):
            f(pool, 0, k, v, torch.zeros(n, dtype=torch.int32), None, torch.zeros(1, dtype=torch.int32), ws_bytes=0, stream=0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_token_or_one_head(lib, dtype):  # noqa: F811
    """A step's rotated keys are a tensor of their own, its values a slice of the projection."""
    def pool(H):
        return kvx.Layout(2, H, 64, kvx.Q4, 64, base=A, plane_stride=64 * H * 40)
    qkv = torch.zeros(3, 8, 64, dtype=dtype)
    reaches_the_library(pool(2), torch.zeros(1, 2, 64, dtype=dtype), qkv[:1, 4:6], 1)
    reaches_the_library(pool(2), torch.zeros(1, 2, 64, dtype=dtype)[None], qkv[None, 1:2, 4:6], 1)
    reaches_the_library(pool(1), torch.zeros(3, 8, 64, dtype=dtype)[:, :1], torch.zeros(1, 3, 8 * 64, dtype=dtype)[0].view(3, 4, 128)[:, 1:2, :64], 3)
    refused(pool(2), torch.zeros(3, 2, 64, dtype=dtype), qkv[:, 4:6], 3)
    refused(pool(2), torch.zeros(1, 2, 64, dtype=dtype), qkv.view(3, 4, 128)[:1, :2, :64], 1)
